// The 8-bit cache: tokens written with their blocks' scales, and read back
// (include/cfp32.h).  Both are bounded by the memory: writing reads 4 bytes and
// writes one for each value, reading back the other way (8190 tokens of 8 x 128
// INT8 written in 19 us, 4.4 TB/s, 8574 read to FP32 in 17, 5.1 TB/s).  One token of
// 64 sequences takes 5 us: sequence, page and values, one after the other.
#include "attention_device.h"
#include "cache8.h"
#include "codes8.h"
#include "lanes.h"

namespace cfp32 {

namespace {

__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFF; }

// One block of a sequence's tokens and one head of K or V: a unit.  Sequence s
// owns the blocks from cu[s] / block + 2 s on: one more than its new tokens make
// of whole blocks, and one because they may begin inside a block.  A unit is a
// wave's (GROUP 64, four to a thread block), or a whole thread block's where it
// has more values than a wave holds in registers between finding the largest
// and writing: what a unit waits for (its sequence, its page, its values) then
// has more units beside it to hide it (6001 tokens of 12 x 64 E4M3 21 -> 14.7 us).
// FOUR: four values at a time (16-byte loads, 4-byte stores).
template <bool E4M3, int GROUP, bool FOUR>
__global__ __launch_bounds__(256) void cache8_append_kernel(HeadsView k, HeadsView v, const int32_t *cu, const int32_t *lens,
                                                            int32_t *lens_out, Cache8 c, const int32_t *table, int64_t ld, int S,
                                                            int W, int T, int64_t units)
{
    constexpr int kHeld = 8, E = FOUR ? 4 : 1;  // a thread's values that stay in registers, by E
    __shared__ uint32_t largest[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int me = GROUP == 64 ? lane : threadIdx.x;
    for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s < S; s += (int64_t)gridDim.x * 256)
        lens_out[s] = lens[s] + (cu[s + 1] - cu[s]);
    const int64_t total = units * c.Hkv * 2;
    const int per = c.D / E;
    auto start = [&](int s) { return (int64_t)(cu[s] >> c.block_log2) + 2 * (int64_t)s; };
    const int64_t first = GROUP == 64 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x, step = GROUP == 64 ? (int64_t)gridDim.x * 4 : gridDim.x;
    // A unit's index in scalar registers, and with it all of its addresses' common part: with that and the walks
    // made anew a thread needs 70 registers, not 118 (8190 tokens of 8 x 128 INT8 21 -> 19 us, 6001 of 12 x 64 E4M3
    // 14.5 -> 12.4).
    for (int64_t next_u = first; next_u < total; next_u += step) {
        const int64_t u = (int64_t)__builtin_amdgcn_readfirstlane((int)(next_u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)next_u);
        const int64_t uh = over(u, c.Hkv), id = uh >> 1;
        const int h = (int)(u - uh * c.Hkv);
        const bool second = uh & 1;
        const int s = find_last(S, id, start);
        const int64_t c0 = cu[s], j = id - start(s), len = lens[s];
        const int64_t n = min((int64_t)cu[s + 1], (int64_t)T) - c0;
        if (len < 0 || c0 < 0 || n <= 0 || j < 0) continue;
        const int64_t p0 = ((len >> c.block_log2) + j) << c.block_log2;
        const int64_t a = max(p0, len), e = min(p0 + ((int64_t)1 << c.block_log2), len + n);
        const int64_t entry = p0 >> c.page_log2;
        if (a >= e || entry >= W) continue;
        const int page = table[s * ld + entry];
        if (page < 0 || page >= c.P) continue;
        const HeadsView &x = second ? v : k;
        const PagesView &pool = second ? c.v : c.k;
        const ScalesView &sv = second ? c.vs : c.ks;
        const int off = (int)(p0 & (((int64_t)1 << c.page_log2) - 1));
        float *scale = sv.data + page * sv.page + h * sv.head + (off >> c.block_log2);
        const float *in = (const float *)x.data + (c0 + (a - len)) * x.tok + h * x.head;
        uint8_t *base = (uint8_t *)pool.data + page * pool.page + h * pool.head + off * pool.tok;
        const int old = (int)(a - p0), m = (int)(e - a);  // tokens that are there, and new ones
        const bool begun = p0 < len;
        const float had = begun ? *scale : 0.0f;

        const int items = m * per;
        uint32_t most = 0;
        float held[kHeld][E];
        // A thread's items: item i is token i / per and dims E (i % per) of the unit, GROUP further each time.
        const int by_t = GROUP / per, by_d = GROUP - by_t * per;
        struct Walk {
            int t, d;
        };
        auto begin = [&]() {
            int i = me;
            asm volatile("" : "+v"(i));  // made anew where values are written, not held since they were loaded
            const int t = i / per;
            return Walk{t, i - t * per};
        };
        auto next = [&](Walk &w) {
            w.t += by_t, w.d += by_d;
            if (w.d >= per) w.d -= per, ++w.t;
        };
        auto load = [&](const Walk &at, float (&y)[E]) {
            typedef float vec __attribute__((ext_vector_type(E)));
            const vec w = __builtin_nontemporal_load(reinterpret_cast<const vec *>(in + at.t * x.tok + E * at.d));
#pragma unroll
            for (int q = 0; q < E; ++q) y[q] = w[q];
        };
        auto look = [&](const float (&y)[E]) {
#pragma unroll
            for (int q = 0; q < E; ++q) most = max(most, magnitude(y[q]));
        };
        Walk at = begin();
#pragma unroll
        for (int r = 0; r < kHeld; ++r, next(at))
            if (at.t < m) load(at, held[r]);
#pragma unroll
        for (int r = 0; r < kHeld; ++r)
            if (me + r * GROUP < items) look(held[r]);
        for (; at.t < m; next(at)) {
            float y[E];
            load(at, y);
            look(y);
        }
        most = max(most, from_lane<1>(most));
        most = max(most, from_lane<2>(most));
        most = max(most, from_lane<4>(most));
        most = max(most, from_lane<8>(most));
        most = max(most, from_lane<16>(most));
        most = max(most, from_lane<32>(most));
        if constexpr (GROUP == 256) {
            if (lane == 0) largest[wave] = most;
            __syncthreads();  // every thread has read the block's scale, too
            most = max(max(largest[0], largest[1]), max(largest[2], largest[3]));
        }

        float sc = NAN;
        int up = 0;
        if (most < 0x7F800000u) {
            if (!begun) {
                sc = fresh_scale<E4M3>(most);
            } else if (had >= kLeastScale && had < INFINITY) {
                // Not in a scalar register, where it would go as soon as it is asked for, with a wait of its own (8190
                // tokens of 8 x 128 INT8 written in 19 -> 22 us).
                float before = had;
                asm("" : "+v"(before));
                up = growth<E4M3>(before, most);
                sc = __builtin_amdgcn_ldexpf(before, up);
            }
        }
        if (me == 0) *scale = sc;
        const bool known = sc == sc;
        const float inv = 1.0f / sc;
        auto store = [&](const Walk &at, const float (&y)[E]) {
            uint8_t *p = base + (old + at.t) * pool.tok;
            float w[4] = {};
#pragma unroll
            for (int q = 0; q < E; ++q) w[q] = y[q];
            const uint32_t codes = known ? encode<E4M3>(w, sc, inv) : 0u;
            if constexpr (FOUR) *reinterpret_cast<uint32_t *>(p + 4 * at.d) = codes;
            else p[at.d] = (uint8_t)codes;
        };
        at = begin();
#pragma unroll
        for (int r = 0; r < kHeld; ++r, next(at))
            if (at.t < m) store(at, held[r]);
        for (; at.t < m; next(at)) {
            float y[E];
            load(at, y);
            store(at, y);
        }
        if (known && up) {
            for (at = begin(); at.t < old; next(at)) {
                uint8_t *p = base + at.t * pool.tok;
                if constexpr (FOUR) {
                    uint32_t *w = reinterpret_cast<uint32_t *>(p + 4 * at.d);
                    *w = shifted<E4M3>(*w, up);
                } else {
                    p[at.d] = (uint8_t)shifted<E4M3>(p[at.d], up);
                }
            }
        }
        if constexpr (GROUP == 256) __syncthreads();  // largest has been read
    }
}

constexpr int kReadTokens = 64;

// A block takes `tokens` rows; a thread E codes of a head, the same for all of
// its tokens, so that a wave's stores are whole lines (with 16 codes to a
// thread, whose results lay 64 bytes apart, 8574 tokens of 8 x 128 to FP32 took
// 27 us) and few threads have to find out where they are.
template <bool E4M3, class Out, int E>
__global__ __launch_bounds__(256) void cache8_read_kernel(Cache8 c, const int32_t *table, int64_t ld, const int32_t *first,
                                                          const int32_t *cu, HeadsOut k, HeadsOut v, int S, int W, int T,
                                                          int tokens)
{
    constexpr int kAtOnce = 8;
    __shared__ int64_t codes_at[kReadTokens], scales_at[kReadTokens];  // element offsets; codes -1: no page, -2: no row of a sequence
    __shared__ int starts[64];                 // of the sequences from the first token's on
    const int per = c.D / E;
    const bool second = blockIdx.y;
    const PagesView &pool = second ? c.v : c.k;
    const ScalesView &sv = second ? c.vs : c.ks;
    const HeadsOut &to = second ? v : k;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < T; t0 += (int64_t)gridDim.x * tokens) {
        const int nt = (int)min((int64_t)tokens, T - t0);
        if (threadIdx.x < 64) {
            const int s0 = find_last(S, t0, [&](int s) { return (int64_t)cu[s]; });
            starts[threadIdx.x] = s0 + (int)threadIdx.x < S ? cu[s0 + threadIdx.x] : 0x7FFFFFFF;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int64_t t = t0 + threadIdx.x;
            // The last sequence that begins at t or before: among these 64, or (many empty ones) beyond.
            int lo = 0, hi = 64;
            while (hi - lo > 1) {
                const int m = (lo + hi) / 2;
                if (starts[m] <= t) lo = m;
                else hi = m;
            }
            lo += s0;
            if (lo == s0 + 63) {
                hi = S;
                while (hi - lo > 1) {
                    const int m = lo + (hi - lo) / 2;
                    if (cu[m] <= t) lo = m;
                    else hi = m;
                }
            }
            int page = -2, off = 0;
            if ((int)threadIdx.x < nt && cu[lo] <= t && t < cu[lo + 1]) {
                const int64_t pos = (first ? first[lo] : 0) + (t - cu[lo]), entry = pos >> c.page_log2;
                off = (int)(pos & (((int64_t)1 << c.page_log2) - 1));
                page = -1;
                if (pos >= 0 && entry < W) page = table[lo * ld + entry];
                if (page < 0 || page >= c.P) page = -1;
            }
            if ((int)threadIdx.x < nt) {
                codes_at[threadIdx.x] = page < 0 ? page : page * pool.page + off * pool.tok;
                scales_at[threadIdx.x] = page * sv.page + (off >> c.block_log2);
            }
        }
        __syncthreads();
        const int wide = c.Hkv * per, slots = wide < 256 ? 256 / wide : 1;  // threads of a token; tokens at a time
        const int slot = wide < 256 ? (int)threadIdx.x / wide : 0;
        for (int i = (int)threadIdx.x - slot * wide; i < wide && slot < slots; i += 256) {
            const int h = i / per, d = (i - h * per) * E;
            const uint8_t *from = (const uint8_t *)pool.data + h * pool.head + d;
            const float *scales = sv.data + h * sv.head;
            Out *out = (Out *)to.data + t0 * to.tok + h * to.head + d;
            for (int u = slot; u < nt; u += slots * kAtOnce) {
                typedef uint32_t vec __attribute__((ext_vector_type(E < 4 ? 1 : E / 4)));
                vec w[kAtOnce];
                float s[kAtOnce];
                int64_t at[kAtOnce];
#pragma unroll
                for (int g = 0; g < kAtOnce; ++g) {
                    const int t = u + g * slots;
                    at[g] = t < nt ? codes_at[t] : -2;
                    s[g] = NAN;
                    w[g] = (vec)0;
                    if (at[g] < 0) continue;
                    s[g] = scales[scales_at[t]];
                    if constexpr (E == 1) w[g] = from[at[g]];
                    else w[g] = *reinterpret_cast<const vec *>(from + at[g]);
                }
#pragma unroll
                for (int g = 0; g < kAtOnce; ++g) {
                    if (at[g] == -2) continue;
                    typedef Out piece __attribute__((ext_vector_type(E)));
                    piece y;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const uint32_t word = w[g][e / 4];
                        const float code = e % 4 == 0 ? code_value<E4M3, 0>(word) : e % 4 == 1 ? code_value<E4M3, 1>(word)
                                                      : e % 4 == 2 ? code_value<E4M3, 2>(word) : code_value<E4M3, 3>(word);
                        float x = code * s[g];
                        // Two roundings in every form: else some make one mixed-precision instruction of product and conversion.
                        asm("" : "+v"(x));
                        y[e] = (Out)x;
                    }
                    *reinterpret_cast<piece *>(out + (u + g * slots) * to.tok) = y;
                }
            }
        }
        __syncthreads();  // the offsets have been read
    }
}

}  // namespace

hipError_t launch_cache8_append(const HeadsView &k, const HeadsView &v, const int32_t *cu, const int32_t *lens, int32_t *lens_out,
                                const Cache8 &c, const int32_t *table, int64_t ld, int S, int W, int T, hipStream_t stream)
{
    const int64_t in = (int64_t)((uintptr_t)k.data | (uintptr_t)v.data) | 4 * (k.tok | k.head | v.tok | v.head);
    const int64_t to = (int64_t)((uintptr_t)c.k.data | (uintptr_t)c.v.data) | c.k.page | c.k.head | c.k.tok | c.v.page | c.v.head |
                       c.v.tok;
    const bool four = c.D % 4 == 0 && in % 16 == 0 && to % 4 == 0;
    const int64_t units = T > 0 && c.P > 0 && c.D > 0 ? ((int64_t)T >> c.block_log2) + 2 * (int64_t)S : 0;
    // A unit's values: of whole blocks, or of the new tokens where they are fewer.
    int64_t tokens = S > 0 ? ((int64_t)T + S - 1) / S : 0;
    if (tokens > (int64_t)1 << c.block_log2) tokens = (int64_t)1 << c.block_log2;
    const bool wave = tokens * c.D <= 64 * 8 * (four ? 4 : 1);
    int64_t blocks = units * c.Hkv * 2;
    if (wave) blocks = (blocks + 3) / 4;
    if (blocks < 1) blocks = 1;
    if (blocks > 1 << 20) blocks = 1 << 20;
#define CFP32_APPEND8(E4M3, GROUP, FOUR) \
    cache8_append_kernel<E4M3, GROUP, FOUR><<<(unsigned)blocks, 256, 0, stream>>>(k, v, cu, lens, lens_out, c, table, ld, S, W, T, units)
#define CFP32_APPEND8_TYPE(GROUP, FOUR)                 \
    do {                                                \
        if (c.e4m3) CFP32_APPEND8(true, GROUP, FOUR);   \
        else CFP32_APPEND8(false, GROUP, FOUR);         \
    } while (0)
    if (wave) {
        if (four) CFP32_APPEND8_TYPE(64, true);
        else CFP32_APPEND8_TYPE(64, false);
    } else {
        if (four) CFP32_APPEND8_TYPE(256, true);
        else CFP32_APPEND8_TYPE(256, false);
    }
#undef CFP32_APPEND8_TYPE
#undef CFP32_APPEND8
    return hipGetLastError();
}

hipError_t launch_cache8_read(const Cache8 &c, const int32_t *table, int64_t ld, const int32_t *first, const int32_t *cu,
                              const HeadsOut &k, const HeadsOut &v, bool f16, int S, int W, int T, hipStream_t stream)
{
    if (T == 0 || S == 0 || c.Hkv == 0 || c.D == 0) return hipSuccess;
    const int64_t eb = f16 ? 2 : 4;
    // Codes to a thread: results of 16 bytes, or fewer where an address does not allow them.
    int64_t m = (f16 ? 8 : 4) | c.D;
    if (c.P > 0) m |= (int64_t)((uintptr_t)c.k.data | (uintptr_t)c.v.data) | c.k.page | c.k.head | c.k.tok | c.v.page | c.v.head | c.v.tok;
    const int64_t to = (int64_t)((uintptr_t)k.data | (uintptr_t)v.data) | eb * (k.tok | k.head | v.tok | v.head);
    m &= -m;
    while (m > 1 && to % (m * eb)) m >>= 1;
    const int E = m >= 8 ? 8 : m >= 4 ? 4 : 1;
    // Some 512 blocks for K and as many for V: the sequences' lookups are few, and what a block waits for is hidden by
    // the others (tokens to a block of T / 128, / 512 and / 1500: 8574 x 8 x 128 INT8 to FP32 29, 17 and 18 us, 6769 x
    // 12 x 64 E4M3 to FP16 15, 10 and 15).
    int64_t tokens = (int64_t)T / 512;
    tokens = tokens < 4 ? 4 : tokens > kReadTokens ? kReadTokens : tokens;
    int64_t blocks = (T + tokens - 1) / tokens;
    if (blocks > 1 << 20) blocks = 1 << 20;
    const dim3 grid((unsigned)blocks, 2);
#define CFP32_READ8(E4M3, OUT, E) \
    cache8_read_kernel<E4M3, OUT, E><<<grid, 256, 0, stream>>>(c, table, ld, first, cu, k, v, S, W, T, (int)tokens)
#define CFP32_READ8_TYPE(OUT, E)                    \
    do {                                            \
        if (c.e4m3) CFP32_READ8(true, OUT, E);      \
        else CFP32_READ8(false, OUT, E);            \
    } while (0)
    if (f16) {
        if (E == 8) CFP32_READ8_TYPE(_Float16, 8);
        else if (E == 4) CFP32_READ8_TYPE(_Float16, 4);
        else CFP32_READ8_TYPE(_Float16, 1);
    } else {
        if (E == 4) CFP32_READ8_TYPE(float, 4);
        else CFP32_READ8_TYPE(float, 1);
    }
#undef CFP32_READ8_TYPE
#undef CFP32_READ8
    return hipGetLastError();
}

}  // namespace cfp32
