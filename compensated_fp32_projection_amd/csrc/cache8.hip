// The 8-bit cache: tokens written with their blocks' scales, and read back
// (include/cfp32.h).  Both are bounded by the memory: writing reads 4 bytes and
// writes one for each value, reading back the other way.
#include "attention_device.h"
#include "cache8.h"
#include "codes8.h"

namespace cfp32 {

namespace {

__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFF; }

// One block of a sequence's tokens and one head of K or V at a time.  Sequence s
// owns the units from cu[s] / block + 2 s on: one more than its new tokens make
// of whole blocks, and one because they may begin inside a block.
// FOUR: four values at a time (16-byte loads, 4-byte stores).
template <bool E4M3, int NT, bool FOUR>
__global__ __launch_bounds__(NT) void cache8_append_kernel(HeadsView k, HeadsView v, const int32_t *cu, const int32_t *lens,
                                                           int32_t *lens_out, Cache8 c, const int32_t *table, int64_t ld, int S,
                                                           int W, int T, int64_t units)
{
    constexpr int kHeld = 8;  // values of a thread that stay in registers between the two passes, by four
    __shared__ uint32_t largest[NT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t s = (int64_t)blockIdx.x * NT + threadIdx.x; s < S; s += (int64_t)gridDim.x * NT)
        lens_out[s] = lens[s] + (cu[s + 1] - cu[s]);
    const int64_t total = units * c.Hkv * 2;
    const int per = FOUR ? c.D / 4 : c.D;
    auto start = [&](int s) { return (int64_t)(cu[s] >> c.block_log2) + 2 * (int64_t)s; };
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int h = (int)(u % c.Hkv);
        const bool second = (u / c.Hkv) & 1;
        const int64_t id = u / c.Hkv >> 1;
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
        float held[kHeld][FOUR ? 4 : 1];
        auto load = [&](int i, float (&y)[FOUR ? 4 : 1]) {
            const int t = i / per, d = i - t * per;
            const float *p = in + t * x.tok;
            if constexpr (FOUR) {
                const floatx4_t w = *reinterpret_cast<const floatx4_t *>(p + 4 * d);
#pragma unroll
                for (int q = 0; q < 4; ++q) y[q] = w[q];
            } else {
                y[0] = p[d];
            }
        };
#pragma unroll
        for (int r = 0; r < kHeld; ++r) {
            const int i = threadIdx.x + r * NT;
            if (i < items) {
                load(i, held[r]);
#pragma unroll
                for (int q = 0; q < (FOUR ? 4 : 1); ++q) most = max(most, magnitude(held[r][q]));
            }
        }
        for (int i = threadIdx.x + kHeld * NT; i < items; i += NT) {
            float y[FOUR ? 4 : 1];
            load(i, y);
#pragma unroll
            for (int q = 0; q < (FOUR ? 4 : 1); ++q) most = max(most, magnitude(y[q]));
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o));
        if (lane == 0) largest[wave] = most;
        __syncthreads();  // every thread has read the block's scale, too
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) most = max(most, largest[w]);

        float sc = NAN;
        int up = 0;
        if (most < 0x7F800000u) {
            if (!begun) {
                sc = fresh_scale<E4M3>(most);
            } else if (had >= kLeastScale && had < INFINITY) {
                up = growth<E4M3>(had, most);
                sc = __builtin_amdgcn_ldexpf(had, up);
            }
        }
        if (threadIdx.x == 0) *scale = sc;
        const bool known = sc == sc;
        const float inv = 1.0f / sc;
        auto store = [&](int i, const float (&y)[FOUR ? 4 : 1]) {
            const int t = i / per, d = i - t * per;
            uint8_t *p = base + (old + t) * pool.tok;
            float w[4] = {};
#pragma unroll
            for (int q = 0; q < (FOUR ? 4 : 1); ++q) w[q] = y[q];
            const uint32_t codes = known ? encode<E4M3>(w, sc, inv) : 0u;
            if constexpr (FOUR) *reinterpret_cast<uint32_t *>(p + 4 * d) = codes;
            else p[d] = (uint8_t)codes;
        };
#pragma unroll
        for (int r = 0; r < kHeld; ++r) {
            const int i = threadIdx.x + r * NT;
            if (i < items) store(i, held[r]);
        }
        for (int i = threadIdx.x + kHeld * NT; i < items; i += NT) {
            float y[FOUR ? 4 : 1];
            load(i, y);
            store(i, y);
        }
        if (known && up) {
            for (int i = threadIdx.x; i < old * per; i += NT) {
                const int t = i / per, d = i - t * per;
                uint8_t *p = base + t * pool.tok;
                if constexpr (FOUR) {
                    uint32_t *w = reinterpret_cast<uint32_t *>(p + 4 * d);
                    *w = shifted<E4M3>(*w, up);
                } else {
                    p[d] = (uint8_t)shifted<E4M3>(p[d], up);
                }
            }
        }
        __syncthreads();  // largest has been read
    }
}

// E codes of a token and head at a time; a block takes `tokens` rows.
template <bool E4M3, class Out, int E>
__global__ __launch_bounds__(256) void cache8_read_kernel(Cache8 c, const int32_t *table, int64_t ld, const int32_t *first,
                                                          const int32_t *cu, HeadsOut k, HeadsOut v, int S, int W, int T,
                                                          int tokens)
{
    constexpr int kMost = 64;
    __shared__ int pages[kMost], offs[kMost];  // page -1: none, -2: no row of a sequence
    const int per = c.D / E;
    const bool second = blockIdx.y;
    const PagesView &pool = second ? c.v : c.k;
    const ScalesView &sv = second ? c.vs : c.ks;
    const HeadsOut &to = second ? v : k;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < T; t0 += (int64_t)gridDim.x * tokens) {
        const int nt = (int)min((int64_t)tokens, T - t0);
        if (threadIdx.x < nt) {
            const int64_t t = t0 + threadIdx.x;
            int lo = 0, hi = S;  // the largest s < S with cu[s] <= t
            while (hi - lo > 1) {
                const int m = lo + (hi - lo) / 2;
                if (cu[m] <= t) lo = m;
                else hi = m;
            }
            int page = -2, off = 0;
            if (cu[lo] <= t && t < cu[lo + 1]) {
                const int64_t pos = (first ? first[lo] : 0) + (t - cu[lo]), entry = pos >> c.page_log2;
                off = (int)(pos & (((int64_t)1 << c.page_log2) - 1));
                page = -1;
                if (pos >= 0 && entry < W) page = table[lo * ld + entry];
                if (page < 0 || page >= c.P) page = -1;
            }
            pages[threadIdx.x] = page;
            offs[threadIdx.x] = off;
        }
        __syncthreads();
        const int n = nt * c.Hkv * per;
        for (int i = threadIdx.x; i < n; i += 256) {
            const int th = i / per, d = (i - th * per) * E, t = th / c.Hkv, h = th - t * c.Hkv;
            const int page = pages[t], off = offs[t];
            if (page == -2) continue;
            float y[E];
            if (page < 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = NAN;
            } else {
                const float s = sv.data[page * sv.page + h * sv.head + (off >> c.block_log2)];
                const uint8_t *p = (const uint8_t *)pool.data + page * pool.page + h * pool.head + off * pool.tok + d;
                if constexpr (E == 1) {
                    y[0] = code_value<E4M3, 0>(*p) * s;
                } else {
                    typedef uint32_t vec __attribute__((ext_vector_type(E / 4)));
                    const vec w = *reinterpret_cast<const vec *>(p);
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        y[e] = code_value<E4M3, 0>(w[e / 4]) * s;
                        y[e + 1] = code_value<E4M3, 1>(w[e / 4]) * s;
                        y[e + 2] = code_value<E4M3, 2>(w[e / 4]) * s;
                        y[e + 3] = code_value<E4M3, 3>(w[e / 4]) * s;
                    }
                }
            }
            Out *out = (Out *)to.data + (t0 + t) * to.tok + h * to.head + d;
            constexpr int O = E * sizeof(Out) <= 16 ? E : 16 / sizeof(Out);
            typedef Out piece __attribute__((ext_vector_type(O)));
#pragma unroll
            for (int e = 0; e < E; e += O) {
                piece w;
#pragma unroll
                for (int q = 0; q < O; ++q) {
                    // Two roundings in every form: else some make one mixed-precision instruction of product and conversion.
                    asm("" : "+v"(y[e + q]));
                    w[q] = (Out)y[e + q];
                }
                *reinterpret_cast<piece *>(out + e) = w;
            }
        }
        __syncthreads();  // pages have been read
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
    const bool small = T <= 8 * (int64_t)S;  // few tokens to a block
    int64_t blocks = units * c.Hkv * 2;
    if (blocks < 1) blocks = 1;
    if (blocks > 1 << 20) blocks = 1 << 20;
#define CFP32_APPEND8(NT, FOUR)                                                                                                    do {                                                                                                                               if (c.e4m3) cache8_append_kernel<true, NT, FOUR><<<(unsigned)blocks, NT, 0, stream>>>(k, v, cu, lens, lens_out, c, table, ld, S, W, T, units);         else cache8_append_kernel<false, NT, FOUR><<<(unsigned)blocks, NT, 0, stream>>>(k, v, cu, lens, lens_out, c, table, ld, S, W, T, units);           } while (0)
    if (small) {
        if (four) CFP32_APPEND8(64, true);
        else CFP32_APPEND8(64, false);
    } else {
        if (four) CFP32_APPEND8(256, true);
        else CFP32_APPEND8(256, false);
    }
#undef CFP32_APPEND8
    return hipGetLastError();
}

hipError_t launch_cache8_read(const Cache8 &c, const int32_t *table, int64_t ld, const int32_t *first, const int32_t *cu,
                              const HeadsOut &k, const HeadsOut &v, bool f16, int S, int W, int T, hipStream_t stream)
{
    if (T == 0 || S == 0 || c.Hkv == 0 || c.D == 0) return hipSuccess;
    const int64_t eb = f16 ? 2 : 4;
    // Codes to a load: what divides every address; results are stored 16 bytes at a time, or as many as these are.
    int64_t m = 16 | c.D;
    if (c.P > 0) m |= (int64_t)((uintptr_t)c.k.data | (uintptr_t)c.v.data) | c.k.page | c.k.head | c.k.tok | c.v.page | c.v.head | c.v.tok;
    m &= -m;
    const int64_t to = (int64_t)((uintptr_t)k.data | (uintptr_t)v.data) | eb * (k.tok | k.head | v.tok | v.head);
    while (m > 1 && to % (m * eb < 16 ? m * eb : 16)) m >>= 1;
    const int E = m >= 16 ? 16 : m >= 8 ? 8 : m >= 4 ? 4 : 1;
    const int64_t per = (int64_t)c.Hkv * (c.D / E);
    int64_t tokens = per >= 1024 ? 1 : 1024 / per;
    if (tokens > 64) tokens = 64;
    int64_t blocks = (T + tokens - 1) / tokens;
    if (blocks > 1 << 20) blocks = 1 << 20;
    const dim3 grid((unsigned)blocks, 2);
#define CFP32_READ8(E4M3, OUT, E)     cache8_read_kernel<E4M3, OUT, E><<<grid, 256, 0, stream>>>(c, table, ld, first, cu, k, v, S, W, T, (int)tokens)
#define CFP32_READ8_TYPE(E)                                     do {                                                            if (c.e4m3) {                                                   if (f16) CFP32_READ8(true, _Float16, E);                    else CFP32_READ8(true, float, E);                       } else {                                                        if (f16) CFP32_READ8(false, _Float16, E);                   else CFP32_READ8(false, float, E);                      }                                                       } while (0)
    switch (E) {
    case 16: CFP32_READ8_TYPE(16); break;
    case 8: CFP32_READ8_TYPE(8); break;
    case 4: CFP32_READ8_TYPE(4); break;
    default: CFP32_READ8_TYPE(1); break;
    }
#undef CFP32_READ8_TYPE
#undef CFP32_READ8
    return hipGetLastError();
}

}  // namespace cfp32
