// Attention of many rows that see the same keys: long packed prompts, and the
// prefix that a decoded batch shares.
//
// A block's waves hold 32 rows each (tokens x heads of one K/V head: grouped
// heads are rows like others) and go through the keys 64 at a time.  A tile
// of K and V comes from memory straight into LDS (16 bytes a lane) while the
// tile before it is multiplied.
//   * Products: v_mfma_f32_32x32x16_f16 with FP32 sums.  An FP32 operand is
//     scaled by a power of two to the top of FP16's range and split into two
//     FP16 parts of 22 bits together (rows on the way in, weights as they are
//     made, FP32 K and V in a pass over them beforehand, by tile or by key);
//     high x high, high x low and low x high are summed, low x low (below
//     2^-22) is not.  FP16 K and V are exact: two products.  The parts share
//     one scale, so all products go to the same accumulators.
//   * S^T = K Q^T leaves a lane with 32 scores of one row (column lane % 32):
//     its maximum and sum need one exchange, with lane + 32.  O^T = V^T P^T
//     takes the weights where the scores lay: keys 16 s + 4 (lane / 32) + j
//     and + 8, j < 4, are its s-th step's, and V is read in that order.
//   * V lies in LDS as in memory, a row to a key; ds_read_b64_tr_b16 gives
//     lane j of 16 the j-th column of four rows, so nothing is transposed.
//   * 16-byte chunks of a row are XORed with the row, for K (32 rows, one
//     chunk) so that 16 neighbours fall in different banks, for V (8 rows,
//     64 bytes) so that four rows do.
//   * The running maximum is followed lazily (kLazy), so that most tiles do
//     not touch the output sums.
// Bound by the matrix units' power where there is enough to do: 8192 x 32/8 x
// 128 FP32, causal, takes 1.27 ms (1.40 on the warmest card), 1300 TFLOP/s of
// products (three for one) with the units busy 77% of a clock that falls to 1.5
// GHz.  8 x 750 of these with FP16 keys take 110 to 120 us, 680 to 740 TFLOP/s
// (two for one): blocks of up to 18 tiles spend much of their time on their
// first one and their last stores.
#include <type_traits>

#include "attention_rows.h"

#define CFP32_GLOBAL __attribute__((address_space(1)))
#define CFP32_CONSTANT __attribute__((address_space(4)))

namespace cfp32 {

namespace {

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

constexpr int kTopWeight = 11;  // weights are multiplied at 2^kTopWeight: up to 2^(kTopWeight + kLazy) = 2^15
constexpr int kNoValues = 1 << 20;  // shift of a tile or key whose values are all zero
constexpr int kKeyShifts = 1 << 21; // shift of K: the tile's keys have shifts of their own

// One shift for 64 keys where the largest magnitudes of those that are not zero
// are within 1 / kSpread of each other (see Planes).
constexpr float kSpread = 0x1p-12f;

// ---- Where a tile's rows are ------------------------------------------------------

// Row row0 + lr of a tile (row0 the same for the wave), 16-byte chunk `chunk`:
// where it is, as an address of the tile's, an offset of the wave's and one of
// the lane's (32 bits each).
struct PlaneSource {
    static constexpr bool kWaveBase = true;
    const char *keys;       // of this head and sequence
    const int32_t *shifts, *key_shifts;
    int last;               // a tile beyond the last repeats it: no row sees it
    __device__ __forceinline__ int page(int, int, int) const { return 0; }
    template <int DP>
    __device__ __forceinline__ const char *base(int, int tile) const
    {
        return keys + (int64_t)min(tile, last) * (kTile * plane_key_bytes(DP));
    }
    template <int DP>
    __device__ __forceinline__ uint32_t wave_offset(int value, int plane, int row0) const
    {
        return row0 * plane_key_bytes(DP) + (value * 2 + plane) * (DP * 2);
    }
    template <int DP>
    __device__ __forceinline__ uint32_t offset(int, int, int, int lr, int chunk) const { return lr * plane_key_bytes(DP) + chunk * 16; }
    // A scalar load: a vector load would be waited for behind the tiles on their way.
    __device__ __forceinline__ int shift(int value, int tile) const
    {
        return ((const CFP32_CONSTANT int32_t *)shifts)[2 * min(tile, last) + value];
    }
    // Tile t0 + lane's shifts, asked for before what else a block begins with.
    __device__ __forceinline__ int2 ask(int t0) const
    {
        return *reinterpret_cast<const int2 *>(shifts + 2 * min(t0 + (int)(threadIdx.x & 63), last));
    }
    // No tile from t0 on has keys with shifts of their own, and those of V are
    // within 60 of each other (weights at one tile's scale are then within
    // FP32's range at another's).
    __device__ __forceinline__ bool alike(int t0, int2 s) const
    {
        const int first = __builtin_amdgcn_readfirstlane(s.y);
        bool other = false;
        for (int t = t0;;) {
            other |= s.x == kKeyShifts || (s.y != kNoValues && abs(s.y - first) > 30);
            t += 64;
            if (t > last) return !__any(other);
            s = ask(t);
        }
    }
    // [64], K and V in turn
    __device__ __forceinline__ const int32_t *shifts_of(int tile) const { return key_shifts + 2 * kTile * (int64_t)min(tile, last); }
};

struct PackedSource {
    static constexpr bool kWaveBase = true;
    const char *k, *v;      // key 0
    uint32_t k_tok, v_tok;  // bytes, below 2^26: a tile's rows are within 2^32 of each other
    int last, chunks;       // a key or chunk beyond the last repeats one: it meets a weight or an element of 0
    __device__ __forceinline__ int page(int, int, int) const { return 0; }
    template <int DP>
    __device__ __forceinline__ const char *base(int value, int tile) const
    {
        const int64_t j0 = min(tile, last / kTile) * kTile;
        return value ? v + j0 * v_tok : k + j0 * k_tok;
    }
    template <int DP>
    __device__ __forceinline__ uint32_t wave_offset(int, int, int) const { return 0; }
    template <int DP>
    __device__ __forceinline__ uint32_t offset(int value, int tile, int row0, int lr, int chunk) const
    {
        const uint32_t row = min(row0 + lr, last - min(tile, last / kTile) * kTile);
        return row * (value ? v_tok : k_tok) + (chunk < chunks ? chunk : 0) * 16;
    }
    __device__ __forceinline__ int shift(int, int) const { return 0; }
};

// A row has the address of its page, looked up (page) before the loads of several rows.
struct PagedSource {
    static constexpr bool kWaveBase = false;
    const char *k, *v;      // the head in page 0
    int64_t k_page, v_page;
    uint32_t k_tok, v_tok;  // bytes
    const int *ids;         // LDS: the pages from that of key `first` on
    int first, last, chunks, lg;
    __device__ __forceinline__ int page(int tile, int row0, int lr) const
    {
        return ids[(min(tile * kTile + row0 + lr, last) >> lg) - (first >> lg)];
    }
    template <int DP>
    __device__ __forceinline__ const char *at(int value, int tile, int row0, int lr, int chunk, int page) const
    {
        const int j = min(tile * kTile + row0 + lr, last);
        const uint32_t o = j & ((1 << lg) - 1);
        const char *base = (value ? v : k) + (int64_t)page * (value ? v_page : k_page) + (uint64_t)o * (value ? v_tok : k_tok);
        return base + (chunk < chunks ? chunk : 0) * 16;
    }
    __device__ __forceinline__ int shift(int, int) const { return 0; }
};

// Two values as high and low FP16 parts (to nearest even; p - high is exact).
// The difference takes the FP16 operand as it is, which the compiler does not
// find by itself (it converts back first).  Only that is written out: what
// reads an exponential's result too early is for the compiler to see.
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t &hi, uint32_t &lo)
{
    hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{p0, p1}, half2_t));
    float r0, r1;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r0) : "v"(hi), "v"(p0));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r1) : "v"(hi), "v"(p1));
    lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{r0, r1}, half2_t));
}

// A wave's rows on their way between memory and registers: [32 rows][64 bytes]
// of LDS, chunks of 16 bytes XORed with the row.
__device__ __forceinline__ CFP32_LDS char *stage_of(int wave, uint4 *a, uint4 *b)
{
    return (CFP32_LDS char *)(wave < 4 ? a : b) + (wave & 3) * 2048;
}
__device__ __forceinline__ int stage_at(int row, int chunk) { return row * 64 + (chunk ^ ((row >> 2) & 3)) * 16; }

// ---- The rows of a wave -------------------------------------------------------------

template <int DP>
struct WaveRows {
    floatx16_t o[DP / 32];  // O^T: this lane's column; row r of block b is dim 32 b + 8 (r / 4) + 4 (lane / 32) + r % 4
    float m, l;             // in powers of two; l of this lane's keys
    int scale;              // o is at 2^scale
};

// Keys of tiles [t0, t1), at least one, for the wave's rows q_row(0 .. 31); this
// lane's sees the first `limit` keys.  Tiles go in pairs (one body of code for each pair of
// buffers): after an odd number, one that no row sees.
template <int DP, int PL, int NW, int R, class Source, class Row>
__device__ __forceinline__ void attend_tiles(Row q_row, bool q_wide, int D, int limit, float scale, int t0, int t1,
                                             const Source &src, uint4 *k0, uint4 *k1, uint4 *v0, uint4 *v1, WaveRows<DP> &to)
{
    constexpr int CH = DP / 8;         // 16-byte chunks of a row
    constexpr int PLANE = kTile * CH;  // of a plane
    constexpr int KK = DP / 16, DB = DP / 32;
    constexpr int PER = CH / 4;        // loads of a loading wave and plane
    constexpr int LOADS = PL * PER;     // and of K or V of a tile
    static_assert(PER * (64 / CH) == 16, "a wave's rows begin where the swizzles do");
    static_assert(NW == 4 || NW == 8, "one or two groups of four waves");
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // A row's chunks are XORed with these.
    auto k_swizzle = [](int row) { return CH == 16 ? row & 15 : (row >> 1) & 7; };
    auto v_swizzle = [](int row) { return CH == 16 ? (row & 3) << 2 | ((row >> 2) & 3) : (row & 2) << 1 | ((row >> 2) & 3); };

    // Loads are 64 chunks each, PER of each of the first four waves to a plane:
    // load n of a tile's K or V.
    auto page = [&](int tile, int n) { return src.page(tile, (wave * PER + n % PER) * (64 / CH), lane / CH); };
    auto fetch = [&](int value, int tile, uint4 *buf, int n, int at_page) {
        const int i = n % PER, p = n / PER, piece = wave * PER + i, row0 = piece * (64 / CH);
        int from_lane = lane;
        asm("" : "+v"(from_lane));  // the addresses are made again each time: kept, they would cost the products registers
        const int lr = from_lane / CH;
        const int c = (from_lane % CH) ^ (value ? v_swizzle(lr) ^ v_swizzle(i * (64 / CH)) : k_swizzle(lr) ^ k_swizzle(i * (64 / CH)));
        CFP32_LDS void *to_lds = (CFP32_LDS void *)(buf + p * PLANE + piece * 64);
        if constexpr (Source::kWaveBase) {
            // (A global load to LDS would make the compiler wait for every read of LDS before it uses one.)
            const char *base = src.template base<DP>(value, tile);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void *)base, 0, -1, 0x00020000), to_lds, 16,
                                                     src.template offset<DP>(value, tile, row0, lr, c),
                                                     src.template wave_offset<DP>(value, p, row0), 0, 0);
        } else {
            __builtin_amdgcn_global_load_lds((const CFP32_GLOBAL void *)src.template at<DP>(value, tile, row0, lr, c, at_page),
                                             to_lds, 16, 0, 0);
        }
    };
    t1 += (t1 - t0) & 1;
    int2 shifts = {};
    if constexpr (PL == 2) shifts = src.ask(t0);
    if (wave < 4) {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) fetch(0, t0, k0, n, page(t0, n));
    }

    float x[KK][8];  // the row's values 16 i + 8 half ..
    if (q_wide) {
        // Four lanes to 64 bytes of a row, and to their places through LDS
        // (a lane for itself, 16 bytes of 64 rows at a time, spent 4 us).
        CFP32_LDS char *stage = stage_of(wave, v0, v1);
        const float *qa = q_row(lane >> 2), *qb = q_row(16 + (lane >> 2));
        float y[KK][2][4];
#pragma unroll
        for (int i = 0; i < KK; ++i) {
            load_floats<4, true>(qa, 16 * i + 4 * (lane & 3), D, y[i][0]);
            load_floats<4, true>(qb, 16 * i + 4 * (lane & 3), D, y[i][1]);
        }
#pragma unroll
        for (int i = 0; i < KK; ++i) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                *(CFP32_LDS floatx4_t *)(stage + stage_at(16 * s + (lane >> 2), lane & 3)) =
                    floatx4_t{y[i][s][0], y[i][s][1], y[i][s][2], y[i][s][3]};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const floatx4_t z = *(CFP32_LDS floatx4_t *)(stage + stage_at(col, 2 * half + s));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][4 * s + e] = z[e];
            }
        }
    } else {
        const float *q = q_row(col);
#pragma unroll
        for (int i = 0; i < KK; ++i) load_floats<8, false>(q, 16 * i + 8 * half, D, x[i]);
    }
    // The row, at 2^e2, as the right operand of the scores.
    half8_t qh[KK], ql[KK];
    const float f = fabsf(scale) * kLog2e;  // the sign goes into the row
    int e2;  // (scores are taken back from the row's and the keys' shifts at once: one after the other may leave FP32's range)
    auto split_row = [&] {
        float mx = 0.0f;
        // (A row that is not finite has no finite result, whatever its scale.)
#pragma unroll
        for (int i = 0; i < KK; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[i][e]));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        e2 = top_shift(mx);
#pragma unroll
        for (int i = 0; i < KK; ++i) {
            uint32_t h[4], w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p0 = __builtin_amdgcn_ldexpf(scale < 0.0f ? -x[i][2 * e] : x[i][2 * e], e2);
                const float p1 = __builtin_amdgcn_ldexpf(scale < 0.0f ? -x[i][2 * e + 1] : x[i][2 * e + 1], e2);
                split_pair(p0, p1, h[e], w[e]);
            }
            qh[i] = __builtin_bit_cast(half8_t, uint4_t{h[0], h[1], h[2], h[3]});
            ql[i] = __builtin_bit_cast(half8_t, uint4_t{w[0], w[1], w[2], w[3]});
        }
    };
    float m = -INFINITY, l = 0.0f;
    int cv = kNoValues;  // values are summed at 2^(kTopWeight + cv); kNoValues: none yet
    floatx16_t o[DB];
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] = 0.0f;

    // This lane's byte in a plane: K's row col, chunk `half`; V's row 4 half +
    // (lane % 16) / 4, columns 16 ((lane / 16) % 2) + 4 (lane % 4).
    const int k_at = (col * CH + (half ^ k_swizzle(col))) * 16;
    const int i16 = lane & 15, v_row = 4 * half + (i16 >> 2), v_chunk = 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
    const int v_at = (v_row * CH + (v_chunk ^ v_swizzle(v_row))) * 16 + 8 * (i16 & 1);

    floatx16_t s[2];
    half8_t ph[4], pl[4];
    // The running maximum after a tile whose largest score is mx, and the
    // sums' scale after its largest weight times value, `comes` beside the
    // maximum (in powers of two, FP32 V): at 2^-cv beside the weights' 2^-m,
    // it is lowered only by a tile that weighs more with its values than all
    // before it (lazily, as m is).  A tile that the row does not see, or gives
    // no weight, leaves it.  m and cv are integers there, so what the sums are
    // multiplied by is exact.
    auto above = [&](float mx) { return fmaxf(m, PL == 2 ? ceilf(mx) : mx); };
    auto follow = [&](float mx, float mn, float comes) {
        const float held = (m - (mn == -INFINITY ? 0.0f : mn)) - (float)cv;  // what was summed, as `comes`
        if (__any(mx > m + kLazy || (PL == 2 && comes > held + kLazy))) {
            const float d = mn == -INFINITY ? 1.0f : exp2_raw(m - mn);
            float c = d;
            if (PL == 2) {
                const float top = fmaxf(held, ceilf(comes));
                cv = top > -(float)kNoValues ? -(int)top : kNoValues;
                c = exp2_raw(held + (float)cv);
            }
            m = mn;
            l *= d;
#pragma unroll
            for (int b = 0; b < DB; ++b) o[b] *= c;
        }
    };
    auto zero_if_none = [](float x) { return x == -INFINITY ? 0.0f : x; };
    // `each`: K and V have a scale for each key, for what one scale for 64 keys,
    // or tiles whose scales are alike, does not hold.  A loop of its own, chosen
    // once for a block from shifts asked for before the row (a test in each
    // tile cost the usual inputs 3 to 5%, the shifts asked for by themselves 1
    // to 3%); 8192 x 32/8 x 128 whose blocks all take it 2.26 ms against 1.34,
    // 1000 x 12 x 64 57 us against 36.
    auto weights = [&](int tile, int k_shift, int v_shift, auto each) {
        constexpr bool EACH = decltype(each)::value;
        const int j0 = tile * kTile, n = limit - j0 - 4 * half;
        float ft, base;
        int up = 0;  // this tile's values beside the sums' scale
        if constexpr (EACH) {
            // Key by key, and the weights' sum by itself: those for the values may leave FP32's range.
            auto by_key = [&](int value, auto change) {
                const CFP32_GLOBAL int32_t *shifts = nullptr;
                if constexpr (PL == 2) shifts = (const CFP32_GLOBAL int32_t *)src.shifts_of(tile) + 8 * half + value;
                asm("" : "+v"(shifts));  // read again each time, four at a time: kept, they would need registers
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = 32 * b + 8 * (r / 4) + r % 4;
                        s[b][r] = change(s[b][r], key, shifts[2 * key]);
                        if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    }
            };
            float mx = -INFINITY, comes = -INFINITY;
            by_key(0, [&](float x, int key, int shift) {
                const float fk = __builtin_amdgcn_ldexpf(f, -e2 - shift);
                x = key < n ? x * fk : -INFINITY;
                mx = fmaxf(mx, key < n && fk == INFINITY ? INFINITY : x);
                return x;
            });
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = above(mx), from = zero_if_none(mn);
            by_key(1, [&](float x, int, int shift) {
                comes = fmaxf(comes, (x - from) - (float)shift);
                return x;
            });
            follow(mx, mn, fmaxf(comes, __shfl_xor(comes, 32)));
            const float top = zero_if_none(m);
            by_key(1, [&](float x, int, int shift) {
                x -= top;
                l += exp2_raw(x + (float)kTopWeight);
                return x - (float)shift;
            });
            ft = 1.0f;
            base = (float)(kTopWeight + cv);
        } else {
            ft = __builtin_amdgcn_ldexpf(f, -e2 - (PL == 2 ? k_shift : 0));
            const bool far = ft == INFINITY;
            if (__any(j0 + kTile > limit)) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float x = s[b][r] * ft;
                        s[b][r] = 32 * b + 8 * (r / 4) + r % 4 < n ? x : -INFINITY;
                    }
                ft = 1.0f;
            }
            float mx = fmaxf(s[0][0], s[1][0]);
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, fmaxf(s[0][r], s[1][r]));
            mx = far ? INFINITY : mx * ft;  // ft >= 0
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = above(mx);
            follow(mx, mn, v_shift == kNoValues ? -INFINITY : (mx - zero_if_none(mn)) - (float)v_shift);
            if (PL == 2) up = v_shift == kNoValues ? 0 : v_shift - cv;
            base = (float)(kTopWeight - up) - zero_if_none(m);
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t h[4], w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p0 = exp2_raw(fmaf(s[t / 2][8 * (t % 2) + 2 * e], ft, base));
                const float p1 = exp2_raw(fmaf(s[t / 2][8 * (t % 2) + 2 * e + 1], ft, base));
                sum[0] += p0;
                sum[1] += p1;
                split_pair(p0, p1, h[e], w[e]);
            }
            ph[t] = __builtin_bit_cast(half8_t, uint4_t{h[0], h[1], h[2], h[3]});
            pl[t] = __builtin_bit_cast(half8_t, uint4_t{w[0], w[1], w[2], w[3]});
            __builtin_amdgcn_sched_barrier(0);  // eight at a time: more would need registers the products hold
        }
        const float add = sum[0] + sum[1];
        if (!EACH) l = PL == 2 ? fmaf(add, __builtin_amdgcn_ldexpf(1.0f, up), l) : l + add;
    };
    // The products of a phase: V of one tile with its weights (VALUES), K of
    // the next with the row (SCORES).  Fragments (4 registers) go through a
    // ring of R, each requested R - 2 ahead of its use; in between,
    // also(n) is called for n = 0, 1, ... 2 LOADS - 1 (the next loads).
    constexpr int NV = 4 * DB * PL, NK = 2 * KK * PL;
    auto products = [&](const uint4 *vb, const uint4 *kb, auto with_values, auto with_scores, auto also) {
        constexpr bool VALUES = decltype(with_values)::value, SCORES = decltype(with_scores)::value;
        constexpr int from = VALUES ? 0 : NV, to = SCORES ? NV + NK : NV;
        constexpr int every = (to - from) / (2 * LOADS);
        half8_t ring[R];
        int v_lane = v_at, k_lane = k_at;
        asm("" : "+v"(v_lane), "+v"(k_lane));  // addresses are made where they are used: kept, they would cost registers
        // Fragments in pairs of accumulators b, b + 1: the low parts, then the high ones.
        auto part = [](int k) { return PL - 1 - k / 2 % PL; };
        auto read = [&](int n) -> half8_t {
            if (n < NV) {  // keys 16 t, dims 32 b
                const int p = part(n), b = n / (2 * PL) * 2 % DB + n % 2, t = n / PL / DB;
                short4_t y[2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    y[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CFP32_LDS short4_t *)(
                        (CFP32_LDS char *)vb + ((v_lane ^ (b * 64) ^ (u * 32)) + (p * PLANE + (16 * t + 8 * u) * CH) * 16)));
                return __builtin_bit_cast(half8_t, __builtin_shufflevector(y[0], y[1], 0, 1, 2, 3, 4, 5, 6, 7));
            }
            const int k = n - NV, p = part(k), b = k % 2, i = k / PL / 2;  // dims 16 i, keys 32 b
            return *reinterpret_cast<const half8_t *>((const char *)kb + ((k_lane ^ (i * 32)) + (b * 32 * CH + p * PLANE) * 16));
        };
#pragma unroll
        for (int n = from; n < from + R - 2; ++n) ring[n % R] = read(n);
        if (SCORES)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
#pragma unroll
        for (int n = from; n < to; ++n) {
            if (n + R - 2 < to) ring[(n + R - 2) % R] = read(n + R - 2);
            if ((n - from) % every == 0 && (n - from) / every < 2 * LOADS) also((n - from) / every);
            __builtin_amdgcn_sched_barrier(0);
            // Neighbouring products go to different accumulators: the high
            // fragments meet the low weights one by one, and the high ones together.
            const bool value = n < NV;
            const int k = value ? n : n - NV, p = part(k), t = k / PL / DB, i = k / PL / 2;
            const int b = value ? k / (2 * PL) * 2 % DB + k % 2 : k % 2;
            auto multiply = [&](const half8_t &x, int to_b, bool low) {
                if (value) o[to_b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, low ? pl[t] : ph[t], o[to_b], 0, 0, 0);
                else s[to_b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, low ? ql[i] : qh[i], s[to_b], 0, 0, 0);
            };
            multiply(ring[n % R], b, p == 0);
            if (p == 0 && k % 2) {
                multiply(ring[(n - 1) % R], b - 1, false);
                multiply(ring[n % R], b, false);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // With eight waves: two groups, one of each on every SIMD, half a tile
    // apart: while one multiplies (values of the tile before, scores of this one), the
    // other turns scores into weights on the vector units.  Phases end with a
    // barrier; the first group multiplies in even ones, the second in odd ones.
    // K(t) and V(t - 1) are read in phases 2 t and 2 t + 1, so their buffers
    // can be filled from phase 2 t + 2 on, and must be full when phase 2 t + 4
    // begins.  The first group does that: it asks for the loads between its
    // products in phase 2 t + 2 and waits for them at the end of 2 t + 3.
    // With four waves there is one group, often beside another block's, and a
    // barrier before its products (asking for the loads before the weights
    // instead, for a longer flight, was slower: 8192 x 32/8 x 128 FP16 955 ->
    // 1011 us).
    auto sync = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto drain = [] { __builtin_amdgcn_s_waitcnt(0x0F70); };  // vmcnt(0)
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    // The groups run separate copies of the loop: which loads are on their way
    // at which read is then plain to the compiler, which would wait otherwise.
    // All waves go through all tiles (those of the block's last row): the
    // barriers hold them that long anyway.
    auto run = [&](auto group, auto each) {
        constexpr bool second = decltype(group)::value;
        int t = t0;
        // K(u), V(u - 1); beyond the last tile, where no one reads them, the last again.
        auto refill = [&](int u, uint4 *kb, uint4 *vb) {
            return [=, &fetch, &page](int n) {
                const int tile = n >= LOADS ? u - 1 : u;
                if (!second) fetch(n >= LOADS, tile, n >= LOADS ? vb : kb, n % LOADS, page(tile, n % LOADS));
            };
        };
        // Weights of tile t, its values, the next one's scores (unless it is the last).
        auto step = [&](uint4 *k_now, uint4 *k_next, uint4 *v_now, uint4 *v_next, auto last) {
            constexpr bool more = !decltype(last)::value;
            weights(t, src.shift(0, t), src.shift(1, t), each);
            if (!second) drain();
            if (!second || more) sync();
            if constexpr (more) {
                products(v_now, k_next, yes, yes, refill(t + 2, k_now, v_next));
                if (NW == 8) sync();
            } else {
                products(v_now, k_next, yes, no, [](int) {});
            }
            ++t;
        };
        if (second) sync();
        products(v0, k0, no, yes, refill(t0 + 1, k1, v0));
        if (NW == 8) sync();
        while (t + 2 < t1) {
            step(k0, k1, v0, v1, no);
            step(k1, k0, v1, v0, no);
        }
        step(k0, k1, v0, v1, no);
        step(k1, k0, v1, v0, yes);
    };
    auto run_groups = [&](auto each) {
        split_row();
        drain();
        sync();
        if (NW == 8 && wave >= 4) run(yes, each);
        else run(no, each);
    };
    if constexpr (PL == 2) {
        if (src.alike(t0, shifts)) {
            run_groups(no);
        } else {
            // (The row is split in both places, so that what one loop has no
            // registers for is not spilled in the other.)
            asm volatile("" ::: "memory");
            run_groups(yes);
        }
    } else {
        run_groups(no);
    }
#pragma unroll
    for (int b = 0; b < DB; ++b) to.o[b] = o[b];
    to.m = m;
    // Scores (in powers of two) beyond FP32's range, the lowest of them for
    // all keys included: whether they are finite as such is for the slow form.
    l += __shfl_xor(l, 32);
    to.l = m == INFINITY || (l == 0.0f && limit > t0 * kTile) ? NAN : l;
    to.scale = kTopWeight + (cv == kNoValues ? 0 : PL == 2 ? cv : 0);
}

// A wave's 32 rows y(b, 4 c + e) (laid out as o) to row_to(0 .. 31) (null: no
// such row), the first D values of each, through LDS: four lanes to 64 bytes
// of a row.  `wide`: rows allow 16-byte stores.
template <int DP, class Value, class Row>
__device__ __forceinline__ void store_rows(CFP32_LDS char *stage, Value y, Row row_to, int D, bool wide)
{
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    float *to[2] = {row_to(lane >> 2), row_to(16 + (lane >> 2))};
#pragma unroll
    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
        for (int c2 = 0; c2 < 4; c2 += 2) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                floatx4_t x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = y(b, 4 * (c2 + c) + e);
                *(CFP32_LDS floatx4_t *)(stage + stage_at(col, 2 * c + half)) = x;
            }
            const int d = 32 * b + 8 * c2 + 4 * (lane & 3);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const floatx4_t x = *(CFP32_LDS floatx4_t *)(stage + stage_at(16 * s + (lane >> 2), lane & 3));
                if (!to[s]) continue;
                if (wide && d + 4 <= D) {
                    *reinterpret_cast<floatx4_t *>(to[s] + d) = x;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (d + e < D) to[s][d + e] = x[e];
                }
            }
        }
}

template <int DP>
__device__ __forceinline__ void no_rows(WaveRows<DP> &w)
{
    w.m = -INFINITY, w.l = 0.0f, w.scale = 0;
#pragma unroll
    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) w.o[b][e] = 0.0f;
}

// A wave's rows into their slots (slot_of(row) < 0: no such row).
template <int DP, class Slot>
__device__ __forceinline__ void leave_rows(const WaveRows<DP> &w, const Partials &to, Slot slot_of, CFP32_LDS char *stage)
{
    const int lane = threadIdx.x & 63;
    const int64_t slot = slot_of(lane & 31);
    if (lane < 32 && slot >= 0) {
        to.m[slot] = w.m;
        to.l[slot] = __builtin_amdgcn_ldexpf(w.l, -kTopWeight);
    }
    if (!__any(w.l != 0.0f)) return;
    store_rows<DP>(stage, [&](int b, int r) { return __builtin_amdgcn_ldexpf(w.o[b][r], -w.scale); },
                   [&](int row) {
                       const int64_t s = slot_of(row);
                       return s < 0 ? (float *)nullptr : to.o + s * DP;
                   }, DP, true);
}

// Tiles [0, n) in parts of an even number.
__device__ __forceinline__ void part_tiles(int n, int part, int parts, int &t0, int &t1)
{
    const int per = ((n + parts - 1) / parts + 1) & ~1;
    t0 = (int)min((int64_t)n, (int64_t)part * per);
    t1 = min(n, t0 + per);
}

// ---- Long prompts -------------------------------------------------------------------

template <class T, int DP, int NW>
__global__ __launch_bounds__(64 * NW, 2) void prompt_tile_kernel(PromptArgs a, Planes planes, Partials to)
{
    constexpr int PL = sizeof(T) == 4 ? 2 : 1;
    constexpr int kBlockRows = NW * kWaveRows;
    __shared__ uint4 k0[PL * kTile * DP / 8], k1[PL * kTile * DP / 8], v0[PL * kTile * DP / 8], v1[PL * kTile * DP / 8];
    const int g = a.Hq / a.Hkv;
    const int kh = blockIdx.x % a.Hkv, part = blockIdx.y;
    const int64_t id = (gridDim.x - 1 - blockIdx.x) / a.Hkv;  // the rows that see most first
    int64_t start;
    const int sid = find_unit(a.cu_q, a.S, g, kBlockRows, id, start);
    const Sequence sq = sequence(a, sid);
    const int64_t n = (int64_t)sq.nq * g, r0 = (id - start) * kBlockRows;
    if (id < start || r0 >= n) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = r0 + wave * kWaveRows;
    const int own = (int)over(min(first + (lane & 31), n - 1), g);  // this lane's row of the sequence
    const bool rows = first < n;
    const int keys = sq.limit((int)over(min(r0 + kBlockRows, n) - 1, g));
    const int limit = sq.limit(own);
    // Row of the wave -> token, head.
    auto q_row = [&](int row) {
        const int64_t r = min(first + row, n - 1), i = over(r, g);
        return (const float *)a.q.data + (sq.q0 + i) * a.q.tok + (kh * g + (r - i * g)) * a.q.head;
    };
    const bool q_wide = rows_wide(a.q.data, a.q.tok | a.q.head, a.D);
    WaveRows<DP> w;
    int t0, t1;
    part_tiles((keys + kTile - 1) / kTile, part, to.slots, t0, t1);
    if (t0 >= t1) {
        no_rows<DP>(w);
    } else if constexpr (PL == 2) {
        const int64_t key = kh * planes.count + sq.k0;
        const PlaneSource src = {planes.keys + key * plane_key_bytes(DP), planes.shifts + 2 * (kh * planes.slots + sq.k0 / kTile + sid),
                                 planes.key_shifts + 2 * key, t1 - 1};
        attend_tiles<DP, PL, NW, 7>(q_row, q_wide, a.D, limit, a.scale, t0, t1, src, k0, k1, v0, v1, w);
    } else {
        const PackedSource src = {(const char *)((const T *)a.k.data + sq.k0 * a.k.tok + kh * a.k.head),
                                  (const char *)((const T *)a.v.data + sq.k0 * a.v.tok + kh * a.v.head),
                                  (uint32_t)(a.k.tok * 2), (uint32_t)(a.v.tok * 2), sq.nk - 1, a.D / 8};
        attend_tiles<DP, PL, NW, 7>(q_row, q_wide, a.D, limit, a.scale, t0, t1, src, k0, k1, v0, v1, w);
    }
    if (!rows) return;
    // K's buffers have been read by now (V's last may be in use).
    CFP32_LDS char *stage = stage_of(wave, k0, k1);
    if (to.o)
        return leave_rows<DP>(w, to, [&](int row) -> int64_t {
            const int64_t r = first + row, i = over(r, g);
            return r < n ? ((sq.q0 + i) * a.Hq + kh * g + (r - i * g)) * to.slots + part : -1;
        }, stage);
    // l is summed at 2^kTopWeight, o at 2^scale: one factor where that is no
    // extreme power of two.
    const float inv = w.l == 0.0f ? 0.0f : 1.0f / w.l;
    const int shift = kTopWeight - w.scale;
    const bool once = PL == 1 || (shift > -60 && shift < 60);
    const float factor = __builtin_amdgcn_ldexpf(inv, once ? shift : 0);
    const int then = once ? 0 : shift;
    float finite = 0.0f;  // NaN once a result is not
#pragma unroll
    for (int b = 0; b < DP / 32; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            w.o[b][r] *= factor;
            if (then) w.o[b][r] = __builtin_amdgcn_ldexpf(w.o[b][r], then);
            finite = fmaf(w.o[b][r], 0.0f, finite);
        }
    const bool live = first + (lane & 31) < n, odd = finite != finite;
    store_rows<DP>(stage, [&](int b, int r) { return w.o[b][r]; },
                   [&](int row) {
                       const int64_t r = first + row, i = over(r, g);
                       return r < n ? a.out + (sq.q0 + i) * a.out_tok + (kh * g + (r - i * g)) * a.out_head : (float *)nullptr;
                   }, a.D, ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)((a.out_tok | a.out_head) * 4)) & 15) == 0);
    uint64_t redo = __ballot(odd && live);
    redo = (redo | redo >> 32) & 0xFFFFFFFFull;
    for (; redo; redo &= redo - 1) {
        const int64_t rr = first + __builtin_ctzll(redo);
        const int ri = (int)over(rr, g);
        attend_prompt_row<T>(a, sq, ri, kh * g + (int)(rr - (int64_t)ri * g));
    }
}

// ---- A prefix that all sequences of a decode share -----------------------------------

// The first blocks take 128 rows (sequences x heads of a K/V head) against one
// part of the shared keys each, into slot `part`; the others
// (attention_rows.h) the rows of a sequence against a part of its own keys.
// The former are bounded by their products, the latter by memory: with one
// of the former to a CU and the latter beside them 32 x 32/8 x 128 behind 65536
// keys takes 123 us, in two launches of two blocks to a CU 131, and 20 behind
// 20480 44 against 54 (mixed evenly 151 and 57: some CUs then get three of the
// long blocks).
template <int DP>
__global__ __launch_bounds__(256, 2) void decode_tile_kernel(DecodeArgs a, DecodeParts c, unsigned tile_blocks)
{
    __shared__ uint4 k0[kTile * DP / 8], k1[kTile * DP / 8], v0[kTile * DP / 8], v1[kTile * DP / 8];
    __shared__ int ids[kPageIds];
    __shared__ int first_bad;
    const unsigned id = blockIdx.x;
    if (id >= tile_blocks) {
        static_assert(sizeof k0 >= 4 * Joined<DP, 4>::kWave && sizeof ids >= (8 + 1) * 4 * kRows, "its sums fit");
        Joined<DP, 4> sh;
        sh.o[0] = (CFP32_LDS float *)k0;
        sh.o[1] = (CFP32_LDS float *)k1;
        sh.o[2] = (CFP32_LDS float *)v0;
        sh.o[3] = (CFP32_LDS float *)v1;
        sh.m = (CFP32_LDS float *)ids;
        sh.l = sh.m + 4 * kRows;
        sh.unfinished = (CFP32_LDS int *)(sh.l + 4 * kRows);
        const int other = (int)(id - tile_blocks);
        decode_rows<_Float16, DP, true, 4, true>(a, c, other / a.Hkv, other % a.Hkv, sh);
        return;
    }
    const Partials &to = c.to;
    const int parts = c.tiles, g = a.Hq / a.Hkv, part = id % parts, kh = id / parts % a.Hkv;
    const int64_t n = (int64_t)a.B * g, r0 = (int64_t)(id / parts / a.Hkv) * 128;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = r0 + wave * kWaveRows, b = over(min(first + (lane & 31), n - 1), g);
    const int shared = a.shared_pages << a.page_log2;
    const int limit = min(decode_length(a, (int)b), shared);
    int t0, t1;
    part_tiles((shared + kTile - 1) / kTile, part, parts, t0, t1);
    WaveRows<DP> w;
    if (t0 < t1) {
        const int j0 = t0 * kTile, last = min(t1 * kTile, shared) - 1, p0 = j0 >> a.page_log2, p1 = last >> a.page_log2;
        if (threadIdx.x == 0) first_bad = 0x7FFFFFFF;
        __syncthreads();
        for (int i = threadIdx.x; i <= p1 - p0; i += 256) {
            int id = a.table[p0 + i];
            if (id < 0 || id >= a.P) {  // page 0 instead; rows that see it become NaN
                id = 0;
                atomicMin(&first_bad, (p0 + i) << a.page_log2);
            }
            ids[i] = id;
        }
        __syncthreads();
        const PagedSource src = {(const char *)((const _Float16 *)a.k.data + kh * a.k.head),
                                 (const char *)((const _Float16 *)a.v.data + kh * a.v.head), a.k.page * 2, a.v.page * 2,
                                 (uint32_t)(a.k.tok * 2), (uint32_t)(a.v.tok * 2), ids, j0, last, a.D / 8, a.page_log2};
        attend_tiles<DP, 1, 4, DP == 128 ? 5 : 7>([&](int row) {
            const int64_t r = min(first + row, n - 1), s = over(r, g);
            return a.q + s * a.q_seq + (kh * g + (r - s * g)) * a.q_head;
        }, rows_wide(a.q, a.q_seq | a.q_head, a.D), a.D, limit, a.scale,
                               t0, t1, src, k0, k1, v0, v1, w);
        if (limit > first_bad) w.l = NAN;
    } else {
        no_rows<DP>(w);
    }
    leave_rows<DP>(w, to, [&](int row) -> int64_t {
        const int64_t r = first + row, s = over(r, g);
        return r < n ? (s * a.Hq + kh * g + (r - s * g)) * to.slots + part : -1;
    }, stage_of(wave, k0, k1));
}

// The largest x >= 0 of each N (8 or 16) neighbouring lanes, to all of them:
// lanes exchanged by quad_perm 1 0 3 2 and 2 3 0 1, halves and rows mirrored.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float x)
{
    return fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true)));
}
template <int N>
__device__ __forceinline__ float max_of_lanes(float x)
{
    static_assert(N == 8 || N == 16, "half a row of lanes, or a row");
    x = max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(x)));
    return N == 16 ? max_dpp<0x140>(x) : x;
}

// FP32 K and V of one tile and head as two FP16 planes each.
template <int DP>
__global__ __launch_bounds__(256) void prompt_planes_kernel(PromptArgs a, Planes planes)
{
    constexpr int CH = DP / 8, PER = kTile * CH / 256;
    __shared__ float most[2][4], least[2][4];
    const int kh = blockIdx.y;
    int64_t start;
    const int sid = find_unit(a.cu_k, a.S, 1, kTile, blockIdx.x, start);
    const Sequence sq = sequence(a, sid);
    const int64_t j0 = (blockIdx.x - start) * kTile;
    if (blockIdx.x < start || j0 >= sq.nk) return;
    const int64_t slot = kh * planes.slots + blockIdx.x, key0 = kh * planes.count + sq.k0 + j0;
    const int64_t behind = min(max(a.cu_k[a.S], 0), a.Tk) - sq.k0 - j0;  // rows from here on are no sequence's
    const bool wide = a.D % 4 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.k.data) | reinterpret_cast<uintptr_t>(a.v.data) |
                        (uintptr_t)((a.k.tok | a.k.head | a.v.tok | a.v.head) * 4)) & 15) == 0;
    float x[2][PER][8], key_mx[2][PER];  // of the key's CH lanes
#pragma unroll
    for (int value = 0; value < 2; ++value)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x + 256 * i, row = at / CH, d = at % CH * 8;
            const HeadsView &t = value ? a.v : a.k;
            const float *p = (const float *)t.data + (sq.k0 + j0 + row) * t.tok + kh * t.head + d;
            const bool there = j0 + row < sq.nk;
            float mx = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                if (wide) {
                    floatx4_t y = {0, 0, 0, 0};
                    if (there && d + e < a.D) y = *reinterpret_cast<const floatx4_t *>(p + e);
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[value][i][e + u] = y[u];
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[value][i][e + u] = there && d + e + u < a.D ? p[e + u] : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float ax = fabsf(x[value][i][e + u]);
                    mx = fmaxf(mx, ax < INFINITY ? ax : 0.0f);
                }
            }
            key_mx[value][i] = max_of_lanes<CH>(mx);
        }
#pragma unroll
    for (int value = 0; value < 2; ++value) {
        float hi = 0.0f, lo = INFINITY;  // of the keys that are not zero
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            hi = fmaxf(hi, key_mx[value][i]);
            lo = fminf(lo, key_mx[value][i] > 0.0f ? key_mx[value][i] : INFINITY);
        }
#pragma unroll
        for (int o = 32; o >= CH; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor(hi, o));
            lo = fminf(lo, __shfl_xor(lo, o));
        }
        if ((threadIdx.x & 63) == 0) {
            most[value][threadIdx.x >> 6] = hi;
            least[value][threadIdx.x >> 6] = lo;
        }
    }
    __syncthreads();
    float top[2];
    bool each = false;
#pragma unroll
    for (int value = 0; value < 2; ++value) {
        top[value] = fmaxf(fmaxf(most[value][0], most[value][1]), fmaxf(most[value][2], most[value][3]));
        each |= fminf(fminf(least[value][0], least[value][1]), fminf(least[value][2], least[value][3])) < top[value] * kSpread;
    }
#pragma unroll
    for (int value = 0; value < 2; ++value) {
        const int all = top_shift(top[value]);
        if (threadIdx.x == 0)
            planes.shifts[2 * slot + value] = each ? (value ? 0 : kKeyShifts) : value && top[1] == 0.0f ? kNoValues : all;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = threadIdx.x + 256 * i, row = at / CH;
            if (j0 + row >= sq.nk && row < behind) continue;  // the next sequence's
            const int e2 = each ? top_shift(key_mx[value][i]) : all;
            if (at % CH == 0)
                planes.key_shifts[2 * (key0 + row) + value] = value && key_mx[1][i] == 0.0f ? kNoValues : e2;
            half8_t hi, lo;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                _Float16 h, w;
                split_scaled(x[value][i][e], e2, h, w);
                hi[e] = h, lo[e] = w;
            }
            char *to = planes.keys + (key0 + row) * plane_key_bytes(DP) + value * 2 * (DP * 2) + at % CH * 16;
            *reinterpret_cast<half8_t *>(to) = hi;
            *reinterpret_cast<half8_t *>(to + DP * 2) = lo;
        }
    }
}

}  // namespace

hipError_t launch_prompt_tile(const PromptArgs &a, const PromptPlan &p, hipStream_t stream)
{
    if (!a.kv_f16) {
        const dim3 grid((unsigned)p.planes.slots, (unsigned)a.Hkv);
        if (a.D <= 64) prompt_planes_kernel<64><<<grid, 256, 0, stream>>>(a, p.planes);
        else prompt_planes_kernel<128><<<grid, 256, 0, stream>>>(a, p.planes);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)p.blocks, (unsigned)p.to.slots);
#define CFP32_PROMPT(T, DP)                                                                            \
    do {                                                                                               \
        if (p.eight) prompt_tile_kernel<T, DP, 8><<<grid, 512, 0, stream>>>(a, p.planes, p.to);        \
        else prompt_tile_kernel<T, DP, 4><<<grid, 256, 0, stream>>>(a, p.planes, p.to);                \
    } while (0)
    if (a.kv_f16) {
        if (a.D <= 64) CFP32_PROMPT(_Float16, 64);
        else CFP32_PROMPT(_Float16, 128);
    } else {
        if (a.D <= 64) CFP32_PROMPT(float, 64);
        else CFP32_PROMPT(float, 128);
    }
#undef CFP32_PROMPT
    return hipGetLastError();
}

hipError_t launch_decode_tile(const DecodeArgs &a, const DecodePlan &p, hipStream_t stream)
{
    const unsigned blocks = (unsigned)p.blocks, tiles = (unsigned)p.tile_blocks;
    if (a.D <= 64) decode_tile_kernel<64><<<blocks, 256, 0, stream>>>(a, p.parts, tiles);
    else decode_tile_kernel<128><<<blocks, 256, 0, stream>>>(a, p.parts, tiles);
    return hipGetLastError();
}

}  // namespace cfp32
