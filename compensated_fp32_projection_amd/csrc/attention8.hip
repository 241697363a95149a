// Attention of new tokens over an 8-bit cache (include/cfp32.h:
// cfp32_attention8_decode).
//
// The form of attention_rows.h: a block of four waves takes 16 query heads of
// one sequence and K/V head, its keys are dealt to the waves in steps of 32 or
// 64, scores are S^T = K Q^T, so that a lane holds scores of one row, and
// outputs O^T = V^T P^T.  Codes are exact in FP16, so both products run on
// v_mfma_f32_16x16x32_f16, with q and the weights cut into two FP16 parts.
//   * Codes become FP16 in registers: an integer's byte under the exponent of
//     1024 (a byte permutation), less 1152; a float's bits where FP16's are
//     (2^-8 of the value).  The permutation that picks V's bytes also puts two
//     keys' side by side, which is the transposition that V^T needs.
//   * A score is scaled by its key's scale.  A weight is multiplied by its
//     key's scale of V in FP32, and a step's products by a power of two of
//     their own for each row before they are cut, so that neither a large
//     scale beside them nor a small weight costs them bits.
// A step of 32 keys x 128 costs a wave some 650 vector and 32 matrix
// instructions for its 8 KiB, which with two waves to a SIMD is 7 TB/s over the
// chip; its codes are asked for a step ahead, 64 KiB to a compute unit.  Long
// contexts are bounded by the memory (64 x 4000 to 8000 keys x 32/8 x 128 INT8 162
// us, 4.9 TB/s), short ones by what they wait for one after the other: a length, a
// page, codes, the join (130 keys 7.6 us).
#include "attention8.h"
#include "attention_join.h"
#include "attention_rows.h"
#include "lanes.h"

namespace cfp32 {

namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef short short2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

// Bytes I of `a` and J of `b` as FP16: integers, or floats times 2^-8.  An
// integer c goes, as c + 128, into the last bits of 1024, which leaves 1152 + c.
template <bool E4M3, int I, int J>
__device__ __forceinline__ half2_t two_codes(uint32_t a, uint32_t b)
{
    if constexpr (E4M3) {
        const uint32_t x = __builtin_amdgcn_perm(b, a, 0x0C000C | (uint32_t)I << 8 | (uint32_t)(4 + J) << 24);
        const uint32_t y = __builtin_bit_cast(uint32_t, (short2_t)(__builtin_bit_cast(short2_t, x) >> 1)) & 0xBF80BF80u;
        return __builtin_bit_cast(half2_t, y);
    } else {
        const uint32_t x = __builtin_amdgcn_perm(b, a, 0x0C000C00 | (uint32_t)I | (uint32_t)(4 + J) << 16) ^ 0x64806480u;
        return __builtin_bit_cast(half2_t, x) - (half2_t)(_Float16)1152;
    }
}

// Four codes of a key, one after the other.
template <bool E4M3>
__device__ __forceinline__ void four_codes(uint32_t w, half2_t &x, half2_t &y)
{
    if constexpr (E4M3) {
        x = two_codes<true, 0, 1>(w, w);
        y = two_codes<true, 2, 3>(w, w);
    } else {  // the exponent's byte from the permutation, too
        const uint32_t u = w ^ 0x80808080u;
        x = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - (half2_t)(_Float16)1152;
        y = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - (half2_t)(_Float16)1152;
    }
}

// Eight codes of a key.
template <bool E4M3>
__device__ __forceinline__ half8_t eight_codes(uint32_t a, uint32_t b)
{
    half2_t p[4];
    four_codes<E4M3>(a, p[0], p[1]);
    four_codes<E4M3>(b, p[2], p[3]);
    half8_t h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = p[e / 2][e % 2];
    return h;
}

// Byte C of eight keys' words.
template <bool E4M3, int C>
__device__ __forceinline__ half8_t column(const uint32_t (&w)[8])
{
    half8_t h;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const half2_t p = two_codes<E4M3, C, C>(w[e], w[e + 1]);
        h[e] = p[0], h[e + 1] = p[1];
    }
    return h;
}

// Two values below 2^15 as FP16 parts: high, and what is left of each (exact in
// FP32, a mixed-precision difference), rounded to nearest even both.
__device__ __forceinline__ void two_parts(float x, float y, half2_t &hi, half2_t &lo)
{
    typedef float float2_t __attribute__((ext_vector_type(2)));
    hi = __builtin_convertvector(float2_t{x, y}, half2_t);
    float r, s;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(hi), "v"(x));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(s) : "v"(hi), "v"(y));
    lo = __builtin_convertvector(float2_t{r, s}, half2_t);
}

// Where a sequence's keys are.  A page id outside the pool is replaced by page 0
// (the pool has pages) and remembered: rows that see it become NaN.  What is
// the same for a block's lanes (the sequence, its pages) is in scalar registers.
struct Keys8 {
    const char *k, *v;       // the head in page 0
    const float *ks, *vs;
    int64_t k_page, v_page, k_tok, v_tok, ks_page, vs_page;
    const int32_t *row;
    int lg, blg, P, bad;
    __device__ __forceinline__ int page_of(int j)
    {
        const int p = row[j >> lg];
        if (p >= 0 && p < P) return p;
        bad = min(bad, j >> lg << lg);
        return 0;
    }
    __device__ __forceinline__ int page(int j, int p) { return lg >= 4 ? p : page_of(j); }
    __device__ __forceinline__ int inside(int j) const { return j & ((1 << lg) - 1); }
    __device__ __forceinline__ const char *key(int j, int p) { return k + page(j, p) * k_page + inside(j) * k_tok; }
    __device__ __forceinline__ const char *value(int j, int p) { return v + page(j, p) * v_page + inside(j) * v_tok; }
    __device__ __forceinline__ float k_scale(int j, int p) { return ks[page(j, p) * ks_page + (inside(j) >> blg)]; }
    __device__ __forceinline__ float v_scale(int j, int p) { return vs[page(j, p) * vs_page + (inside(j) >> blg)]; }
};

// N bytes at p + at of a row of n, as words; zeros, or the row's first bytes
// (which meet zeros of q, or dims that are not written), from byte n on.
// A: what divides addresses and n.
template <int N, int A>
__device__ __forceinline__ void load_codes(const char *p, int at, int n, uint32_t (&w)[N / 4])
{
    if constexpr (A >= N) {
        typedef uint32_t vec __attribute__((ext_vector_type(N / 4)));
        const vec t = *reinterpret_cast<const vec *>(p + (at < n ? at : 0));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = t[i];
    } else if constexpr (A == 8) {
        static_assert(N == 16, "");
        const uint2_t t = *reinterpret_cast<const uint2_t *>(p + (at < n ? at : 0));
        const uint2_t u = *reinterpret_cast<const uint2_t *>(p + (at + 8 < n ? at + 8 : 0));
        w[0] = t[0], w[1] = t[1], w[2] = u[0], w[3] = u[1];
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            w[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + 4 * i + e < n) w[i] |= (uint32_t)(uint8_t)p[at + 4 * i + e] << (8 * e);
        }
    }
}

// The codes and scales of a step's keys that a lane takes.  FAST: pages of 16
// tokens or more and blocks of 4 or more, so that 16 keys have one page and the
// four keys of a lane's scores one scale; and offsets within 16 tokens fit 31
// bits, so that addresses are a scalar and a lane's offset that never changes.
template <int DP, bool FAST>
struct Tile8 {
    static constexpr int NB = row_step<DP>() / 16, KL = DP / 64, NV = DP / 16;
    uint32_t k[NB][KL][4], v[NB][4][NV / 4];
    float ks[NB][FAST ? 1 : 4], vs[NB][FAST ? 1 : 4];
};

// One wave's share: keys [kb, hi), NW steps further each time, all of which
// this lane's row q sees.
template <bool E4M3, int DP, int A, bool FAST, int NW>
__device__ __forceinline__ void attend_share8(const float *q, bool q_wide, int D, float scale, int kb, int hi, Keys8 keys,
                                              const Joined<DP, NW> &to)
{
    using Tile = Tile8<DP, FAST>;
    constexpr int kStep = row_step<DP>(), NB = Tile::NB, KL = Tile::KL, NV = Tile::NV;
    constexpr float kCode = E4M3 ? 256.0f : 1.0f;  // of a value's FP16 form
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    float m = -INFINITY, l = 0.0f;
    floatx4_t o[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) o[c] = floatx4_t{0, 0, 0, 0};

    if (kb < hi) {
        // The row: dims 64 i + 16 quad + e, as K's are loaded.
        float x[KL][16];
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            if (q_wide) load_floats<16, true>(q, 64 * i + 16 * quad, D, x[i]);
            else load_floats<16, false>(q, 64 * i + 16 * quad, D, x[i]);
        }
        const int last = hi - 1;
        int page[NB], next[NB];
        auto ask = [&](int b0) {  // for the pages of a step
#pragma unroll
            for (int b = 0; b < NB; ++b) next[b] = FAST || keys.lg >= 4 ? keys.row[min(b0 + 16 * b, last) >> keys.lg] : 0;
        };
        auto take = [&](int b0) {  // ... which have come
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                page[b] = __builtin_amdgcn_readfirstlane(next[b]);
                if (page[b] < 0 || page[b] >= keys.P) {
                    const int j = min(b0 + 16 * b, last);
                    keys.bad = min(keys.bad, j >> keys.lg << keys.lg);
                    page[b] = 0;
                }
            }
        };
        // A lane's bytes of 16 keys: its key's of K, and of each of its four keys of V.  Dims beyond D: the row's first
        // (where q is 0, or nothing is written).
        uint32_t k_dim[KL], v_dim = col * NV < D ? col * NV : 0, k_off, v_off[4];
#pragma unroll
        for (int i = 0; i < KL; ++i) k_dim[i] = 64 * i + 16 * quad < D ? 64 * i + 16 * quad : 0;
        k_off = (uint32_t)col * (uint32_t)keys.k_tok + k_dim[0];
#pragma unroll
        for (int r = 0; r < 4; ++r) v_off[r] = (uint32_t)(4 * quad + r) * (uint32_t)keys.v_tok + v_dim;
        // ALL: every key of the step is there.  Of others, keys beyond the last are the last's place, or the first sixteen's.
        auto load_fast = [&](int b0, Tile &t, auto all) {
            constexpr bool ALL = decltype(all)::value;
            int64_t pg[NB];
            int in[NB], room[NB];
            const char *kp[NB], *vp[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const bool some = ALL || b0 + 16 * b <= last;
                const int j = some ? b0 + 16 * b : b0;
                pg[b] = some ? page[b] : page[0];
                in[b] = keys.inside(j);
                room[b] = last - j;
                kp[b] = keys.k + pg[b] * keys.k_page + in[b] * keys.k_tok;
                vp[b] = keys.v + pg[b] * keys.v_page + in[b] * keys.v_tok;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t off = ALL ? k_off : (uint32_t)min(col, room[b]) * (uint32_t)keys.k_tok + k_dim[0];
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const uint32_t at = off + (k_dim[i] - k_dim[0]);
                    if constexpr (A == 16) {
                        const uint4_t w = __builtin_nontemporal_load(reinterpret_cast<const uint4_t *>(kp[b] + at));
                        t.k[b][i][0] = w[0], t.k[b][i][1] = w[1], t.k[b][i][2] = w[2], t.k[b][i][3] = w[3];
                    } else {
                        const uint32_t more = 64 * i + 16 * quad + 8 < D ? 8u : 0u;
                        const uint2_t w = *reinterpret_cast<const uint2_t *>(kp[b] + at);
                        const uint2_t u = *reinterpret_cast<const uint2_t *>(kp[b] + (at + more));
                        t.k[b][i][0] = w[0], t.k[b][i][1] = w[1], t.k[b][i][2] = u[0], t.k[b][i][3] = u[1];
                    }
                }
                t.ks[b][0] = (keys.ks + pg[b] * keys.ks_page)[(uint32_t)(in[b] + 4 * quad) >> keys.blg];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t off = ALL ? v_off[r] : (uint32_t)min(4 * quad + r, room[b]) * (uint32_t)keys.v_tok + v_dim;
                    typedef uint32_t vec __attribute__((ext_vector_type(NV / 4)));
                    const vec w = __builtin_nontemporal_load(reinterpret_cast<const vec *>(vp[b] + off));
#pragma unroll
                    for (int i = 0; i < NV / 4; ++i) t.v[b][r][i] = w[i];
                }
                t.vs[b][0] = (keys.vs + pg[b] * keys.vs_page)[(uint32_t)(in[b] + 4 * quad) >> keys.blg];
            }
        };
        auto load = [&](int b0, Tile &t) {
            if constexpr (FAST) {
                if (b0 + kStep <= hi) load_fast(b0, t, std::integral_constant<bool, true>{});
                else load_fast(b0, t, std::integral_constant<bool, false>{});
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const char *p = keys.key(min(b0 + 16 * b + col, last), page[b]);
#pragma unroll
                    for (int i = 0; i < KL; ++i) load_codes<16, A>(p, 64 * i + 16 * quad, D, t.k[b][i]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) t.ks[b][r] = keys.k_scale(min(b0 + 16 * b + 4 * quad + r, last), page[b]);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = min(b0 + 16 * b + 4 * quad + r, last);
                        load_codes<NV, A>(keys.value(j, page[b]), col * NV, D, t.v[b][r]);
                        t.vs[b][r] = keys.v_scale(j, page[b]);
                    }
            }
        };

        Tile tiles[2];
        ask(kb);
        take(kb);
        if (kb + NW * kStep < hi) ask(kb + NW * kStep);
        load(kb, tiles[0]);

        half8_t qh[2 * KL], ql[2 * KL];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < KL; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(x[i][e]));  // of a row with an infinity none is needed
        mx = max_of_quads(mx);
        const int e2 = top_shift(mx);
#pragma unroll
        for (int i = 0; i < KL; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                half2_t h, w;
                two_parts(__builtin_amdgcn_ldexpf(x[i][e], e2), __builtin_amdgcn_ldexpf(x[i][e + 1], e2), h, w);
                qh[2 * i + e / 8][e % 8] = h[0], qh[2 * i + e / 8][e % 8 + 1] = h[1];
                ql[2 * i + e / 8][e % 8] = w[0], ql[2 * i + e / 8][e % 8 + 1] = w[1];
            }
        // What scores are multiplied by, but for their keys' scales: scale log2 e 2^-e2, as two factors of which neither is
        // beyond FP32's range, where very small rows, large scales of theirs or of the scores bring each other back.
        const int up = __builtin_amdgcn_frexp_expf(scale) - e2 + (E4M3 ? 8 : 0), half = up / 2;
        const float f = __builtin_amdgcn_ldexpf(__builtin_amdgcn_frexp_mantf(scale) * kLog2e, half), f2 = __builtin_amdgcn_ldexpf(1.0f, up - half);

        // A step's work on one tile, while the next one's is on its way into the other.
        auto step = [&](Tile &t, Tile &ahead) {
            const int nb = kb + NW * kStep;
            if (nb < hi) {
                take(nb);
                if (nb + NW * kStep < hi) ask(nb + NW * kStep);
                load(nb, ahead);
            }
            const bool ends = kb + kStep > hi;
            const int room = hi - kb - 4 * quad;  // of this lane's keys 16 b + r
            floatx4_t s[NB];
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < NB; ++b) s[b] = floatx4_t{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2 * KL; ++i) {
                half8_t a[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) a[b] = eight_codes<E4M3>(t.k[b][i / 2][2 * (i % 2)], t.k[b][i / 2][2 * (i % 2) + 1]);
#pragma unroll
                for (int b = 0; b < NB; ++b) s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b], ql[i], s[b], 0, 0, 0);
#pragma unroll
                for (int b = 0; b < NB; ++b) s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b], qh[i], s[b], 0, 0, 0);
            }
            // One factor for a scale's four scores, unless it is beyond FP32's range (a product of 0 may be among them).
            constexpr int R = FAST ? 1 : 4;
            float fk[NB][R], peak = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    fk[b][r] = f * t.ks[b][r] * f2;
                    // A scale that no key of the row has may be anything, and must not choose the form either.
                    if (ends) fk[b][r] = 16 * b + r < room ? fk[b][r] : 0.0f;
                    peak = fmaxf(peak, fabsf(fk[b][r]));
                }
            if (__any(peak == INFINITY)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[b][r] = s[b][r] * f * t.ks[b][r % R] * f2;
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[b][r] *= fk[b][r % R];
            }
            if (ends) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[b][r] = 16 * b + r < room ? s[b][r] : -INFINITY;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, s[b][r]);
            top = max_of_quads(top);
            if (__any(top > m + kLazy)) {
                const float mn = fmaxf(m, top);
                const float c = mn == -INFINITY ? 1.0f : exp2_raw(m - mn);
                m = mn;
                l *= c;
#pragma unroll
                for (int i = 0; i < NV; ++i) o[i] *= c;
            }
            const float base = m == -INFINITY ? 0.0f : m;
            float w[NB][4], most = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = exp2_raw(s[b][r] - base);
                    l += p;
                    w[b][r] = p * t.vs[b][FAST ? 0 : r];
                }
            if (ends) {  // what lies beyond the last key has a scale that may be anything
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[b][r] = 16 * b + r < room ? w[b][r] : 0.0f;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) most = fmaxf(most, fabsf(w[b][r]));
            // Up to 2^-149 and back, both in FP32's range: no weight is too small to keep its bits.
            const int e = min(top_shift(max_of_quads(most)), 149);
            half8_t wh[NB / 2], wl[NB / 2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    half2_t h, u;
                    two_parts(__builtin_amdgcn_ldexpf(w[b][r], e), __builtin_amdgcn_ldexpf(w[b][r + 1], e), h, u);
                    wh[b / 2][b % 2 * 4 + r] = h[0], wh[b / 2][b % 2 * 4 + r + 1] = h[1];
                    wl[b / 2][b % 2 * 4 + r] = u[0], wl[b / 2][b % 2 * 4 + r + 1] = u[1];
                }
            const float g = __builtin_amdgcn_ldexpf(kCode, -e);
#pragma unroll
            for (int i = 0; i < NV / 4; ++i) {
                floatx4_t add[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) add[c] = floatx4_t{0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < NB / 2; ++u) {
                    uint32_t word[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n) word[n] = t.v[2 * u + n / 4][n % 4][i];
                    const half8_t a[4] = {column<E4M3, 0>(word), column<E4M3, 1>(word), column<E4M3, 2>(word), column<E4M3, 3>(word)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) add[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[c], wl[u], add[c], 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) add[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[c], wh[u], add[c], 0, 0, 0);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[4 * i + c][r] = fmaf(add[c][r], g, o[4 * i + c][r]);
            }
            kb = nb;
        };
        for (;;) {
            step(tiles[0], tiles[1]);
            if (kb >= hi) break;
            step(tiles[1], tiles[0]);
            if (kb >= hi) break;
        }
        int bad = keys.bad;
        if (__any(bad != 0x7FFFFFFF)) {
#pragma unroll
            for (int t = 32; t; t >>= 1) bad = min(bad, __shfl_xor(bad, t));
            if (hi > bad) l = NAN;
        }
        l += from_lane<16>(l);
        l += from_lane<32>(l);
    }
    // O^T: this lane's column, dims NV (4 quad + r) + c.
    // Not to.o[wave]: an index would put the pointers into private memory (16 x 4000 keys x 32/8 x 128 31 -> 34 us).
    CFP32_LDS float *sums = to.o[0] + wave * Joined<DP, NW>::kWave;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < NV; c += 4) {
            floatx4_t t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = o[c + e][r];
            *reinterpret_cast<CFP32_LDS floatx4_t *>(sums + col * (DP + 4) + NV * (4 * quad + r) + c) = t;
        }
    if (quad == 0) {
        to.m[wave * kRows + col] = m;
        to.l[wave * kRows + col] = l;
    }
}

template <bool E4M3, int DP, int A, bool FAST, int NW>
__global__ __launch_bounds__(64 * NW, 2) void decode8_kernel(Decode8Args a, Decode8Plan p)
{
    __shared__ float sums[NW][kRows * (DP + 4)], maxima[NW * kRows], weights[NW * kRows];
    __shared__ int unfinished[kRows];
    Joined<DP, NW> sh;
#pragma unroll
    for (int w = 0; w < NW; ++w) sh.o[w] = (CFP32_LDS float *)sums[w];
    sh.m = (CFP32_LDS float *)maxima;
    sh.l = (CFP32_LDS float *)weights;
    sh.unfinished = (CFP32_LDS int *)unfinished;
    const Cache8 &c = a.c;
    const int kh = blockIdx.y, g = a.Hq / c.Hkv;
    const int part = blockIdx.x % p.parts, group = blockIdx.x / p.parts;
    const int b = group / p.groups, h0 = group % p.groups * kRows, live = min(kRows, g - h0);
    const int n = __builtin_amdgcn_readfirstlane(min(max(a.lens[b], 0), a.W << c.page_log2));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int lo, hi;
    part_range(0, n, part, p.parts, NW * row_step<DP>(), lo, hi);
    const int h = kh * g + h0 + min((int)(threadIdx.x & 15), live - 1);
    const Keys8 keys = {(const char *)c.k.data + kh * c.k.head, (const char *)c.v.data + kh * c.v.head,
                        c.ks.data + kh * c.ks.head, c.vs.data + kh * c.vs.head, c.k.page, c.v.page, c.k.tok, c.v.tok,
                        c.ks.page, c.vs.page, a.table + b * a.ld_table, c.page_log2, c.block_log2, c.P, 0x7FFFFFFF};
    attend_share8<E4M3, DP, A, FAST, NW>(a.q + b * a.q_seq + h * a.q_head, rows_wide(a.q, a.q_seq | a.q_head, c.D), c.D, a.scale,
                                   lo + wave * row_step<DP>(), hi, keys, sh);
    __syncthreads();
    const int row = threadIdx.x >> 4, rh = kh * g + h0 + row;
    leave_row<false>(sh, p.to, ((int64_t)b * a.Hq + rh) * p.parts + part, a.out + b * a.out_seq + rh * a.out_head, c.D, row < live);
}

// Rows for the join.  Codes are finite, so a result that is not is as it should be.
struct Decode8Rows {
    float *data;
    int64_t seq, head;
    int heads, dim;
    __device__ __forceinline__ int Hq() const { return heads; }
    __device__ __forceinline__ int D() const { return dim; }
    __device__ __forceinline__ float *out(int64_t i, int h) const { return data + i * seq + h * head; }
    __device__ __forceinline__ void finish(int64_t, int) const {}
};

// Rows against a pool without pages: 0, or NaN where a sequence has tokens.
__global__ __launch_bounds__(256) void decode8_no_pages_kernel(Decode8Args a)
{
    const int64_t n = (int64_t)a.B * a.Hq * a.c.D;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / a.c.D, b = row / a.Hq;
        a.out[b * a.out_seq + (row - b * a.Hq) * a.out_head + (i - row * a.c.D)] = a.lens[b] > 0 && a.W > 0 ? NAN : 0.0f;
    }
}

}  // namespace

hipError_t launch_attention8_decode(const Decode8Args &a, void *workspace, hipStream_t stream)
{
    const Decode8Plan p = plan_decode8(a, workspace);
    if (p.error != hipSuccess) return p.error;
    if (a.c.P == 0) {
        const int64_t n = (int64_t)a.B * a.Hq * a.c.D, blocks = (n + 255) / 256;
        decode8_no_pages_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)p.blocks, (unsigned)a.c.Hkv);
#define CFP32_DECODE8(E4M3, DP, A, FAST) decode8_kernel<E4M3, DP, A, FAST, 4><<<grid, 256, 0, stream>>>(a, p)
#define CFP32_DECODE8_ALIGN(E4M3, DP)                                     \
    do {                                                                  \
        if (p.fast && p.align == 16) CFP32_DECODE8(E4M3, DP, 16, true);   \
        else if (p.fast) CFP32_DECODE8(E4M3, DP, 8, true);                \
        else if (p.align >= 8) CFP32_DECODE8(E4M3, DP, 8, false);         \
        else CFP32_DECODE8(E4M3, DP, 1, false);                           \
    } while (0)
    if (a.c.e4m3) {
        if (a.c.D <= 64) CFP32_DECODE8_ALIGN(true, 64);
        else CFP32_DECODE8_ALIGN(true, 128);
    } else {
        if (a.c.D <= 64) CFP32_DECODE8_ALIGN(false, 64);
        else CFP32_DECODE8_ALIGN(false, 128);
    }
#undef CFP32_DECODE8_ALIGN
#undef CFP32_DECODE8
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.to.o) return e;
    return launch_join(Decode8Rows{a.out, a.out_seq, a.out_head, a.Hq, a.c.D}, p.to, (int64_t)a.B * a.Hq, stream);
}

}  // namespace cfp32
