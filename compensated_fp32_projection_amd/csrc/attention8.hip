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
// A byte of K or V costs some two vector instructions and a sixteenth of a
// matrix instruction for four, so what bounds it is the memory.
#include "attention8.h"
#include "attention_join.h"
#include "attention_rows.h"

namespace cfp32 {

namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef short short2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

// Bytes I of `a` and J of `b` as FP16: integers, or floats times 2^-8.  The
// bytes of integers have their signs turned (see turned).
template <bool E4M3, int I, int J>
__device__ __forceinline__ half2_t two_codes(uint32_t a, uint32_t b)
{
    if constexpr (E4M3) {
        const uint32_t x = __builtin_amdgcn_perm(b, a, 0x0C000C | (uint32_t)I << 8 | (uint32_t)(4 + J) << 24);
        const uint32_t y = __builtin_bit_cast(uint32_t, (short2_t)(__builtin_bit_cast(short2_t, x) >> 1)) & 0xBF80BF80u;
        return __builtin_bit_cast(half2_t, y);
    } else {
        const uint32_t x = __builtin_amdgcn_perm(b, a, 0x0C000C00 | (uint32_t)I | (uint32_t)(4 + J) << 16) | 0x64006400u;
        return __builtin_bit_cast(half2_t, x) - (half2_t)(_Float16)1152;
    }
}

template <bool E4M3>
__device__ __forceinline__ uint32_t turned(uint32_t w) { return E4M3 ? w : w ^ 0x80808080u; }

// Eight codes of a key, one after the other.
template <bool E4M3>
__device__ __forceinline__ half8_t eight_codes(uint2_t w)
{
    const uint32_t a = turned<E4M3>(w[0]), b = turned<E4M3>(w[1]);
    const half2_t p[4] = {two_codes<E4M3, 0, 1>(a, a), two_codes<E4M3, 2, 3>(a, a), two_codes<E4M3, 0, 1>(b, b),
                          two_codes<E4M3, 2, 3>(b, b)};
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

// Where a sequence's keys are.  A page id outside the pool is replaced by page 0
// (the pool has pages) and remembered: rows that see it become NaN.
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
    // The page of 16 keys from a multiple of 16 on, where pages hold as many.
    __device__ __forceinline__ int page_step(int j) { return lg >= 4 ? page_of(j) : 0; }
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

// One wave's share: keys [kb, hi), NW steps further each time, all of which
// this lane's row q sees.
template <bool E4M3, int DP, int A, int NW>
__device__ __forceinline__ void attend_share8(const float *q, bool q_wide, int D, float scale, int kb, int hi, Keys8 keys,
                                              const Joined<DP, NW> &to)
{
    constexpr int kStep = row_step<DP>(), NB = kStep / 16, KL = DP / 64, NV = DP / 16;
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
        uint32_t kr[NB][KL][4], vr[NB][4][NV / 4];
        float ks[NB][4], vs[NB][4];
        int page[NB], next[NB];
        const int last = hi - 1;
        auto pages = [&](int b0, int (&p)[NB]) {
#pragma unroll
            for (int b = 0; b < NB; ++b) p[b] = keys.page_step(min(b0 + 16 * b, last));
        };
        auto load_k = [&](int b0) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const char *p = keys.key(min(b0 + 16 * b + col, last), page[b]);
#pragma unroll
                for (int i = 0; i < KL; ++i) load_codes<16, A>(p, 64 * i + 16 * quad, D, kr[b][i]);
                const int j = b0 + 16 * b + 4 * quad;
                if (keys.blg >= 2) {
                    ks[b][0] = ks[b][1] = ks[b][2] = ks[b][3] = keys.k_scale(min(j, last), page[b]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) ks[b][r] = keys.k_scale(min(j + r, last), page[b]);
                }
            }
        };
        auto load_v = [&](int b0) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int j = b0 + 16 * b + 4 * quad;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    load_codes<NV, A>(keys.value(min(j + r, last), page[b]), col * NV, D, vr[b][r]);
                if (keys.blg >= 2) {
                    vs[b][0] = vs[b][1] = vs[b][2] = vs[b][3] = keys.v_scale(min(j, last), page[b]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) vs[b][r] = keys.v_scale(min(j + r, last), page[b]);
                }
            }
        };
        pages(kb, page);
        load_k(kb);
        load_v(kb);
        pages(kb + NW * kStep, next);

        half8_t qh[2 * KL], ql[2 * KL];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < KL; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float ax = fabsf(x[i][e]);
                mx = fmaxf(mx, ax < INFINITY ? ax : 0.0f);
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const int e2 = top_shift(mx);
#pragma unroll
        for (int i = 0; i < KL; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                _Float16 h, w;
                split_scaled(x[i][e], e2, h, w);
                qh[2 * i + e / 8][e % 8] = h, ql[2 * i + e / 8][e % 8] = w;
            }
        const float f = __builtin_amdgcn_ldexpf(scale * kLog2e * kCode, -e2);

        for (; kb < hi;) {
            floatx4_t s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                s[b] = floatx4_t{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 2 * KL; ++i) {
                    const half8_t a = eight_codes<E4M3>(uint2_t{kr[b][i / 2][2 * (i % 2)], kr[b][i / 2][2 * (i % 2) + 1]});
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ql[i], s[b], 0, 0, 0);
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[i], s[b], 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool seen = kb + 16 * b + 4 * quad + r < hi;
                    s[b][r] = seen ? s[b][r] * f * ks[b][r] : -INFINITY;
                }
            }
            const int nb = kb + NW * kStep;
            const bool more = nb < hi;
            if (more) {
                // The next step's pages are known; ask for those after it first.
#pragma unroll
                for (int b = 0; b < NB; ++b) page[b] = next[b];
                if (nb + NW * kStep < hi) pages(nb + NW * kStep, next);
                load_k(nb);
            }
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, s[b][r]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
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
                    // What lies beyond the last key is not multiplied: its scale may be anything.
                    w[b][r] = kb + 16 * b + 4 * quad + r < hi ? p * vs[b][r] : 0.0f;
                    most = fmaxf(most, fabsf(w[b][r]));
                }
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            const int e = top_shift(most);
            half8_t wh[NB / 2], wl[NB / 2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    _Float16 h, t;
                    split_scaled(w[b][r], e, h, t);
                    wh[b / 2][b % 2 * 4 + r] = h, wl[b / 2][b % 2 * 4 + r] = t;
                }
            floatx4_t add[NV];
#pragma unroll
            for (int c = 0; c < NV; ++c) add[c] = floatx4_t{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < NB / 2; ++u)
#pragma unroll
                for (int i = 0; i < NV / 4; ++i) {
                    uint32_t word[8];
#pragma unroll
                    for (int t = 0; t < 8; ++t) word[t] = turned<E4M3>(vr[2 * u + t / 4][t % 4][i]);
                    const half8_t a[4] = {column<E4M3, 0>(word), column<E4M3, 1>(word), column<E4M3, 2>(word), column<E4M3, 3>(word)};
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        add[4 * i + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[t], wl[u], add[4 * i + t], 0, 0, 0);
                        add[4 * i + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[t], wh[u], add[4 * i + t], 0, 0, 0);
                    }
                }
            if (__any(e > 120 || e < -120)) {  // the power of two is beyond FP32's, the products may not be
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[c][r] += __builtin_amdgcn_ldexpf(add[c][r] * kCode, -e);
            } else {
                const float g = __builtin_amdgcn_ldexpf(kCode, -e);
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[c][r] = fmaf(add[c][r], g, o[c][r]);
            }
            if (more) load_v(nb);
            kb = nb;
        }
        int bad = keys.bad;
        if (__any(bad != 0x7FFFFFFF)) {
#pragma unroll
            for (int t = 32; t; t >>= 1) bad = min(bad, __shfl_xor(bad, t));
            if (hi > bad) l = NAN;
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
    }
    // O^T: this lane's column, dims NV (4 quad + r) + c.
    CFP32_LDS float *sums = to.o[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) sums = wave == w ? to.o[w] : sums;
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

template <bool E4M3, int DP, int A, int NW>
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
    const int n = min(max(a.lens[b], 0), a.W << c.page_log2);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int lo, hi;
    part_range(0, n, part, p.parts, NW * row_step<DP>(), lo, hi);
    const int h = kh * g + h0 + min((int)(threadIdx.x & 15), live - 1);
    const Keys8 keys = {(const char *)c.k.data + kh * c.k.head, (const char *)c.v.data + kh * c.v.head,
                        c.ks.data + kh * c.ks.head, c.vs.data + kh * c.vs.head, c.k.page, c.v.page, c.k.tok, c.v.tok,
                        c.ks.page, c.vs.page, a.table + b * a.ld_table, c.page_log2, c.block_log2, c.P, 0x7FFFFFFF};
    attend_share8<E4M3, DP, A, NW>(a.q + b * a.q_seq + h * a.q_head, rows_wide(a.q, a.q_seq | a.q_head, c.D), c.D, a.scale,
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
#define CFP32_DECODE8_ALIGN(E4M3, DP)                                                          \
    do {                                                                                       \
        if (p.align == 16) decode8_kernel<E4M3, DP, 16, 4><<<grid, 256, 0, stream>>>(a, p);    \
        else if (p.align == 8) decode8_kernel<E4M3, DP, 8, 4><<<grid, 256, 0, stream>>>(a, p); \
        else decode8_kernel<E4M3, DP, 1, 4><<<grid, 256, 0, stream>>>(a, p);                   \
    } while (0)
    if (a.c.e4m3) {
        if (a.c.D <= 64) CFP32_DECODE8_ALIGN(true, 64);
        else CFP32_DECODE8_ALIGN(true, 128);
    } else {
        if (a.c.D <= 64) CFP32_DECODE8_ALIGN(false, 64);
        else CFP32_DECODE8_ALIGN(false, 128);
    }
#undef CFP32_DECODE8_ALIGN
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.to.o) return e;
    return launch_join(Decode8Rows{a.out, a.out_seq, a.out_head, a.Hq, a.c.D}, p.to, (int64_t)a.B * a.Hq, stream);
}

}  // namespace cfp32
