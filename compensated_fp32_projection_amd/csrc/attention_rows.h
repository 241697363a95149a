// Attention of few rows: new tokens against the paged cache, and short
// packed prompts (the kernels' bodies).
//
// A block of four waves works on 16 rows (tokens x heads of one K/V head, so
// grouped heads share what is read); its keys are dealt to the waves in steps
// of 32 or 64, and the waves' sums are joined in LDS.  Everything a wave
// multiplies goes from memory straight into the registers the matrix
// instructions read:
//   * scores as S^T = K Q^T, so that a lane holds scores of one row (column
//     lane % 16) and keeps that row's maximum and sum: FP16 keys by
//     v_mfma_f32_16x16x32_f16 with the row split into two FP16 parts, FP32
//     keys by v_mfma_f32_16x16x4_f32;
//   * O^T = V^T P^T by v_mfma_f32_16x16x4_f32, in FP32: with keys 4 (lane /
//     16) + r in its r-th step it takes the weights from where the scores
//     were left, and V as rows, as it lies in memory (no transposition, no
//     split).
// K of the next step is requested when its registers have been multiplied,
// V when its have, so a step's loads are in flight during the step before.
// 16 rows against FP32 keys need 1024 cycles of a SIMD for 8 KiB at D = 64,
// which is 19 TB/s over the chip: a decode, whose keys come from memory, is
// bounded by that and by its latency.  A prompt's keys come from the caches,
// again for each 16 rows, and its FP32 products are much of its time: 512 x
// 12 x 64 FP32 takes 15 us, of which 4 to 8 are a SIMD's matrix instructions
// (64 keys of a wave: 128 of 32 cycles).
#pragma once

#include "attention_device.h"

namespace cfp32 {

namespace {

// Where a block's keys are: packed rows, ...
struct PackedKeys {
    const char *k, *v;       // key 0 of the head
    int64_t k_tok, v_tok;    // bytes
    __device__ __forceinline__ int page_step(int) { return 0; }
    __device__ __forceinline__ const char *key(int j, int) const { return k + j * k_tok; }
    __device__ __forceinline__ const char *value(int j, int) const { return v + j * v_tok; }
    __device__ __forceinline__ int first_bad() const { return 0x7FFFFFFF; }
};

// ... or pages of a table row.  A page id outside the pool is replaced by
// page 0 (the pool has pages) and remembered: rows that see it become NaN.
struct PagedKeys {
    const char *k, *v;  // the head in page 0
    int64_t k_page, v_page, k_tok, v_tok;
    const int32_t *row;
    int lg, P, bad;
    __device__ __forceinline__ int page_of(int j)
    {
        const int p = row[j >> lg];
        if (p >= 0 && p < P) return p;
        bad = min(bad, j >> lg << lg);
        return 0;
    }
    // The page of 16 keys from a multiple of 16 on, where pages hold as many.
    __device__ __forceinline__ int page_step(int j) { return lg >= 4 ? page_of(j) : 0; }
    __device__ __forceinline__ const char *key(int j, int p)
    {
        if (lg < 4) p = page_of(j);
        return k + p * k_page + (j & ((1 << lg) - 1)) * k_tok;
    }
    __device__ __forceinline__ const char *value(int j, int p)
    {
        if (lg < 4) p = page_of(j);
        return v + p * v_page + (j & ((1 << lg) - 1)) * v_tok;
    }
    __device__ __forceinline__ int first_bad() const { return bad; }
};

// N elements from p + at, zeros from element n on.  WIDE: aligned, and n a
// multiple of a load; a load that lies beyond n repeats the first (what it
// meets is zero or not used).
template <class T, int N, bool WIDE>
__device__ __forceinline__ void load_row(const char *p, int at, int n, T (&x)[N])
{
    constexpr int E = 16 / sizeof(T) < N ? 16 / sizeof(T) : N;
    if (WIDE) {
        typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
        for (int i = 0; i < N; i += E) {
            const vec t = *reinterpret_cast<const vec *>(p + (at + i < n ? at + i : 0) * (int)sizeof(T));
#pragma unroll
            for (int e = 0; e < E; ++e) x[i + e] = t[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = at + i < n ? reinterpret_cast<const T *>(p)[at + i] : (T)0;
    }
}

// What the waves of a block leave in LDS: a wave's sums [kRows][DP + 4], and
// maxima, weights and rows to do again.
template <int DP, int NW>
struct Joined {
    static constexpr int kWave = kRows * (DP + 4);  // floats of a wave
    CFP32_LDS float *o[NW], *m, *l;   // m, l: [NW][kRows]
    CFP32_LDS int *unfinished;        // [kRows]
};

template <int DP>
constexpr int row_step() { return DP == 128 ? 32 : 64; }  // keys a wave takes at a time

// One wave's share of 16 rows: this lane's row q sees the first `limit` keys;
// the wave takes keys [kb, hi), row_step at a time, NW steps further each
// time.  FEW: there is one step, of which blocks of 16 keys may be missing.
template <class T, int DP, bool WIDE, int NW, bool FEW, class Keys>
__device__ __forceinline__ void attend_share(const float *q, bool q_wide, int D, int limit, float scale, int kb, int hi, Keys keys,
                                             const Joined<DP, NW> &to)
{
    constexpr bool F16 = sizeof(T) == 2;
    constexpr int kStep = row_step<DP>(), NB = kStep / 16;
    constexpr int KK = F16 ? DP / 32 : DP / 16;  // key loads (16 bytes) of a lane and block
    constexpr int KE = F16 ? 8 : 4;
    constexpr int NV = DP / 16;                // value elements of a lane and key
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    float m = -INFINITY, l = 0.0f;
    floatx4_t o[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) o[c] = floatx4_t{0, 0, 0, 0};

    if (kb < hi) {
        float x[KK][KE];
        if (q_wide) {
#pragma unroll
            for (int i = 0; i < KK; ++i) load_floats<KE, true>(q, (i * 4 + quad) * KE, D, x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < KK; ++i) load_floats<KE, false>(q, (i * 4 + quad) * KE, D, x[i]);
        }
        T kr[NB][KK][KE], vr[NB][4][NV];
        int page[NB], next[NB];
        const int last = hi - 1;
        auto pages = [&](int b0, int (&p)[NB]) {
#pragma unroll
            for (int b = 0; b < NB; ++b) p[b] = keys.page_step(min(b0 + 16 * b, last));
        };
        auto load_k = [&](int b0) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (FEW && b && b0 + 16 * b > last) continue;  // no such keys
                const char *p = keys.key(min(b0 + 16 * b + col, last), page[b]);
#pragma unroll
                for (int i = 0; i < KK; ++i) load_row<T, KE, WIDE>(p, (i * 4 + quad) * KE, D, kr[b][i]);
            }
        };
        auto load_v = [&](int b0) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (FEW && b && b0 + 16 * b > last) continue;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    load_row<T, NV, WIDE>(keys.value(min(b0 + 16 * b + 4 * quad + r, last), page[b]), col * NV, D, vr[b][r]);
            }
        };
        pages(kb, page);
        load_k(kb);
        load_v(kb);
        if (!FEW) pages(kb + NW * kStep, next);

        // The row, as the right operand of the score products.
        float f = scale * kLog2e;
        half8_t qh[F16 ? KK : 1], ql[F16 ? KK : 1];
        if constexpr (F16) {
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < KK; ++i)
#pragma unroll
                for (int e = 0; e < KE; ++e) {
                    const float ax = fabsf(x[i][e]);
                    mx = fmaxf(mx, ax < INFINITY ? ax : 0.0f);
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const int e2 = top_shift(mx);
#pragma unroll
            for (int i = 0; i < KK; ++i)
#pragma unroll
                for (int e = 0; e < KE; ++e) {
                    _Float16 h, w;
                    split_scaled(x[i][e], e2, h, w);
                    qh[i][e] = h, ql[i][e] = w;
                }
            f = __builtin_amdgcn_ldexpf(f, -e2);
        }

        for (bool again = true; again; again = !FEW && kb < hi) {
            floatx4_t s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                s[b] = floatx4_t{0, 0, 0, 0};
                if (FEW && b && kb + 16 * b > last) continue;
#pragma unroll
                for (int i = 0; i < KK; ++i) {
                    if constexpr (F16) {
                        half8_t a;
#pragma unroll
                        for (int e = 0; e < 8; ++e) a[e] = kr[b][i][e];
                        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ql[i], s[b], 0, 0, 0);
                        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[i], s[b], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(kr[b][i][e], x[i][e], s[b], 0, 0, 0);
                    }
                }
            }
            const int nb = kb + NW * kStep;
            const bool more = !FEW && nb < hi;
            if (more) {
                // The next step's pages are known; ask for those after it first.
#pragma unroll
                for (int b = 0; b < NB; ++b) page[b] = next[b];
                if (nb + NW * kStep < hi) pages(nb + NW * kStep, next);
                load_k(nb);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[b][r] = kb + 16 * b + 4 * quad + r < limit ? s[b][r] * f : -INFINITY;
                    mx = fmaxf(mx, s[b][r]);
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            if (__any(mx > m + kLazy)) {
                const float mn = fmaxf(m, mx);
                const float c = mn == -INFINITY ? 1.0f : exp2_raw(m - mn);
                m = mn;
                l *= c;
#pragma unroll
                for (int i = 0; i < NV; ++i) o[i] *= c;
            }
            const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (FEW && b && kb + 16 * b > last) continue;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = exp2_raw(s[b][r] - base);
                    l += p;
#pragma unroll
                    for (int c = 0; c < NV; ++c)
                        o[c] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)vr[b][r][c], p, o[c], 0, 0, 0);
                }
            }
            if (more) load_v(nb);
            kb = nb;
        }
        int bad = keys.first_bad();
        if (__any(bad != 0x7FFFFFFF)) {
#pragma unroll
            for (int x = 32; x; x >>= 1) bad = min(bad, __shfl_xor(bad, x));
            if (limit > bad) l = NAN;
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

// A block's keys [lo, hi) (lo a multiple of 16 if pages are to be read 16 keys
// at a time), dealt to its waves in steps, or, if they make no more than a
// step of each, in equal shares of whole blocks of 16 (37 keys x 64: 7.0 ->
// 5.7 us, all four waves at work).
template <class T, int DP, bool WIDE, int NW, class Keys>
__device__ __forceinline__ void attend_rows(const float *q, bool q_wide, int D, int limit, float scale, int lo, int hi, Keys keys,
                                            const Joined<DP, NW> &to)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (hi - lo <= NW * row_step<DP>()) {
        const int share = (hi - lo + 16 * NW - 1) / (16 * NW) * 16, kb = lo + wave * share, end = min(hi, kb + share);
        attend_share<T, DP, WIDE, NW, true>(q, q_wide, D, min(limit, end), scale, kb, end, keys, to);
    } else {
        attend_share<T, DP, WIDE, NW, false>(q, q_wide, D, min(limit, hi), scale, lo + wave * row_step<DP>(), hi, keys, to);
    }
}

// The waves' sums of a row joined: m, l and DP / 16 values from d0 on
// (unnormalised).
template <int DP, int NW>
__device__ __forceinline__ void join_rows(const Joined<DP, NW> &from, int row, int d0, float &m, float &l, float (&x)[DP / 16])
{
    constexpr int NV = DP / 16;
    m = from.m[row];
#pragma unroll
    for (int w = 1; w < NW; ++w) m = fmaxf(m, from.m[w * kRows + row]);
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) x[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float mw = from.m[w * kRows + row], f = mw == -INFINITY ? 0.0f : exp2_raw(mw - m);
        l = fmaf(f, from.l[w * kRows + row], l);
#pragma unroll
        for (int c = 0; c < NV; ++c) x[c] = fmaf(f, from.o[w][row * (DP + 4) + d0 + c], x[c]);
    }
}

// A row's sums, of what this block has seen: into its slot, or (all there is)
// as its result.  Results that are not finite are marked, and rows of no
// weight: they see nothing, or scores that are too low in powers of two only.
template <bool SLOTS, int DP, int NW>
__device__ __forceinline__ void leave_row(const Joined<DP, NW> &sh, const Partials &to, int64_t slot, float *out, int D, bool live)
{
    if (!live) return;
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (DP / 16);
    float m, l, x[DP / 16];
    join_rows(sh, row, d0, m, l, x);
    if (SLOTS || to.o) {
        if ((threadIdx.x & 15) == 0) {
            to.m[slot] = m;
            to.l[slot] = l;
        }
        if (l != 0.0f)
#pragma unroll
            for (int e = 0; e < DP / 16; e += 4)
                *reinterpret_cast<floatx4_t *>(to.o + slot * DP + d0 + e) = floatx4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < DP / 16; ++e) {
        const float y = x[e] * inv;
        if (d0 + e < D) {
            out[d0 + e] = y;
            if (!(fabsf(y) < INFINITY) || l == 0.0f) sh.unfinished[row] = 1;
        }
    }
}

// Keys [lo, hi) in `parts` of equal lengths (in whole units).
__device__ __forceinline__ void part_range(int lo, int hi, int part, int parts, int unit, int &a, int &b)
{
    const int n = max(hi - lo, 0), u = (n + unit - 1) / unit, per = (u + parts - 1) / parts;
    a = lo + (int)min((int64_t)n, (int64_t)part * per * unit);
    b = lo + (int)min((int64_t)n, (int64_t)(part + 1) * per * unit);
}

// Block `id` of a decode's rows, of K/V head kh.  SLOTS: its rows are known to
// go into slots.
template <class T, int DP, bool WIDE, int NW, bool SLOTS>
__device__ __forceinline__ void decode_rows(const DecodeArgs &a, const DecodeParts &c, int id, int kh, const Joined<DP, NW> &sh)
{
    constexpr int kUnit = NW * row_step<DP>();
    const int g = a.Hq / a.Hkv;
    const int shared_len = c.own_from;
    const bool common = id < c.shared * c.shared_groups;
    if (!common) id -= c.shared * c.shared_groups;
    const int parts = common ? c.shared : c.own, part = id % parts, group = id / parts;
    // Rows r0 + i: sequence r / g, head kh g + r % g.
    const int64_t r0 = common ? (int64_t)group * kRows : (int64_t)(group / c.own_groups) * g + group % c.own_groups * kRows;
    const int64_t end = common ? (int64_t)a.B * g : (int64_t)(group / c.own_groups + 1) * g;
    const int live = (int)min((int64_t)kRows, end - r0);
    const int64_t r = r0 + min((int)(threadIdx.x & 15), live - 1);
    const int64_t b = over(r, g);
    const int h = kh * g + (int)(r - b * g);
    const int n = decode_length(a, (int)b);
    int lo, hi;
    if (common) {
        int most = min(n, shared_len);  // of the block's rows
#pragma unroll
        for (int x = 8; x; x >>= 1) most = max(most, __shfl_xor(most, x));
        part_range(0, shared_len, part, parts, kUnit, lo, hi);
        hi = min(hi, most);
    } else {
        part_range(shared_len, n, part, parts, kUnit, lo, hi);
    }
    hi = __builtin_amdgcn_readfirstlane(hi);
    const PagedKeys keys = {(const char *)((const T *)a.k.data + kh * a.k.head),
                            (const char *)((const T *)a.v.data + kh * a.v.head),
                            a.k.page * (int64_t)sizeof(T), a.v.page * (int64_t)sizeof(T),
                            a.k.tok * (int64_t)sizeof(T), a.v.tok * (int64_t)sizeof(T),
                            a.table + (common ? 0 : b * a.ld_table), a.page_log2, a.P, 0x7FFFFFFF};
    attend_rows<T, DP, WIDE, NW>(a.q + b * a.q_seq + h * a.q_head, rows_wide(a.q, a.q_seq | a.q_head, a.D), a.D,
                                 common ? min(n, shared_len) : n, a.scale, lo, hi, keys, sh);
    if (threadIdx.x < kRows) sh.unfinished[threadIdx.x] = 0;
    __syncthreads();
    const int row = threadIdx.x >> 4;
    const int64_t rb = over(r0 + row, g);
    const int rh = kh * g + (int)(r0 + row - rb * g);
    leave_row<SLOTS>(sh, c.to, (rb * a.Hq + rh) * c.to.slots + (common ? part : c.to.slots - c.own + part),
                  a.out + rb * a.out_seq + rh * a.out_head, a.D, row < live);
    if (SLOTS || c.to.o) return;
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += NW)
        if (sh.unfinished[w]) {
            const int64_t wb = over(r0 + w, g);
            attend_decode_row<T>(a, wb, kh * g + (int)(r0 + w - wb * g));
        }
}

}  // namespace

}  // namespace cfp32
