// Attention of few rows: new tokens against the paged cache, and short
// packed prompts.
//
// A block of four waves works on 16 rows (tokens x heads of one K/V head, so
// grouped heads share what is read); its keys are dealt to the waves in steps
// of kStep, and the waves' sums are joined in LDS.  Everything a wave
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
// These products are bounded by memory, not by the matrix units: 16 rows
// against FP32 keys need 1024 cycles of a SIMD for 8 KiB at D = 64, which is
// 19 TB/s over the chip.
#include <stdlib.h>
#include "attention_device.h"

namespace cfp32 {

namespace {

constexpr int kWaves = 4;
constexpr int kRows = 16;

// Where a block's keys are: packed rows, ...
struct PackedKeys {
    const char *k, *v;       // key 0 of the head
    int64_t k_tok, v_tok;    // bytes
    __device__ __forceinline__ int page_of(int) { return 0; }
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

struct Joined {
    float o[kWaves][kRows][kAttnMaxDim + 4];
    float m[kWaves][kRows], l[kWaves][kRows];
    int unfinished[kRows];
};

// One wave's share of 16 rows: this lane's row q sees the first
// `limit` keys; keys [lo, hi) (lo a multiple of 16 if pages are to be read
// 16 keys at a time), every kWaves-th step of them.
template <class T, int DP, bool WIDE, class Keys>
__device__ __forceinline__ void attend_rows(const float *q, bool q_wide, int D, int limit, float scale, int lo, int hi, Keys keys,
                                            Joined &to)
{
    constexpr bool F16 = sizeof(T) == 2;
    constexpr int NB = DP == 128 ? 2 : 4;      // 16-key blocks of a step
    constexpr int kStep = 16 * NB;
    constexpr int KK = F16 ? DP / 32 : DP / 16;  // key loads (16 bytes) of a lane and block
    constexpr int KE = F16 ? 8 : 4;
    constexpr int NV = DP / 16;                // value elements of a lane and key
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    float m = -INFINITY, l = 0.0f;
    floatx4_t o[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) o[c] = floatx4_t{0, 0, 0, 0};

    int kb = lo + wave * kStep;
    if (kb < hi) {
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
                const char *p = keys.key(min(b0 + 16 * b + col, last), page[b]);
#pragma unroll
                for (int i = 0; i < KK; ++i) load_row<T, KE, WIDE>(p, (i * 4 + quad) * KE, D, kr[b][i]);
            }
        };
        auto load_v = [&](int b0) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    load_row<T, NV, WIDE>(keys.value(min(b0 + 16 * b + 4 * quad + r, last), page[b]), col * NV, D, vr[b][r]);
        };
        pages(kb, page);
        load_k(kb);
        load_v(kb);
        pages(kb + kWaves * kStep, next);

        // The row, as the right operand of the score products.
        float f = scale * kLog2e;
        half8_t qh[F16 ? KK : 1], ql[F16 ? KK : 1];
        float x[KK][KE];
        if (q_wide) {
#pragma unroll
            for (int i = 0; i < KK; ++i) load_floats<KE, true>(q, (i * 4 + quad) * KE, D, x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < KK; ++i) load_floats<KE, false>(q, (i * 4 + quad) * KE, D, x[i]);
        }
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

        for (; kb < hi; kb += kWaves * kStep) {
            floatx4_t s[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                s[b] = floatx4_t{0, 0, 0, 0};
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
            const int nb = kb + kWaves * kStep;
            const bool more = nb < hi;
            if (more) {
                // The next step's pages are known; ask for those after it first.
#pragma unroll
                for (int b = 0; b < NB; ++b) page[b] = next[b];
                if (nb + kWaves * kStep < hi) pages(nb + kWaves * kStep, next);
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
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = exp2_raw(s[b][r] - base);
                    l += p;
#pragma unroll
                    for (int c = 0; c < NV; ++c)
                        o[c] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)vr[b][r][c], p, o[c], 0, 0, 0);
                }
            if (more) load_v(nb);
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
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < NV; c += 4) {
            floatx4_t t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = o[c + e][r];
            *reinterpret_cast<floatx4_t *>(&to.o[wave][col][NV * (4 * quad + r) + c]) = t;
        }
    if (quad == 0) {
        to.m[wave][col] = m;
        to.l[wave][col] = l;
    }
}

// The waves' sums of row threadIdx.x / 16 joined: m, l and this thread's DP /
// 16 values (unnormalised).
template <int DP>
__device__ __forceinline__ void join_rows(const Joined &from, float &m, float &l, float (&x)[DP / 16])
{
    constexpr int NV = DP / 16;
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * NV;
    m = from.m[0][row];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, from.m[w][row]);
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) x[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float mw = from.m[w][row], f = mw == -INFINITY ? 0.0f : exp2_raw(mw - m);
        l = fmaf(f, from.l[w][row], l);
#pragma unroll
        for (int c = 0; c < NV; ++c) x[c] = fmaf(f, from.o[w][row][d0 + c], x[c]);
    }
}

template <class T, int DP, bool WIDE>
__global__ __launch_bounds__(64 * kWaves, 2) void prompt_rows_kernel(PromptArgs a)
{
    __shared__ Joined sh;
    const int g = a.Hq / a.Hkv, kh = blockIdx.y;
    int64_t start;
    const int64_t id = gridDim.x - 1 - blockIdx.x;  // the rows that see most first
    const int sid = find_unit(a.cu_q, a.S, g, kRows, id, start);
    const Sequence sq = sequence(a, sid);
    const int64_t n = (int64_t)sq.nq * g;
    if (id < start || (id - start) * kRows >= n) return;
    const int64_t r0 = (id - start) * kRows;
    const int live = (int)min((int64_t)kRows, n - r0);
    const int64_t r = r0 + min((int)(threadIdx.x & 15), live - 1);
    const int i = (int)(r / g), h = kh * g + (int)(r - (int64_t)i * g);
    const PackedKeys keys = {(const char *)((const T *)a.k.data + sq.k0 * a.k.tok + kh * a.k.head),
                             (const char *)((const T *)a.v.data + sq.k0 * a.v.tok + kh * a.v.head),
                             a.k.tok * (int64_t)sizeof(T), a.v.tok * (int64_t)sizeof(T)};
    const int hi = sq.limit((int)((r0 + live - 1) / g));
    attend_rows<T, DP, WIDE>((const float *)a.q.data + (sq.q0 + i) * a.q.tok + h * a.q.head,
                             rows_wide(a.q.data, a.q.tok | a.q.head, a.D), a.D, sq.limit(i), a.scale, 0,
                             hi, keys, sh);
    if (threadIdx.x < kRows) sh.unfinished[threadIdx.x] = 0;
    __syncthreads();
    float m, l, x[DP / 16];
    join_rows<DP>(sh, m, l, x);
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (DP / 16);
    if (row < live) {
        const int ri = (int)((r0 + row) / g), rh = kh * g + (int)(r0 + row - (int64_t)ri * g);
        float *out = a.out + (sq.q0 + ri) * a.out_tok + rh * a.out_head;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const float y = x[c] * inv;
            if (d0 + c < a.D) {
                out[d0 + c] = y;
                if (!(fabsf(y) < INFINITY)) sh.unfinished[row] = 1;
            }
        }
    }
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += kWaves)
        if (sh.unfinished[w]) {
            const int ri = (int)((r0 + w) / g);
            attend_prompt_row<T>(a, sq, ri, kh * g + (int)(r0 + w - (int64_t)ri * g));
        }
}

// How the keys of a decode are cut: the shared ones into `shared` parts (0:
// none are shared), each sequence's others into `own`, of equal lengths (in
// whole steps of all waves).  Row groups: 16 rows of the batch's for the
// shared keys, 16 of a sequence's heads for its own.
struct DecodeParts {
    int shared, own, shared_groups, own_groups;
    Partials to;  // slots: shared + own; null o: straight to the output
};

__device__ __forceinline__ void part_range(int lo, int hi, int part, int parts, int unit, int &a, int &b)
{
    const int n = max(hi - lo, 0), u = (n + unit - 1) / unit, per = (u + parts - 1) / parts;
    a = lo + (int)min((int64_t)n, (int64_t)part * per * unit);
    b = lo + (int)min((int64_t)n, (int64_t)(part + 1) * per * unit);
}

template <class T, int DP, bool WIDE>
__global__ __launch_bounds__(64 * kWaves, 2) void decode_rows_kernel(DecodeArgs a, DecodeParts c)
{
    __shared__ Joined sh;
    constexpr int kUnit = kWaves * (DP == 128 ? 32 : 64);
    const int g = a.Hq / a.Hkv, kh = blockIdx.y;
    const int shared_len = c.shared ? a.shared_pages << a.page_log2 : 0;
    int id = blockIdx.x;
    const bool common = id < c.shared * c.shared_groups;
    if (!common) id -= c.shared * c.shared_groups;
    const int parts = common ? c.shared : c.own, part = id % parts, group = id / parts;
    // Rows r0 + i: sequence r / g, head kh g + r % g.
    const int64_t r0 = common ? (int64_t)group * kRows : (int64_t)(group / c.own_groups) * g + group % c.own_groups * kRows;
    const int64_t end = common ? (int64_t)a.B * g : (int64_t)(group / c.own_groups + 1) * g;
    const int live = (int)min((int64_t)kRows, end - r0);
    const int64_t r = r0 + min((int)(threadIdx.x & 15), live - 1);
    const int64_t b = r / g;
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
    attend_rows<T, DP, WIDE>(a.q + b * a.q_seq + h * a.q_head, rows_wide(a.q, a.q_seq | a.q_head, a.D), a.D, common ? min(n, shared_len) : n, a.scale, lo, hi, keys,
                             sh);
    if (threadIdx.x < kRows) sh.unfinished[threadIdx.x] = 0;
    __syncthreads();
    float m, l, x[DP / 16];
    join_rows<DP>(sh, m, l, x);
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (DP / 16);
    const int64_t rb = (r0 + row) / g;
    const int rh = kh * g + (int)(r0 + row - rb * g);
    if (c.to.o) {
        if (row < live) {
            const int64_t slot = (rb * a.Hq + rh) * c.to.slots + (common ? part : c.shared + part);
            if ((threadIdx.x & 15) == 0) {
                c.to.m[slot] = m;
                c.to.l[slot] = l;
            }
            if (l != 0.0f)
#pragma unroll
                for (int e = 0; e < DP / 16; e += 4)
                    *reinterpret_cast<floatx4_t *>(c.to.o + slot * DP + d0 + e) = floatx4_t{x[e], x[e + 1], x[e + 2], x[e + 3]};
        }
        return;
    }
    if (row < live) {
        float *out = a.out + rb * a.out_seq + rh * a.out_head;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
            const float y = x[e] * inv;
            if (d0 + e < a.D) {
                out[d0 + e] = y;
                if (!(fabsf(y) < INFINITY)) sh.unfinished[row] = 1;
            }
        }
    }
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += kWaves)
        if (sh.unfinished[w]) {
            const int64_t wb = (r0 + w) / g;
            attend_decode_row<T>(a, wb, kh * g + (int)(r0 + w - wb * g));
        }
}

// Rows from their parts, a wave to a row.
template <class T, int DP>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs a, Partials from)
{
    constexpr int E = DP / 64;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= (int64_t)a.B * a.Hq) return;
    const int lane = threadIdx.x & 63;
    const int64_t s0 = row * from.slots;
    float m = -INFINITY;
    for (int i = lane; i < from.slots; i += 64) m = fmaxf(m, from.m[s0 + i]);
#pragma unroll
    for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = 0.0f, o[E] = {};
    for (int i0 = 0; i0 < from.slots; i0 += 64) {
        const int i = i0 + lane;
        float f = 0.0f, li = 0.0f;
        if (i < from.slots) {
            const float mi = from.m[s0 + i];
            f = mi == -INFINITY ? 0.0f : exp2_raw(mi - m);
            li = from.l[s0 + i];
        }
        float t = f * li;
#pragma unroll
        for (int x = 32; x; x >>= 1) t += __shfl_xor(t, x);
        l += t;
        if (li == 0.0f) f = 0.0f;  // nothing was written there
        uint64_t used = __ballot(f != 0.0f);
        while (used) {
            constexpr int U = 8;  // loads in flight
            float w[U], x[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = used ? __builtin_ctzll(used) : -1;
                w[u] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) x[u][e] = 0.0f;
                if (k >= 0) {
                    used &= used - 1;
                    w[u] = __shfl(f, k);
#pragma unroll
                    for (int e = 0; e < E; ++e) x[u][e] = from.o[(s0 + i0 + k) * DP + lane * E + e];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(w[u], x[u][e], o[e]);
        }
    }
    const int64_t b = row / a.Hq;
    const int h = (int)(row - b * a.Hq);
    float *out = a.out + b * a.out_seq + h * a.out_head;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = o[e] * inv;
        if (lane * E + e < a.D) {
            out[lane * E + e] = y;
            odd |= !(fabsf(y) < INFINITY);
        }
    }
    odd |= !(fabsf(l) < INFINITY);
    if (__any(odd)) attend_decode_row<T>(a, b, h);
}

// Rows against a pool without pages: 0, or NaN where a sequence has tokens.
__global__ __launch_bounds__(64) void decode_no_pages_kernel(DecodeArgs a)
{
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x)
        for (int h = blockIdx.y; h < a.Hq; h += gridDim.y) attend_decode_row<float>(a, b, h);
}

bool wide(const void *p, int64_t strides, int D, bool f16)
{
    const int64_t eb = f16 ? 2 : 4;
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(strides * eb)) & 15) == 0 && D % (16 / eb) == 0;
}

}  // namespace

#define CFP32_BY_TYPE(KERNEL, F16, D, WIDE, GRID, BLOCK, ...)                                           \
    do {                                                                                              \
        if (F16) {                                                                                    \
            if ((D) <= 64) {                                                                          \
                if (WIDE) KERNEL<_Float16, 64, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);        \
                else KERNEL<_Float16, 64, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);            \
            } else {                                                                                  \
                if (WIDE) KERNEL<_Float16, 128, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);       \
                else KERNEL<_Float16, 128, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);           \
            }                                                                                         \
        } else {                                                                                      \
            if ((D) <= 64) {                                                                          \
                if (WIDE) KERNEL<float, 64, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);           \
                else KERNEL<float, 64, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);               \
            } else {                                                                                  \
                if (WIDE) KERNEL<float, 128, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);          \
                else KERNEL<float, 128, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);              \
            }                                                                                         \
        }                                                                                             \
    } while (0)

size_t attention_prompt_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16)
{
    return prompt_tile_workspace(S, Tk, Hkv, D, kv_f16);
}

hipError_t launch_attention_prompt(const PromptArgs &a, void *workspace, hipStream_t stream)
{
    const int g = a.Hq / a.Hkv;
    const int64_t units = (int64_t)a.Tq * g / kRows + a.S;
    if (a.Hkv > 65535 || units > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const bool w = wide(a.k.data, a.k.tok | a.k.head, a.D, a.kv_f16) && wide(a.v.data, a.v.tok | a.v.head, a.D, a.kv_f16);
    static const int force = getenv("CF_FORCE") ? atoi(getenv("CF_FORCE")) : 0;
    if (a.Tk > 0 && (!a.kv_f16 || (w && a.k.tok < ((int64_t)1 << 31) && a.v.tok < ((int64_t)1 << 31))) && (force == 2 || (force == 0 && a.Tq >= 1024))) return launch_prompt_tile(a, workspace, stream);
    const dim3 grid((unsigned)units, (unsigned)a.Hkv);
    CFP32_BY_TYPE(prompt_rows_kernel, a.kv_f16, a.D, w, grid, 64 * kWaves, a);
    return hipGetLastError();
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts are made until the grid has kTargetBlocks blocks (2 of 4 waves to a
// CU, twice over), of at least one step of all waves each.
DecodeParts decode_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages)
{
    constexpr int64_t kTargetBlocks = 1024;
    DecodeParts c = {};
    const int64_t g = Hq / Hkv, unit = kWaves * (D <= 64 ? 64 : 32);
    const int64_t n_shared = B > 1 ? shared_pages << lg : 0;
    const int64_t n_own = (W << lg) - n_shared;
    c.shared_groups = (int)ceil_div(B * g, kRows);
    c.own_groups = (int)ceil_div(g, kRows);
    auto parts = [&](int64_t keys, int64_t blocks) {
        const int64_t most = ceil_div(keys, unit), want = ceil_div(kTargetBlocks, blocks);
        return (int)(most < want ? most : want);
    };
    if (n_shared) c.shared = parts(n_shared, c.shared_groups * Hkv);
    c.own = n_own > 0 ? parts(n_own, B * c.own_groups * Hkv) : 0;
    if (c.shared + c.own == 0) c.own = 1;
    c.to.slots = c.shared + c.own;
    c.to.dim = D <= 64 ? 64 : 128;
    return c;
}

}  // namespace

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg,
                                  int64_t shared_pages, bool)
{
    if (Hkv == 0) return 0;
    const DecodeParts c = decode_parts(B, Hq, Hkv, D, W, lg, shared_pages);
    return c.to.slots > 1 ? (size_t)(B * Hq) * c.to.slots * (c.to.dim + 2) * 4 : 0;
}

hipError_t launch_attention_decode(const DecodeArgs &a, void *workspace, hipStream_t stream)
{
    if (a.Hkv > 65535) return hipErrorInvalidConfiguration;
    if (a.P == 0) {
        const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)(a.Hq < 65535 ? a.Hq : 65535));
        decode_no_pages_kernel<<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    DecodeParts c = decode_parts(a.B, a.Hq, a.Hkv, a.D, a.W, a.page_log2, a.shared_pages);
    const int64_t rows = (int64_t)a.B * a.Hq, n = rows * c.to.slots;
    const int64_t blocks = (int64_t)c.shared * c.shared_groups + (int64_t)a.B * c.own_groups * c.own;
    if (blocks > 0x7FFFFFFF || (rows + 3) / 4 > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (c.to.slots > 1) {
        c.to.o = (float *)workspace;
        c.to.m = c.to.o + n * c.to.dim;
        c.to.l = c.to.m + n;
    }
    const int64_t eb_k = a.k.page | a.k.head | a.k.tok, eb_v = a.v.page | a.v.head | a.v.tok;
    const bool w = wide(a.k.data, eb_k, a.D, a.kv_f16) && wide(a.v.data, eb_v, a.D, a.kv_f16);
    const dim3 grid((unsigned)blocks, (unsigned)a.Hkv);
    CFP32_BY_TYPE(decode_rows_kernel, a.kv_f16, a.D, w, grid, 64 * kWaves, a, c);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || c.to.slots <= 1) return e;
    const unsigned join = (unsigned)((rows + 3) / 4);
    if (a.kv_f16) {
        if (a.D <= 64) decode_join_kernel<_Float16, 64><<<join, 256, 0, stream>>>(a, c.to);
        else decode_join_kernel<_Float16, 128><<<join, 256, 0, stream>>>(a, c.to);
    } else {
        if (a.D <= 64) decode_join_kernel<float, 64><<<join, 256, 0, stream>>>(a, c.to);
        else decode_join_kernel<float, 128><<<join, 256, 0, stream>>>(a, c.to);
    }
    return hipGetLastError();
}

}  // namespace cfp32
