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
#include "attention_device.h"

namespace cfp32 {

namespace {

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

template <int DP, int NW>
struct Joined {
    float o[NW][kRows][DP + 4];
    float m[NW][kRows], l[NW][kRows];
    int unfinished[kRows];
};

template <int DP>
constexpr int row_step() { return DP == 128 ? 32 : 64; }  // keys a wave takes at a time

// One wave's share of 16 rows: this lane's row q sees the first `limit` keys;
// the wave takes keys [kb, hi), row_step at a time, NW steps further each
// time.  FEW: there is one step, of which blocks of 16 keys may be missing.
template <class T, int DP, bool WIDE, int NW, bool FEW, class Keys>
__device__ __forceinline__ void attend_share(const float *q, bool q_wide, int D, int limit, float scale, int kb, int hi, Keys keys,
                                             Joined<DP, NW> &to)
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

// A block's keys [lo, hi) (lo a multiple of 16 if pages are to be read 16 keys
// at a time), dealt to its waves in steps, or, if they make no more than a
// step of each, in equal shares of whole blocks of 16 (37 keys x 64: 7.0 ->
// 5.7 us, all four waves at work).
template <class T, int DP, bool WIDE, int NW, class Keys>
__device__ __forceinline__ void attend_rows(const float *q, bool q_wide, int D, int limit, float scale, int lo, int hi, Keys keys,
                                            Joined<DP, NW> &to)
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
    m = from.m[0][row];
#pragma unroll
    for (int w = 1; w < NW; ++w) m = fmaxf(m, from.m[w][row]);
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) x[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float mw = from.m[w][row], f = mw == -INFINITY ? 0.0f : exp2_raw(mw - m);
        l = fmaf(f, from.l[w][row], l);
#pragma unroll
        for (int c = 0; c < NV; ++c) x[c] = fmaf(f, from.o[w][row][d0 + c], x[c]);
    }
}

// A row's sums, of what this block has seen: into its slot, or (all there is)
// as its result.  Results that are not finite are marked.
template <int DP, int NW>
__device__ __forceinline__ void leave_row(Joined<DP, NW> &sh, const Partials &to, int64_t slot, float *out, int D, bool live)
{
    if (!live) return;
    const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (DP / 16);
    float m, l, x[DP / 16];
    join_rows(sh, row, d0, m, l, x);
    if (to.o) {
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
            if (!(fabsf(y) < INFINITY)) sh.unfinished[row] = 1;
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

template <class T, int DP, bool WIDE, int NW>
__global__ __launch_bounds__(64 * NW, 2) void prompt_rows_kernel(PromptArgs a, Partials to)
{
    __shared__ Joined<DP, NW> sh;
    constexpr int kUnit = row_step<DP>();
    // The rows that see most first.  Heads vary fastest: blocks go round the
    // eight XCDs, so a head's keys are read by few of them.
    const int g = a.Hq / a.Hkv, kh = blockIdx.x % a.Hkv, part = blockIdx.y;
    int64_t start;
    const int64_t id = (gridDim.x - 1 - blockIdx.x) / a.Hkv;
    const int sid = find_unit(a.cu_q, a.S, g, kRows, id, start);
    const Sequence sq = sequence(a, sid);
    const int64_t n = (int64_t)sq.nq * g;
    if (id < start || (id - start) * kRows >= n) return;
    const int64_t r0 = (id - start) * kRows;
    const int live = (int)min((int64_t)kRows, n - r0);
    const int64_t r = r0 + min((int)(threadIdx.x & 15), live - 1);
    const int i = (int)over(r, g), h = kh * g + (int)(r - (int64_t)i * g);
    const PackedKeys keys = {(const char *)((const T *)a.k.data + sq.k0 * a.k.tok + kh * a.k.head),
                             (const char *)((const T *)a.v.data + sq.k0 * a.v.tok + kh * a.v.head),
                             a.k.tok * (int64_t)sizeof(T), a.v.tok * (int64_t)sizeof(T)};
    int lo, hi;
    part_range(0, sq.limit((int)over(r0 + live - 1, g)), part, to.slots, kUnit, lo, hi);
    attend_rows<T, DP, WIDE, NW>((const float *)a.q.data + (sq.q0 + i) * a.q.tok + h * a.q.head,
                             rows_wide(a.q.data, a.q.tok | a.q.head, a.D), a.D, sq.limit(i), a.scale, lo, hi, keys, sh);
    if (threadIdx.x < kRows) sh.unfinished[threadIdx.x] = 0;
    __syncthreads();
    const int row = threadIdx.x >> 4, ri = (int)over(r0 + row, g), rh = kh * g + (int)(r0 + row - (int64_t)ri * g);
    leave_row(sh, to, ((int64_t)(sq.q0 + ri) * a.Hq + rh) * to.slots + part,
                  a.out + (sq.q0 + ri) * a.out_tok + rh * a.out_head, a.D, row < live);
    if (to.o) return;
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += NW)
        if (sh.unfinished[w]) {
            const int wi = (int)over(r0 + w, g);
            attend_prompt_row<T>(a, sq, wi, kh * g + (int)(r0 + w - (int64_t)wi * g));
        }
}

// How the keys of a decode are cut: the shared ones into `shared` parts (0:
// none are shared), each sequence's others into `own`, of equal lengths (in
// whole steps of all waves).  Row groups: 16 rows of the batch's for the
// shared keys, 16 of a sequence's heads for its own.
struct DecodeParts {
    int shared, own, shared_groups, own_groups;
    int own_from;  // the first key that is not shared
    bool eight;    // waves
    Partials to;  // slots: shared + own; null o: straight to the output
};

template <class T, int DP, bool WIDE, int NW>
__global__ __launch_bounds__(64 * NW, 2) void decode_rows_kernel(DecodeArgs a, DecodeParts c)
{
    __shared__ Joined<DP, NW> sh;
    constexpr int kUnit = NW * row_step<DP>();
    const int g = a.Hq / a.Hkv, kh = blockIdx.y;
    const int shared_len = c.own_from;
    int id = blockIdx.x;
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
    attend_rows<T, DP, WIDE, NW>(a.q + b * a.q_seq + h * a.q_head, rows_wide(a.q, a.q_seq | a.q_head, a.D), a.D, common ? min(n, shared_len) : n, a.scale, lo, hi, keys,
                             sh);
    if (threadIdx.x < kRows) sh.unfinished[threadIdx.x] = 0;
    __syncthreads();
    const int row = threadIdx.x >> 4;
    const int64_t rb = over(r0 + row, g);
    const int rh = kh * g + (int)(r0 + row - rb * g);
    leave_row(sh, c.to, (rb * a.Hq + rh) * c.to.slots + (common ? part : c.to.slots - c.own + part),
                  a.out + rb * a.out_seq + rh * a.out_head, a.D, row < live);
    if (c.to.o) return;
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += NW)
        if (sh.unfinished[w]) {
            const int64_t wb = over(r0 + w, g);
            attend_decode_row<T>(a, wb, kh * g + (int)(r0 + w - wb * g));
        }
}

// Row (i, h) of a call: where its result goes (null: it is no row of a sequence), and its slow form.
__device__ __forceinline__ float *row_out(const DecodeArgs &a, int64_t i, int h) { return a.out + i * a.out_seq + h * a.out_head; }
template <class T>
__device__ __forceinline__ void redo_row(const DecodeArgs &a, int64_t i, int h) { attend_decode_row<T>(a, i, h); }
__device__ __forceinline__ bool prompt_row(const PromptArgs &a, int64_t i, Sequence &sq)
{
    int lo = 0, hi = a.S;  // the largest s < S with cu_q[s] <= i
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a.cu_q[mid] <= i) lo = mid;
        else hi = mid;
    }
    sq = sequence(a, lo);
    return i >= sq.q0 && i < sq.q0 + sq.nq;
}
__device__ __forceinline__ float *row_out(const PromptArgs &a, int64_t i, int h)
{
    Sequence sq;
    return prompt_row(a, i, sq) ? a.out + i * a.out_tok + h * a.out_head : nullptr;
}
template <class T>
__device__ __forceinline__ void redo_row(const PromptArgs &a, int64_t i, int h)
{
    Sequence sq;
    if (prompt_row(a, i, sq)) attend_prompt_row<T>(a, sq, (int)i - sq.q0, h);
}

// Rows from their parts.  WAVES: of a row, each taking every WAVES-th part,
// their sums joined in LDS.  Few parts: a wave to a row (a block to a row made
// 9600 rows of 2 parts cost 15 us).  Many: four (a wave to a row took 10 us
// for 1024 rows of 68 parts x 128, for want of loads in flight; now 6).
template <class T, int DP, int WAVES, class Args>
__global__ __launch_bounds__(256) void join_kernel(Args a, Partials from, int64_t rows)
{
    constexpr int E = DP / 64;
    __shared__ float sums[4][DP], weight[4];
    const int lane = threadIdx.x & 63, w4 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = w4 % WAVES;
    const int64_t row = min((int64_t)blockIdx.x * (4 / WAVES) + w4 / WAVES, rows - 1), b = row / a.Hq;
    const int h = (int)(row - b * a.Hq);
    float *out = row_out(a, b, h);
    const int64_t s0 = row * from.slots;
    const int slots = out ? from.slots : 0;
    float m = -INFINITY;
    for (int i = lane; i < slots; i += 64) m = fmaxf(m, from.m[s0 + i]);
#pragma unroll
    for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = 0.0f, o[E] = {};
    for (int i0 = 0; i0 < slots; i0 += 64 * WAVES) {
        const int i = i0 + WAVES * lane + wave;
        float f = 0.0f, li = 0.0f;
        if (i < slots) {
            const float mi = from.m[s0 + i];
            f = mi == -INFINITY ? 0.0f : exp2_raw(mi - m);
            li = from.l[s0 + i];
        }
        l = fmaf(f, li, l);
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
                    for (int e = 0; e < E; ++e) x[u][e] = from.o[(s0 + i0 + WAVES * k + wave) * DP + lane * E + e];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(w[u], x[u][e], o[e]);
        }
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) l += __shfl_xor(l, x);
    if (WAVES == 4) {
        if (lane == 0) weight[wave] = l;
#pragma unroll
        for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = o[e];
        __syncthreads();
        if (wave) return;
        l = (weight[0] + weight[1]) + (weight[2] + weight[3]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e;
            o[e] = (sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d]);
        }
    }
    if (!out) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    bool odd = !(fabsf(l) < INFINITY);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = o[e] * inv;
        if (lane * E + e < a.D) {
            out[lane * E + e] = y;
            odd |= !(fabsf(y) < INFINITY);
        }
    }
    if (__any(odd)) redo_row<T>(a, b, h);
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

// KERNEL<type, padded D, WIDE, waves>
#define CFP32_BY_WAVES(KERNEL, T, DP, WIDE, EIGHT, GRID, ...)                                        \
    do {                                                                                             \
        if (EIGHT) KERNEL<T, DP, WIDE, 8><<<GRID, 512, 0, stream>>>(__VA_ARGS__);                    \
        else KERNEL<T, DP, WIDE, 4><<<GRID, 256, 0, stream>>>(__VA_ARGS__);                          \
    } while (0)
#define CFP32_BY_TYPE(KERNEL, F16, D, WIDE, EIGHT, GRID, ...)                                        \
    do {                                                                                             \
        if (F16) {                                                                                   \
            if ((D) <= 64) {                                                                         \
                if (WIDE) CFP32_BY_WAVES(KERNEL, _Float16, 64, true, EIGHT, GRID, __VA_ARGS__);      \
                else CFP32_BY_WAVES(KERNEL, _Float16, 64, false, EIGHT, GRID, __VA_ARGS__);          \
            } else {                                                                                 \
                if (WIDE) CFP32_BY_WAVES(KERNEL, _Float16, 128, true, EIGHT, GRID, __VA_ARGS__);     \
                else CFP32_BY_WAVES(KERNEL, _Float16, 128, false, EIGHT, GRID, __VA_ARGS__);         \
            }                                                                                        \
        } else {                                                                                     \
            if ((D) <= 64) {                                                                         \
                if (WIDE) CFP32_BY_WAVES(KERNEL, float, 64, true, EIGHT, GRID, __VA_ARGS__);         \
                else CFP32_BY_WAVES(KERNEL, float, 64, false, EIGHT, GRID, __VA_ARGS__);             \
            } else {                                                                                 \
                if (WIDE) CFP32_BY_WAVES(KERNEL, float, 128, true, EIGHT, GRID, __VA_ARGS__);        \
                else CFP32_BY_WAVES(KERNEL, float, 128, false, EIGHT, GRID, __VA_ARGS__);            \
            }                                                                                        \
        }                                                                                            \
    } while (0)

size_t partial_bytes(int64_t rows, int slots, int dim) { return slots > 1 ? (size_t)rows * slots * (dim + 2) * 4 : 0; }

void place_partials(Partials &to, int64_t rows, void *at)
{
    if (to.slots <= 1) return;
    const int64_t n = rows * to.slots;
    to.o = (float *)at;
    to.m = to.o + n * to.dim;
    to.l = to.m + n;
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded(int64_t D) { return D <= 64 ? 64 : 128; }

template <class Args>
hipError_t join(const Args &a, const Partials &from, int64_t rows, hipStream_t stream)
{
    const bool four = from.slots > 16;
    const unsigned blocks = (unsigned)(four ? rows : ceil_div(rows, 4));
#define CFP32_JOIN(T, DP)                                                            \
    do {                                                                           \
        if (four) join_kernel<T, DP, 4><<<blocks, 256, 0, stream>>>(a, from, rows); \
        else join_kernel<T, DP, 1><<<blocks, 256, 0, stream>>>(a, from, rows);      \
    } while (0)
    if (a.kv_f16) {
        if (a.D <= 64) CFP32_JOIN(_Float16, 64);
        else CFP32_JOIN(_Float16, 128);
    } else {
        if (a.D <= 64) CFP32_JOIN(float, 64);
        else CFP32_JOIN(float, 128);
    }
#undef CFP32_JOIN
    return hipGetLastError();
}

// Parts are made until the grid has `target` blocks (of 4 waves), of a step
// of all waves each (a little more than one makes no parts).
constexpr int64_t kDecodeBlocks = 512, kPromptBlocks = 256;
int key_parts(int64_t keys, int64_t unit, int64_t blocks, int64_t target)
{
    const int64_t most = 4 * keys <= 5 * unit ? 1 : ceil_div(keys, unit), want = target / (blocks ? blocks : 1);
    return (int)(want <= 1 || most <= 1 ? 1 : most < want ? most : want);
}
int64_t wave_step(int64_t D) { return D <= 64 ? 64 : 32; }

// Blocks of eight waves where that makes their keys one step instead of two
// (400 x 12 x 64 FP32 14.4 -> 12.5 us, 130 keys x 32/8 x 128 FP16 11.2 -> 9.3);
// with more keys than that, or fewer, four are as good or better (500 x 16/2 x
// 128 FP16 20 against 26 us).
bool eight_waves(int64_t keys, int64_t D) { return keys > 4 * wave_step(D) && keys <= 8 * wave_step(D); }

// How many parts the keys of a short prompt make: by the average sequence's.
int prompt_parts(int64_t S, int64_t Tk, int64_t blocks, int64_t D)
{
    return key_parts(ceil_div(Tk, S), 4 * wave_step(D), blocks, kPromptBlocks);
}

// Which kernel a prompt goes through, by estimates in microseconds beyond what
// both have in common: here FP32 matrix products (45 TFLOP/s of the useful
// ones, 75 with FP16 keys) and the blocks, there the way through the longest
// sequence's tiles and what comes before (for FP32 K and V a pass over them).
// Measured, 16 rows to a block against tiles: FP32 500 / 750 / 1000 x 12 x 64
// 17 / 26 / 38 against 25 / 30 / 36 us, 300 / 500 x 32/8 x 128 26 / 48 against
// 31 / 38; FP16 500 / 1500 x 12 x 64 13 / 38 against 17 / 34, 300 / 500 x 32/8 x
// 128 20 / 33 against 21 / 25, 8 x 60 and 4 x 100 of these 19 and 17 against 14
// and 14, 50 after 700 16 against 20.
bool prefer_tiles(const PromptArgs &a, int64_t units)
{
    const double keys = (double)a.Tk / a.S, seen = a.causal ? keys - 0.5 * a.Tq / a.S : keys;
    const double gflop = 4e-9 * a.D * a.Hq * a.Tq * (seen > 0 ? seen : 0), tiles = keys / 64;
    const double rows_us = gflop * (a.kv_f16 ? 1e3 / 75 : 1e3 / 45) + 0.008 * units * a.Hkv;
    const double tiles_us = a.kv_f16 ? (a.D <= 64 ? 4 + 1.1 * tiles : 4 + 2 * tiles) : (a.D <= 64 ? 6 + 1.7 * tiles : 10 + 3 * tiles);
    return rows_us > tiles_us;
}

}  // namespace

hipError_t launch_join(const PromptArgs &a, const Partials &from, hipStream_t stream)
{
    return join(a, from, (int64_t)a.Tq * a.Hq, stream);
}
hipError_t launch_join(const DecodeArgs &a, const Partials &from, hipStream_t stream)
{
    return join(a, from, (int64_t)a.B * a.Hq, stream);
}

size_t attention_prompt_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16)
{
    // Whatever the rows are, blocks of kRows of them and parts make no more than kPromptBlocks.
    const size_t parts = prompt_parts(S, Tk, 1, D) > 1 ? partial_bytes(kPromptBlocks * kRows / 2, 2, padded(D)) : 0;
    const size_t tiles = prompt_tile_workspace(S, Tk, Hkv, D, kv_f16);
    return parts > tiles ? parts : tiles;
}

hipError_t launch_attention_prompt(const PromptArgs &a, void *workspace, hipStream_t stream)
{
    const int g = a.Hq / a.Hkv;
    const int64_t units = (int64_t)a.Tq * g / kRows + a.S, rows = (int64_t)a.Tq * a.Hq;
    if (units > 0x7FFFFFFF / a.Hkv || rows > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    const bool w = wide(a.k.data, a.k.tok | a.k.head, a.D, a.kv_f16) && wide(a.v.data, a.v.tok | a.v.head, a.D, a.kv_f16);
    const bool can = a.Tk > 0 && (!a.kv_f16 || (w && a.k.tok < ((int64_t)1 << 31) && a.v.tok < ((int64_t)1 << 31)));
    if (can && prefer_tiles(a, units)) return launch_prompt_tile(a, workspace, stream);
    Partials to = {nullptr, nullptr, nullptr, prompt_parts(a.S, a.Tk, units * a.Hkv, a.D), padded(a.D)};
    const bool eight = eight_waves(ceil_div(a.Tk, (int64_t)a.S * to.slots), a.D);
    place_partials(to, rows, workspace);
    const dim3 grid((unsigned)(units * a.Hkv), (unsigned)to.slots);
    CFP32_BY_TYPE(prompt_rows_kernel, a.kv_f16, a.D, w, eight, grid, a, to);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !to.o ? e : launch_join(a, to, stream);
}

namespace {

// Which kernel takes the keys that all sequences share: estimates in
// microseconds, of this one by its groups of 16 rows, of attention_tile.hip's
// by its blocks of 128.  Measured, this against that, FP16 pages: 32 x 32/8 x
// 128 behind 1280 / 5120 / 20480 keys 33 / 50 / 112 against 35 / 39 / 58 us; 12
// of these 18 / 33 / 63 against 27 / 31 / 46; 10 x 16/2 x 128 behind 5120 /
// 20480 / 61440 18 / 34 / 67 against 29 / 34 / 47; 16 x 14/2 x 64 behind the
// same 16 / 29 / 52 against 23 / 26 / 38.
bool prefer_tiles(int64_t rows, int64_t Hkv, int64_t D, int64_t keys)
{
    const double k = 1e-3 * (double)keys * Hkv, groups = (double)ceil_div(rows, kRows), blocks = (double)ceil_div(rows, 128);
    return D <= 64 ? 0.05 * groups * k > 10 + 0.13 * blocks * k : 0.1 * groups * k > 13 + 0.16 * blocks * k;
}

// `tiled`: the shared keys are cut for the other kernel, and c.shared is 0.
DecodeParts decode_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages, bool tiles,
                         int &tiled)
{
    DecodeParts c = {};
    const int64_t g = Hq / Hkv, unit = 4 * wave_step(D);
    const int64_t n_shared = B > 1 ? shared_pages << lg : 0, n_own = (W << lg) - n_shared;
    c.shared_groups = (int)ceil_div(B * g, kRows);
    c.own_groups = (int)ceil_div(g, kRows);
    c.own_from = (int)n_shared;
    tiled = 0;
    if (n_shared) {
        if (tiles && prefer_tiles(B * g, Hkv, D, n_shared)) tiled = decode_tile_parts(B, Hq, Hkv, n_shared, lg);
        else c.shared = key_parts(n_shared, unit, c.shared_groups * Hkv, kDecodeBlocks);
    }
    if (n_own > 0) c.own = key_parts(n_own, unit, B * c.own_groups * Hkv, kDecodeBlocks);
    if (tiled + c.shared + c.own == 0) c.own = 1;
    c.eight = c.shared == 0 && c.own == 1 && eight_waves(n_own, D);
    c.to.slots = tiled + c.shared + c.own;
    if (tiled && c.to.slots == 1) c.to.slots = 2;  // always by way of slots; the second is an empty part
    if (tiled && c.own == 0) c.own = c.to.slots - tiled;
    c.to.dim = padded(D);
    return c;
}

}  // namespace

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages,
                                  bool kv_f16)
{
    if (Hkv == 0) return 0;
    int tiled;
    const size_t a = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, false, tiled).to.slots, padded(D));
    if (!kv_f16) return a;
    const size_t b = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, true, tiled).to.slots, padded(D));
    return a > b ? a : b;
}

hipError_t launch_attention_decode(const DecodeArgs &a, void *workspace, hipStream_t stream)
{
    if (a.Hkv > 65535) return hipErrorInvalidConfiguration;
    if (a.P == 0) {
        const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)(a.Hq < 65535 ? a.Hq : 65535));
        decode_no_pages_kernel<<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    const bool w = wide(a.k.data, a.k.page | a.k.head | a.k.tok, a.D, a.kv_f16) &&
                   wide(a.v.data, a.v.page | a.v.head | a.v.tok, a.D, a.kv_f16);
    const bool tiles = a.kv_f16 && w && a.k.tok < ((int64_t)1 << 31) && a.v.tok < ((int64_t)1 << 31);
    int tiled;
    DecodeParts c = decode_parts(a.B, a.Hq, a.Hkv, a.D, a.W, a.page_log2, a.shared_pages, tiles, tiled);
    const int64_t rows = (int64_t)a.B * a.Hq;
    const int64_t blocks = (int64_t)c.shared * c.shared_groups + (int64_t)a.B * c.own_groups * c.own;
    if (blocks > 0x7FFFFFFF || rows > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    place_partials(c.to, rows, workspace);
    if (tiled) {
        const hipError_t e = launch_decode_tile(a, c.to, tiled, stream);
        if (e != hipSuccess) return e;
    }
    hipError_t e = hipSuccess;
    if (blocks) {  // none where every key is shared and goes through tiles
        const dim3 grid((unsigned)blocks, (unsigned)a.Hkv);
        CFP32_BY_TYPE(decode_rows_kernel, a.kv_f16, a.D, w, c.eight, grid, a, c);
        e = hipGetLastError();
    }
    return e != hipSuccess || !c.to.o ? e : launch_join(a, c.to, stream);
}

}  // namespace cfp32
