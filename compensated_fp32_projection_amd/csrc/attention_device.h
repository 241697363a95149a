// Device code shared by the attention kernels.
#pragma once

#include "attention.h"
#include "device_common.h"

#define CFP32_LDS __attribute__((address_space(3)))

namespace cfp32 {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }  // results below 2^-126: 0

// The running maximum follows the scores only where they exceed it by more
// than this (in powers of two): weights are then at most 2^kLazy, and most
// steps leave the sums as they are.
constexpr float kLazy = 4.0f;

// a / b for 0 <= a, in 32 bits where they do (a 64-bit division costs a
// thread half a microsecond).
__device__ __forceinline__ int64_t over(int64_t a, int b)
{
    return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The largest s < S with start(s) <= id (0 if none), by all lanes of a wave:
// 64 starts at a time (one after the other, three lookups took 1.5 us).
template <class Start>
__device__ __forceinline__ int find_last(int S, int64_t id, Start start)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, n = S;  // it is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64, at = lane * step;
        const uint64_t below = __ballot(at < n && start(lo + at) <= id);
        const int k = below ? 63 - __builtin_clzll(below) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The sequence that owns unit `id` of a packed batch, where sequence s starts
// at unit cu[s] * mul / div + s (so sequences of n tokens own up to
// ceil(n * mul / div) units, and some units belong to none).
__device__ __forceinline__ int find_unit(const int32_t *cu, int S, int mul, int div, int64_t id, int64_t &start)
{
    auto at = [&](int s) { return (int64_t)cu[s] * mul / div + s; };
    const int s = find_last(S, id, at);
    start = at(s);
    return s;
}

// A sequence of a packed batch: rows [q0, q0 + nq) and keys [k0, k0 + nk),
// within the tensors whatever the offsets say.
struct Sequence {
    int q0, nq, k0, nk;
    bool causal;
    // How many keys row i sees.
    __device__ __forceinline__ int limit(int i) const { return causal ? max(0, min(nk, nk - nq + i + 1)) : nk; }
};

__device__ __forceinline__ Sequence sequence(const PromptArgs &a, int s)
{
    Sequence r;
    r.q0 = min(max(a.cu_q[s], 0), a.Tq);
    r.nq = min(max(a.cu_q[s + 1], r.q0), a.Tq) - r.q0;
    r.k0 = min(max(a.cu_k[s], 0), a.Tk);
    r.nk = min(max(a.cu_k[s + 1], r.k0), a.Tk) - r.k0;
    r.causal = a.causal;
    return r;
}

__device__ __forceinline__ int decode_length(const DecodeArgs &a, int b)
{
    return min(max(a.lens[b], 0), a.W << a.page_log2);
}

// Where one row's keys are, for attend_row: packed rows of a head, ...
template <class T>
struct PackedRow {
    const T *k, *v;  // key 0
    int64_t k_tok, v_tok;
    __device__ __forceinline__ bool operator()(int j, const T *&kj, const T *&vj) const
    {
        kj = k + j * k_tok;
        vj = v + j * v_tok;
        return true;
    }
};
// ... or pages.
template <class T>
struct PagedRow {
    PagesView k, v;  // of the head
    const int32_t *table, *shared_table;
    int shared_pages, lg, P;
    __device__ __forceinline__ bool operator()(int j, const T *&kj, const T *&vj) const
    {
        const int e = j >> lg, o = j - (e << lg), page = (e < shared_pages ? shared_table : table)[e];
        if (page < 0 || page >= P) return false;
        kj = (const T *)k.data + page * k.page + o * k.tok;
        vj = (const T *)v.data + page * v.page + o * v.tok;
        return true;
    }
};

// One row as it is written, by one wave: a lane scores a key, 64 at a time;
// FP32 throughout.  What a row does not see is never multiplied, so it serves
// the rows whose result is not finite (matrix instructions multiply masked
// values by a weight of 0, which NaN and infinities survive), and pools
// without pages.  `key` gives the addresses of a key and its value, or false
// where they cannot be read.  Not inlined: it is rare, and would cost the
// kernels that call it registers.
template <class T, class Key>
__device__ __attribute__((noinline)) void attend_row(const float *q, int D, int n, float scale, Key key, float *out)
{
    constexpr int kPer = kAttnMaxDim / 64;
    const int lane = threadIdx.x & 63;
    float m = -INFINITY, l = 0.0f, o[kPer] = {};
    for (int64_t j0 = 0; j0 < n; j0 += 64) {
        const int64_t j = j0 + lane;
        const T *k = nullptr, *v = nullptr;
        float s = -INFINITY;
        if (j < n) {
            s = NAN;
            if (key((int)j, k, v)) {
                s = 0.0f;
                for (int d = 0; d < D; ++d) s = fmaf(q[d], (float)k[d], s);
                s *= scale;
            }
        }
        float mx = s;
#pragma unroll
        for (int x = 32; x; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x));
        const float mn = __any(s != s) ? NAN : fmaxf(m, mx);
        const float c = m == -INFINITY ? 0.0f : exp2f((m - mn) * kLog2e);
        const float p = s == -INFINITY ? 0.0f : exp2f((s - mn) * kLog2e);
        float t = p;
#pragma unroll
        for (int x = 32; x; x >>= 1) t += __shfl_xor(t, x);
        l = l * c + t;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] *= c;
        m = mn;
        for (int u = 0; u < 64 && j0 + u < n; ++u) {
            const float pu = __shfl(p, u);
            const T *vu = (const T *)__shfl((unsigned long long)v, u);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 64 * i < D) o[i] = vu ? fmaf(pu, (float)vu[lane + 64 * i], o[i]) : NAN;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (lane + 64 * i < D) out[lane + 64 * i] = l == 0.0f ? 0.0f : o[i] / l;
}

// Row i of a packed sequence, and sequence b's row, of head h.
template <class T>
__device__ __forceinline__ void attend_prompt_row(const PromptArgs &a, const Sequence &sq, int i, int h)
{
    const int kh = h / (a.Hq / a.Hkv);
    const int64_t t = sq.q0 + i;
    attend_row<T>((const float *)a.q.data + t * a.q.tok + h * a.q.head, a.D, sq.limit(i), a.scale,
                  PackedRow<T>{(const T *)a.k.data + sq.k0 * a.k.tok + kh * a.k.head,
                               (const T *)a.v.data + sq.k0 * a.v.tok + kh * a.v.head, a.k.tok, a.v.tok},
                  a.out + t * a.out_tok + h * a.out_head);
}

template <class T>
__device__ __forceinline__ void attend_decode_row(const DecodeArgs &a, int64_t b, int h)
{
    const int kh = h / (a.Hq / a.Hkv);
    PagedRow<T> key = {a.k, a.v, a.table + b * a.ld_table, a.table, a.shared_pages, a.page_log2, a.P};
    key.k.data = (T *)a.k.data + kh * a.k.head;
    key.v.data = (T *)a.v.data + kh * a.v.head;
    attend_row<T>(a.q + b * a.q_seq + h * a.q_head, a.D, decode_length(a, (int)b), a.scale, key,
                  a.out + b * a.out_seq + h * a.out_head);
}

// N values of a row of D from p + d on, zeros from D on.  WIDE: p is a
// multiple of 16 bytes, d, N and D of 4.
template <int N, bool WIDE>
__device__ __forceinline__ void load_floats(const float *p, int d, int D, float (&x)[N])
{
    if (WIDE) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const floatx4_t t = *reinterpret_cast<const floatx4_t *>(p + (d + e < D ? d + e : 0));
#pragma unroll
            for (int u = 0; u < 4; ++u) x[e + u] = d + e < D ? t[u] : 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float t = p[d + e < D ? d + e : 0];
            x[e] = d + e < D ? t : 0.0f;
        }
    }
}

__device__ __forceinline__ bool rows_wide(const void *p, int64_t strides, int D)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(strides * 4)) & 15) == 0 && D % 4 == 0;
}

// The power of two that brings `mx` (the largest magnitude of a group, >= 0)
// to [2^14, 2^15), the top of FP16's range; 0 for zero.
__device__ __forceinline__ int top_shift(float mx)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, mx);
    if (u == 0 || u >= 0x7F800000u) return 0;
    return 14 - (__builtin_amdgcn_frexp_expf(mx) - 1);
}

// x scaled by 2^e as two FP16 parts with 22 significant bits together (at the
// same scale: hi is below 2^15, so lo keeps its bits down to 2^-24).
__device__ __forceinline__ void split_scaled(float x, int e, _Float16 &hi, _Float16 &lo)
{
    const float y = __builtin_amdgcn_ldexpf(x, e);
    hi = (_Float16)y;
    lo = (_Float16)(y - (float)hi);
}

}  // namespace cfp32
