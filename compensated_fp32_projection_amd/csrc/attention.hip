// Attention over packed prompts and against the paged cache, as written: one
// wave per query row and head, 64 keys at a time (a lane scores one key),
// FP32 throughout, one pass with the running maximum and sum of the softmax.
#include "attention.h"

namespace cfp32 {

namespace {

constexpr int kDimsPerLane = kAttnMaxDim / 64;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// out[0, D) = softmax(scale q . k_j) v_j over keys j < n; key(j, k, v) gives
// a key's and a value's addresses, or false where they cannot be read.
template <class T, class Key>
__device__ void attend_row(const float *q, int D, int n, float scale, float *qs, Key key, float *out)
{
    const int lane = threadIdx.x & 63;
    for (int d = lane; d < D; d += 64) qs[d] = q[d];
    __syncthreads();  // one wave to a block
    float m = -INFINITY, l = 0.0f, o[kDimsPerLane] = {};
    for (int j0 = 0; j0 < n; j0 += 64) {
        const int j = j0 + lane;
        const T *k = nullptr, *v = nullptr;
        float s = -INFINITY;
        if (j < n) {
            s = NAN;
            if (key(j, k, v)) {
                s = 0.0f;
                for (int d = 0; d < D; ++d) s = fmaf(qs[d], (float)k[d], s);
                s *= scale;
            }
        }
        const bool bad = __any(s != s);
        const float mn = bad ? NAN : fmaxf(m, wave_max(s));
        const float c = m == -INFINITY ? 0.0f : exp2f((m - mn) * kLog2e);
        const float p = s == -INFINITY ? 0.0f : exp2f((s - mn) * kLog2e);
        l = l * c + wave_sum(p);
#pragma unroll
        for (int i = 0; i < kDimsPerLane; ++i) o[i] *= c;
        m = mn;
        for (int t = 0; t < 64 && j0 + t < n; ++t) {
            const float pt = __shfl(p, t);
            const T *vt = (const T *)__shfl((unsigned long long)v, t);
#pragma unroll
            for (int i = 0; i < kDimsPerLane; ++i)
                if (lane + 64 * i < D) o[i] = vt ? fmaf(pt, (float)vt[lane + 64 * i], o[i]) : NAN;
        }
    }
#pragma unroll
    for (int i = 0; i < kDimsPerLane; ++i)
        if (lane + 64 * i < D) out[lane + 64 * i] = l == 0.0f ? 0.0f : o[i] / l;
}

template <class T>
__global__ __launch_bounds__(64) void prompt_kernel(PromptArgs a)
{
    __shared__ float qs[kAttnMaxDim];
    const int h = blockIdx.y, kh = h / (a.Hq / a.Hkv);
    for (int t = blockIdx.x; t < a.Tq; t += gridDim.x) {
        int lo = 0, hi = a.S;
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (a.cu_q[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1];
        if (t < q0 || t >= q1) continue;
        const int k0 = min(max(a.cu_k[lo], 0), a.Tk), k1 = min(max(a.cu_k[lo + 1], k0), a.Tk);
        int n = k1 - k0;
        if (a.causal) n = max(0, min(n, t - q0 + n - (q1 - q0) + 1));
        __syncthreads();
        attend_row<T>(
            (const float *)a.q.data + t * a.q.tok + h * a.q.head, a.D, n, a.scale, qs,
            [&](int j, const T *&k, const T *&v) {
                k = (const T *)a.k.data + (int64_t)(k0 + j) * a.k.tok + kh * a.k.head;
                v = (const T *)a.v.data + (int64_t)(k0 + j) * a.v.tok + kh * a.v.head;
                return true;
            },
            a.out + t * a.out_tok + h * a.out_head);
    }
}

template <class T>
__global__ __launch_bounds__(64) void decode_kernel(DecodeArgs a)
{
    __shared__ float qs[kAttnMaxDim];
    const int h = blockIdx.y, kh = h / (a.Hq / a.Hkv);
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = min(max(a.lens[b], 0), a.W << a.page_log2);
        __syncthreads();
        attend_row<T>(
            a.q + b * a.q_seq + h * a.q_head, a.D, n, a.scale, qs,
            [&](int j, const T *&k, const T *&v) {
                const int e = j >> a.page_log2, o = j - (e << a.page_log2);
                const int page = a.table[(e < a.shared_pages ? 0 : b) * a.ld_table + e];
                if (page < 0 || page >= a.P) return false;
                k = (const T *)a.k.data + page * a.k.page + kh * a.k.head + o * a.k.tok;
                v = (const T *)a.v.data + page * a.v.page + kh * a.v.head + o * a.v.tok;
                return true;
            },
            a.out + b * a.out_seq + h * a.out_head);
    }
}

}  // namespace

size_t attention_prompt_workspace(int64_t, int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_attention_prompt(const PromptArgs &a, void *, hipStream_t stream)
{
    if (a.Hq > 65535) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(a.Tq < 65536 ? a.Tq : 65536), (unsigned)a.Hq);
    if (a.kv_f16) prompt_kernel<_Float16><<<grid, 64, 0, stream>>>(a);
    else prompt_kernel<float><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

size_t attention_decode_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int, int64_t, bool) { return 0; }

hipError_t launch_attention_decode(const DecodeArgs &a, void *, hipStream_t stream)
{
    if (a.Hq > 65535) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)a.Hq);
    if (a.kv_f16) decode_kernel<_Float16><<<grid, 64, 0, stream>>>(a);
    else decode_kernel<float><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace cfp32
