// Launches of the attention calls (as attention_plans.hip has them): the
// kernels of few rows (attention_rows.h), and the joining of parts.
#include "attention_join.h"
#include "attention_rows.h"

namespace cfp32 {

namespace {

template <class T, int DP, bool WIDE, int NW>
__global__ __launch_bounds__(64 * NW, 2) void prompt_rows_kernel(PromptArgs a, Partials to)
{
    __shared__ float sums[NW][kRows * (DP + 4)], maxima[NW * kRows], weights[NW * kRows];
    __shared__ int unfinished[kRows];
    Joined<DP, NW> sh;
#pragma unroll
    for (int w = 0; w < NW; ++w) sh.o[w] = (CFP32_LDS float *)sums[w];
    sh.m = (CFP32_LDS float *)maxima;
    sh.l = (CFP32_LDS float *)weights;
    sh.unfinished = (CFP32_LDS int *)unfinished;
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
    leave_row<false>(sh, to, ((int64_t)(sq.q0 + ri) * a.Hq + rh) * to.slots + part,
                  a.out + (sq.q0 + ri) * a.out_tok + rh * a.out_head, a.D, row < live);
    if (to.o) return;
    __syncthreads();
    for (int w = threadIdx.x >> 6; w < live; w += NW)
        if (sh.unfinished[w]) {
            const int wi = (int)over(r0 + w, g);
            attend_prompt_row<T>(a, sq, wi, kh * g + (int)(r0 + w - (int64_t)wi * g));
        }
}

template <class T, int DP, bool WIDE, int NW>
__global__ __launch_bounds__(64 * NW, 2) void decode_rows_kernel(DecodeArgs a, DecodeParts c)
{
    __shared__ float sums[NW][kRows * (DP + 4)], maxima[NW * kRows], weights[NW * kRows];
    __shared__ int unfinished[kRows];
    Joined<DP, NW> sh;
#pragma unroll
    for (int w = 0; w < NW; ++w) sh.o[w] = (CFP32_LDS float *)sums[w];
    sh.m = (CFP32_LDS float *)maxima;
    sh.l = (CFP32_LDS float *)weights;
    sh.unfinished = (CFP32_LDS int *)unfinished;
    decode_rows<T, DP, WIDE, NW, false>(a, c, blockIdx.x, blockIdx.y, sh);
}

// A call's rows for the join: where their results go, and their slow form.
template <class T>
struct DecodeRows {
    DecodeArgs a;
    __device__ __forceinline__ int Hq() const { return a.Hq; }
    __device__ __forceinline__ int D() const { return a.D; }
    __device__ __forceinline__ float *out(int64_t i, int h) const { return a.out + i * a.out_seq + h * a.out_head; }
    __device__ __forceinline__ void finish(int64_t i, int h) const { attend_decode_row<T>(a, i, h); }
};
template <class T>
struct PromptRows {
    PromptArgs a;
    __device__ __forceinline__ int Hq() const { return a.Hq; }
    __device__ __forceinline__ int D() const { return a.D; }
    __device__ __forceinline__ bool row(int64_t i, Sequence &sq) const
    {
        const int lo = find_last(a.S, i, [&](int s) { return (int64_t)a.cu_q[s]; });
        sq = sequence(a, lo);
        return i >= sq.q0 && i < sq.q0 + sq.nq;
    }
    __device__ __forceinline__ float *out(int64_t i, int h) const
    {
        Sequence sq;
        return row(i, sq) ? a.out + i * a.out_tok + h * a.out_head : nullptr;
    }
    __device__ __forceinline__ void finish(int64_t i, int h) const
    {
        Sequence sq;
        if (row(i, sq)) attend_prompt_row<T>(a, sq, (int)i - sq.q0, h);
    }
};

// Rows against a pool without pages: 0, or NaN where a sequence has tokens.
__global__ __launch_bounds__(64) void decode_no_pages_kernel(DecodeArgs a)
{
    for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x)
        for (int h = blockIdx.y; h < a.Hq; h += gridDim.y) attend_decode_row<float>(a, b, h);
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

namespace {

template <template <class> class Rows, class Args>
hipError_t join(const Args &a, const Partials &from, int64_t rows, hipStream_t stream)
{
    return a.kv_f16 ? launch_join(Rows<_Float16>{a}, from, rows, stream) : launch_join(Rows<float>{a}, from, rows, stream);
}

}  // namespace

hipError_t launch_attention_prompt(const PromptArgs &a, void *workspace, hipStream_t stream)
{
    const PromptPlan p = plan_prompt(a, workspace);
    if (p.error != hipSuccess) return p.error;
    hipError_t e;
    if (p.tiles) {
        e = launch_prompt_tile(a, p, stream);
    } else {
        const dim3 grid((unsigned)p.blocks, (unsigned)p.to.slots);
        CFP32_BY_TYPE(prompt_rows_kernel, a.kv_f16, a.D, p.wide, p.eight, grid, a, p.to);
        e = hipGetLastError();
    }
    return e != hipSuccess || !p.to.o ? e : join<PromptRows>(a, p.to, (int64_t)a.Tq * a.Hq, stream);
}

hipError_t launch_attention_decode(const DecodeArgs &a, void *workspace, hipStream_t stream)
{
    const DecodePlan p = plan_decode(a, workspace);
    if (p.error != hipSuccess) return p.error;
    if (a.P == 0) {
        const dim3 grid((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)(a.Hq < 65535 ? a.Hq : 65535));
        decode_no_pages_kernel<<<grid, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    hipError_t e;
    if (p.parts.tiles) {
        e = launch_decode_tile(a, p, stream);
    } else {
        const dim3 grid((unsigned)p.blocks, (unsigned)a.Hkv);
        CFP32_BY_TYPE(decode_rows_kernel, a.kv_f16, a.D, p.wide, p.parts.eight, grid, a, p.parts);
        e = hipGetLastError();
    }
    return e != hipSuccess || !p.parts.to.o ? e : join<DecodeRows>(a, p.parts.to, (int64_t)a.B * a.Hq, stream);
}

}  // namespace cfp32
