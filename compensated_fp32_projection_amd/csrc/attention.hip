// Launches of the attention calls (as attention_plans.hip has them): the
// kernels of few rows (attention_rows.h), and the joining of parts.
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

// Row (i, h) of a call: where its result goes (null: it is no row of a sequence), and its slow form.
__device__ __forceinline__ float *row_out(const DecodeArgs &a, int64_t i, int h) { return a.out + i * a.out_seq + h * a.out_head; }
template <class T>
__device__ __forceinline__ void redo_row(const DecodeArgs &a, int64_t i, int h) { attend_decode_row<T>(a, i, h); }
__device__ __forceinline__ bool prompt_row(const PromptArgs &a, int64_t i, Sequence &sq)
{
    const int lo = find_last(a.S, i, [&](int s) { return (int64_t)a.cu_q[s]; });
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
        // Nothing was written where li is 0; what is has to be read also where
        // f is 0, for the NaN of an infinite value.
        uint64_t used = __ballot(li != 0.0f);
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
    bool odd = !(fabsf(l) < INFINITY) || l == 0.0f;
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

template <class Args>
hipError_t join(const Args &a, const Partials &from, int64_t rows, hipStream_t stream)
{
    const bool four = from.slots > kJoinByWave;
    const unsigned blocks = (unsigned)join_blocks(from, rows);
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
    return e != hipSuccess || !p.to.o ? e : join(a, p.to, (int64_t)a.Tq * a.Hq, stream);
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
    return e != hipSuccess || !p.parts.to.o ? e : join(a, p.parts.to, (int64_t)a.B * a.Hq, stream);
}

}  // namespace cfp32
