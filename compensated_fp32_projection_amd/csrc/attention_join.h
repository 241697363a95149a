// Rows that several blocks have worked on, joined (a launch of its own).
#pragma once

#include "attention_device.h"

namespace cfp32 {

namespace {

// Rows from their parts.  WAVES: of a row, each taking every WAVES-th part,
// their sums joined in LDS.  Few parts: a wave to a row (a block to a row made
// 9600 rows of 2 parts cost 15 us).  Many: four (a wave to a row took 10 us
// for 1024 rows of 68 parts x 128, for want of loads in flight; now 6).
// Rows: Hq and D of the call, out(i, h), where the result of row (i, h) goes (null:
// it is no row of a sequence), and finish(i, h), for a result that is not finite
// or a row without weight.
template <int DP, int WAVES, class Rows>
__global__ __launch_bounds__(256) void join_kernel(Rows a, Partials from, int64_t rows)
{
    constexpr int E = DP / 64;
    __shared__ float sums[4][DP], weight[4];
    const int lane = threadIdx.x & 63, w4 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = w4 % WAVES;
    const int64_t row = min((int64_t)blockIdx.x * (4 / WAVES) + w4 / WAVES, rows - 1), b = row / a.Hq();
    const int h = (int)(row - b * a.Hq());
    float *out = a.out(b, h);
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
        if (lane * E + e < a.D()) {
            out[lane * E + e] = y;
            odd |= !(fabsf(y) < INFINITY);
        }
    }
    if (__any(odd)) a.finish(b, h);
}

template <class Rows>
hipError_t launch_join(const Rows &a, const Partials &from, int64_t rows, hipStream_t stream)
{
    const bool four = from.slots > kJoinByWave;
    const unsigned blocks = (unsigned)join_blocks(from, rows);
    if (from.dim == 64) {
        if (four) join_kernel<64, 4><<<blocks, 256, 0, stream>>>(a, from, rows);
        else join_kernel<64, 1><<<blocks, 256, 0, stream>>>(a, from, rows);
    } else {
        if (four) join_kernel<128, 4><<<blocks, 256, 0, stream>>>(a, from, rows);
        else join_kernel<128, 1><<<blocks, 256, 0, stream>>>(a, from, rows);
    }
    return hipGetLastError();
}

}  // namespace

}  // namespace cfp32
