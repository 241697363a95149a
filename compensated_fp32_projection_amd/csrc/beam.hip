// Beam search (include/cfp32.h: cfp32_beam_select, cfp32_beam_reorder).
//
// A beam's offers are ordered as its logits are, so the n best of a sequence are
// among the n largest logits of each beam.  One launch passes over the logits:
// a wave takes 512 or 2048 of a row, holds them in registers, and leaves
//   * the sum of exp(x - c), c next to the largest of its logits, and c;
//   * its n largest logits with their tokens, in order.  The n-th largest of
//     the lanes' own largest is a lower bound of the n-th largest of all, so
//     few logits but the wanted ones reach the sort.
// The second launch, a block to a sequence, joins a row's sums and lists, a wave
// to a beam, and merges the beams' lists.  The logits are read once; that
// bounds the first launch (256 x 128000 27 us, 4.8 TB/s), latency the second (10 us
// for 8 beams of 63 lists, 6.5 for 4 of them).
#include <cfloat>

#include "beam.h"
#include "device_common.h"
#include "lanes.h"

namespace cfp32 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// A logit and its token as one number: larger logits first, of equal ones the
// lower token.  0: none.
__device__ __forceinline__ uint64_t offer_key(float x, int token)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // one zero
    const uint32_t o = b >> 31 ? ~b : b | 0x80000000u;
    return (uint64_t)o << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float key_logit(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __builtin_bit_cast(float, o >> 31 ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

// A wave's values, sorted by a bitonic network whose exchanges stay out of LDS
// (they took a third of the join's time there).
template <int J, class V>
__device__ __forceinline__ V exchange(V v, bool keep_larger)
{
    const V o = from_lane<J>(v);
    return (v > o) == keep_larger ? v : o;
}
template <int J, class V>
__device__ __forceinline__ V merge_steps(V v, bool down)
{
    const int lane = threadIdx.x & 63;
    v = exchange<J>(v, ((lane & J) == 0) == down);
    if constexpr (J > 1) return merge_steps<J / 2>(v, down);
    else return v;
}
template <int K, class V>
__device__ __forceinline__ V sort_steps(V v)
{
    if constexpr (K > 2) v = sort_steps<K / 2>(v);
    return merge_steps<K / 2>(v, (threadIdx.x & K & 63) == 0);
}

// In order, the largest in lane 0.
template <class V>
__device__ __forceinline__ V sort_wave(V v) { return sort_steps<64>(v); }

// The 64 largest of two wave's lists that are in order, in order.
__device__ __forceinline__ uint64_t merge_wave(uint64_t a, uint64_t b)
{
    const uint64_t r = __shfl_xor(b, 63);
    return merge_steps<32>(a > r ? a : r, true);
}

// A wave's sum, and its maximum.
template <class V>
__device__ __forceinline__ V wave_sum(V v)
{
    v += from_lane<1>(v);
    v += from_lane<2>(v);
    v += from_lane<4>(v);
    v += from_lane<8>(v);
    v += from_lane<16>(v);
    return v + from_lane<32>(v);
}
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, from_lane<1>(v));
    v = fmaxf(v, from_lane<2>(v));
    v = fmaxf(v, from_lane<4>(v));
    v = fmaxf(v, from_lane<8>(v));
    return max_of_quads(v);
}

// Terms exp(x) of a sum, relative to a power of two next to the largest.  x log2 e = n + f to the nearest integer n; f is
// formed by two fused multiply-adds, the second with what FP32 leaves of log2 e, so that rounding takes bits off f (2^-26
// each time) and not off x log2 e.  2^f is off by its instruction's last place; two terms are added in FP32, pairs in
// FP64, and their sum becomes FP32: 4.03 x 2^-24 of it in all.  (Rounded products x log2 e and FP32 sums left 2^-19 of a
// row of 2048 logits all but one of which are equal; 256 x 128000 took 25.5 us with them.)
struct Terms {
    static constexpr float kRound = 0x1.8p23f;  // what is added to it loses its fraction
    float least, round;
    // Of x up to `top` (below 2^20 in magnitude), 2^power being the unit.
    __device__ __forceinline__ Terms(float top, float power) : least(top - 80.0f), round(kRound - power) {}
    // x as two factors: 2^f, and the power of two.  Below `least` the power stays, and 2^f goes on to 0.
    __device__ __forceinline__ void factors(float x, float &p, float &s) const
    {
        constexpr float kRest = 1.9259629911e-8f;  // log2 e - kLog2e
        // Not fmaxf, or the median with infinity, which take two instructions (256 x 128000 27.2 -> 28 us).
        const float up = __builtin_amdgcn_fmed3f(x, least, 0x1p20f);
        const float r = fmaf(up, kLog2e, round), n = r - round;
        p = __builtin_amdgcn_exp2f(fmaf(x, kRest, fmaf(x, kLog2e, -n)));
        s = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, r) << 23) + 0x3F800000u);
    }
    __device__ __forceinline__ float two(float x, float y) const
    {
        float p, q, s, t;
        factors(x, p, s);
        factors(y, q, t);
        return fmaf(q, t, p * s);
    }
};

// The largest keys seen by a wave, in order, and those that wait to be sorted
// into them (in LDS, of this wave alone).
struct Best {
    uint64_t top;       // lane i: the i-th largest
    uint64_t *waiting;  // [128]
    int count;
    bool any;
    __device__ __forceinline__ void sync() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }
    // `mine`: this lane's key is to be taken.  All lanes call.
    __device__ __forceinline__ void add(bool mine, uint64_t key)
    {
        const uint64_t mask = __ballot(mine);
        if (!mask) return;
        const int lane = threadIdx.x & 63;
        if (mine) waiting[count + __popcll(mask & (((uint64_t)1 << lane) - 1))] = key;
        count += __popcll(mask);
        if (count >= 64) flush();
    }
    __device__ __forceinline__ void flush()
    {
        const int lane = threadIdx.x & 63;
        sync();
        const uint64_t k = sort_wave(lane < count ? waiting[lane] : (uint64_t)0);
        top = any ? merge_wave(top, k) : k;
        any = true;
        const uint64_t rest = waiting[64 + lane];
        sync();
        count = count > 64 ? count - 64 : 0;
        if (lane < count) waiting[lane] = rest;
    }
};

// E logits of a lane, VEC at a time (4: rows allow loads of 16 bytes).
template <int E, int VEC>
__global__ __launch_bounds__(256) void beam_rows_kernel(BeamArgs a, int chunks, float2 *stats, uint64_t *lists)
{
    __shared__ uint64_t waiting[4][128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave, row = unit / chunks;
    const int chunk = (int)(unit - row * chunks);
    if (row >= (int64_t)a.S * a.beams) return;
    if (a.done && a.done[row]) return;
    const float score = a.scores[row];
    if (!(fabsf(score) < INFINITY)) return;

    // Which logits a lane takes does not depend on where the row lies, so equal
    // rows have equal sums, and equal offers stay equal.
    const float *x0 = a.logits + row * a.ld;
    auto token = [&](int e) { return (int64_t)chunk * (64 * E) + (64 * (e / VEC) + lane) * VEC + e % VEC; };
    float x[E];
#pragma unroll
    for (int e = 0; e < E; e += VEC) {
        const int64_t t = token(e);
        if (VEC == 4 && t + 4 <= a.V) {
            const floatx4_t w = *reinterpret_cast<const floatx4_t *>(x0 + t);
#pragma unroll
            for (int u = 0; u < VEC; ++u) x[e + u] = w[u];
        } else {
#pragma unroll
            for (int u = 0; u < VEC; ++u) x[e + u] = t + u < a.V ? x0[t + u] : -INFINITY;
        }
    }
    float mine = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) mine = fmaxf(mine, x[e]);
    const float sorted = sort_wave(mine);
    const float most = __shfl(sorted, 0), least = __shfl(sorted, a.n - 1);
    const float bar = fmaxf(least, -FLT_MAX);  // -infinity is not offered
    Best best = {0, waiting[wave], 0, false};
#pragma unroll
    for (int e = 0; e < E; ++e) best.add(x[e] >= bar, offer_key(x[e], (int)token(e)));
    if (best.count) best.flush();
    if (lane < a.n) lists[unit * a.n + lane] = best.top;

    // A NaN, or infinity less itself, leaves a sum of NaN; of nothing but -infinity (and no NaN) it is 0.
    if (most == -INFINITY) {
        float odd = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) odd = x[e] != x[e] ? NAN : odd;
        if (lane == 0) stats[unit] = make_float2(most, __any(odd != odd) ? NAN : 0.0f);
        return;
    }
    // Far from 0 only differences from the largest have a fraction to be kept, and those that count are exact.
    const bool far = fabsf(most) >= 1024.0f;
    if (far) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] -= most;
    }
    const float power = far ? 0.0f : rintf(most * kLog2e);
    const Terms terms(far ? 0.0f : most, power);
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < E; e += 2) sum += (double)terms.two(x[e], x[e + 1]);
    sum = wave_sum(sum);
    // The unit, 2^power, as e to the power of an FP32 number and a factor next to 1.
    const double unit_log = (double)power * 0.693147180559945309417232;
    const float from = far ? most : (float)unit_log;
    const double rest = far ? 0.0 : unit_log - (double)from;
    if (lane == 0) stats[unit] = make_float2(from, (float)(sum * (1.0 + rest * (1.0 + 0.5 * rest))));
}

// An offer of a beam: larger totals first, of equal ones the lower place (beam,
// then the order of its logits).
struct Offer {
    double total;
    uint32_t place;
    __device__ __forceinline__ bool operator>(const Offer &o) const { return total > o.total || (total == o.total && place < o.place); }
};
template <int J>
__device__ __forceinline__ Offer from_lane(Offer v) { return {cfp32::from_lane<J>(v.total), cfp32::from_lane<J>(v.place)}; }

template <int J>
__device__ __forceinline__ Offer best_offer(Offer v)
{
    const Offer o = from_lane<J>(v);
    if (o > v) v = o;
    if constexpr (J > 1) return best_offer<J / 2>(v);
    else return v;
}

__global__ __launch_bounds__(1024) void beam_join_kernel(BeamArgs a, int chunks, const float2 *stats, const uint64_t *lists)
{
    constexpr int kKeys = 8;                          // of a lane at a time
    extern __shared__ double totals[];                // [beams][n]
    int *tokens = (int *)(totals + a.beams * a.n);    // [beams][n]
    __shared__ uint64_t waiting[16][128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int64_t s = blockIdx.x;
    for (int b = wave; b < a.beams; b += waves) {
        const int64_t row = s * a.beams + b;
        const float score = a.scores[row];
        const bool done = a.done && a.done[row];
        double total = -INFINITY;
        int token = -1;
        if (!(fabsf(score) < INFINITY)) {
        } else if (done) {
            if (lane == 0) {
                total = score;
                token = a.eos;
            }
        } else {
            // The n largest of the row's lists, as of its logits.
            Best best = {0, waiting[wave], 0, false};
            const uint64_t *keys = lists + row * chunks * a.n;
            const int64_t count = (int64_t)chunks * a.n;
            const float2 *st = stats + row * chunks;
            const float2 first = lane < chunks ? st[lane] : make_float2(-INFINITY, 0.0f);
            for (int64_t i0 = 0; i0 < count; i0 += 64 * kKeys) {
                uint64_t k[kKeys], mine = 0;
#pragma unroll
                for (int e = 0; e < kKeys; ++e) {
                    const int64_t i = i0 + 64 * e + lane;
                    k[e] = i < count ? keys[i] : 0;
                }
#pragma unroll
                for (int e = 0; e < kKeys; ++e) mine = k[e] > mine ? k[e] : mine;
                uint64_t least = __shfl(sort_wave(mine), a.n - 1);
                if (best.any) {
                    const uint64_t have = __shfl(best.top, a.n - 1);
                    least = have > least ? have : least;
                }
#pragma unroll
                for (int e = 0; e < kKeys; ++e) best.add(k[e] >= least && k[e], k[e]);
                if (best.count) best.flush();
            }
            float most = first.x;
            for (int i = lane + 64; i < chunks; i += 64) most = fmaxf(most, st[i].x);
            most = wave_max(most);
            double sum = first.y != 0.0f ? (double)first.y * exp((double)first.x - (double)most) : 0.0;
            for (int i = lane + 64; i < chunks; i += 64) {
                const float2 c = st[i];
                if (c.y != 0.0f) sum += (double)c.y * exp((double)c.x - (double)most);
            }
            sum = wave_sum(sum);
            if (sum > 0.0 && sum < INFINITY && lane < a.n && best.any && best.top) {
                const double lse = (double)most + log(sum);
                total = (double)score + ((double)key_logit(best.top) - lse);
                token = key_token(best.top);
            }
        }
        if (lane < a.n) {
            totals[b * a.n + lane] = total;
            tokens[b * a.n + lane] = token;
        }
    }
    __syncthreads();
    if (wave) return;
    auto put = [&](int i, const Offer &o) {
        const int64_t out = s * a.n + i;
        const bool some = o.total > -INFINITY;
        const int b = some ? (int)(o.place / (uint32_t)a.n) : 0, token = some ? tokens[o.place] : a.eos;
        const int64_t row = s * a.beams + b;
        a.parents[out] = some ? (int)row : -1;
        a.tokens[out] = token;
        a.scores_out[out] = (float)o.total;
        if (a.done_out) a.done_out[out] = !some || (a.done && a.done[row]) || (a.eos >= 0 && token == a.eos);
    };
    const int count = a.beams * a.n;
    if (count <= 64) {
        const Offer o = sort_wave(Offer{lane < count ? totals[lane] : -INFINITY, (uint32_t)lane});
        if (lane < a.n) put(lane, o);
        return;
    }
    // Lane b holds the best offer of beam b that is left.
    int at = 0;
    for (int i = 0; i < a.n; ++i) {
        const uint32_t place = lane * a.n + at;
        const Offer o = best_offer<32>(Offer{lane < a.beams && at < a.n ? totals[place] : -INFINITY, place});
        if (lane == 0) put(i, o);
        at += o.place == place;
    }
}

template <class V>
__global__ __launch_bounds__(256) void beam_reorder_kernel(const char *states, int64_t stride, char *out, int64_t out_stride,
                                                           const int32_t *parents, int rows, int n, int64_t vecs)
{
    const int64_t total = n * vecs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / vecs, c = i - r * vecs;
        const int p = parents[r];
        V v = {};
        if (p >= 0 && p < rows) v = *reinterpret_cast<const V *>(states + p * stride + c * (int64_t)sizeof(V));
        *reinterpret_cast<V *>(out + r * out_stride + c * (int64_t)sizeof(V)) = v;
    }
}

}  // namespace

hipError_t launch_beam_select(const BeamArgs &a, void *workspace, hipStream_t stream)
{
    const BeamPlan p = plan_beam(a.S, a.beams, a.V, a.n);
    const int64_t units = (int64_t)a.S * a.beams * p.chunks, blocks = (units + 3) / 4;
    const int waves = a.beams < 16 ? a.beams : 16;
    if (blocks > 0x7FFFFFFF || blocks * 256 > 0xFFFFFFFF || (int64_t)a.S * 64 * waves > 0xFFFFFFFF) return hipErrorInvalidConfiguration;
    float2 *stats = (float2 *)workspace;
    uint64_t *lists = (uint64_t *)(stats + units);
    const bool wide = ((reinterpret_cast<uintptr_t>(a.logits) | (uintptr_t)(a.ld * 4)) & 15) == 0;
#define CFP32_BEAM_ROWS(E, VEC) beam_rows_kernel<E, VEC><<<(unsigned)blocks, 256, 0, stream>>>(a, p.chunks, stats, lists)
    if (p.each == 32) {
        if (wide) CFP32_BEAM_ROWS(32, 4);
        else CFP32_BEAM_ROWS(32, 1);
    } else {
        if (wide) CFP32_BEAM_ROWS(8, 4);
        else CFP32_BEAM_ROWS(8, 1);
    }
#undef CFP32_BEAM_ROWS
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t lds = (size_t)a.beams * a.n * (sizeof(double) + sizeof(int));
    beam_join_kernel<<<(unsigned)a.S, 64 * waves, lds, stream>>>(a, p.chunks, stats, lists);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const void *states, int64_t stride, void *out, int64_t out_stride, const int32_t *parents,
                               int rows, int n, int64_t row_bytes, hipStream_t stream)
{
    typedef uint32_t vec4_t __attribute__((ext_vector_type(4)));
    const int64_t m = 16 | row_bytes | stride | out_stride | (int64_t)((uintptr_t)states | (uintptr_t)out);
    const int vec = (int)(m & -m);
    const int64_t vecs = row_bytes / vec, blocks = (n * vecs + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 16384 ? blocks : 16384);
#define CFP32_REORDER(V) \
    beam_reorder_kernel<V><<<grid, 256, 0, stream>>>((const char *)states, stride, (char *)out, out_stride, parents, rows, n, vecs)
    switch (vec) {
    case 16: CFP32_REORDER(vec4_t); break;
    case 8: CFP32_REORDER(uint64_t); break;
    case 4: CFP32_REORDER(uint32_t); break;
    case 2: CFP32_REORDER(uint16_t); break;
    default: CFP32_REORDER(uint8_t); break;
    }
#undef CFP32_REORDER
    return hipGetLastError();
}

}  // namespace cfp32
