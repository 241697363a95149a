// Rotary positions of q and k (include/cfp32.h: cfp32_rotary).
//
// Pair i of a token at position p turns by the angle p f_i, the same in every
// head.  A block takes some tokens: it makes their sines and cosines once,
// into LDS, and then passes over all of their heads.  What bounds it is the
// memory: each value is read and written once (8192 x 32/8 x 128 FP32 62 us, 5.4
// TB/s; 64 tokens of these 4 us, mostly a position's, a value's and the launch's
// latency).
//
// Angles: p f_i / 2 pi in FP64 is reduced to a quarter turn there, since the
// whole turns of a far position leave FP32 nothing (2^20 positions of 1 radian
// are off by 0.03 in it); the remainder, within an eighth of a turn, is FP32
// with 2^-25 radians at most lost, and goes through the Taylor polynomials of sine and
// cosine (terms to x^9 and x^10: 1.8e-9 left at pi / 4).
#include "device_common.h"
#include "rotary.h"

namespace cfp32 {

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559, kPerTurn = 1.0 / kTwoPi;

// Sine and cosine of `turns` whole turns.
__device__ __forceinline__ void sincos_turns(double turns, float &s, float &c)
{
    const double q = rint(turns * 4.0);                       // quarters; huge and NaN turns give NaN below
    const float x = (float)((turns - q * 0.25) * kTwoPi), z = x * x;
    const float sn = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
    const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const int n = (int)(q - 4.0 * floor(q * 0.25)) & 3;
    s = n & 1 ? cs : sn;
    c = n & 1 ? sn : cs;
    if (n & 2) s = -s;
    if (n == 1 || n == 2) c = -c;
}

// VEC consecutive elements as FP32, one load or store (16 bytes at most).
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *x)
{
    typedef T vec __attribute__((ext_vector_type(VEC)));
    const vec v = *reinterpret_cast<const vec *>(p);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = (float)v[e];
}

template <class T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *x)
{
    typedef T vec __attribute__((ext_vector_type(VEC)));
    vec v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = (T)x[e];
    *reinterpret_cast<vec *>(p) = v;
}

// An item is VEC pairs of a token and head, or, from `turned` on, VEC elements
// that are copied.
template <class T, int VEC, bool INTER>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int tokens, int heads, int turned, int per)
{
    extern __shared__ float table[];  // of each token and pair: cosine, sine
    const int pairs = a.R / 2;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
        const int nt = (int)min((int64_t)tokens, a.T - t0);
        for (int i = threadIdx.x; i < nt * pairs; i += 256) {
            const int t = i / pairs, p = i - t * pairs;
            const double pos = (double)(a.positions ? a.positions[t0 + t] : t0 + t);
            float s, c;
            sincos_turns(pos * (a.frequencies[p] * kPerTurn), s, c);
            table[2 * i] = c * a.amplitude;
            table[2 * i + 1] = (a.transpose ? -s : s) * a.amplitude;
        }
        __syncthreads();
        const int n = nt * heads * per;
        for (int i = threadIdx.x; i < n; i += 256) {
            const int th = i / per, item = i - th * per, t = th / heads, h = th - t * heads;
            const bool second = h >= a.q.heads;
            const RotaryTensor &x = second ? a.k : a.q;
            const int hh = second ? h - a.q.heads : h;
            const T *in = (const T *)x.in + (t0 + t) * x.in_tok + hh * x.in_head;
            T *out = (T *)x.out + (t0 + t) * x.out_tok + hh * x.out_head;
            float u[VEC], v[VEC];
            if (item < turned) {
                const int p = item * VEC;
                if constexpr (INTER) {
                    float w[2 * VEC];
                    load_vec<T, VEC>(in + 2 * p, w);
                    load_vec<T, VEC>(in + 2 * p + VEC, w + VEC);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) u[e] = w[2 * e], v[e] = w[2 * e + 1];
                } else {
                    load_vec<T, VEC>(in + p, u);
                    load_vec<T, VEC>(in + pairs + p, v);
                }
                const float *cs = table + 2 * (t * pairs + p);
                float y[VEC], z[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float c = cs[2 * e], s = cs[2 * e + 1];
                    y[e] = fmaf(u[e], c, -(v[e] * s));
                    z[e] = fmaf(v[e], c, u[e] * s);
                }
                if constexpr (INTER) {
                    float w[2 * VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[2 * e] = y[e], w[2 * e + 1] = z[e];
                    store_vec<T, VEC>(out + 2 * p, w);
                    store_vec<T, VEC>(out + 2 * p + VEC, w + VEC);
                } else {
                    store_vec<T, VEC>(out + p, y);
                    store_vec<T, VEC>(out + pairs + p, z);
                }
            } else {
                float w[VEC];
                const int d = a.R + (item - turned) * VEC;
                load_vec<T, VEC>(in + d, w);
                store_vec<T, VEC>(out + d, w);
            }
        }
        __syncthreads();  // the table is read
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream)
{
    const int heads = a.q.heads + a.k.heads, rest = a.D - a.R;
    // Elements to a load: what divides every address.
    const int64_t size = a.f16 ? 2 : 4;
    int64_t m = 16 / size | a.R / 2 | rest;
    for (const RotaryTensor *x : {&a.q, &a.k})
        if (x->heads) m |= x->in_tok | x->in_head | x->out_tok | x->out_head | ((uintptr_t)x->in | (uintptr_t)x->out) / size;
    const int vec = (int)(m & -m);
    const int turned = a.R / 2 / vec, per = turned + rest / vec;
    // Tokens to a block: some 1024 items, as long as there are blocks enough.
    int tokens = 1024 / (heads * per) < 16 ? 1024 / (heads * per) : 16;
    if (tokens > a.T / 1024) tokens = a.T / 1024;
    if (tokens < 1) tokens = 1;
    const int64_t blocks = ((int64_t)a.T + tokens - 1) / tokens;
    const unsigned grid = (unsigned)(blocks < 65536 ? blocks : 65536);
    const size_t lds = (size_t)tokens * a.R * sizeof(float);
#define CFP32_ROTARY(T, VEC)                                                                                      \
    do {                                                                                                          \
        if (a.interleaved) rotary_kernel<T, VEC, true><<<grid, 256, lds, stream>>>(a, tokens, heads, turned, per); \
        else rotary_kernel<T, VEC, false><<<grid, 256, lds, stream>>>(a, tokens, heads, turned, per);              \
    } while (0)
    if (a.f16) {
        switch (vec) {
        case 8: CFP32_ROTARY(_Float16, 8); break;
        case 4: CFP32_ROTARY(_Float16, 4); break;
        case 2: CFP32_ROTARY(_Float16, 2); break;
        default: CFP32_ROTARY(_Float16, 1); break;
        }
    } else {
        switch (vec) {
        case 4: CFP32_ROTARY(float, 4); break;
        case 2: CFP32_ROTARY(float, 2); break;
        default: CFP32_ROTARY(float, 1); break;
        }
    }
#undef CFP32_ROTARY
    return hipGetLastError();
}

}  // namespace cfp32
