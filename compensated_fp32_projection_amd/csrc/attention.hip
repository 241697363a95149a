// Launches of the attention calls: the kernels of few rows (attention_rows.h),
// the joining of parts, and the choice between these and attention_tile.hip's.
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
    const bool can = a.Tk > 0 && (!a.kv_f16 || (w && a.k.tok < ((int64_t)1 << 25) && a.v.tok < ((int64_t)1 << 25)));
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
// 128 behind 320 / 1280 / 5120 / 20480 keys 22 / 33 / 50 / 117 against 29 / 30 /
// 33 / 45 us; 12 of these behind 1280 / 5120 18 / 35 against 24 / 26; 10 x 16/2
// x 128 behind 5120 / 20480 18 / 34 against 20 / 25; 16 x 14/2 x 64 behind 1280 /
// 5120 / 20480 12 / 16 / 29 against 15 / 16 / 18.
bool prefer_tiles(int64_t rows, int64_t Hkv, int64_t D, int64_t keys)
{
    const double k = 1e-3 * (double)keys * Hkv, groups = (double)ceil_div(rows, kRows), blocks = (double)ceil_div(rows, 128);
    return D <= 64 ? 0.06 * groups * k > 3 + 0.1 * blocks * k : 0.13 * groups * k > 8 + 0.13 * blocks * k;
}

// `tiles`: the pages allow the other kernel.
DecodeParts decode_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages, bool tiles)
{
    DecodeParts c = {};
    const int64_t g = Hq / Hkv, unit = 4 * wave_step(D);
    const int64_t n_shared = B > 1 ? shared_pages << lg : 0, n_own = (W << lg) - n_shared;
    c.shared_groups = (int)ceil_div(B * g, kRows);
    c.own_groups = (int)ceil_div(g, kRows);
    c.own_from = (int)n_shared;
    if (n_shared) {
        if (tiles && prefer_tiles(B * g, Hkv, D, n_shared)) c.tiles = decode_tile_parts(B, Hq, Hkv, n_shared, lg);
        else c.shared = key_parts(n_shared, unit, c.shared_groups * Hkv, kDecodeBlocks);
    }
    if (n_own > 0) c.own = key_parts(n_own, unit, B * c.own_groups * Hkv, kDecodeBlocks);
    // Tiles always leave their rows in slots: beside a single part, an empty one.
    if (c.shared + c.own == 0 && c.tiles <= 1) c.own = 1;
    c.eight = c.tiles == 0 && c.shared == 0 && c.own == 1 && eight_waves(n_own, D);
    c.to.slots = c.tiles + c.shared + c.own;
    c.to.dim = padded(D);
    return c;
}

}  // namespace

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int lg, int64_t shared_pages,
                                  bool kv_f16)
{
    if (Hkv == 0) return 0;
    const size_t a = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, false).to.slots, padded(D));
    if (!kv_f16) return a;
    const size_t b = partial_bytes(B * Hq, decode_parts(B, Hq, Hkv, D, W, lg, shared_pages, true).to.slots, padded(D));
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
    DecodeParts c = decode_parts(a.B, a.Hq, a.Hkv, a.D, a.W, a.page_log2, a.shared_pages, tiles);
    const int64_t rows = (int64_t)a.B * a.Hq;
    const int64_t blocks = (int64_t)c.shared * c.shared_groups + (int64_t)a.B * c.own_groups * c.own;
    if (blocks > 0x7FFFFFFF || rows > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    place_partials(c.to, rows, workspace);
    hipError_t e;
    if (c.tiles) {
        e = launch_decode_tile(a, c, stream);
    } else {
        const dim3 grid((unsigned)blocks, (unsigned)a.Hkv);
        CFP32_BY_TYPE(decode_rows_kernel, a.kv_f16, a.D, w, c.eight, grid, a, c);
        e = hipGetLastError();
    }
    return e != hipSuccess || !c.to.o ? e : launch_join(a, c.to, stream);
}

}  // namespace cfp32
