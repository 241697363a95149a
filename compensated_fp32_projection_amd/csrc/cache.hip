// The paged cache: reserving pages, writing tokens, copying, forking, freeing
// and compacting (include/cfp32.h).
//
// The bookkeeping (which free page goes where) is a prefix sum over the
// pool's counts and one over the wanted entries, in one block of 1024
// threads: its results are needed by everything after it, and pools hold
// thousands of pages, so one block reads them in microseconds and needs no
// hand-over between blocks.  Data moves in a grid over 16 KiB pieces.
// Counts are integers, so atomics on them give the same results in any
// order.
#include "attention.h"
#include "cache8.h"

namespace cfp32 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRun = 4;                           // consecutive entries per thread
constexpr int kPlanChunk = kPlanThreads * kPlanRun;
constexpr int kListCap = 2 * kPlanChunk;              // free pages held at a time (32 KiB of LDS)

// Exclusive prefix sum over the block of one count per thread, and the total.
__device__ __forceinline__ int block_scan(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();  // the previous call's reads of sums are done
    if (lane == 63) sums[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        const int x = sums[w];
        before += w < wave ? x : 0;
        all += x;
    }
    total = all;
    return before + s - v;
}

// Gives the lowest free pages of refs[P] to the wanted ones of n entries, in
// order: give(i, page).  wanted(i) must be false once entry i was given a
// page.  Returns how many entries got none (to every thread).
template <class Wanted, class Give>
__device__ int assign_free(const int32_t *refs, int P, int64_t n, Wanted wanted, Give give)
{
    __shared__ int list[kListCap];
    __shared__ int sums[kPlanThreads / 64];
    int pos = 0, left = 0;
    for (;;) {
        int have = 0, total;
        while (pos < P && have + kPlanChunk <= kListCap) {
            const int64_t i0 = (int64_t)pos + threadIdx.x * kPlanRun;
            bool f[kPlanRun];
            int c = 0;
#pragma unroll
            for (int e = 0; e < kPlanRun; ++e) {
                f[e] = i0 + e < P && refs[i0 + e] <= 0;
                c += f[e];
            }
            int r = have + block_scan(c, sums, total);
#pragma unroll
            for (int e = 0; e < kPlanRun; ++e)
                if (f[e]) list[r++] = (int)(i0 + e);
            have += total;
            pos = P - pos > kPlanChunk ? pos + kPlanChunk : P;
        }
        __syncthreads();
        int64_t base = 0;
        for (int64_t b = 0; b < n; b += kPlanChunk) {
            const int64_t i0 = b + threadIdx.x * kPlanRun;
            bool f[kPlanRun];
            int c = 0;
#pragma unroll
            for (int e = 0; e < kPlanRun; ++e) {
                f[e] = i0 + e < n && wanted(i0 + e);
                c += f[e];
            }
            int64_t r = base + block_scan(c, sums, total);
#pragma unroll
            for (int e = 0; e < kPlanRun; ++e)
                if (f[e]) {
                    if (r < have) give(i0 + e, list[r]);
                    ++r;
                }
            base += total;
        }
        left = base > have ? (int)(base - have < 0x7FFFFFFF ? base - have : 0x7FFFFFFF) : 0;
        __syncthreads();  // the list is read, the given entries are written
        if (left == 0 || pos >= P) return left;
    }
}

__device__ __forceinline__ int64_t pages_for(int64_t tokens, int lg) { return tokens <= 0 ? 0 : (tokens + ((int64_t)1 << lg) - 1) >> lg; }

__global__ __launch_bounds__(kPlanThreads) void cache_reserve_kernel(const int32_t *table, int64_t ld,
                                                                     const int32_t *lens, const int32_t *cu,
                                                                     const int32_t *refs, int32_t *table_out,
                                                                     int64_t ld_out, int32_t *refs_out,
                                                                     int32_t *missing, int S, int W, int P, int lg)
{
    __shared__ unsigned long long beyond;
    if (threadIdx.x == 0) beyond = 0;
    for (int64_t i = threadIdx.x; i < P; i += kPlanThreads) refs_out[i] = refs[i];
    const int64_t n = (int64_t)S * W;
    if (table != table_out)
        for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
            const int64_t s = i / W, j = i - s * W;
            table_out[s * ld_out + j] = table[s * ld + j];
        }
    __syncthreads();
    auto need = [&](int64_t s) { return pages_for((int64_t)lens[s] + cu[s + 1] - cu[s], lg); };
    const int left = assign_free(
        refs_out, P, n,
        [&](int64_t i) {
            const int64_t s = i / W, j = i - s * W;
            return table_out[s * ld_out + j] < 0 && j < need(s);
        },
        [&](int64_t i, int p) {
            const int64_t s = i / W, j = i - s * W;
            table_out[s * ld_out + j] = p;
            refs_out[p] = 1;
        });
    if (missing) {
        unsigned long long b = 0;
        for (int64_t s = threadIdx.x; s < S; s += kPlanThreads) {
            const int64_t m = need(s) - W;
            b += m > 0 ? m : 0;
        }
        atomicAdd(&beyond, b);
        __syncthreads();
        if (threadIdx.x == 0) *missing = (int)min(beyond + left, 0x7FFFFFFFull);
    }
}

// Children's lengths and last pages; src/dst: the pages to copy, -1 where none.
__global__ __launch_bounds__(kPlanThreads) void cache_fork_plan_kernel(const int32_t *table, int64_t ld,
                                                                       const int32_t *lens, const int32_t *refs,
                                                                       const int32_t *parents, int32_t *lens_out,
                                                                       int32_t *refs_out, int32_t *missing, int S,
                                                                       int W, int C, int P, int lg, int32_t *src,
                                                                       int32_t *dst)
{
    for (int64_t i = threadIdx.x; i < P; i += kPlanThreads) refs_out[i] = refs[i];
    const int mask = (1 << lg) - 1;
    for (int64_t c = threadIdx.x; c < C; c += kPlanThreads) {
        const int p = parents[c];
        int len = p >= 0 && p < S ? lens[p] : 0;
        len = len < 0 ? 0 : len;
        if ((len >> lg) >= W) len = W << lg;
        int from = -1;
        if (len & mask) from = table[(int64_t)p * ld + (len >> lg)];
        src[c] = from >= 0 && from < P ? from : -1;
        dst[c] = -1;
        lens_out[c] = src[c] >= 0 ? len : len & ~mask;
    }
    __syncthreads();
    const int left = assign_free(
        refs_out, P, C, [&](int64_t c) { return src[c] >= 0 && dst[c] < 0; },
        [&](int64_t c, int p) {
            dst[c] = p;
            refs_out[p] = 1;
        });
    for (int64_t c = threadIdx.x; c < C; c += kPlanThreads)
        if (src[c] >= 0 && dst[c] < 0) {
            lens_out[c] &= ~mask;
            src[c] = -1;
        }
    if (missing && threadIdx.x == 0) *missing = left;
}

// ---- Moving pages --------------------------------------------------------------

typedef uint32_t vec4_t __attribute__((ext_vector_type(4)));
typedef uint32_t vec2_t __attribute__((ext_vector_type(2)));

// Non-temporal: what is moved is not read again soon, and as ordinary loads
// and stores it went through the L2s at two thirds of the speed (compaction
// of 1024 pages of 256 KiB 37 -> 25 us, fork of 256 35 -> 29).
template <class V>
__device__ __forceinline__ void copy_piece(const PageShape &g, int src, int dst, int64_t piece, int64_t pieces)
{
    const bool second = piece >= pieces;
    const PageRows &t = second ? g.v : g.k;
    const int64_t total = g.vecs * g.rows;
    const int64_t v0 = (second ? piece - pieces : piece) * 1024 + threadIdx.x;
    const char *from = t.data + src * t.page;
    char *to = t.data + dst * t.page;
    V x[4];
    int64_t off[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t u = v0 + 256 * e;
        off[e] = -1;
        if (u < total) {
            const int64_t r = g.rows == 1 ? 0 : u / g.vecs, i = u - r * g.vecs;
            off[e] = (g.rows == 1 ? 0 : r / g.n2 * t.s1 + r % g.n2 * t.s2) + i * (int64_t)sizeof(V);
            x[e] = __builtin_nontemporal_load(reinterpret_cast<const V *>(from + off[e]));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (off[e] >= 0) __builtin_nontemporal_store(x[e], reinterpret_cast<V *>(to + off[e]));
}

// Table entries to be made beside the copies, by the first blocks of their
// launch (of their own they took 2 to 4 us of a fork's or a compaction's).
struct NoTables {
    __device__ __forceinline__ void operator()(int64_t) const {}
};

// Pairs (src, dst), each cut into 2 * pieces pieces (K, then V); pairs with
// an id outside the pool are passed over.  `count`: how many pairs (null: n).
// Blocks below `table_blocks` make the `entries` table entries instead.
template <class V, class Tables>
__global__ __launch_bounds__(256) void cache_copy_kernel(PageShape g, const int32_t *src, const int32_t *dst, int n,
                                                         const int32_t *count, int P, int64_t pieces, Tables tables,
                                                         int64_t entries, unsigned table_blocks)
{
    if (blockIdx.x < table_blocks) {
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)table_blocks * 256) tables(i);
        return;
    }
    const int64_t units = (int64_t)(count ? *count : n) * 2 * pieces;
    for (int64_t u = blockIdx.x - table_blocks; u < units; u += gridDim.x - table_blocks) {
        const int64_t i = u / (2 * pieces);
        const int a = src[i], b = dst[i];
        if (a < 0 || b < 0 || a >= P || b >= P) continue;
        copy_piece<V>(g, a, b, u - i * 2 * pieces, pieces);
    }
}

template <class Tables>
hipError_t launch_copy(const Pool &pool, const int32_t *src, const int32_t *dst, int n, const int32_t *count,
                       const Tables &tables, int64_t entries, hipStream_t stream)
{
    const unsigned table_blocks = (unsigned)(entries < 256 * 4096 ? (entries + 255) / 256 : 4096);
    if (pool.Hkv == 0 || pool.D == 0) n = 0;
    PageShape g = {};
    g.vec_bytes = 16;
    if (n > 0) g = page_shape(pool);
    const int64_t pieces = n > 0 ? (g.vecs * g.rows + 1023) / 1024 : 0, units = (int64_t)n * 2 * pieces;
    const unsigned blocks = (unsigned)(units < 16384 ? units : 16384) + table_blocks;
    if (blocks == 0) return hipSuccess;
#define CFP32_COPY(V) \
    cache_copy_kernel<V><<<blocks, 256, 0, stream>>>(g, src, dst, n, count, pool.P, pieces, tables, entries, table_blocks)
    switch (g.vec_bytes) {
    case 16: CFP32_COPY(vec4_t); break;
    case 8: CFP32_COPY(vec2_t); break;
    case 4: CFP32_COPY(uint32_t); break;
    case 2: CFP32_COPY(uint16_t); break;
    default: CFP32_COPY(uint8_t); break;
    }
#undef CFP32_COPY
    return hipGetLastError();
}

// Children's tables, and the counts of the pages they share.
struct ForkTables {
    const int32_t *table, *lens_out, *parents, *dst;
    int32_t *table_out, *refs_out;
    int64_t ld, ld_out;
    int W, P, lg;
    __device__ __forceinline__ void operator()(int64_t i) const
    {
        const int64_t c = i / W, j = i - c * W;
        const int whole = lens_out[c] >> lg;
        int e = -1;
        if (j < whole) {  // a child with pages has a parent in [0, S)
            e = table[(int64_t)parents[c] * ld + j];
            if (e >= 0 && e < P) atomicAdd(&refs_out[e], 1);
        } else if (j == whole && dst[c] >= 0) {
            e = dst[c];
        }
        table_out[c * ld_out + j] = e;
    }
};

// Tables after a compaction.
struct MovedTables {
    const int32_t *table, *map;
    int32_t *table_out;
    int64_t ld, ld_out;
    int W, P;
    __device__ __forceinline__ void operator()(int64_t i) const
    {
        const int64_t s = i / W, j = i - s * W;
        const int e = table[s * ld + j];
        table_out[s * ld_out + j] = e >= 0 && e < P ? map[e] : e;
    }
};

// ---- Writing tokens --------------------------------------------------------------

// The sequence s with cu[s] <= t < cu[s + 1], or -1.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int S, int t)
{
    int lo = 0, hi = S;  // the largest s < S with cu[s] <= t
    while (hi - lo > 1) {
        const int m = lo + (hi - lo) / 2;
        if (cu[m] <= t) lo = m;
        else hi = m;
    }
    return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

template <class Out, int E>
__global__ __launch_bounds__(256) void cache_append_kernel(HeadsView k, HeadsView v, const int32_t *cu,
                                                           const int32_t *lens, int32_t *lens_out, Pool pool,
                                                           const int32_t *table, int64_t ld, int S, int W, int T)
{
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t s = first; s < S; s += step) lens_out[s] = lens[s] + (cu[s + 1] - cu[s]);
    const int per = pool.D / E;
    const int64_t n = (int64_t)T * pool.Hkv * per;
    for (int64_t i = first; i < n; i += step) {
        const int d = (int)(i % per) * E;
        const int64_t th = i / per;
        const int h = (int)(th % pool.Hkv), t = (int)(th / pool.Hkv);
        const int s = find_sequence(cu, S, t);
        if (s < 0) continue;
        const int64_t pos = (int64_t)lens[s] + (t - cu[s]);
        const int64_t j = pos >> pool.page_log2;
        if (pos < 0 || j >= W) continue;
        const int page = table[s * ld + j];
        if (page < 0 || page >= pool.P) continue;
        const int64_t o = pos & (((int64_t)1 << pool.page_log2) - 1);
        // In pieces of 16 bytes at most, which is what the pointers are aligned
        // to; non-temporal (4 x 2048 tokens 29 -> 26 us).
        auto put = [&](const HeadsView &x, const PagesView &to) {
            constexpr int IN = E < 4 ? E : 4, OUT = E < 16 / (int)sizeof(Out) ? E : 16 / (int)sizeof(Out);
            typedef float in_piece __attribute__((ext_vector_type(IN)));
            typedef Out out_piece __attribute__((ext_vector_type(OUT)));
            float a[E];
#pragma unroll
            for (int e = 0; e < E; e += IN) {
                const in_piece p = __builtin_nontemporal_load(reinterpret_cast<const in_piece *>((const float *)x.data + t * x.tok + h * x.head + d + e));
#pragma unroll
                for (int u = 0; u < IN; ++u) a[e + u] = p[u];
            }
            Out *out = (Out *)to.data + page * to.page + h * to.head + o * to.tok + d;
#pragma unroll
            for (int e = 0; e < E; e += OUT) {
                out_piece p;
#pragma unroll
                for (int u = 0; u < OUT; ++u) p[u] = (Out)a[e + u];
                __builtin_nontemporal_store(p, reinterpret_cast<out_piece *>(out + e));
            }
        };
        put(k, pool.k);
        put(v, pool.v);
    }
}

// ---- Freeing and compacting --------------------------------------------------------

__global__ __launch_bounds__(256) void cache_counts_kernel(const int32_t *refs, int32_t *refs_out, int P)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < P) refs_out[i] = refs[i];
}

__global__ __launch_bounds__(256) void cache_free_kernel(const int32_t *rows, int64_t ld, int32_t *refs_out, int R, int W,
                                                         int P)
{
    const int64_t n = (int64_t)R * W;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / W;
        const int e = rows[r * ld + (i - r * W)];
        if (e >= 0 && e < P) atomicSub(&refs_out[e], 1);
    }
}

// The same of a small pool in one launch: what is given up is counted in LDS.
constexpr int kSmallPool = 16384;
__global__ __launch_bounds__(kPlanThreads) void cache_free_small_kernel(const int32_t *rows, int64_t ld, const int32_t *refs,
                                                                        int32_t *refs_out, int R, int W, int P)
{
    __shared__ int gone[kSmallPool];
    for (int i = threadIdx.x; i < P; i += kPlanThreads) gone[i] = 0;
    __syncthreads();
    const int n = R * W;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int r = i / W, e = rows[r * ld + (i - r * W)];
        if (e >= 0 && e < P) atomicAdd(&gone[e], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += kPlanThreads) refs_out[i] = refs[i] - gone[i];
}

// map[p]: where page p goes (itself unless it moves); src/dst: the moves; *moves: how many.
__global__ __launch_bounds__(kPlanThreads) void cache_compact_plan_kernel(const int32_t *refs, int32_t *refs_out,
                                                                          int32_t *live, int P, int32_t *map,
                                                                          int32_t *src, int32_t *dst, int32_t *moves)
{
    __shared__ int sums[kPlanThreads / 64];
    int c = 0, n;
    for (int64_t i = threadIdx.x; i < P; i += kPlanThreads) c += refs[i] > 0;
    block_scan(c, sums, n);
    // The free pages below n and the live ones from n on, each in order:
    // equally many.
    int holes = 0, total;
    for (int64_t b = 0; b < n; b += kPlanThreads) {
        const int64_t i = b + threadIdx.x;
        const bool free = i < n && refs[i] <= 0;
        const int r = holes + block_scan(free, sums, total);
        if (i < n) map[i] = (int)i;
        if (free) dst[r] = (int)i;
        else if (i < n) refs_out[i] = refs[i];
        holes += total;
    }
    __syncthreads();
    int at = 0;
    for (int64_t b = n; b < P; b += kPlanThreads) {
        const int64_t i = b + threadIdx.x;
        const int count = i < P ? refs[i] : 0;
        const int r = at + block_scan(count > 0, sums, total);
        const int to = count > 0 ? dst[r] : (int)i;
        if (i < P) {
            map[i] = to;
            refs_out[i] = 0;
        }
        if (count > 0) {
            src[r] = (int)i;
            refs_out[to] = count;
        }
        at += total;
    }
    if (threadIdx.x == 0) {
        *live = n;
        if (P > 0) *moves = holes;
    }
}

unsigned grid_for(int64_t n) { return (unsigned)(n <= 0 ? 1 : (n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192); }

}  // namespace

hipError_t launch_cache_reserve(const int32_t *table, int64_t ld, const int32_t *lens, const int32_t *cu,
                                const int32_t *refs, int32_t *table_out, int64_t ld_out, int32_t *refs_out,
                                int32_t *missing, int S, int W, int P, int page_log2, hipStream_t stream)
{
    cache_reserve_kernel<<<1, kPlanThreads, 0, stream>>>(table, ld, lens, cu, refs, table_out, ld_out, refs_out, missing,
                                                         S, W, P, page_log2);
    return hipGetLastError();
}

hipError_t launch_cache_append(const HeadsView &k, const HeadsView &v, const int32_t *cu, const int32_t *lens,
                               int32_t *lens_out, const Pool &pool, const int32_t *table, int64_t ld, int S, int W,
                               int T, hipStream_t stream)
{
    const int64_t eb = pool.elem_bytes;
    const int64_t in = (int64_t)((uintptr_t)k.data | (uintptr_t)v.data) | 4 * (k.tok | k.head | v.tok | v.head);
    const int64_t to = (int64_t)((uintptr_t)pool.k.data | (uintptr_t)pool.v.data) |
                       eb * (pool.k.page | pool.k.head | pool.k.tok | pool.v.page | pool.v.head | pool.v.tok);
    // Elements of a thread: 32 bytes of FP32 in, and 16 or 32 out.
    const bool wide = pool.D % 8 == 0 && in % 16 == 0 && to % 16 == 0, four = pool.D % 4 == 0 && in % 16 == 0 && to % (4 * eb) == 0;
    const int64_t n = (int64_t)T * pool.Hkv * (pool.D / (wide ? 8 : four ? 4 : 1));
    const unsigned blocks = grid_for(n > S ? n : S);
#define CFP32_APPEND(OUT, E) \
    cache_append_kernel<OUT, E><<<blocks, 256, 0, stream>>>(k, v, cu, lens, lens_out, pool, table, ld, S, W, T)
    if (pool.elem_bytes == 2) {
        if (wide) CFP32_APPEND(_Float16, 8);
        else if (four) CFP32_APPEND(_Float16, 4);
        else CFP32_APPEND(_Float16, 1);
    } else {
        if (wide) CFP32_APPEND(float, 8);
        else if (four) CFP32_APPEND(float, 4);
        else CFP32_APPEND(float, 1);
    }
#undef CFP32_APPEND
    return hipGetLastError();
}

hipError_t launch_cache_copy_pages(const Pool &pool, const int32_t *src, const int32_t *dst, int n, hipStream_t stream)
{
    return launch_copy(pool, src, dst, n, nullptr, NoTables{}, 0, stream);
}

hipError_t launch_cache_fork(const Pool &pool, const int32_t *table, int64_t ld, const int32_t *lens,
                             const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out,
                             int32_t *lens_out, int32_t *refs_out, int32_t *missing, int S, int W, int C,
                             int32_t *workspace, hipStream_t stream)
{
    int32_t *src = workspace, *dst = workspace + C;
    cache_fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(table, ld, lens, refs, parents, lens_out, refs_out, missing,
                                                           S, W, C, pool.P, pool.page_log2, src, dst);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || C == 0) return e;
    const ForkTables tables = {table, lens_out, parents, dst, table_out, refs_out, ld, ld_out, W, pool.P, pool.page_log2};
    return launch_copy(pool, src, dst, C, nullptr, tables, (int64_t)C * W, stream);
}

hipError_t launch_cache8_copy_pages(const Pool &codes, const Pool &scales, const int32_t *src, const int32_t *dst, int n,
                                    hipStream_t stream)
{
    const hipError_t e = launch_cache_copy_pages(codes, src, dst, n, stream);
    return e != hipSuccess ? e : launch_cache_copy_pages(scales, src, dst, n, stream);
}

hipError_t launch_cache8_fork(const Pool &codes, const Pool &scales, const int32_t *table, int64_t ld, const int32_t *lens,
                              const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out,
                              int32_t *lens_out, int32_t *refs_out, int32_t *missing, int S, int W, int C,
                              int32_t *workspace, hipStream_t stream)
{
    const hipError_t e = launch_cache_fork(codes, table, ld, lens, refs, parents, table_out, ld_out, lens_out, refs_out, missing,
                                           S, W, C, workspace, stream);
    return e != hipSuccess || C == 0 ? e : launch_copy(scales, workspace, workspace + C, C, nullptr, NoTables{}, 0, stream);
}

hipError_t launch_cache_free(const int32_t *rows, int64_t ld, const int32_t *refs, int32_t *refs_out, int R, int W,
                             int P, hipStream_t stream)
{
    if (P <= kSmallPool && (int64_t)R * W <= 65536) {
        cache_free_small_kernel<<<1, kPlanThreads, 0, stream>>>(rows, ld, refs, refs_out, R, W, P);
        return hipGetLastError();
    }
    if (refs != refs_out) {
        cache_counts_kernel<<<(unsigned)(((int64_t)P + 255) / 256), 256, 0, stream>>>(refs, refs_out, P);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if ((int64_t)R * W == 0) return hipSuccess;
    cache_free_kernel<<<grid_for((int64_t)R * W), 256, 0, stream>>>(rows, ld, refs_out, R, W, P);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const Pool &pool, const int32_t *table, int64_t ld, const int32_t *refs,
                                int32_t *table_out, int64_t ld_out, int32_t *refs_out, int32_t *live, int S, int W,
                                int32_t *workspace, hipStream_t stream)
{
    int32_t *map = workspace, *src = map + pool.P, *dst = src + pool.P, *moves = dst + pool.P;
    cache_compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(refs, refs_out, live, pool.P, map, src, dst, moves);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const MovedTables tables = {table, map, table_out, ld, ld_out, W, pool.P};
    return launch_copy(pool, src, dst, pool.P / 2, moves, tables, (int64_t)S * W, stream);
}

hipError_t launch_cache8_compact(const Pool &codes, const Pool &scales, const int32_t *table, int64_t ld, const int32_t *refs,
                                 int32_t *table_out, int64_t ld_out, int32_t *refs_out, int32_t *live, int S, int W,
                                 int32_t *workspace, hipStream_t stream)
{
    const hipError_t e = launch_cache_compact(codes, table, ld, refs, table_out, ld_out, refs_out, live, S, W, workspace, stream);
    if (e != hipSuccess) return e;
    const int32_t *src = workspace + codes.P, *dst = src + codes.P, *moves = dst + codes.P;
    return launch_copy(scales, src, dst, codes.P / 2, moves, NoTables{}, 0, stream);
}

}  // namespace cfp32
