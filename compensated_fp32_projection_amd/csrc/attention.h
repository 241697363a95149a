// Arguments and launchers of the attention and cache kernels (internal to
// libcfp32).  Arguments are validated by attention_api.hip; every launcher
// only enqueues kernels on `stream` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cfp32 {

constexpr int kAttnMaxDim = 128;  // largest head size
constexpr int kRows = 16;         // rows of a block of attention_rows.h
constexpr int kTile = 64;         // keys of a tile of attention_tile.hip, ...
constexpr int kWaveRows = 32;     // ... rows of a wave, ...
constexpr int kPageIds = 2048;    // ... and pages of a block's keys

// [tokens, heads, D] with unit stride along D: element strides of a token and a head.
struct HeadsView {
    const void *data;
    int64_t tok, head;
};

// Cache pages [P, Hkv, page, D] with unit stride along D.
struct PagesView {
    void *data;
    int64_t page, head, tok;  // element strides
};

struct PromptArgs {
    HeadsView q, k, v;
    float *out;
    int64_t out_tok, out_head;
    const int32_t *cu_q, *cu_k;  // [S + 1]
    int S, Tq, Tk, Hq, Hkv, D;
    bool kv_f16, causal;
    float scale;
};

struct DecodeArgs {
    const float *q;
    int64_t q_seq, q_head;
    PagesView k, v;
    const int32_t *table;
    int64_t ld_table;
    const int32_t *lens;
    float *out;
    int64_t out_seq, out_head;
    int B, Hq, Hkv, D, P, page_log2, W, shared_pages;
    bool kv_f16;
    float scale;
};

// What several blocks contribute to one row: unnormalised sums, their maxima
// (in powers of two) and weights.  Part i of row r is entry r * slots + i.
// Null o: one part, which goes straight to the output.
struct Partials {
    float *o;   // [rows * slots, dim]
    float *m, *l;
    int slots, dim;
};
// How the keys of a decode are cut: the shared ones into `shared` parts (0:
// none are shared), each sequence's others into `own`, of equal lengths (in
// whole steps of all waves).  Row groups: 16 rows of the batch's for the
// shared keys, 16 of a sequence's heads for its own.
struct DecodeParts {
    int shared, own, shared_groups, own_groups;
    int own_from;  // the first key that is not shared
    bool eight;    // waves
    int tiles;     // shared parts that attention_tile.hip's kernel takes (then `shared` is 0): slots [0, tiles)
    Partials to;   // slots: tiles + shared + own; null o: straight to the output
};

// Rows of up to this many parts are joined by a wave each, of more by a block.
constexpr int kJoinByWave = 16;
inline int64_t join_blocks(const Partials &from, int64_t rows) { return from.slots > kJoinByWave ? rows : (rows + 3) / 4; }

// FP32 K and V, cut in two: of each K/V head and key, in the order of the packed
// keys, [K hi, K lo, V hi, V lo][DP] FP16, zeros beyond D; each sequence's tiles
// begin with its first key, and what its last one holds beyond its end are the
// next sequence's keys, or zeros behind the last.  And the shifts of K and V of
// each tile (sequence s's begin at cu_k[s] / 64 + s).  One shift for 64 keys
// leaves each its bits as long as their largest magnitudes are within 2^12 of
// each other: an element is then off by no more than 2^-22 of itself or 2^-27
// of its key's largest.  Tiles whose keys differ by more, of which a row may
// see the small ones alone, or weigh them alone, have a shift for each key.
// key_shifts has every key's, also those of a tile that are alike.
struct Planes {
    char *keys;                    // [Hkv][count]
    int32_t *shifts, *key_shifts;  // [Hkv][slots][K, V], [Hkv][count][K, V]
    int64_t count, slots;
};
constexpr int plane_key_bytes(int dp) { return 4 * 2 * dp; }

// What attention_plans.hip decides about a call.  error: a grid that cannot be
// launched.
struct PromptPlan {
    hipError_t error;
    bool tiles;      // attention_tile.hip's kernel, else attention_rows.h's
    bool wide;       // K and V allow 16-byte loads
    bool eight;      // waves
    int64_t blocks;  // of each part
    Partials to;
    Planes planes;   // FP32 K and V of tiles
};
struct DecodePlan {
    hipError_t error;
    bool wide;
    DecodeParts parts;
    int64_t blocks, tile_blocks;  // of each K/V head; with tiles, of all, and those for shared keys
};
PromptPlan plan_prompt(const PromptArgs &a, void *workspace);
DecodePlan plan_decode(const DecodeArgs &a, void *workspace);
size_t attention_prompt_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16);
size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int page_log2,
                                  int64_t shared_pages, bool kv_f16);

hipError_t launch_attention_prompt(const PromptArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_attention_decode(const DecodeArgs &a, void *workspace, hipStream_t stream);

// The forms for many rows (attention_tile.hip), without the join.  FP16 K and V
// have to allow 16-byte loads, a token's stride to be below 2^26 bytes (pages:
// 2^32).
hipError_t launch_prompt_tile(const PromptArgs &a, const PromptPlan &p, hipStream_t stream);
hipError_t launch_decode_tile(const DecodeArgs &a, const DecodePlan &p, hipStream_t stream);

// A pool of K pages and of V pages.
struct Pool {
    PagesView k, v;
    int P, page_log2, Hkv, D, elem_bytes;
};

// How pages are moved: a tensor of a pool as rows of `vecs` vectors, n1 x n2 rows to a page.
struct PageRows {
    char *data;
    int64_t page, s1, s2;  // bytes
};
struct PageShape {
    PageRows k, v;
    int64_t rows;          // of a page: n1 * n2
    int n2;
    int64_t vecs;          // vectors of a row
    int vec_bytes;
};
PageShape page_shape(const Pool &p);

hipError_t launch_cache_reserve(const int32_t *table, int64_t ld, const int32_t *lens, const int32_t *cu,
                                const int32_t *refs, int32_t *table_out, int64_t ld_out, int32_t *refs_out,
                                int32_t *missing, int S, int W, int P, int page_log2, hipStream_t stream);
hipError_t launch_cache_append(const HeadsView &k, const HeadsView &v, const int32_t *cu, const int32_t *lens,
                               int32_t *lens_out, const Pool &pool, const int32_t *table, int64_t ld, int S, int W,
                               int T, hipStream_t stream);
hipError_t launch_cache_copy_pages(const Pool &pool, const int32_t *src, const int32_t *dst, int n,
                                   hipStream_t stream);
// workspace: 2 x C int32 (the pages copied, as sources and destinations)
hipError_t launch_cache_fork(const Pool &pool, const int32_t *table, int64_t ld, const int32_t *lens,
                             const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out,
                             int32_t *lens_out, int32_t *refs_out, int32_t *missing, int S, int W, int C,
                             int32_t *workspace, hipStream_t stream);
hipError_t launch_cache_free(const int32_t *rows, int64_t ld, const int32_t *refs, int32_t *refs_out, int R, int W,
                             int P, hipStream_t stream);
// workspace: 3 P + 1 int32 (where each page goes; the moves, as sources and destinations; their number)
hipError_t launch_cache_compact(const Pool &pool, const int32_t *table, int64_t ld, const int32_t *refs,
                                int32_t *table_out, int64_t ld_out, int32_t *refs_out, int32_t *live, int S, int W,
                                int32_t *workspace, hipStream_t stream);

}  // namespace cfp32
