// Arguments and launchers of the attention and cache kernels (internal to
// libcfp32).  Arguments are validated by attention_api.hip; every launcher
// only enqueues kernels on `stream` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cfp32 {

constexpr int kAttnMaxDim = 128;  // largest head size

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

size_t attention_prompt_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16);
hipError_t launch_attention_prompt(const PromptArgs &a, void *workspace, hipStream_t stream);

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

size_t partial_bytes(int64_t rows, int slots, int dim);
void place_partials(Partials &to, int64_t rows, void *at);
hipError_t launch_join(const PromptArgs &a, const Partials &from, hipStream_t stream);
hipError_t launch_join(const DecodeArgs &a, const Partials &from, hipStream_t stream);

// The form for many rows (attention_tile.hip); FP16 K and V have to allow
// 16-byte loads, and a token's stride to be below 2^26 bytes.
size_t prompt_tile_workspace(int64_t S, int64_t Tk, int64_t Hkv, int64_t D, bool kv_f16);
hipError_t launch_prompt_tile(const PromptArgs &a, void *workspace, hipStream_t stream);

// How many parts the shared keys of a decode make there, and the launch of
// all of a decode whose shared keys go there (FP16 pages that allow 16-byte
// loads, a token's stride below 2^32 bytes).
int decode_tile_parts(int64_t B, int64_t Hq, int64_t Hkv, int64_t keys, int page_log2);
hipError_t launch_decode_tile(const DecodeArgs &a, const DecodeParts &c, hipStream_t stream);

size_t attention_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int page_log2,
                                  int64_t shared_pages, bool kv_f16);
hipError_t launch_attention_decode(const DecodeArgs &a, void *workspace, hipStream_t stream);

// A pool of K pages and of V pages.
struct Pool {
    PagesView k, v;
    int P, page_log2, Hkv, D, elem_bytes;
};

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
