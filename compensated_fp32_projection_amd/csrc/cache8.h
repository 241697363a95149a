// Arguments and launchers of the 8-bit cache's kernels (internal to libcfp32).
// Arguments are validated by serving_api.hip.
#pragma once

#include "attention.h"

namespace cfp32 {

// Scales [P, Hkv, blocks of a page], contiguous blocks.
struct ScalesView {
    float *data;
    int64_t page, head;
};

struct Cache8 {
    PagesView k, v;  // codes
    ScalesView ks, vs;
    int P, Hkv, D, page_log2, block_log2;
    bool e4m3;
};

hipError_t launch_cache8_append(const HeadsView &k, const HeadsView &v, const int32_t *cu, const int32_t *lens, int32_t *lens_out,
                                const Cache8 &c, const int32_t *table, int64_t ld, int S, int W, int T, hipStream_t stream);

// Packed rows that are written.
struct HeadsOut {
    void *data;
    int64_t tok, head;
};
hipError_t launch_cache8_read(const Cache8 &c, const int32_t *table, int64_t ld, const int32_t *first, const int32_t *cu,
                              const HeadsOut &k, const HeadsOut &v, bool f16, int S, int W, int T, hipStream_t stream);

// Codes and scales as pools (cache.hip); workspaces as launch_cache_fork's and launch_cache_compact's.
hipError_t launch_cache8_copy_pages(const Pool &codes, const Pool &scales, const int32_t *src, const int32_t *dst, int n,
                                    hipStream_t stream);
hipError_t launch_cache8_fork(const Pool &codes, const Pool &scales, const int32_t *table, int64_t ld, const int32_t *lens,
                              const int32_t *refs, const int32_t *parents, int32_t *table_out, int64_t ld_out,
                              int32_t *lens_out, int32_t *refs_out, int32_t *missing, int S, int W, int C,
                              int32_t *workspace, hipStream_t stream);
hipError_t launch_cache8_compact(const Pool &codes, const Pool &scales, const int32_t *table, int64_t ld, const int32_t *refs,
                                 int32_t *table_out, int64_t ld_out, int32_t *refs_out, int32_t *live, int S, int W,
                                 int32_t *workspace, hipStream_t stream);

}  // namespace cfp32
