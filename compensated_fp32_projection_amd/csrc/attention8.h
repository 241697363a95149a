// Attention over an 8-bit cache: arguments, plan and launcher (internal to
// libcfp32).
#pragma once

#include "cache8.h"

namespace cfp32 {

struct Decode8Args {
    const float *q;
    int64_t q_seq, q_head;
    Cache8 c;
    const int32_t *table;
    int64_t ld_table;
    const int32_t *lens;
    float *out;
    int64_t out_seq, out_head;
    int B, Hq, W;
    float scale;
};

// What attention8_plans.hip decides about a call.  error: a grid that cannot be
// launched.
struct Decode8Plan {
    hipError_t error;
    int align;       // bytes that divide every address and the head size: 16, 8 or 1
    bool fast;       // see Tile8
    int groups;      // of 16 query heads to a K/V head
    int parts;       // of a sequence's keys
    int64_t blocks;  // of each K/V head
    Partials to;     // null o: straight to the output
};
Decode8Plan plan_decode8(const Decode8Args &a, void *workspace);
size_t attention8_decode_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t W, int page_log2);

hipError_t launch_attention8_decode(const Decode8Args &a, void *workspace, hipStream_t stream);

}  // namespace cfp32
