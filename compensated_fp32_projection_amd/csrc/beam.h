// Arguments, plan and launchers of beam search (internal to libcfp32).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cfp32 {

constexpr int kMaxBeams = 64;  // of a sequence, and selected: a lane each

struct BeamArgs {
    const float *logits;
    int64_t ld;
    const float *scores;
    const uint8_t *done;
    int S, beams, V, n, eos;
    int32_t *parents, *tokens;
    float *scores_out;
    uint8_t *done_out;
};

// How a row's logits are cut among waves: `each` of a lane.
struct BeamPlan {
    int each, chunks;
    size_t bytes;  // of the chunks' sums and best logits
};
BeamPlan plan_beam(int64_t S, int64_t beams, int64_t V, int64_t n);

hipError_t launch_beam_select(const BeamArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_beam_reorder(const void *states, int64_t stride, void *out, int64_t out_stride, const int32_t *parents,
                               int rows, int n, int64_t row_bytes, hipStream_t stream);

}  // namespace cfp32
