// Host-side planning of beam search (no device code).
#include "beam.h"

namespace cfp32 {

BeamPlan plan_beam(int64_t S, int64_t beams, int64_t V, int64_t n)
{
    BeamPlan p = {};
    const int64_t rows = S * beams;
    // Waves of 2048 logits where there are enough of them, else of 512.
    p.each = rows * ((V + 2047) / 2048) >= 2048 ? 32 : 8;
    p.chunks = (int)((V + 64 * p.each - 1) / (64 * p.each));
    p.bytes = (size_t)(rows * p.chunks) * (8 + 8 * (size_t)n);
    return p;
}

}  // namespace cfp32
