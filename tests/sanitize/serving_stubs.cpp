// Launcher stubs of the rotary, 8-bit cache and beam calls for the host-only
// sanitizer build (see attention_stubs.cpp).  No check gets as far as a launch,
// so every stub aborts.
#include <cstdio>
#include <cstdlib>

#include "../../compensated_fp32_projection_amd/csrc/attention8.h"
#include "../../compensated_fp32_projection_amd/csrc/beam.h"
#include "../../compensated_fp32_projection_amd/csrc/rotary.h"

namespace cfp32 {

[[noreturn]] static void reached(const char *name)
{
    std::fprintf(stderr, "launcher stub reached: %s\n", name);
    std::abort();
}

hipError_t launch_rotary(const RotaryArgs &, hipStream_t) { reached("launch_rotary"); }
hipError_t launch_cache8_append(const HeadsView &, const HeadsView &, const int32_t *, const int32_t *, int32_t *, const Cache8 &,
                                const int32_t *, int64_t, int, int, int, hipStream_t)
{
    reached("launch_cache8_append");
}
hipError_t launch_cache8_read(const Cache8 &, const int32_t *, int64_t, const int32_t *, const int32_t *, const HeadsOut &,
                              const HeadsOut &, bool, int, int, int, hipStream_t)
{
    reached("launch_cache8_read");
}
hipError_t launch_cache8_copy_pages(const Pool &, const Pool &, const int32_t *, const int32_t *, int, hipStream_t)
{
    reached("launch_cache8_copy_pages");
}
hipError_t launch_cache8_fork(const Pool &, const Pool &, const int32_t *, int64_t, const int32_t *, const int32_t *, const int32_t *,
                              int32_t *, int64_t, int32_t *, int32_t *, int32_t *, int, int, int, int32_t *, hipStream_t)
{
    reached("launch_cache8_fork");
}
hipError_t launch_cache8_compact(const Pool &, const Pool &, const int32_t *, int64_t, const int32_t *, int32_t *, int64_t,
                                 int32_t *, int32_t *, int, int, int32_t *, hipStream_t)
{
    reached("launch_cache8_compact");
}
hipError_t launch_attention8_decode(const Decode8Args &, void *, hipStream_t) { reached("launch_attention8_decode"); }
hipError_t launch_beam_select(const BeamArgs &, void *, hipStream_t) { reached("launch_beam_select"); }
hipError_t launch_beam_reorder(const void *, int64_t, void *, int64_t, const int32_t *, int, int, int64_t, hipStream_t)
{
    reached("launch_beam_reorder");
}

}  // namespace cfp32
