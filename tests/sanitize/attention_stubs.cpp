// Launcher stubs of the attention and cache calls for the host-only sanitizer
// build: attention_api.hip and attention_plans.hip are built with
// AddressSanitizer and UndefinedBehaviorSanitizer and linked against these
// instead of the kernels.  No check gets as far as a launch, so every stub aborts.
#include <cstdio>
#include <cstdlib>

#include "../../compensated_fp32_projection_amd/csrc/attention.h"

namespace cfp32 {

[[noreturn]] static void reached(const char *name)
{
    std::fprintf(stderr, "launcher stub reached: %s\n", name);
    std::abort();
}

hipError_t launch_attention_prompt(const PromptArgs &, void *, hipStream_t) { reached("launch_attention_prompt"); }
hipError_t launch_attention_decode(const DecodeArgs &, void *, hipStream_t) { reached("launch_attention_decode"); }
hipError_t launch_cache_reserve(const int32_t *, int64_t, const int32_t *, const int32_t *, const int32_t *, int32_t *, int64_t,
                                int32_t *, int32_t *, int, int, int, int, hipStream_t)
{
    reached("launch_cache_reserve");
}
hipError_t launch_cache_append(const HeadsView &, const HeadsView &, const int32_t *, const int32_t *, int32_t *, const Pool &,
                               const int32_t *, int64_t, int, int, int, hipStream_t)
{
    reached("launch_cache_append");
}
hipError_t launch_cache_copy_pages(const Pool &, const int32_t *, const int32_t *, int, hipStream_t)
{
    reached("launch_cache_copy_pages");
}
hipError_t launch_cache_fork(const Pool &, const int32_t *, int64_t, const int32_t *, const int32_t *, const int32_t *,
                             int32_t *, int64_t, int32_t *, int32_t *, int32_t *, int, int, int, int32_t *, hipStream_t)
{
    reached("launch_cache_fork");
}
hipError_t launch_cache_free(const int32_t *, int64_t, const int32_t *, int32_t *, int, int, int, hipStream_t)
{
    reached("launch_cache_free");
}
hipError_t launch_cache_compact(const Pool &, const int32_t *, int64_t, const int32_t *, int32_t *, int64_t, int32_t *,
                                int32_t *, int, int, int32_t *, hipStream_t)
{
    reached("launch_cache_compact");
}

}  // namespace cfp32
