// Arguments and launcher of the rotary kernel (internal to libcfp32).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cfp32 {

constexpr int kRotaryMaxDim = 1024;

struct RotaryTensor {
    const void *in;
    void *out;
    int64_t in_tok, in_head, out_tok, out_head;  // element strides
    int heads;
};

struct RotaryArgs {
    RotaryTensor q, k;
    const int64_t *positions;
    const double *frequencies;
    float amplitude;
    bool f16, interleaved, transpose;
    int T, D, R;
};

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream);

}  // namespace cfp32
