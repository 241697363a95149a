// Argument checks shared by the C-ABI files of the attention, cache and
// serving calls (host code).
#pragma once

#include <cmath>

#include "api_common.h"
#include "attention.h"

namespace cfp32 {

constexpr int64_t kMaxDim = kApiMaxDim;
constexpr int64_t kMaxSize = 0x7FFFFFFF;  // dimensions: int32 offsets and lengths
constexpr int64_t kMaxKeys = kMaxSize - 65535;  // of attention: int32 indices, and steps beyond the last
constexpr size_t kAlign = 256;            // slack for rounding a workspace pointer up

inline bool size_ok(int64_t v) { return v >= 0 && v <= kMaxSize; }
inline bool heads_ok(int64_t Hq, int64_t Hkv, int64_t D)
{
    return size_ok(Hq) && size_ok(Hkv) && size_ok(D) && D <= kAttnMaxDim && (Hkv == 0 ? Hq == 0 : Hq % Hkv == 0);
}
inline bool scale_ok(double scale) { return std::isfinite((float)scale); }  // as the kernels take it
inline bool type_ok(int t) { return t == CFP32_KV_F32 || t == CFP32_KV_F16; }

// log2 of a page size, -1 if it is not a power of two up to 65536.
inline int page_log2(int64_t page)
{
    if (page < 1 || page > 65536 || (page & (page - 1))) return -1;
    return __builtin_ctzll((unsigned long long)page);
}

inline bool term_ok(int64_t n, int64_t stride) { return stride >= 0 && (n <= 1 || stride <= kMaxDim / (n - 1)); }

// [n1, n2, n3, D] elements with these strides: non-negative, all within 2^48.
inline bool view_ok(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3, int64_t s3, int64_t D)
{
    if (!term_ok(n1, s1) || !term_ok(n2, s2) || !term_ok(n3, s3)) return false;
    const int64_t a = n1 > 1 ? (n1 - 1) * s1 : 0, b = n2 > 1 ? (n2 - 1) * s2 : 0, c = n3 > 1 ? (n3 - 1) * s3 : 0;
    return a + b + c + D <= kMaxDim;  // each term is below 2^48
}

// The rows of D elements of a written [n1, n2, n3, D] tensor do not overlap:
// in order of their strides, each dimension steps over all of the one below.
inline bool distinct_ok(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3, int64_t s3, int64_t D)
{
    int64_t n[3] = {n1, n2, n3}, s[3] = {s1, s2, s3};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i] || (s[j] == s[i] && n[j] < n[i])) {
                const int64_t ts = s[i], tn = n[i];
                s[i] = s[j], n[i] = n[j], s[j] = ts, n[j] = tn;
            }
    int64_t span = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < span) return false;
        span = (n[i] - 1) * s[i] + span;
    }
    return true;
}

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline void *align_up(void *p) { return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + kAlign - 1) & ~(uintptr_t)(kAlign - 1)); }

// one: of a table that is only read, all rows may be one (ld 0).
inline bool table_ok(const void *t, int64_t ld, int64_t rows, int64_t W, bool one = false)
{
    return (ld >= W || (one && ld == 0)) && term_ok(rows, ld) && (t || rows == 0 || W == 0);
}

}  // namespace cfp32
