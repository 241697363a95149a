// Exchanges between the lanes of a wave by data-parallel moves, without LDS
// (device code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace cfp32 {

// The value of lane ^ J.
template <int J>
__device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    static_assert(J == 1 || J == 2 || J == 4 || J == 8 || J == 16 || J == 32, "");
    constexpr int kSwapPairs = 0xB1, kSwapTwos = 0x4E, kReverseFour = 0x1B, kReverseEight = 0x141, kTurnHalf = 0x128;
    auto move = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, true);
    };
    if constexpr (J == 1) return move(v, std::integral_constant<int, kSwapPairs>{});
    if constexpr (J == 2) return move(v, std::integral_constant<int, kSwapTwos>{});
    if constexpr (J == 4)  // ^ 7, then ^ 3
        return move(move(v, std::integral_constant<int, kReverseEight>{}), std::integral_constant<int, kReverseFour>{});
    if constexpr (J == 8) return move(v, std::integral_constant<int, kTurnHalf>{});
    if constexpr (J == 16) {
        // Of two copies, the first's odd rows of 16 change places with the second's even ones.
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return threadIdx.x & 16 ? r[0] : r[1];
    }
    if constexpr (J == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    }
}

template <int J>
__device__ __forceinline__ float from_lane(float v) { return __builtin_bit_cast(float, from_lane<J>(__builtin_bit_cast(uint32_t, v))); }
template <int J>
__device__ __forceinline__ uint64_t from_lane(uint64_t v)
{
    return (uint64_t)from_lane<J>((uint32_t)(v >> 32)) << 32 | from_lane<J>((uint32_t)v);
}
template <int J>
__device__ __forceinline__ double from_lane(double v) { return __builtin_bit_cast(double, from_lane<J>(__builtin_bit_cast(uint64_t, v))); }

// The largest over the lanes of equal lane % 16.
__device__ __forceinline__ float max_of_quads(float v)
{
    v = fmaxf(v, from_lane<16>(v));
    return fmaxf(v, from_lane<32>(v));
}

}  // namespace cfp32
