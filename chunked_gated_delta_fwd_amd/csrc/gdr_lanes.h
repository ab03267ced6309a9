// Sums over the lanes of a wave without LDS, shared by the kernels of the
// operators around the recurrence.
#pragma once

#include "gdr_device.h"

namespace gdr {
namespace {

// Sum over LANES (a power of two from 8 to 64) neighbouring lanes, in each of
// them: within 8 by neighbours, pairs and a mirror, within 16 by another
// mirror, over the four rows of 16 by lane swaps.
template <int LANES>
__device__ __forceinline__ float lane_sum(float x) {
    x = dpp_add<0xB1, 0xF>(x);    // quad_perm 1 0 3 2
    x = dpp_add<0x4E, 0xF>(x);    // quad_perm 2 3 0 1
    x = dpp_add<0x141, 0xF>(x);   // mirror within 8
    if constexpr (LANES >= 16) x = dpp_add<0x140, 0xF>(x);   // mirror within 16
    if constexpr (LANES >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if constexpr (LANES >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    return x;
}
// Sum over the four rows of 16 lanes, in every lane.
__device__ __forceinline__ float sum_rows(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}


// The same in fp64, for sums whose differences count.
// x plus the value that DPP control CTRL moves in (0 where none is), in fp64
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add64(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(b), CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(b >> 32), CTRL, ROW_MASK, 0xF, false);
    return x + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double row_sum64(double x) {   // over a row of 16 lanes
    x = dpp_add64<0xB1, 0xF>(x);
    x = dpp_add64<0x4E, 0xF>(x);
    x = dpp_add64<0x141, 0xF>(x);
    return dpp_add64<0x140, 0xF>(x);
}
__device__ __forceinline__ double sum_rows64(double x) {
    auto join = [](uint32_t lo, uint32_t hi) {
        return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
    };
    uint64_t v = __builtin_bit_cast(uint64_t, x);
    const auto lo = __builtin_amdgcn_permlane16_swap(static_cast<uint32_t>(v), static_cast<uint32_t>(v), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(v >> 32), false, false);
    x = join(lo[0], hi[0]) + join(lo[1], hi[1]);
    v = __builtin_bit_cast(uint64_t, x);
    const auto lo2 = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(v), static_cast<uint32_t>(v), false, false);
    const auto hi2 = __builtin_amdgcn_permlane32_swap(static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(v >> 32), false, false);
    return join(lo2[0], hi2[0]) + join(lo2[1], hi2[1]);
}

}  // namespace
}  // namespace gdr
