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

}  // namespace
}  // namespace gdr
