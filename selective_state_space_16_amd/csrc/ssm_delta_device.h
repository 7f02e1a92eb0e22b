// What the prompts and the single tokens of the gated delta rule share.
#pragma once

#include "ssm_common.h"
#include "ssm_internal.h"

namespace ssm {

// 1 / sqrt(sum of squares + eps) of a key or query, or 1 where they are taken as they are.
__device__ __forceinline__ float unit_scale(float squares, float eps) { return eps >= 0.0f ? rsqrtf(squares + eps) : 1.0f; }

__device__ __forceinline__ float delta_gate(float raw) { return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-raw * kLog2e)); }

// v summed over groups of 8 lanes, in all of them: the neighbour, the other pair of
// four lanes, the other four.
__device__ __forceinline__ float sum8(float v) {
    auto dpp = [](float u, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(u), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
    v += dpp(v, std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
    return v + dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
}

}  // namespace ssm
