// Device helpers of the layer operators' kernels: sums and maxima over lanes
// with DPP moves (register to register, no LDS traffic).
#pragma once

#include "ep_device.h"
#include "moe_kernels.h"

namespace moe {
namespace dev {

// DPP controls: lanes swapped inside a quad, a half row (8) and a row (16)
// mirrored. Applied in this order to a commutative operation, every lane of a
// row of 16 ends up with the row's result.
constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, true));
}

__device__ __forceinline__ float row16_max(float v)
{
    v = __builtin_fmaxf(v, dpp<kDppXor1>(v));
    v = __builtin_fmaxf(v, dpp<kDppXor2>(v));
    v = __builtin_fmaxf(v, dpp<kDppHalfMirror>(v));
    return __builtin_fmaxf(v, dpp<kDppMirror>(v));
}

__device__ __forceinline__ float row16_sum(float v)
{
    v = v + dpp<kDppXor1>(v);
    v = v + dpp<kDppXor2>(v);
    v = v + dpp<kDppHalfMirror>(v);
    return v + dpp<kDppMirror>(v);
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Sum over the wave, the same in every lane; each addition's operands are
// fixed, so the result depends on the values alone.
__device__ __forceinline__ float wave_sum(float v)
{
    v = row16_sum(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Scale and its inverse factor of a block with largest magnitude amax.
__device__ __forceinline__ void block_scale(float amax, float* scale, float* factor)
{
    const float u = __builtin_fmaxf(amax, kTinyAmax);
    *scale = amax > 0.0f ? __fdiv_rn(u, ep::dev::kE4M3Max) : 1.0f;
    *factor = __fdiv_rn(ep::dev::kE4M3Max, u);
}

}  // namespace dev
}  // namespace moe
