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

// exp(-g) to 4 half steps (2 of v_exp_f32, a rounding of each factor) wherever it
// is normal: 2 to the power of -g log2(e), which one float holds only to |g| half
// steps of the result, as t + r, and 2^(t + r) = 2^t (1 + r ln 2). r is no number
// or anything where t is infinite or 2^t is 0 or infinite: held to [-1, 1] (a NaN
// to -1), it changes neither.
__device__ __forceinline__ float exp_minus(float g)
{
    constexpr double kLog2e = 1.4426950408889634;
    constexpr float hi = (float)kLog2e, lo = (float)(kLog2e - (double)hi);
    const float t = -g * hi;
    const float r = __builtin_fmaf(-g, lo, __builtin_fmaf(-g, hi, -t));
    return __builtin_amdgcn_exp2f(t) *
           __builtin_fmaf(__builtin_amdgcn_fmed3f(r, -1.0f, 1.0f), 0.6931471805599453f, 1.0f);
}

// silu(g) * u. Both sides of the quotient over 16, so that the reciprocal stays
// in the normal range wherever the exponential is finite.
__device__ __forceinline__ float silu_times(float g, float u)
{
    const float d = __builtin_fmaf(exp_minus(g), 0.0625f, 0.0625f);
    return g * 0.0625f * __builtin_amdgcn_rcpf(d) * u;
}

}  // namespace dev
}  // namespace moe
