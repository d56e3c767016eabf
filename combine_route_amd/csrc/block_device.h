// Device helpers of the kernels of a whole MoE block.
#pragma once

#include "block_kernels.h"
#include "moe_device.h"

namespace block {
namespace dev {

using namespace ep::dev;
using namespace moe::dev;
using ep::kWave;

// Largest of the wave's values as bit patterns: of magnitudes (sign clear)
// the largest magnitude, a NaN above every number.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v)
{
    auto step = [&](auto ctrl) {
        const int i = (int)v;
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xF,
                                                                 0xF, true);
        v = v > o ? v : o;
    };
    step(std::integral_constant<int, kDppXor1>());
    step(std::integral_constant<int, kDppXor2>());
    step(std::integral_constant<int, kDppHalfMirror>());
    step(std::integral_constant<int, kDppMirror>());
    uint32_t m = 0;
#pragma unroll
    for (int l = 0; l < kWave; l += 16) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, l);
        m = m > o ? m : o;
    }
    return m;
}

__device__ __forceinline__ uint32_t magnitude(float v)
{
    return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}

// Scale and its inverse factor of an INT8 row whose largest magnitude has
// these bits. NaN and infinity stay in the scale (and give codes of 0).
__device__ __forceinline__ void int8_scale(uint32_t amax_bits, float* scale, float* factor)
{
    const float amax = __builtin_bit_cast(float, amax_bits);
    const float u = amax <= moe::kTinyAmax ? moe::kTinyAmax : amax;
    *scale = amax_bits ? __fdiv_rn(u, 127.0f) : 1.0f;
    *factor = __fdiv_rn(127.0f, u);
}

// 4 INT8 codes, one a byte in order: nearest whole number, ties to even, NaN
// 0. The factor keeps |v| under 127.5.
__device__ __forceinline__ uint32_t int8x4(float f0, float f1, float f2, float f3)
{
    auto code = [](float v) {
        return (uint32_t)(int)__builtin_rintf(v == v ? v : 0.0f) & 0xFFu;
    };
    return code(f0) | code(f1) << 8 | code(f2) << 16 | code(f3) << 24;
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

// 8 weights as they lie. WT: 0 bf16, 1 fp16, 2 fp32.
template <int WT>
struct Weights8 {
    static constexpr int kBytes = WT == 2 ? 4 : 2;
    u32x4 v[WT == 2 ? 2 : 1];

    // From element e on; zeros past the resource.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int e)
    {
#pragma unroll
        for (int i = 0; i < (WT == 2 ? 2 : 1); ++i)
            v[i] = bload16<0>(r, (uint32_t)e * kBytes + 16u * i);
    }

    __device__ __forceinline__ void widen8(float (&w)[8]) const
    {
        if constexpr (WT == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = v[i / 4][i % 4];  // bit_cast reads a vector's element 0
                w[i] = __builtin_bit_cast(float, u);
            }
        } else {
            widen<WT>(v[0], w);
        }
    }
};

template <int WT>
__device__ __forceinline__ void weights8(__amdgpu_buffer_rsrc_t r, int e, float (&w)[8])
{
    Weights8<WT> v;
    v.load(r, e);
    v.widen8(w);
}

}  // namespace dev
}  // namespace block
