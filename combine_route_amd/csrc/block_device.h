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
