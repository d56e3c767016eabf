// gfx950 (MI355X, CDNA4) kernel of moe_rms_norm (include/moe.h): RMS norm of
// token rows with the residual's addition, to rows of the input's type and /
// or FP8 rows with a scale per 128 elements.
//
// One pass over HBM: a row is held in registers (16 bytes a lane and chunk of
// 512 elements, up to 8 chunks a wave, up to 16 waves a row) between the sum
// of squares and the scaling, so x and the residual are read once and every
// output is written once. The bound is HBM bandwidth in large calls and load
// latency in small ones, so a row is shared by more waves the fewer rows
// there are. Measured on MI355X with the residual and both outputs: 8 x 4096
// rows of 7168 bf16 370 us for 2.12 GB (5.7 TB/s; a 2 GB copy reaches 4.9),
// 128 rows 5 us, of which the launch is most.
//
// The mean of squares is summed the same way whatever the number of waves:
// FP32 sums of chunks of 512 elements (8 elements a lane in order, then a
// fixed tree over the lanes), added in chunk order. A row's result therefore
// does not depend on the other rows of the call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {
namespace {

using namespace ep::dev;
using namespace moe::dev;
using ep::kWave;

// DT: 0 bf16, 1 fp16 rows. WT: 0 bf16, 1 fp16, 2 fp32 weight. C: chunks a
// wave holds.
template <int C, int DT, int WT, bool kStream>
__global__ __launch_bounds__(kNormMaxWaves * kWave) void moe_norm_kernel(NormArgs a)
{
    constexpr int ld = Policy<kStream>::combine_load;
    constexpr int st = Policy<kStream>::combine_store;
    __shared__ float s_sum[kNormMaxWaves * kNormChunks];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int block_rows = (int)(blockDim.x / kWave) / a.row_waves;
    const int local = wave / a.row_waves;         // the block's row of this wave
    const int part = wave - local * a.row_waves;  // and its share of it
    const int64_t row = (int64_t)blockIdx.x * block_rows + local;
    bool mine = row < a.rows;
    if (mine && a.counts != nullptr) {
        const int64_t g = row / a.group_rows;
        mine = row - g * a.group_rows < (int64_t)a.counts[g];
    }
    // Only a row with one wave may leave here: waves that share a row meet at
    // the barrier below, and so do the waves of the block's other rows.
    if (!mine && a.row_waves == 1)
        return;

    const uint32_t bytes = mine ? (uint32_t)a.H * 2u : 0u;  // 0: nothing is read or written
    const int64_t at = mine ? row * a.H * 2 : 0;
    const __amdgpu_buffer_rsrc_t rx = row_rsrc(a.x + at, bytes);
    const int e0 = part * C * kNormChunk + lane * 8;  // first element of this lane
    u32x4 raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        raw[c] = bload16<ld>(rx, (uint32_t)(e0 + c * kNormChunk) * 2u);
    float h[C][8];
    if (a.res != nullptr) {
        const __amdgpu_buffer_rsrc_t rr = row_rsrc(a.res + at, bytes);
        const __amdgpu_buffer_rsrc_t ro = row_rsrc(a.res_out + at, bytes);
        u32x4 res[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            res[c] = bload16<ld>(rr, (uint32_t)(e0 + c * kNormChunk) * 2u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float f[8], r[8];
            widen<DT>(raw[c], f);
            widen<DT>(res[c], r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = f[i] + r[i];
            // the stream's stored value, which is also what is normalised
            const u32x4 v = narrow<DT>(f);
            bstore16<st>(v, ro, (uint32_t)(e0 + c * kNormChunk) * 2u);
            widen<DT>(v, h[c]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            widen<DT>(raw[c], h[c]);
    }

    float sums[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float v = h[c][0] * h[c][0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v = __builtin_fmaf(h[c][i], h[c][i], v);
        sums[c] = wave_sum(v);
    }
    // chunks past the row are zeros and change nothing
    float total = 0.0f;
    if (a.row_waves == 1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            total = total + sums[c];
    } else {
        float* s = s_sum + local * a.row_waves * C;
        if (lane == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                s[part * C + c] = sums[c];
        }
        __syncthreads();
        if (!mine)
            return;
        for (int i = 0; i < a.row_waves * C; ++i)
            total = total + s[i];
    }
    const float rms = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(total, (float)a.H) + a.eps));

    const uint32_t wbytes = (uint32_t)a.H * (WT == 2 ? 4u : 2u);
    const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.w, wbytes);
    const bool plain = a.out != nullptr, quant = a.codes != nullptr;
    const __amdgpu_buffer_rsrc_t rout = row_rsrc(a.out + at, plain ? bytes : 0u);
    const __amdgpu_buffer_rsrc_t rcode = row_rsrc(a.codes + at / 2, quant ? bytes / 2 : 0u);
    const uint32_t sbytes = (uint32_t)(a.H / 128) * 4u;
    const __amdgpu_buffer_rsrc_t rscale =
        row_rsrc(a.scales + (mine ? row * sbytes : 0), quant ? sbytes : 0u);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = e0 + c * kNormChunk;
        float w[8], y[8];
        if constexpr (WT == 2) {
            const u32x4 lo = bload16<0>(rw, (uint32_t)e * 4u);
            const u32x4 hi = bload16<0>(rw, (uint32_t)e * 4u + 16u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t l = lo[i], u = hi[i];  // bit_cast reads a vector's element 0
                w[i] = __builtin_bit_cast(float, l);
                w[4 + i] = __builtin_bit_cast(float, u);
            }
        } else {
            widen<WT>(bload16<0>(rw, (uint32_t)e * 2u), w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = h[c][i] * rms * w[i];
        if (plain)
            bstore16<st>(narrow<DT>(y), rout, (uint32_t)e * 2u);
        if (quant) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                amax = __builtin_fmaxf(amax, __builtin_fabsf(y[i]));
            float s, f;
            block_scale(row16_max(amax), &s, &f);
            const u32x2 q = {e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                             e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f)};
            __builtin_amdgcn_raw_buffer_store_b64(q, rcode, e, 0, st);
            if ((lane & 15) == 0)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, s), rscale,
                                                      (e / 128) * 4, 0, 0);
        }
    }
}

template <int C, int DT, int WT>
void norm_with(const NormArgs& a, dim3 grid, dim3 block, bool stream, hipStream_t s)
{
    if (stream)
        hipLaunchKernelGGL((moe_norm_kernel<C, DT, WT, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((moe_norm_kernel<C, DT, WT, false>), grid, block, 0, s, a);
}

template <int C>
void norm_types(const NormArgs& a, int dtype, int wtype, dim3 grid, dim3 block, bool stream,
                hipStream_t s)
{
    if (dtype == 0) {
        if (wtype == 2)
            norm_with<C, 0, 2>(a, grid, block, stream, s);
        else
            norm_with<C, 0, 0>(a, grid, block, stream, s);
    } else {
        if (wtype == 2)
            norm_with<C, 1, 2>(a, grid, block, stream, s);
        else
            norm_with<C, 1, 1>(a, grid, block, stream, s);
    }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, int wtype, bool stream, hipStream_t s)
{
    // a.chunks rounded up to a compiled count; the row has to fit its waves
    const int C = a.chunks <= 1 ? 1 : a.chunks <= 2 ? 2 : a.chunks <= 4 ? 4 : 8;
    if (a.rows < 1 || a.chunks < 1 || a.chunks > kNormChunks || a.row_waves < 1 ||
        a.row_waves > kNormMaxWaves || (int64_t)a.row_waves * C * kNormChunk < a.H)
        return hipErrorInvalidValue;
    const int waves = a.row_waves > 4 ? a.row_waves : 4;
    const int block_rows = waves / a.row_waves;
    const dim3 grid((unsigned)((a.rows + block_rows - 1) / block_rows));
    const dim3 block(waves * kWave);
    switch (C) {
    case 1: norm_types<1>(a, dtype, wtype, grid, block, stream, s); break;
    case 2: norm_types<2>(a, dtype, wtype, grid, block, stream, s); break;
    case 4: norm_types<4>(a, dtype, wtype, grid, block, stream, s); break;
    default: norm_types<8>(a, dtype, wtype, grid, block, stream, s); break;
    }
    return hipGetLastError();
}

}  // namespace moe
