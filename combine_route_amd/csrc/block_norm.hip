// gfx950 (MI355X, CDNA4) kernel of moe_block_norm (include/moe_block.h): the
// norm after a block, its gate and scaled residual, and the norm before the
// next block, to rows of the input's type and / or FP8 or INT8 rows.
//
// One pass over HBM: a row is held in registers (16 bytes a lane and chunk of
// 512 elements, up to 4 chunks a wave, up to 16 waves a row) from its load to
// the last store, through the two sums of squares and, of INT8 rows, the
// largest magnitude. The bound is HBM bandwidth in large calls and load
// latency in small ones, so a row is shared by more waves the fewer rows
// there are. Measured on MI355X: 8 x 4096 rows of 7168 bf16 with a gate a rank
// to INT8 rows 286 us for 1.64 GB (5.8 TB/s; a 2 GB copy reaches 4.95), 128 rows
// to bf16 and FP8 rows 6 us. (Weights asked for together with the row instead
// of where they are used: 6.0 -> 6.2 us there, and a third more registers.)
//
// Each mean of squares is summed the same way whatever the number of waves:
// FP32 sums of chunks of 512 elements (8 elements a lane in order, then a
// fixed tree over the lanes), added by a fixed tree over the chunks. A row's
// result therefore does not depend on the other rows of the call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_device.h"

namespace block {
namespace {

using namespace block::dev;

// Sum of squares of a row, the waves that share it adding their chunks'
// sums through s (an array of this sum's own).
template <int C>
__device__ __forceinline__ float square_sum(const float (&h)[C][8], float* s, int part,
                                            int row_waves, int lane)
{
    float sums[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float q = h[c][0] * h[c][0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            q = __builtin_fmaf(h[c][i], h[c][i], q);
        sums[c] = wave_sum(q);
    }
    // the chunks' sums by a fixed tree over 64 of them; those past the row are
    // zeros and change nothing
    if (row_waves == 1) {
        if constexpr (C == 1)
            return sums[0];
        else if constexpr (C == 2)
            return sums[0] + sums[1];
        else
            return (sums[0] + sums[1]) + (sums[2] + sums[3]);
    }
    static_assert(kNormMaxWaves * C <= kWave && C <= 4, "a lane a chunk");
    if (lane == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            s[part * C + c] = sums[c];
    }
    __syncthreads();
    const float v = s[lane < row_waves * C ? lane : 0];
    return wave_sum(lane < row_waves * C ? v : 0.0f);
}

__device__ __forceinline__ float inverse_rms(float total, int H, float eps)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(total, (float)H) + eps));
}

// DT: 0 bf16, 1 fp16 rows. WT: 0 bf16, 1 fp16, 2 fp32 weights. C: chunks a
// wave holds.
template <int C, int DT, int WT, bool kStream>
__global__ __launch_bounds__(kNormMaxWaves * kWave) void block_norm_kernel(NormArgs a)
{
    constexpr int ld = Policy<kStream>::combine_load;
    constexpr int st = Policy<kStream>::combine_store;
    constexpr int kSums = kNormMaxWaves * kNormChunks;
    __shared__ float s_sum[2][kSums];
    __shared__ uint32_t s_max[kNormMaxWaves];
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
    // the barriers below, and so do the waves of the block's other rows.
    if (!mine && a.row_waves == 1)
        return;

    const uint32_t bytes = mine ? (uint32_t)a.H * 2u : 0u;  // 0: nothing is read or written
    const int64_t at = mine ? row * a.H * 2 : 0;
    const __amdgpu_buffer_rsrc_t ry = row_rsrc(a.y + at, bytes);
    const __amdgpu_buffer_rsrc_t rr = row_rsrc(a.res + at, bytes);
    const int e0 = part * C * kNormChunk + lane * 8;  // first element of this lane
    u32x4 raw[C], res[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        raw[c] = bload16<ld>(ry, (uint32_t)(e0 + c * kNormChunk) * 2u);
#pragma unroll
    for (int c = 0; c < C; ++c)
        res[c] = bload16<ld>(rr, (uint32_t)(e0 + c * kNormChunk) * 2u);
    const uint32_t wbytes = (uint32_t)a.H * (WT == 2 ? 4u : 2u);
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
        widen<DT>(raw[c], h[c]);
    if (a.post != nullptr) {
        const float rms = inverse_rms(
            square_sum<C>(h, s_sum[0] + local * a.row_waves * C, part, a.row_waves, lane), a.H,
            a.eps);
        const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.post, wbytes);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            weights8<WT>(rw, e0 + c * kNormChunk, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] = h[c][i] * rms * w[i];
        }
    }
    if (a.gate != nullptr) {
        const __amdgpu_buffer_rsrc_t rw =
            row_rsrc(a.gate + (mine ? row / a.gate_rows : 0) * wbytes, wbytes);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            weights8<WT>(rw, e0 + c * kNormChunk, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[c][i] = h[c][i] * w[i];
        }
    }
    const __amdgpu_buffer_rsrc_t ro = row_rsrc(a.res_out + at, bytes);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float r[8];
        widen<DT>(res[c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[c][i] = __builtin_fmaf(a.res_scale, r[i], h[c][i]);
        bstore16<st>(narrow<DT>(h[c]), ro, (uint32_t)(e0 + c * kNormChunk) * 2u);
    }
    if (a.pre == nullptr)
        return;

    const float rms = inverse_rms(
        square_sum<C>(h, s_sum[1] + local * a.row_waves * C, part, a.row_waves, lane), a.H, a.eps);
    const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.pre, wbytes);
    uint32_t amax = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float w[8];
        weights8<WT>(rw, e0 + c * kNormChunk, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[c][i] = h[c][i] * rms * w[i];
            // (past the row: zeros, unless the row holds no number at all)
            const uint32_t m = magnitude(h[c][i]);
            amax = amax > m ? amax : m;
        }
    }
    if (a.out != nullptr) {
        const __amdgpu_buffer_rsrc_t rout = row_rsrc(a.out + at, bytes);
#pragma unroll
        for (int c = 0; c < C; ++c)
            bstore16<st>(narrow<DT>(h[c]), rout, (uint32_t)(e0 + c * kNormChunk) * 2u);
    }
    if (a.kind == kNoCodes)
        return;
    const __amdgpu_buffer_rsrc_t rcode = row_rsrc(a.codes + at / 2, bytes / 2);
    if (a.kind == kFp8Codes) {
        const uint32_t sbytes = (uint32_t)(a.H / 128) * 4u;
        const __amdgpu_buffer_rsrc_t rscale =
            row_rsrc(a.scales + (mine ? row * sbytes : 0), mine ? sbytes : 0u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = e0 + c * kNormChunk;
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = __builtin_fmaxf(m, __builtin_fabsf(h[c][i]));
            float s, f;
            block_scale(row16_max(m), &s, &f);
            const u32x2 q = {e4m3x4(h[c][0] * f, h[c][1] * f, h[c][2] * f, h[c][3] * f),
                             e4m3x4(h[c][4] * f, h[c][5] * f, h[c][6] * f, h[c][7] * f)};
            __builtin_amdgcn_raw_buffer_store_b64(q, rcode, e, 0, st);
            if ((lane & 15) == 0)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, s), rscale,
                                                      (e / 128) * 4, 0, 0);
        }
        return;
    }
    uint32_t top = wave_umax(amax);
    if (a.row_waves > 1) {
        uint32_t* s = s_max + local * a.row_waves;
        if (lane == 0)
            s[part] = top;
        __syncthreads();
        top = wave_umax(s[lane < a.row_waves ? lane : 0]);
    }
    float s, f;
    int8_scale(top, &s, &f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const u32x2 q = {int8x4(h[c][0] * f, h[c][1] * f, h[c][2] * f, h[c][3] * f),
                         int8x4(h[c][4] * f, h[c][5] * f, h[c][6] * f, h[c][7] * f)};
        __builtin_amdgcn_raw_buffer_store_b64(q, rcode, e0 + c * kNormChunk, 0, st);
    }
    if (mine && part == 0 && lane == 0)
        reinterpret_cast<float*>(a.scales)[row] = s;
}

template <int C, int DT, int WT>
void norm_with(const NormArgs& a, dim3 grid, dim3 block, bool stream, hipStream_t s)
{
    if (stream)
        hipLaunchKernelGGL((block_norm_kernel<C, DT, WT, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((block_norm_kernel<C, DT, WT, false>), grid, block, 0, s, a);
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
    const int C = a.chunks <= 1 ? 1 : a.chunks <= 2 ? 2 : 4;
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
    default: norm_types<4>(a, dtype, wtype, grid, block, stream, s); break;
    }
    return hipGetLastError();
}

}  // namespace block
