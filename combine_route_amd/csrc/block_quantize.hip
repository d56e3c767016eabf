// gfx950 (MI355X, CDNA4) kernel of moe_quantize_int8 (include/moe_block.h):
// rows of bf16 / fp16 to INT8 codes with a scale per row.
//
// One pass over HBM: a row is held in registers (16 bytes a lane and chunk of
// 512 elements, up to 8 chunks a wave, up to 16 waves a row) between its
// largest magnitude and its codes. Bound by HBM bandwidth in large calls and
// by the launch in small ones. Measured on MI355X: 32768 rows of 2048 bf16 in
// groups 35 us (5.8 TB/s), 1024 rows 5.5 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_device.h"

namespace block {
namespace {

using namespace block::dev;

// DT: 0 bf16, 1 fp16 rows. C: chunks a wave holds.
template <int C, int DT, bool kStream>
__global__ __launch_bounds__(kQuantMaxWaves * kWave) void block_quantize_kernel(QuantizeArgs a)
{
    constexpr int ld = Policy<kStream>::combine_load;
    constexpr int st = Policy<kStream>::combine_store;
    __shared__ uint32_t s_max[kQuantMaxWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int block_rows = (int)(blockDim.x / kWave) / a.row_waves;
    const int local = wave / a.row_waves;         // the block's row of this wave
    const int part = wave - local * a.row_waves;  // and its share of it
    const int64_t row = (int64_t)blockIdx.x * block_rows + local;
    bool mine = row < a.n_rows;
    if (mine && a.counts != nullptr) {
        const int64_t g = row / a.group_rows;
        mine = row - g * a.group_rows < (int64_t)a.counts[g];
    }
    if (!mine && a.row_waves == 1)  // (waves that share a row meet at the barrier)
        return;
    const uint32_t bytes = mine ? (uint32_t)a.H * 2u : 0u;  // 0: nothing is read or written
    const int64_t at = mine ? row * a.H : 0;
    const __amdgpu_buffer_rsrc_t rx = row_rsrc(a.rows + at * 2, bytes);
    const int e0 = part * C * kNormChunk + lane * 8;
    u32x4 raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        raw[c] = bload16<ld>(rx, (uint32_t)(e0 + c * kNormChunk) * 2u);
    uint32_t amax = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float f[8];
        widen<DT>(raw[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = magnitude(f[i]);
            amax = amax > m ? amax : m;
        }
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
    const __amdgpu_buffer_rsrc_t rcode = row_rsrc(a.codes + at, bytes / 2);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float v[8];
        widen<DT>(raw[c], v);
        const u32x2 q = {int8x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                         int8x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f)};
        __builtin_amdgcn_raw_buffer_store_b64(q, rcode, e0 + c * kNormChunk, 0, st);
    }
    if (mine && part == 0 && lane == 0)
        a.scales[row] = s;
}

template <int C>
void quantize_with(const QuantizeArgs& a, int dtype, dim3 grid, dim3 block, bool stream,
                   hipStream_t s)
{
    if (dtype == 0) {
        if (stream)
            hipLaunchKernelGGL((block_quantize_kernel<C, 0, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_quantize_kernel<C, 0, false>), grid, block, 0, s, a);
    } else {
        if (stream)
            hipLaunchKernelGGL((block_quantize_kernel<C, 1, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_quantize_kernel<C, 1, false>), grid, block, 0, s, a);
    }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, int dtype, bool stream, hipStream_t s)
{
    // a.chunks rounded up to a compiled count; the row has to fit its waves
    const int C = a.chunks <= 1 ? 1 : a.chunks <= 2 ? 2 : a.chunks <= 4 ? 4 : 8;
    if (a.n_rows < 1 || a.chunks < 1 || a.chunks > kQuantChunks || a.row_waves < 1 ||
        a.row_waves > kQuantMaxWaves || (int64_t)a.row_waves * C * kNormChunk < a.H)
        return hipErrorInvalidValue;
    const int waves = a.row_waves > 4 ? a.row_waves : 4;
    const int block_rows = waves / a.row_waves;
    const dim3 grid((unsigned)((a.n_rows + block_rows - 1) / block_rows));
    const dim3 block(waves * kWave);
    switch (C) {
    case 1: quantize_with<1>(a, dtype, grid, block, stream, s); break;
    case 2: quantize_with<2>(a, dtype, grid, block, stream, s); break;
    case 4: quantize_with<4>(a, dtype, grid, block, stream, s); break;
    default: quantize_with<8>(a, dtype, grid, block, stream, s); break;
    }
    return hipGetLastError();
}

}  // namespace block
