// Argument structs and launch entry points of the layer operators' kernels
// (include/moe.h): RMS norm, the grouped FP8 product and the gradients of the
// fused dispatch and combine. Internal; the host side is moe_host.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_kernels.h"

namespace moe {

// Block maxima below this are quantized as if they were it, so that 448 over
// the maximum stays finite.
constexpr float kTinyAmax = 0x1p-100f;

// moe_norm.hip: chunks of kNormChunk elements, 16 bytes a lane; a wave keeps
// up to kNormChunks of its row in registers.
constexpr int kNormChunk = 512;
constexpr int kNormChunks = 8;
constexpr int kNormMaxWaves = 16;
constexpr int kNormMaxHidden = kNormChunk * kNormChunks * kNormMaxWaves;

struct NormArgs {
    const uint8_t* x;
    const uint8_t* res;          // or null
    uint8_t* res_out;
    const uint8_t* w;
    uint8_t* out;                // or null
    uint8_t* codes;              // or null
    uint8_t* scales;
    const int32_t* counts;       // or null
    int64_t rows, group_rows;
    int32_t H;
    int32_t row_waves;           // waves a row: a power of two up to kNormMaxWaves
    int32_t chunks;              // chunks a wave, <= kNormChunks
    float eps;
};

// dtype, wtype: 0 bf16, 1 fp16 (wtype also 2: fp32).
hipError_t launch_norm(const NormArgs& a, int dtype, int wtype, bool stream, hipStream_t s);

}  // namespace moe
