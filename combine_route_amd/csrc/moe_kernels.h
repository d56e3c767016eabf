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

// moe_backward.hip: gradients of the fused dispatch and combine, through the
// per-slot map of the expert plan's last fused dispatch.
constexpr int kBackChunks = 4;       // 512-element chunks a wave holds at a time
constexpr int kBackMaxWaves = 16;

struct CombineBackwardArgs {
    const uint8_t* go;           // [W][M][H] gradient of the combined rows
    const int32_t* idx;          // [W][M][k]
    const float* w;              // [W][M][k] or null
    const uint8_t* py;           // [W * Er][cap][H], null without grad_w
    const int32_t* fslot;        // [W][M][k]
    uint8_t* gy;                 // [W * Er][cap][H]
    float* gw;                   // [W][M][k] or null
    int32_t row_vecs;            // 16-byte vectors a row
    int32_t row_waves;           // waves a token: a power of two up to kBackMaxWaves
    int32_t wave_vecs;           // vectors of a wave's share of the row
    int32_t group_slots;         // slots a wave handles, 1 .. 64
    int32_t M, k, E;
};

struct DispatchBackwardArgs {
    const uint8_t* gp;           // [W * Er][cap][H] gradient of the packed rows
    const int32_t* fslot;        // [W][M][k]
    uint8_t* gx;                 // [W][M][H]
    int32_t row_vecs;
    int32_t pieces;              // of 64 vectors, a wave each
    int32_t M, k;
};

hipError_t launch_combine_backward(const CombineBackwardArgs& a, const ep::TokenMap& tk, int dtype,
                                   bool stream, hipStream_t s);
hipError_t launch_dispatch_backward(const DispatchBackwardArgs& a, const ep::TokenMap& tk,
                                    int dtype, int waves, bool stream, hipStream_t s);

// moe_gemm.hip: the grouped FP8 product.
struct GemmArgs {
    const uint8_t* a;            // [groups][cap][k] E4M3
    const uint8_t* as;           // [groups][cap][k / 128] float
    const uint8_t* b;            // [groups][n][k] E4M3
    const float* bs;             // [groups][ceil(n / 128)][k / 128]
    const int32_t* counts;       // [groups] or null
    uint8_t* out;                // [groups][cap][n] bf16 / fp16, or [groups][cap][n / 2] E4M3
    uint8_t* osc;                // [groups][cap][n / 256] float (swiglu)
    int32_t groups, cap, n, k;
    int32_t col_tiles;           // ceil(n / 256)
};

hipError_t launch_gemm(const GemmArgs& a, int dtype, bool swiglu, int blocks, hipStream_t s);

}  // namespace moe
