// Argument structs and launch entry points of the kernels of a whole MoE
// block (include/moe_block.h). Internal; the host side is block_host.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_kernels.h"
#include "moe_kernels.h"

namespace block {

// block_norm.hip: chunks of 512 elements, 16 bytes a lane; a wave keeps up to
// kNormChunks of each of its rows in registers.
constexpr int kNormChunk = moe::kNormChunk;
constexpr int kNormChunks = 4;
constexpr int kNormMaxWaves = 16;
constexpr int kNormMaxHidden = kNormChunk * kNormChunks * kNormMaxWaves;

enum { kNoCodes = 0, kFp8Codes = 1, kInt8Codes = 2 };

struct NormArgs {
    const uint8_t* y;
    const uint8_t* res;
    uint8_t* res_out;
    const uint8_t* post;         // or null
    const uint8_t* gate;         // or null
    const uint8_t* pre;          // null without out and codes
    uint8_t* out;                // or null
    uint8_t* codes;              // or null
    uint8_t* scales;
    const int32_t* counts;       // or null
    int64_t rows, group_rows;
    int64_t gate_rows;           // rows a gate, `rows` for one gate
    int32_t H;
    int32_t row_waves;           // waves a row: a power of two up to kNormMaxWaves
    int32_t chunks;              // chunks a wave, <= kNormChunks
    int32_t kind;                // of the codes
    float res_scale, eps;
};

// dtype, wtype: 0 bf16, 1 fp16 (wtype also 2: fp32).
hipError_t launch_norm(const NormArgs& a, int dtype, int wtype, bool stream, hipStream_t s);

// block_backward.hip. A block of row_waves waves walks rows of one group, or
// whole groups, and holds the sums over its rows.
constexpr int kBackChunks = 4;

struct NormBackwardArgs {
    const uint8_t* y;
    const uint8_t* h;            // or null
    const uint8_t* gh;           // or null
    const uint8_t* go;           // or null
    const uint8_t* post;         // or null
    const uint8_t* gate;         // or null
    const uint8_t* pre;          // null iff go is
    uint8_t* gy;
    uint8_t* gres;               // or null
    float* gpost;                // or null
    float* ggate;                // or null
    float* gpre;                 // or null
    float* part;                 // [3][blocks][H]: post, gate, pre
    const int32_t* counts;       // or null
    int64_t groups, group_rows;
    int32_t group_blocks;        // blocks a group; 1 if a block walks several
    int32_t block_groups;        // groups a block
    int32_t blocks;
    int32_t gates;               // gates: 1, or `groups`
    int32_t H;
    int32_t row_waves;
    int32_t chunks;              // chunks a wave, <= kBackChunks
    float res_scale, eps;
};

hipError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, int wtype, bool stream,
                                hipStream_t s);

// block_quantize.hip: rows to INT8 rows. A wave keeps up to kQuantChunks
// chunks of its row in registers.
constexpr int kQuantChunks = 8;
constexpr int kQuantMaxWaves = 16;
constexpr int kQuantMaxHidden = kNormChunk * kQuantChunks * kQuantMaxWaves;

struct QuantizeArgs {
    const uint8_t* rows;
    uint8_t* codes;
    float* scales;
    const int32_t* counts;       // or null
    int64_t n_rows, group_rows;
    int32_t H;
    int32_t row_waves;           // waves a row: a power of two up to kQuantMaxWaves
    int32_t chunks;              // chunks a wave, <= kQuantChunks
};

hipError_t launch_quantize(const QuantizeArgs& a, int dtype, bool stream, hipStream_t s);

// block_gemm.hip: the grouped INT8 product.
struct GemmArgs {
    const uint8_t* a;            // [groups][cap][k] int8
    const float* as;             // [groups][cap]
    const uint8_t* b;            // [groups][n][k] int8
    const float* bs;             // [groups][n]
    const int32_t* counts;       // [groups] or null
    uint8_t* out;                // [groups][cap][n or n / 2] bf16 / fp16
    int32_t groups, cap, n, k;
    int32_t col_tiles;           // of 256 weight rows: ceil(n / 256), ceil(n / 2 / 128) of swiglu
};

hipError_t launch_gemm(const GemmArgs& a, int dtype, bool swiglu, int blocks, hipStream_t s);

// block_few.hip: a layer's experts for a few tokens.
constexpr int kFewMaxTokens = 64;
constexpr int kFewMaxSlots = 1024;   // tokens * topk
constexpr int kFewMaxExperts = 65536;

struct FewArgs {
    const uint8_t* x;            // [T][H] bf16 / fp16
    const int32_t* ids;          // [T][topk]
    const float* w;              // [T][topk] or null
    const uint8_t* up;           // [E][2 I][H] E4M3 or int8
    const float* ups;
    const uint8_t* down;         // [E][H][I]
    const float* downs;
    uint8_t* out;                // [T][H]
    uint8_t* act;                // [2][T * topk][I] bf16: hidden values, their rests
    int32_t T, topk, E, H, I;
    int32_t hits;                // most experts a call of these sizes can hit
    int32_t splits;              // pieces of I in the down product
};

// dtype: 0 bf16, 1 fp16; wtype: 0 E4M3, 1 int8.
hipError_t launch_few(const FewArgs& a, int dtype, int wtype, hipStream_t s);

}  // namespace block
