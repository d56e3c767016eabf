// gfx950 (MI355X, CDNA4) kernels of the gradients of the fused expert-major
// path (include/moe.h): moe_combine_backward and moe_dispatch_backward.
//
// Both go through the per-slot map the fused dispatch wrote: the packed row of
// each slot that is its expert's first in the token and was kept, else -1.
//   combine backward   The combine's output row of token t is sum over its
//            kept pairs of c_p * y_p, so the gradient of pair p's row is
//            c_p * go_t and that of c_p is <go_t, y_p>; c_p sums the weights
//            of every slot naming the expert, so each of those slots gets the
//            same dot. A token's row of go is read once into registers by the
//            waves that share it; every pair's row of y is read once and its
//            gradient row written once while it is at hand.
//   dispatch backward  A token's packed rows are copies of it, so its
//            gradient is their gradients' sum: FP32, in slot order, from the
//            first, rounded once.
// Both move bytes: the bound is HBM bandwidth. Measured on MI355X, 8 ranks x
// 2048 tokens x 7168 bf16, top-8: combine backward 778 us for 3.99 GB, half
// read and half written (5.1 TB/s; a 2 GB copy reaches 4.9), dispatch backward
// 362 us for 2.11 GB, 8 of 9 read (5.8 TB/s). Tried and no faster: 2 or 7
// chunks a wave instead of 4 (780, 793 us), stores or loads through the caches
// (808, 789 us), row pieces of 2 KB or 4 and 8 waves a block in the dispatch's
// (377, 368, 373 us). Nothing depends on the launch:
// a dot is summed over fixed shares of the row (chosen by the row's length
// alone) and a row's sum runs in slot order whatever the pieces.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {
namespace {

using namespace ep::dev;
using namespace moe::dev;
using ep::kWave;
using ep::TokenMap;

// kDot: the weights' gradient is asked for (and the pairs' rows are read). A
// block row of the grid takes group_slots of the tokens' slots: the pairs of a
// token are independent of each other.
template <int DT, bool kDot, bool kStream>
__global__ __launch_bounds__(kBackMaxWaves * kWave) void moe_combine_backward_kernel(
    CombineBackwardArgs a, TokenMap tk)
{
    constexpr int C = kBackChunks;
    constexpr int ld = Policy<kStream>::combine_load;
    constexpr int st = Policy<kStream>::combine_store;
    __shared__ float s_dot[kBackMaxWaves][ep::kMaxTopk];  // [wave][slot]
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int block_tokens = (int)(blockDim.x / kWave) / a.row_waves;
    const int local = wave / a.row_waves;
    const int part = wave - local * a.row_waves;
    const int flat = (int)blockIdx.x * block_tokens + local;
    const bool mine = flat < tk.total;
    const int r = rank_of_token(tk, mine ? flat : 0);
    const int64_t tok = (int64_t)r * a.M + (flat - tk.tok_start[r]);

    // lane j < k: slot j of the token
    const bool has = mine && lane < a.k;
    const int32_t id = has ? a.idx[tok * a.k + lane] : -1;
    const bool valid = has && id >= 0 && id < a.E;
    const int32_t row = has ? a.fslot[tok * a.k + lane] : -1;
    float c = 1.0f;
    int first = lane;  // the first slot naming this slot's expert
    if (a.w != nullptr) {
        const float own = has ? a.w[tok * a.k + lane] : 0.0f;
        c = own;
        for (int j = a.k - 1; j >= 0; --j) {
            const int ij = __builtin_amdgcn_readlane(id, j);
            if (ij == id && j < lane)
                first = j;
        }
        // weights of the later slots naming the expert, in slot order (as the
        // combine sums them)
        for (int j = 0; j < a.k; ++j) {
            const int ij = __builtin_amdgcn_readlane(id, j);
            const float wj = lane_value(own, j);
            if (j > lane && ij == id)
                c = c + wj;
        }
    }
    if constexpr (kDot)
        s_dot[wave][lane] = 0.0f;

    const uint32_t bytes = (uint32_t)a.row_vecs * 16u;
    const __amdgpu_buffer_rsrc_t rgo = row_rsrc(a.go + (mine ? tok : 0) * (int64_t)bytes,
                                                mine ? bytes : 0u);
    const int slot0 = (int)blockIdx.y * a.group_slots;
    const uint64_t group = (~0ull >> (kWave - a.group_slots)) << slot0;
    const uint64_t kept = __ballot(row >= 0) & group;
    const int vbeg = part * a.wave_vecs;
    const int vend = min(a.row_vecs, vbeg + a.wave_vecs);
    for (int v0 = vbeg; v0 < vend && kept != 0; v0 += kWave * C) {
        // a column past the share reads zeros from the row's end
        uint32_t off[C];
        u32x4 raw[C];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int v = v0 + u * kWave + lane;
            off[u] = v < vend ? (uint32_t)v * 16u : bytes;
            raw[u] = bload16<ld>(rgo, off[u]);
        }
        u32x4 y[2][C];
        auto load = [&](uint64_t left, u32x4 (&b)[C]) {
            const int64_t p = left ? __builtin_amdgcn_readlane(row, __builtin_ctzll(left)) : 0;
            const __amdgpu_buffer_rsrc_t ry = row_rsrc(a.py + p * bytes, left ? bytes : 0u);
#pragma unroll
            for (int u = 0; u < C; ++u)
                b[u] = bload16<ld>(ry, off[u]);
        };
        auto pair = [&](uint64_t left, const u32x4 (&b)[C]) {
            const int slot = __builtin_ctzll(left);
            const int64_t p = __builtin_amdgcn_readlane(row, slot);
            const float cp = lane_value(c, slot);
            const __amdgpu_buffer_rsrc_t rg = row_rsrc(a.gy + p * bytes, bytes);
            float dot = 0.0f;
#pragma unroll
            for (int u = 0; u < C; ++u) {
                float g[8], f[8];
                widen<DT>(raw[u], g);
                if constexpr (kDot) {
                    widen<DT>(b[u], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dot = __builtin_fmaf(g[e], f[e], dot);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = cp * g[e];
                bstore16<st>(narrow<DT>(f), rg, off[u]);
            }
            if constexpr (kDot) {
                const float sum = wave_sum(dot);
                if (lane == slot)
                    s_dot[wave][slot] += sum;
            }
        };
        uint64_t left = kept;
        if constexpr (kDot)
            load(left, y[0]);
        while (left) {  // uniform: two pairs a pass, the next one's row in flight
            const uint64_t next = left & (left - 1);
            if constexpr (kDot)
                load(next, y[1]);
            pair(left, y[0]);
            if (!next)
                break;
            left = next & (next - 1);
            if constexpr (kDot)
                load(left, y[0]);
            pair(next, y[1]);
        }
    }
    if constexpr (kDot) {
        __syncthreads();
        if (part == 0 && has && (group >> first & 1)) {
            float g = 0.0f;
            for (int i = 0; i < a.row_waves; ++i)
                g = g + s_dot[wave + i][first];
            a.gw[tok * a.k + lane] = valid ? g : 0.0f;
        }
    }
}

// A wave per (token, row piece of 1 KB); pieces of a token run in neighbouring
// waves, so its rows are read whole at about the same time.
template <int DT, bool kStream>
__global__ __launch_bounds__(1024) void moe_dispatch_backward_kernel(DispatchBackwardArgs a,
                                                                     TokenMap tk)
{
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t item = blockIdx.x * (blockDim.x / kWave) + uniform(threadIdx.x / kWave);
    const uint32_t flat_u = item / (uint32_t)a.pieces;
    if (flat_u >= (uint32_t)tk.total)
        return;  // whole waves only
    const int flat = (int)flat_u;
    const int piece = (int)(item - flat_u * (uint32_t)a.pieces);
    const int r = rank_of_token(tk, flat);
    const int64_t tok = (int64_t)r * a.M + (flat - tk.tok_start[r]);
    const int32_t row = lane < a.k ? a.fslot[tok * a.k + lane] : -1;
    // the kept rows moved to lanes 0 .. n - 1 in slot order, the others behind
    const uint64_t kept = __ballot(row >= 0);
    const int n = __popcll(kept);
    const int to = row >= 0 ? lanes_below(kept) : n + lanes_below(~kept);
    const int32_t gl = __builtin_amdgcn_ds_permute(to * 4, row);

    const uint32_t bytes = (uint32_t)a.row_vecs * 16u;
    const __amdgpu_buffer_rsrc_t rdst = row_rsrc(a.gx + tok * bytes, bytes);
    const int vbeg = piece * kWave;
    const int vend = min(a.row_vecs, vbeg + kWave);
    fold_rows_streamed<1, DT, kStream>(a.gp, bytes, gl, n, rdst, vbeg, vend, lane);
}

template <int DT, bool kDot>
void combine_backward_with(const CombineBackwardArgs& a, const TokenMap& tk, dim3 grid, dim3 block,
                           bool stream, hipStream_t s)
{
    if (stream)
        hipLaunchKernelGGL((moe_combine_backward_kernel<DT, kDot, true>), grid, block, 0, s, a, tk);
    else
        hipLaunchKernelGGL((moe_combine_backward_kernel<DT, kDot, false>), grid, block, 0, s, a,
                           tk);
}

template <int DT>
void dispatch_backward_with(const DispatchBackwardArgs& a, const TokenMap& tk, dim3 grid,
                            dim3 block, bool stream, hipStream_t s)
{
    if (stream)
        hipLaunchKernelGGL((moe_dispatch_backward_kernel<DT, true>), grid, block, 0, s, a, tk);
    else
        hipLaunchKernelGGL((moe_dispatch_backward_kernel<DT, false>), grid, block, 0, s, a, tk);
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs& a, const TokenMap& tk, int dtype,
                                   bool stream, hipStream_t s)
{
    if (tk.total == 0)
        return hipSuccess;
    if (a.row_waves < 1 || a.row_waves > kBackMaxWaves || a.k > ep::kMaxTopk ||
        a.group_slots < 1 || a.group_slots > kWave ||
        (int64_t)a.row_waves * a.wave_vecs < a.row_vecs)
        return hipErrorInvalidValue;
    const int waves = a.row_waves > 4 ? a.row_waves : 4;
    const int block_tokens = waves / a.row_waves;
    const dim3 grid((unsigned)((tk.total + block_tokens - 1) / block_tokens),
                    (unsigned)((a.k + a.group_slots - 1) / a.group_slots));
    const dim3 block(waves * kWave);
    if (dtype == 0) {
        if (a.gw)
            combine_backward_with<0, true>(a, tk, grid, block, stream, s);
        else
            combine_backward_with<0, false>(a, tk, grid, block, stream, s);
    } else {
        if (a.gw)
            combine_backward_with<1, true>(a, tk, grid, block, stream, s);
        else
            combine_backward_with<1, false>(a, tk, grid, block, stream, s);
    }
    return hipGetLastError();
}

hipError_t launch_dispatch_backward(const DispatchBackwardArgs& a, const TokenMap& tk, int dtype,
                                    int waves, bool stream, hipStream_t s)
{
    if (tk.total == 0)
        return hipSuccess;
    if (a.pieces < 1 || (int64_t)a.pieces * kWave < a.row_vecs)
        return hipErrorInvalidValue;
    const int64_t items = (int64_t)tk.total * a.pieces;
    const dim3 grid((unsigned)((items + waves - 1) / waves));
    const dim3 block(waves * kWave);
    if (dtype == 0)
        dispatch_backward_with<0>(a, tk, grid, block, stream, s);
    else
        dispatch_backward_with<1>(a, tk, grid, block, stream, s);
    return hipGetLastError();
}

}  // namespace moe
