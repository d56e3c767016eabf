// gfx950 (MI355X, CDNA4) kernels of moe_block_norm_backward
// (include/moe_block.h): the gradients of the norm after a block, its gate and
// scaled residual, and the norm before the next block.
//
// One pass over the rows and a small second kernel. A block walks rows; the
// waves of a block share a row (16 bytes a lane and chunk of 512 elements), so
// every lane meets the same columns in each row and holds their sums for the
// gradients of the weights and the gate in registers. Those go to the
// workspace once a block, and the second kernel adds the blocks' in order: no
// atomics, and a column's sum depends on the call's sizes alone, not on timing.
//
// The two norms' means would be taken one after the other, the second of
// values that hold the first; but d is linear in the first mean, so
//   sum d1 y = sum gh q + r2 (sum d2 q - mean(d2 n2) r2 sum h q),
//   q = gate * post_weight * y, d2 = go * pre_weight,
// and one exchange of six sums a row serves both. What bounds it is HBM
// bandwidth: the next row is on its way while a row is worked on, and the
// weights stay in registers, as a load of them between two rows would wait for
// all of the next row. Measured on MI355X: 8 x 2048 rows of 7168 bf16 310 us (1.41
// GB, 4.5 TB/s; 488 with the weights loaded each row and the waves' sums read one
// by one) and 7 us for the second kernel, 4 x 256 rows of 4096 fp16, half of them
// there, 15 and 4 us. Rows of more than 8192 elements leave no registers for the
// next row and are read twice, the second time from the caches; their 96 sums a
// lane do not fit the registers either (224 to 288 bytes a lane of scratch memory up
// to 16384 elements, 776 to 964 above): 8192 rows of 16384 1116 us (1.4 TB/s), 4096
// of 32768 1954 (0.8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_device.h"

namespace block {
namespace {

using namespace block::dev;

constexpr int kSums = 6;
constexpr int kReduceSlices = 16;  // waves that share a column's blocks

// A row's 16-byte vectors of this lane, as they come.
template <int C>
struct Raw {
    u32x4 y[C], h[C], gh[C], go[C];
};

// DT: 0 bf16, 1 fp16 rows. WT: 0 bf16, 1 fp16, 2 fp32 weights. C: chunks a
// wave holds; W: the most waves a row. kAhead: the next row is loaded while a
// row is worked on (its registers are there up to 2 chunks).
template <int C, int W, int DT, int WT, bool kStream>
__global__ __launch_bounds__(W * kWave) void block_norm_backward_kernel(NormBackwardArgs a)
{
    constexpr int ld = Policy<kStream>::combine_load;
    constexpr int st = Policy<kStream>::combine_store;
    constexpr bool kAhead = C <= 2;
    // longer rows leave no registers for their values: read again for the second pass
    constexpr bool kAgain = !kAhead;
    __shared__ float s_sum[2][kSums][W];  // (those of waves that are not there stay 0)
    const int lane = threadIdx.x & (kWave - 1);
    const int part = uniform(threadIdx.x / kWave);
    const int waves = a.row_waves;
    const int e0 = part * C * kNormChunk + lane * 8;
    const uint32_t bytes = (uint32_t)a.H * 2u;
    const uint32_t wbytes = (uint32_t)a.H * (WT == 2 ? 4u : 2u);
    const bool has_post = a.post != nullptr, has_gate = a.gate != nullptr,
               has_out = a.go != nullptr, has_h = a.gh != nullptr;

    // this block's groups and its rows of each: chunk, chunk + group_blocks ..
    const int64_t g0 = a.group_blocks > 1 ? (int64_t)blockIdx.x / a.group_blocks
                                          : (int64_t)blockIdx.x * a.block_groups;
    const int64_t g1 = a.group_blocks > 1 ? g0 + 1 : min(a.groups, g0 + a.block_groups);
    const int64_t first = a.group_blocks > 1 ? (int64_t)blockIdx.x % a.group_blocks : 0;
    auto rows_of = [&](int64_t g) {
        return a.counts ? min((int64_t)a.counts[g], a.group_rows) : a.group_rows;
    };
    int64_t g = g0, r = first, limit = rows_of(g0);
    auto settle = [&]() {  // the first row at or after (g, r) that is there
        while (r >= limit && g < g1) {
            ++g;
            r = first;
            limit = g < g1 ? rows_of(g) : 0;
        }
    };
    settle();

    float acc_post[C][8], acc_gate[C][8], acc_pre[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc_post[c][i] = acc_gate[c][i] = acc_pre[c][i] = 0.0f;

    // columns [e0 ..) of a float row
    auto store_sums = [&](float* to, const float (&v)[C][8]) {
        const __amdgpu_buffer_rsrc_t rs = row_rsrc(to, (uint32_t)a.H * 4u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t at = (uint32_t)(e0 + c * kNormChunk) * 4u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = __builtin_bit_cast(uint32_t, v[c][half * 4 + i]);
                bstore16<0>(w, rs, at + half * 16u);
            }
        }
    };
    // the gate's gradient of a group that this block alone has walked
    const bool whole_gates = a.ggate != nullptr && a.gates > 1 && a.group_blocks == 1;
    auto close_gate = [&](int64_t which) {
        store_sums(a.ggate + which * a.H, acc_gate);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc_gate[c][i] = 0.0f;
    };

    auto load_chunk = [&](int64_t row, int c, Raw<C>& x) {
        const int64_t at = row * a.H * 2;
        const __amdgpu_buffer_rsrc_t ry = row_rsrc(a.y + at, bytes);
        const __amdgpu_buffer_rsrc_t rh = row_rsrc(a.h + at, has_out ? bytes : 0u);
        const __amdgpu_buffer_rsrc_t rgh = row_rsrc(a.gh + at, has_h ? bytes : 0u);
        const __amdgpu_buffer_rsrc_t rgo = row_rsrc(a.go + at, has_out ? bytes : 0u);
        const uint32_t off = (uint32_t)(e0 + c * kNormChunk) * 2u;
        x.y[c] = bload16<ld>(ry, off);
        x.h[c] = bload16<ld>(rh, off);
        x.gh[c] = bload16<ld>(rgh, off);
        x.go[c] = bload16<ld>(rgo, off);
    };
    auto load = [&](int64_t row, Raw<C>& x) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            load_chunk(row, c, x);
    };
    // The weights of this lane's columns: held over the rows where there are
    // registers, as a load of them between two rows would be waited for with
    // all of the next row's before it; else loaded in each pass.
    Weights8<WT> held_post[kAhead ? C : 1], held_gate[kAhead ? C : 1], held_pre[kAhead ? C : 1];
    auto hold = [&](const uint8_t* w, bool there, Weights8<WT> (&held)[kAhead ? C : 1]) {
        const __amdgpu_buffer_rsrc_t rw = row_rsrc(w, there ? wbytes : 0u);
#pragma unroll
        for (int c = 0; c < (kAhead ? C : 1); ++c)
            held[c].load(rw, e0 + c * kNormChunk);
    };
    auto weight = [&](const uint8_t* w, bool there, const Weights8<WT> (&held)[kAhead ? C : 1],
                      int c, float (&f)[8]) {
        if (!there) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = 1.0f;
        } else if (kAhead) {
            held[c < (kAhead ? C : 1) ? c : 0].widen8(f);
        } else {
            int e = e0 + c * kNormChunk;
            asm volatile("" : "+v"(e));  // (not kept from one pass to the other)
            weights8<WT>(row_rsrc(w, wbytes), e, f);
        }
    };
    if (kAhead) {
        hold(a.post, has_post, held_post);
        hold(a.gate, has_gate && a.gates == 1, held_gate);
        hold(a.pre, has_out, held_pre);
    }
    if (threadIdx.x < 2 * kSums * W)
        (&s_sum[0][0][0])[threadIdx.x] = 0.0f;
    if (waves > 1)
        __syncthreads();
    static_assert(2 * kSums * W <= 3 * kWave, "cleared by 3 waves");

    int64_t gate_group = -1;  // whose gate is held
    int64_t open = g0;  // groups before it have their gate's gradient written
    int parity = 0;
    Raw<C> x;
    if (kAhead && g < g1)
        load(g * a.group_rows + r, x);
    while (g < g1) {
        const int64_t group = g, row = g * a.group_rows + r;
        r += a.group_blocks;
        settle();
        const uint8_t* gate = has_gate ? a.gate + (a.gates > 1 ? group : 0) * wbytes : nullptr;
        if (kAhead && has_gate && a.gates > 1 && gate_group != group) {
            hold(gate, true, held_gate);
            gate_group = group;
        }
        Raw<C> next;
        if (kAhead && g < g1)
            load(g * a.group_rows + r, next);
        if (whole_gates) {
            for (; open < group; ++open)
                close_gate(open);
        }

        float s[kSums] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (C > 2)  // a chunk at a time: the sums take most registers
                __builtin_amdgcn_sched_barrier(0);
            if (kAgain)
                load_chunk(row, c, x);
            float y[8], h[8], gh[8], go[8], wp[8], wg[8], w2[8];
            widen<DT>(x.y[c], y);
            widen<DT>(x.h[c], h);
            widen<DT>(x.gh[c], gh);
            widen<DT>(x.go[c], go);
            weight(a.post, has_post, held_post, c, wp);
            weight(gate, has_gate, held_gate, c, wg);
            weight(a.pre, has_out, held_pre, c, w2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = wg[i] * wp[i] * y[i], d2 = go[i] * w2[i];
                s[0] = __builtin_fmaf(y[i], y[i], s[0]);
                s[1] = __builtin_fmaf(h[i], h[i], s[1]);
                s[2] = __builtin_fmaf(d2, h[i], s[2]);
                s[3] = __builtin_fmaf(gh[i], q, s[3]);
                s[4] = __builtin_fmaf(d2, q, s[4]);
                s[5] = __builtin_fmaf(h[i], q, s[5]);
            }
        }
#pragma unroll
        for (int k = 0; k < kSums; ++k)
            s[k] = wave_sum(s[k]);
        if (waves > 1) {
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < kSums; ++k)
                    s_sum[parity][k][part] = s[k];
            }
            __syncthreads();
            // a lane a wave and sum: one read, and a tree over the waves
            static_assert(W == 8 || W == 16, "lanes of a sum");
            constexpr int kEach = kWave / W;  // sums a read
#pragma unroll
            for (int k0 = 0; k0 < kSums; k0 += kEach) {
                const int at = k0 * W + lane;
                float v = (&s_sum[parity][0][0])[at < kSums * W ? at : 0];
                v = v + dpp<kDppXor1>(v);
                v = v + dpp<kDppXor2>(v);
                v = v + dpp<kDppHalfMirror>(v);
                if (W == 16)
                    v = v + dpp<kDppMirror>(v);
#pragma unroll
                for (int k = k0; k < kSums && k < k0 + kEach; ++k)
                    s[k] = lane_value(v, (k - k0) * W);
            }
            parity ^= 1;  // the next row's sums go where no wave reads any more
        }
        const float H = (float)a.H;
        const float r1 =
            has_post ? __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s[0], H) + a.eps)) : 1.0f;
        const float r2 = has_out ? __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(s[1], H) + a.eps)) : 0.0f;
        const float m2 = has_out ? __fdiv_rn(r2 * s[2], H) : 0.0f;
        const float sum1 = has_out ? __builtin_fmaf(r2, s[4] - m2 * (r2 * s[5]), s[3]) : s[3];
        const float m1 = has_post ? __fdiv_rn(r1 * sum1, H) : 0.0f;

        const __amdgpu_buffer_rsrc_t rgy = row_rsrc(a.gy + row * a.H * 2, bytes);
        const __amdgpu_buffer_rsrc_t rgr =
            row_rsrc(a.gres + (a.gres ? row * a.H * 2 : 0), a.gres ? bytes : 0u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (C > 2)
                __builtin_amdgcn_sched_barrier(0);
            const uint32_t off = (uint32_t)(e0 + c * kNormChunk) * 2u;
            if (kAgain)
                load_chunk(row, c, x);
            else  // widened again: kept since the first pass, it would take twice the registers
                asm volatile("" : "+v"(x.y[c]), "+v"(x.h[c]), "+v"(x.gh[c]), "+v"(x.go[c]));
            float y[8], h[8], gh[8], go[8], wp[8], wg[8], w2[8], gr[8], gy[8];
            widen<DT>(x.y[c], y);
            widen<DT>(x.h[c], h);
            widen<DT>(x.gh[c], gh);
            widen<DT>(x.go[c], go);
            weight(a.post, has_post, held_post, c, wp);
            weight(gate, has_gate, held_gate, c, wg);
            weight(a.pre, has_out, held_pre, c, w2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n2 = h[i] * r2;
                const float d =
                    has_out ? __builtin_fmaf(r2, go[i] * w2[i] - n2 * m2, gh[i]) : gh[i];
                acc_pre[c][i] = __builtin_fmaf(go[i], n2, acc_pre[c][i]);
                gr[i] = a.res_scale * d;
                const float n1 = y[i] * r1;
                acc_gate[c][i] = __builtin_fmaf(d, n1 * wp[i], acc_gate[c][i]);
                const float du = d * wg[i];
                acc_post[c][i] = __builtin_fmaf(du, n1, acc_post[c][i]);
                gy[i] = has_post ? r1 * (du * wp[i] - n1 * m1) : du;
            }
            bstore16<st>(narrow<DT>(gr), rgr, off);
            bstore16<st>(narrow<DT>(gy), rgy, off);
        }
        if (kAhead)
            x = next;
    }

    const int64_t size = (int64_t)a.blocks * a.H, mine = (int64_t)blockIdx.x * a.H;
    const bool last = a.blocks == 1;  // its sums are the results
    if (a.gpost)
        store_sums(last ? a.gpost : a.part + mine, acc_post);
    if (whole_gates) {
        for (; open < g1; ++open)
            close_gate(open);
    } else if (a.ggate) {
        store_sums(last ? a.ggate : a.part + size + mine, acc_gate);
    }
    if (a.gpre)
        store_sums(last ? a.gpre : a.part + 2 * size + mine, acc_pre);
}

// Sums of the blocks' parts: 64 columns a block, kReduceSlices waves, each
// adding every kReduceSlices-th part; the waves' sums are added in order.
__global__ __launch_bounds__(kReduceSlices * kWave) void block_norm_reduce_kernel(
    NormBackwardArgs a)
{
    __shared__ float s_sum[kReduceSlices][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int slice = uniform(threadIdx.x / kWave);
    const int col = blockIdx.x * kWave + lane;
    const int64_t size = (int64_t)a.blocks * a.H;
    const int what = blockIdx.y;  // 0: post, 1: pre, 2 ..: gates
    float* out = what == 0 ? a.gpost : what == 1 ? a.gpre : a.ggate;
    if (out == nullptr)
        return;
    const float* from = a.part + (what == 0 ? 0 : what == 1 ? 2 * size : size);
    int parts = a.blocks;
    if (what >= 2) {
        out += (int64_t)(what - 2) * a.H;
        if (a.gates > 1) {
            parts = a.group_blocks;
            from += (int64_t)(what - 2) * parts * a.H;
        }
    }
    float sum = 0.0f;
    if (col < a.H) {
        int b = slice;
        for (; b + 7 * kReduceSlices < parts; b += 8 * kReduceSlices) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = from[(int64_t)(b + i * kReduceSlices) * a.H + col];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = sum + v[i];
        }
        for (; b < parts; b += kReduceSlices)
            sum = sum + from[(int64_t)b * a.H + col];
    }
    s_sum[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && col < a.H) {
        for (int i = 1; i < kReduceSlices; ++i)
            sum = sum + s_sum[i][lane];
        out[col] = sum;
    }
}

template <int C, int W, int DT, int WT>
void backward_with(const NormBackwardArgs& a, bool stream, hipStream_t s)
{
    const dim3 grid(a.blocks), block(a.row_waves * kWave);
    if (stream)
        hipLaunchKernelGGL((block_norm_backward_kernel<C, W, DT, WT, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((block_norm_backward_kernel<C, W, DT, WT, false>), grid, block, 0, s, a);
}

template <int C, int W>
void backward_types(const NormBackwardArgs& a, int dtype, int wtype, bool stream, hipStream_t s)
{
    if (dtype == 0) {
        if (wtype == 2)
            backward_with<C, W, 0, 2>(a, stream, s);
        else
            backward_with<C, W, 0, 0>(a, stream, s);
    } else {
        if (wtype == 2)
            backward_with<C, W, 1, 2>(a, stream, s);
        else
            backward_with<C, W, 1, 1>(a, stream, s);
    }
}

}  // namespace

hipError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, int wtype, bool stream,
                                hipStream_t s)
{
    const int C = a.chunks;
    if ((C != 1 && C != 2 && C != 4) || a.row_waves < 1 ||
        a.row_waves > (C == 4 ? 16 : 8) || a.row_waves * C * kNormChunk < a.H || a.blocks < 1 ||
        a.group_blocks < 1 || a.block_groups < 1 || (a.gates != 1 && a.gates != a.groups) ||
        (a.group_blocks > 1 ? a.groups * a.group_blocks != a.blocks
                            : (a.groups + a.block_groups - 1) / a.block_groups != a.blocks))
        return hipErrorInvalidValue;
    if (C == 1)
        backward_types<1, 8>(a, dtype, wtype, stream, s);
    else if (C == 2)
        backward_types<2, 8>(a, dtype, wtype, stream, s);
    else if (a.row_waves <= 8)
        backward_types<4, 8>(a, dtype, wtype, stream, s);
    else
        backward_types<4, 16>(a, dtype, wtype, stream, s);
    const bool gates_left = a.ggate && !(a.gates > 1 && a.group_blocks == 1);
    if (a.blocks > 1 && (a.gpost || a.gpre || gates_left)) {
        NormBackwardArgs r = a;
        if (!gates_left)
            r.ggate = nullptr;
        const dim3 grid((a.H + kWave - 1) / kWave, 2 + (gates_left ? a.gates : 0));
        hipLaunchKernelGGL(block_norm_reduce_kernel, grid, dim3(kReduceSlices * kWave), 0, s, r);
    }
    return hipGetLastError();
}

}  // namespace block
