// gfx950 (MI355X, CDNA4) kernels of moe_few_tokens (include/moe_block.h): a
// whole layer's experts for a few tokens.
//
// Such a call is its weights' bytes: 3 * inter * hidden for each expert hit,
// against which tokens, hidden rows and arithmetic are nothing. So nothing is
// gathered or packed, every weight byte goes from memory to a register once,
// and the two kernels only see to it that enough loads are in flight.
//
// The first kernel takes gate and up: a block has one expert and 16 hidden
// columns (16 gate rows, 16 up rows), its 4 waves a quarter of k each; the
// quarters are added in order through LDS, and silu(gate) * up goes to the
// workspace as a bf16 value and the bf16 value of its rest. The second takes
// down: a block has 16 or 32 output columns for every expert hit, its waves
// share the experts (and pieces of k), each (token, expert) pair's sums go to
// LDS, and at the end each token's are added in slot order with their weights.
// No sum's order depends on which other tokens are there.
//
// Weights are the matrix instruction's rows, tokens its columns (16 at a
// time; absent ones are zeros that no load touches memory for). A lane's 16
// bytes of weights are widened to two operands of 8 values of the tokens'
// type, which is exact for E4M3 and int8 alike, so that x needs no rounding;
// both sides take k in the same permuted order. FP8 weights: the sum of each
// 128 elements of k is scaled as it joins the FP32 sum.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_device.h"

namespace block {
namespace {

using namespace block::dev;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kMaxWords = kFewMaxExperts / 32;
constexpr int kBlockK = 128;  // elements of k a step
constexpr uint32_t kNowhere = 1u << 31;

// 4 codes as 4 values of the tokens' type (XT 0 bf16, 1 fp16), exact. WT: 0
// E4M3, 1 int8.
template <int WT, int XT>
__device__ __forceinline__ u32x2 widened4(uint32_t c)
{
    if constexpr (WT == 0 && XT == 0) {
        return {__builtin_bit_cast(uint32_t,
                                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false)),
                __builtin_bit_cast(uint32_t,
                                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true))};
    } else if constexpr (WT == 0) {
        return {__builtin_bit_cast(uint32_t,
                                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false)),
                __builtin_bit_cast(uint32_t,
                                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true))};
    } else {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = (float)(int8_t)(c >> (8 * i));
        if constexpr (XT == 0) {
            // whole numbers of 8 bits: the upper halves of the binary32
            return {__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[1]),
                                          __builtin_bit_cast(uint32_t, f[0]), 0x07060302u),
                    __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[3]),
                                          __builtin_bit_cast(uint32_t, f[2]), 0x07060302u)};
        } else {
            return {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[0], f[1])),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2], f[3]))};
        }
    }
}

template <int WT, int XT>
__device__ __forceinline__ u32x4 widened8(uint32_t lo, uint32_t hi)
{
    const u32x2 a = widened4<WT, XT>(lo), b = widened4<WT, XT>(hi);
    return {a[0], a[1], b[0], b[1]};
}

template <int XT>
__device__ __forceinline__ f32x4 product(const u32x4& w, const u32x4& x, const f32x4& c)
{
    if constexpr (XT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                       __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w),
                                                      __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// What a block knows of the routing: the expert of each slot that is its
// token's first to name it (else -1), and the experts hit, by their number.
struct Routing {
    int id[kFewMaxSlots];
    int hit[kFewMaxSlots];
    uint32_t bits[kMaxWords];
    int part[16];
    int hits;
};

// Fills s in a block of N threads. Ends with a barrier.
template <int N>
__device__ __forceinline__ void read_routing(const FewArgs& a, Routing& s)
{
    const int tid = threadIdx.x, P = a.T * a.topk;
    const int words = (a.E + 31) / 32;
    for (int p = tid; p < P; p += N)
        s.hit[p] = a.ids[p];  // (as they come; the list of hits is made later)
    for (int i = tid; i < words; i += N)
        s.bits[i] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += N) {
        const int e = s.hit[p], first = p - p % a.topk;
        bool lead = e >= 0 && e < a.E;
        for (int j = first; j < p; ++j)
            lead = lead && s.hit[j] != e;
        s.id[p] = lead ? e : -1;
        if (lead)
            atomicOr(&s.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    const int share = (words + N - 1) / N;
    const int w0 = min(words, tid * share), w1 = min(words, w0 + share);
    int mine = 0;
    for (int i = w0; i < w1; ++i)
        mine += __popc(s.bits[i]);
    int inc = mine;
    const int lane = tid & (kWave - 1), wave = tid / kWave;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(inc, o);
        if (lane >= o)
            inc += u;
    }
    if (lane == kWave - 1)
        s.part[wave] = inc;
    __syncthreads();
    int at = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < N / kWave; ++w) {
        at += w < wave ? s.part[w] : 0;
        total += s.part[w];
    }
    for (int i = w0; i < w1; ++i)
        for (uint32_t b = s.bits[i]; b; b &= b - 1)
            s.hit[at++] = i * 32 + __ffs(b) - 1;
    if (tid == 0)
        s.hits = total;
    __syncthreads();
}

// The slots of expert e, in order, to list; how many. One wave.
__device__ __forceinline__ int slots_of(const Routing& s, int P, int e, int* list)
{
    const int lane = threadIdx.x & (kWave - 1);
    int n = 0;
    for (int p0 = 0; p0 < P; p0 += kWave) {
        const int p = p0 + lane;
        const bool yes = p < P && s.id[p] == e;
        const uint64_t b = __ballot(yes);
        if (yes)
            list[n + lanes_below(b)] = p;
        n += (int)__popcll(b);
    }
    return n;
}

// The sums over steps [k0, k1) of R operands of 16 weight rows with G groups of
// 16 columns. rsrc[r]: resource of operand r's 16 rows of K bytes; xoff[g]:
// byte offset of this lane's column (kNowhere: none) in X resources rx, of
// which the operand of k is the sum (X = 2: values and their rests). scale(r,
// step): operand r's scale of that step, of FP8 weights. D: steps in flight.
template <int R, int G, int X, int WT, int XT, int D, class Scale>
__device__ __forceinline__ void accumulate(const __amdgpu_buffer_rsrc_t (&rw)[R],
                                           const __amdgpu_buffer_rsrc_t (&rx)[X],
                                           const uint32_t (&xoff)[G], int K, int k0, int k1,
                                           Scale&& scale, f32x4 (&acc)[R][G])
{
    const int lane = threadIdx.x & (kWave - 1);
    const int q = lane >> 4;
    const uint32_t woff = (uint32_t)(lane & 15) * (uint32_t)K + (uint32_t)q * 16u;
    struct Step {
        u32x4 w[R][2], x[G][X][4];
    };
    Step in[D];
    auto load = [&](int k, Step& s) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // 16 elements of k: rows end at K, steps at k1
            const int at = k * kBlockK + half * 64;
            const bool there = k < k1 && at + q * 16 < K;
#pragma unroll
            for (int r = 0; r < R; ++r)
                s.w[r][half] = bload16<2>(rw[r], there ? woff + at : kNowhere);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int v = 0; v < X; ++v)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s.x[g][v][half * 2 + c] = bload16<0>(
                            rx[v], there ? xoff[g] + (uint32_t)(at + q * 16 + c * 8) * 2u : kNowhere);
        }
    };
    auto use = [&](int k, const Step& s) {
        f32x4 sum[R][G];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int g = 0; g < G; ++g)
                sum[r][g] = WT == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[r][g];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const u32x4 w = widened8<WT, XT>(s.w[r][c >> 1][(c & 1) * 2],
                                                 s.w[r][c >> 1][(c & 1) * 2 + 1]);
#pragma unroll
                for (int v = 0; v < X; ++v)
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        sum[r][g] = product<XT>(w, s.x[g][v][c], sum[r][g]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float f = WT == 0 ? scale(r, k) : 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if constexpr (WT == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[r][g][i] = __builtin_fmaf(f, sum[r][g][i], acc[r][g][i]);
                } else {
                    acc[r][g] = sum[r][g];
                }
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(k0 + d, in[d]);
    for (int k = k0; k < k1; k += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (k + d < k1)
                use(k + d, in[d]);
            load(k + d + D, in[d]);
        }
    }
}

// Scales of up to 64 steps from k0 on, one a lane, and one of them.
struct StepScales {
    const float* from;
    int k0, k1, held;
    float v;

    __device__ __forceinline__ StepScales(const float* row, int first, int end)
        : from(row), k0(first), k1(end), held(first)
    {
        fill();
    }
    __device__ __forceinline__ void fill()
    {
        const int k = held + (int)(threadIdx.x & (kWave - 1));
        v = k < k1 ? from[k] : 0.0f;
    }
    __device__ __forceinline__ float at(int k)
    {
        if (k - held >= kWave) {
            held += kWave;
            fill();
        }
        return lane_value(v, k - held);
    }
};

// Runs f with the number of groups of 16 that hold n columns, at most kMost.
template <int kMost, class F>
__device__ __forceinline__ void with_groups(int n, F&& f)
{
    if (kMost == 1 || n <= 16)
        f(std::integral_constant<int, 1>());
    else if (n <= 32)
        f(std::integral_constant<int, kMost == 1 ? 1 : 2>());
    else
        f(std::integral_constant<int, kMost == 1 ? 1 : 4>());
}

// Gate and up. kMost: 1 for calls of up to 16 tokens, else 4.
template <int WT, int XT, int kMost>
__global__ __launch_bounds__(kUpWaves * kWave) __attribute__((amdgpu_waves_per_eu(kMost == 1 ? 4 : 2)))
void block_few_up_kernel(FewArgs a)
{
    __shared__ Routing s;
    __shared__ int s_list[kFewMaxTokens];
    __shared__ int s_n;
    __shared__ f32x4 s_sum[kUpWaves][2][kMost][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int tiles = a.I / 16;
    const int u = (int)blockIdx.x / tiles, tile = (int)blockIdx.x % tiles;
    read_routing<kUpWaves * kWave>(a, s);
    if (u >= s.hits)
        return;  // the whole block
    const int e = uniform(s.hit[u]);
    if (wave == 0) {
        const int n = slots_of(s, a.T * a.topk, e, s_list);
        if (lane == 0)
            s_n = n;
    }
    __syncthreads();
    const int n = uniform(s_n);
    const int64_t row = (int64_t)e * 2 * a.I + tile * 16;
    const __amdgpu_buffer_rsrc_t rw[2] = {
        row_rsrc(a.up + row * a.H, (uint32_t)a.H * 16u),
        row_rsrc(a.up + (row + a.I) * a.H, (uint32_t)a.H * 16u)};
    const __amdgpu_buffer_rsrc_t rx[1] = {row_rsrc(a.x, (uint32_t)a.T * (uint32_t)a.H * 2u)};
    const int steps = (a.H + kBlockK - 1) / kBlockK;
    const int k0 = steps * wave / kUpWaves, k1 = steps * (wave + 1) / kUpWaves;

    with_groups<kMost>(n, [&](auto groups) {
        constexpr int G = decltype(groups)::value;
        uint32_t xoff[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int c = g * 16 + (lane & 15);
            xoff[g] = c < n ? (uint32_t)(s_list[c] / a.topk) * (uint32_t)a.H * 2u : kNowhere;
        }
        f32x4 acc[2][G];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int g = 0; g < G; ++g)
                acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int blocks = a.H / kBlockK;  // of a row's scales (FP8)
        const float* first = a.ups + (row / 128) * blocks;
        StepScales sg(WT == 0 ? first : a.ups, WT == 0 ? k0 : 0, WT == 0 ? k1 : 0);
        StepScales su(WT == 0 ? first + (int64_t)(a.I / 128) * blocks : a.ups, WT == 0 ? k0 : 0,
                      WT == 0 ? k1 : 0);
        accumulate<2, G, 1, WT, XT, G == 1 ? 2 : 1>(
            rw, rx, xoff, a.H, k0, k1, [&](int r, int k) { return r == 0 ? sg.at(k) : su.at(k); },
            acc);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int g = 0; g < G; ++g)
                s_sum[wave][r][g][lane] = acc[r][g];
    });
    __syncthreads();
    // wave g finishes group g: a lane has 4 hidden columns of one token
    if (wave * 16 < n) {
        const int c = wave * 16 + (lane & 15);
        f32x4 v[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            v[r] = s_sum[0][r][wave][lane];
#pragma unroll
            for (int w = 1; w < kUpWaves; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[r][i] = v[r][i] + s_sum[w][r][wave][lane][i];
        }
        const int col = tile * 16 + (lane >> 4) * 4;
        if (c < n) {
            float z[4], rest[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g = v[0][i], up = v[1][i];
                if constexpr (WT == 1) {
                    const int64_t at = (int64_t)e * 2 * a.I + col + i;
                    g = g * a.ups[at];
                    up = up * a.ups[at + a.I];
                }
                const float y = silu_times(g, up);
                z[i] = round_to<0>(y);
                rest[i] = z[i] == y ? 0.0f : y - z[i];  // (an infinity has no rest)
            }
            const int64_t at = (int64_t)s_list[c] * a.I + col;
            const int64_t plane = (int64_t)a.T * a.topk * a.I;
            auto pair = [](float lo, float hi) {
                return (__builtin_bit_cast(uint32_t, round_to<0>(lo)) >> 16) |
                       (__builtin_bit_cast(uint32_t, round_to<0>(hi)) & 0xFFFF0000u);
            };
            *reinterpret_cast<u32x2*>(a.act + at * 2) = u32x2{pair(z[0], z[1]), pair(z[2], z[3])};
            *reinterpret_cast<u32x2*>(a.act + (plane + at) * 2) =
                u32x2{pair(rest[0], rest[1]), pair(rest[2], rest[3])};
        }
    }
}

// Down and the sum over experts, of 16 R output columns.
template <int WT, int XT, int R, int kMost>
__global__ __launch_bounds__(kDownWaves * kWave) __attribute__((amdgpu_waves_per_eu(kMost == 1 ? 4 : 2)))
void block_few_down_kernel(FewArgs a)
{
    extern __shared__ float s_y[];  // [splits][T * topk][16 R]
    __shared__ Routing s;
    __shared__ int s_list[kDownWaves][kFewMaxTokens];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    constexpr int kCols = 16 * R;
    const int h0 = (int)blockIdx.x * kCols;
    const int P = a.T * a.topk;
    read_routing<kDownWaves * kWave>(a, s);
    const uint32_t plane = (uint32_t)P * (uint32_t)a.I * 2u;
    const __amdgpu_buffer_rsrc_t rx[2] = {row_rsrc(a.act, plane), row_rsrc(a.act + plane, plane)};
    const int steps = (a.I + kBlockK - 1) / kBlockK;
    const int items = uniform(s.hits) * a.splits;
    for (int item = wave; item < items; item += kDownWaves) {
        const int e = uniform(s.hit[item / a.splits]), split = item % a.splits;
        const int n = slots_of(s, P, e, s_list[wave]);
        const int k0 = steps * split / a.splits, k1 = steps * (split + 1) / a.splits;
        const int64_t row = (int64_t)e * a.H + h0;
        __amdgpu_buffer_rsrc_t rw[R];
#pragma unroll
        for (int r = 0; r < R; ++r)  // (H may end inside the block)
            rw[r] = row_rsrc(a.down + (row + r * 16) * a.I,
                             h0 + r * 16 < a.H ? (uint32_t)a.I * 16u : 0u);
        with_groups<kMost>(n, [&](auto groups) {
            constexpr int G = decltype(groups)::value;
            uint32_t xoff[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = g * 16 + (lane & 15);
                xoff[g] = c < n ? (uint32_t)s_list[wave][c] * (uint32_t)a.I * 2u : kNowhere;
            }
            f32x4 acc[R][G];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[r][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // (a block's columns lie in one block of 128)
            StepScales sc(WT == 0 ? a.downs + (row / 128) * (a.I / kBlockK) : a.downs,
                          WT == 0 ? k0 : 0, WT == 0 ? k1 : 0);
            accumulate<R, G, 2, WT, 0, G == 1 ? 2 : 1>(
                rw, rx, xoff, a.I, k0, k1, [&](int, int k) { return sc.at(k); }, acc);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int c = g * 16 + (lane & 15);
                if (c < n) {
                    float* y = s_y + ((int64_t)split * P + s_list[wave][c]) * kCols + (lane >> 4) * 4;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        *reinterpret_cast<f32x4*>(y + r * 16) = acc[r][g];
                }
            }
        });
    }
    __syncthreads();
    // a token's pairs in slot order, each the sum of its pieces in order
    for (int i = threadIdx.x; i < a.T * kCols; i += kDownWaves * kWave) {
        const int t = i / kCols, c = i % kCols;
        float sum = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int p = t * a.topk + j, e = s.id[p];
            if (e < 0 || h0 + c >= a.H)
                continue;
            float y = s_y[(int64_t)p * kCols + c];
            for (int k = 1; k < a.splits; ++k)
                y = y + s_y[((int64_t)k * P + p) * kCols + c];
            if constexpr (WT == 1)
                y = y * a.downs[(int64_t)e * a.H + h0 + c];
            float weight = 1.0f;
            if (a.w != nullptr) {
                weight = a.w[p];
                // slots after it that name the expert again
                for (int k = j + 1; k < a.topk; ++k)
                    if (a.ids[t * a.topk + k] == e)
                        weight = weight + a.w[t * a.topk + k];
            }
            sum = __builtin_fmaf(weight, y, sum);
        }
        if (h0 + c < a.H) {
            uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)t * a.H + h0 + c;
            if constexpr (XT == 0)
                *out = (uint16_t)(__builtin_bit_cast(uint32_t, round_to<0>(sum)) >> 16);
            else
                *out = __builtin_bit_cast(uint16_t, (_Float16)sum);
        }
    }
}

template <int WT, int XT, int kMost>
hipError_t few_with(const FewArgs& a, hipStream_t s)
{
    const dim3 up((unsigned)(a.hits * (a.I / 16)));
    hipLaunchKernelGGL((block_few_up_kernel<WT, XT, kMost>), up, dim3(kUpWaves * kWave), 0, s, a);
    const size_t pair = (size_t)a.splits * a.T * a.topk * sizeof(float);
    // 32 columns a block where that leaves half the compute units a block and
    // the pairs' sums fit
    if (a.H >= 32 * 128 && pair * 32 <= 96 * 1024)
        hipLaunchKernelGGL((block_few_down_kernel<WT, XT, 2, kMost>), dim3((a.H + 31) / 32),
                           dim3(kDownWaves * kWave), pair * 32, s, a);
    else
        hipLaunchKernelGGL((block_few_down_kernel<WT, XT, 1, kMost>), dim3(a.H / 16),
                           dim3(kDownWaves * kWave), pair * 16, s, a);
    return hipGetLastError();
}

template <int WT, int XT>
hipError_t few_types(const FewArgs& a, hipStream_t s)
{
    return a.T <= 16 ? few_with<WT, XT, 1>(a, s) : few_with<WT, XT, 4>(a, s);
}

}  // namespace

hipError_t launch_few(const FewArgs& a, int dtype, int wtype, hipStream_t s)
{
    if (a.T < 1 || a.T > kFewMaxTokens || a.topk < 1 || a.T * a.topk > kFewMaxSlots || a.E < 1 ||
        a.E > kFewMaxExperts || a.H % 16 || a.I % 16 || a.splits < 1 ||
        a.splits * a.T * a.topk > kFewMaxSlots || a.hits < 1)
        return hipErrorInvalidValue;
    if (wtype == 0)
        return dtype == 0 ? few_types<0, 0>(a, s) : few_types<0, 1>(a, s);
    return dtype == 0 ? few_types<1, 0>(a, s) : few_types<1, 1>(a, s);
}

}  // namespace block
