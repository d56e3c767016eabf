// gfx950 (MI355X, CDNA4) kernel of moe_grouped_gemm (include/moe.h): each
// expert's product of its expert-major FP8 rows with its FP8 weights, a scale
// per row and 128 elements on one side and per 128 x 128 block on the other,
// to bf16 / fp16 rows or, with gate and up weights, to FP8 rows of
// silu(gate) * up with their own scales.
//
// A work item is a tile of up to 256 rows of one expert by 256 weight rows.
// Row counts are on the GPU, so the launch is a fixed grid of one block a
// compute unit; each block works out every expert's tile range from the
// counts and walks its share of the tiles. An expert's last tile computes as
// few of 64, 128 or 256 rows as hold its rows, so that experts with few rows
// cost their weights' bytes and little else.
//
// The FP8 matrix instruction adds 8 products at a time after aligning them to
// the largest of the 8 and cutting what lies below 2^-13 of it (measured on
// gfx950: 2^16 + 2^2 gives 2^16 among 8 neighbouring k, 2^16 + 2^-7 is kept
// across them; the same in v_mfma_f32_16x16x32_fp8_fp8). Rows of bf16 / fp16
// take it: its error, 1.3e-5 of a row's norm whatever k, is 1/20 of fp16's
// rounding and 1/150 of bf16's. The swiglu form returns its block scales in
// FP32, so there both operands are widened to fp16 (exact) in registers and
// multiplied by v_mfma_f32_16x16x32_f16, whose sums of such products are
// FP32's; the matrix rate is half.
//
// Inside a tile: 8 waves, 2 along the rows x 4 along the weight rows. For
// each 128 elements of k the block holds both operands' slices (128 bytes a
// row) in LDS, loaded there directly from memory while the slices before are
// multiplied. The matrix instruction is v_mfma_f32_16x16x128_f8f6f4 with the
// weights as its rows and the token rows as its columns: one instruction
// takes a whole scale block of k, and a lane then holds one token row's
// partial sums, so the scales' product is one value a lane and the partial
// joins the FP32 sum with a fused multiply-add an element.
//
// LDS slices are 128 bytes a row without padding; the eight 16-byte chunks of
// a row are permuted by a key of the row, so the 16 rows a matrix operand
// reads together fall in different banks. Both operands take the chunks in
// the same order, so the order of k inside an instruction is the same too.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {
namespace {

using namespace ep::dev;
using namespace moe::dev;
using ep::kWave;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kTileN = 256;                     // weight rows a tile
constexpr int kSlice = 128;                     // bytes of k a step
constexpr int kWaveRows = 64;                   // weight rows a wave
constexpr int kSubs = kWaveRows / 16;           // 16-row operands of them
constexpr int kScaleBytes = 2048;               // row scales a stage: 8 waves x 64 floats
constexpr int kLdsBytes = 153600;

// Token rows of a tile whose waves hold TS operands of 16 rows each.
constexpr int tile_rows(int ts) { return 2 * 16 * ts; }
constexpr int stage_bytes(int ts)
{
    return (tile_rows(ts) + kTileN) * kSlice + kScaleBytes;
}
constexpr int stages(int ts) { return kLdsBytes / stage_bytes(ts); }

template <int N>
__device__ __forceinline__ void wait_loads()
{
    // the barrier makes every wave's arrived slices visible; LDS reads of the
    // stage about to be overwritten have returned
    if constexpr (N == 0)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    else
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 or 4 bytes a lane straight to LDS: lane i's to dst + 16 * i or 4 * i. off
// is checked against the resource, soff (the column) moves the address.
typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off,
                                              uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, (int)off, (int)soff, 0, 0);
}

__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off,
                                             uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 4, (int)off, (int)soff, 0, 0);
}

__device__ __forceinline__ i32x8 operand(const uint8_t* lo, const uint8_t* hi)
{
    const i32x4 a = *reinterpret_cast<const i32x4*>(lo);
    const i32x4 b = *reinterpret_cast<const i32x4*>(hi);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The 32 FP8 values of an operand as 4 operands of 8 fp16 values (exact; NaN
// stays NaN).
struct Widened {
    f16x8 v[4];
};

__device__ __forceinline__ Widened widened(const i32x8& o)
{
    Widened r;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(o[2 * h], 1.0f, false);
        const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(o[2 * h], 1.0f, true);
        const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(o[2 * h + 1], 1.0f, false);
        const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(o[2 * h + 1], 1.0f, true);
        r.v[h] = f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    return r;
}

// One tile: the group's first row, how many rows, and the column tile.
struct Tile {
    int64_t row0;   // first row (of [groups * cap])
    int group;
    int rows;       // rows of the tile that exist, 1 .. 256
    int col;        // column tile
};

// kSwiglu: weight rows [0, 128) of the tile are gate rows 128 * col .., rows
// [128, 256) the up rows. Otherwise they are rows 256 * col .. .
template <int TS, int DT, bool kSwiglu>
__device__ __forceinline__ void run_tile(const GemmArgs& a, const Tile& t, uint8_t* lds,
                                         float (*s_amax)[256])
{
    constexpr int S = stages(TS);
    constexpr int kRows = tile_rows(TS);
    constexpr int kB = kRows * kSlice;          // offsets in a stage
    constexpr int kScale = kB + kTileN * kSlice;
    constexpr int kALoads = kRows / 64;         // 16-byte loads a wave and stage
    constexpr int kLoads = kALoads + 4 + 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;
    const int q = lane >> 4, i16 = lane & 15;

    // ---- loads: wave w's i-th 1 KB holds rows 8 * (8 * i + w) .. + 7, a lane
    // one 16-byte chunk of a row
    const uint32_t K = (uint32_t)a.k;
    const int lr = wave * 8 + (lane >> 3);      // row of i = 0; i adds 64
    const int chunk = lane & 7;
    const __amdgpu_buffer_rsrc_t ra = row_rsrc(a.a + t.row0 * K, (uint32_t)t.rows * K);
    const uint32_t aoff = (uint32_t)lr * K + (uint32_t)((chunk ^ (lr & 7)) * 16);
    // the key of a weight row: the bits in which the rows of an operand differ
    constexpr int kKeyShift = kSwiglu ? 3 : 4;
    const int bkey = (lr & 3) | (((lr >> kKeyShift) & 1) << 2);
    const uint32_t boff = (uint32_t)lr * K + (uint32_t)((chunk ^ bkey) * 16);
    const int64_t wrow = (int64_t)t.group * a.n;
    const int r0 = kSwiglu ? t.col * 128 : t.col * kTileN;     // first weight rows of the halves
    const int r1 = kSwiglu ? a.n / 2 + r0 : r0 + 128;
    const __amdgpu_buffer_rsrc_t rb0 =
        row_rsrc(a.b + (wrow + r0) * K, (uint32_t)min(128, a.n - r0) * K);
    const int left1 = a.n - r1;
    const __amdgpu_buffer_rsrc_t rb1 =
        row_rsrc(a.b + (wrow + (left1 > 0 ? r1 : 0)) * K, (uint32_t)max(0, min(128, left1)) * K);
    const int nk = a.k / kSlice;
    const uint32_t srow = (uint32_t)nk * 4u;
    const __amdgpu_buffer_rsrc_t rs = row_rsrc(a.as + t.row0 * srow, (uint32_t)t.rows * srow);
    const uint32_t soff = (uint32_t)(wave * kWave + lane) * srow;
    auto load = [&](int kb, int stage) {
        uint8_t* st = lds + stage * stage_bytes(TS);
        const uint32_t k0 = (uint32_t)kb * kSlice;
#pragma unroll
        for (int i = 0; i < kALoads; ++i)
            load16_to_lds(ra, st + (i * 8 + wave) * 1024, aoff + (uint32_t)(i * 64) * K, k0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load16_to_lds(i < 2 ? rb0 : rb1, st + kB + (i * 8 + wave) * 1024,
                            boff + (uint32_t)((i & 1) * 64) * K, k0);
        load4_to_lds(rs, st + kScale + wave * 256, soff, (uint32_t)kb * 4u);
    };

    // ---- operands: a lane's row of each, its chunk q and q + 4
    // (exclusive-or 4)
    const int wrow0 = kSwiglu ? wn * 32 + 8 * (i16 >> 2) + (i16 & 3)
                              : wn * kWaveRows + 16 * (i16 >> 2) + (i16 & 3);
    const int wkey = (wrow0 & 3) | (((wrow0 >> kKeyShift) & 1) << 2);
    const uint32_t wlo = kB + (uint32_t)wrow0 * kSlice + (uint32_t)((q ^ wkey) * 16);
    const int trow0 = wm * 16 * TS + i16;
    const uint32_t tlo = (uint32_t)trow0 * kSlice + (uint32_t)((q ^ (trow0 & 7)) * 16);
    auto sub_offset = [](int s) {
        return kSwiglu ? (uint32_t)((s & 1) * 4 + (s >> 1) * 128) * kSlice
                       : (uint32_t)(s * 4) * kSlice;
    };
    // weight scales: the 128-row block(s) of the wave's weight rows
    const int nb = (a.n + 127) / 128;
    const float* sb0;
    const float* sb1;
    {
        const float* base = a.bs + (int64_t)t.group * nb * nk;
        if (kSwiglu) {
            sb0 = base + (int64_t)t.col * nk;
            sb1 = base + (int64_t)(nb / 2 + t.col) * nk;
        } else {
            sb0 = base + (int64_t)min(t.col * 2 + (wn >> 1), nb - 1) * nk;
            sb1 = sb0;
        }
    }

    f32x4 acc[TS][kSubs];
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            acc[j][s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        load(min(i, nk - 1), i);
    int stage = 0;
    for (int kb = 0; kb < nk; ++kb) {
        // S - 2 later stages stay in flight; past the end the last slice is
        // loaded again, so that the count holds
        wait_loads<(S - 2) * kLoads>();
        const int into = stage == 0 ? S - 1 : stage - 1;
        load(min(kb + S - 1, nk - 1), into);
        const uint8_t* st = lds + stage * stage_bytes(TS);
        const float wb0 = sb0[kb], wb1 = sb1[kb];
        const float* scale = reinterpret_cast<const float*>(st + kScale) + trow0;
        auto weights = [&](int s) {
            return operand(st + wlo + sub_offset(s), st + (wlo ^ 64) + sub_offset(s));
        };
        auto tokens = [&](int j) {
            return operand(st + tlo + j * 16 * kSlice, st + (tlo ^ 64) + j * 16 * kSlice);
        };
        if constexpr (!kSwiglu) {
            i32x8 w[kSubs];
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
                w[s] = weights(s);
#pragma unroll
            for (int j = 0; j < TS; ++j) {
                const i32x8 x = tokens(j);
                const float c = scale[j * 16] * wb0;
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w[s], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[j][s][r] = __builtin_fmaf(p[r], c, acc[j][s][r]);
                }
            }
        } else {
            Widened w[kSubs];
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
                w[s] = widened(weights(s));
#pragma unroll
            for (int j = 0; j < TS; ++j) {
                const Widened x = widened(tokens(j));
                const float c0 = scale[j * 16] * wb0, c1 = scale[j * 16] * wb1;
                f32x4 p[kSubs];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
#pragma unroll
                    for (int s = 0; s < kSubs; ++s)
                        p[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            w[s].v[h], x.v[h], h == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : p[s], 0, 0,
                            0);
                }
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[j][s][r] = __builtin_fmaf(p[s][r], s < 2 ? c0 : c1, acc[j][s][r]);
                }
            }
        }
        stage = stage + 1 == S ? 0 : stage + 1;
    }

    // ---- epilogue
    if constexpr (!kSwiglu) {
        // a lane holds 16 consecutive columns of each of its rows
        const int col = t.col * kTileN + wn * kWaveRows + q * 16;
        const __amdgpu_buffer_rsrc_t ro =
            row_rsrc(a.out + t.row0 * a.n * 2, (uint32_t)t.rows * (uint32_t)a.n * 2u);
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            const uint32_t at = ((uint32_t)(trow0 + j * 16) * (uint32_t)a.n + (uint32_t)col) * 2u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f[r] = acc[j][2 * h][r];
                    f[4 + r] = acc[j][2 * h + 1][r];
                }
                if (col + h * 8 < a.n)  // rows past the tile's are dropped by the resource
                    bstore16<0>(narrow<DT>(f), ro, at + h * 16u);
            }
        }
    } else {
        // gate in operands 0 and 1, up in 2 and 3: a lane holds 8 consecutive
        // values of each of its rows, the wave 32, the four waves the block
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float g = acc[j][s][r];
                    const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
                    const float z = g * sig * acc[j][2 + s][r];
                    acc[j][s][r] = z;
                    amax = __builtin_fmaxf(amax, __builtin_fabsf(z));
                }
            }
            amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
            amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
            if (q == 0)
                s_amax[wn][trow0 + j * 16] = amax;
        }
        __syncthreads();
        const int inter = a.n / 2;
        const int col = t.col * 128 + wn * 32 + q * 8;
        const __amdgpu_buffer_rsrc_t ro =
            row_rsrc(a.out + t.row0 * inter, (uint32_t)t.rows * (uint32_t)inter);
        const uint32_t orow = (uint32_t)(inter / 128) * 4u;
        const __amdgpu_buffer_rsrc_t rsc =
            row_rsrc(a.osc + t.row0 * orow, (uint32_t)t.rows * orow);
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            const int row = trow0 + j * 16;
            const float amax = __builtin_fmaxf(__builtin_fmaxf(s_amax[0][row], s_amax[1][row]),
                                               __builtin_fmaxf(s_amax[2][row], s_amax[3][row]));
            float s, f;
            block_scale(amax, &s, &f);
            const u32x2 c = {e4m3x4(acc[j][0][0] * f, acc[j][0][1] * f, acc[j][0][2] * f,
                                    acc[j][0][3] * f),
                             e4m3x4(acc[j][1][0] * f, acc[j][1][1] * f, acc[j][1][2] * f,
                                    acc[j][1][3] * f)};
            __builtin_amdgcn_raw_buffer_store_b64(c, ro, row * inter + col, 0, 0);
            if (wn == 0 && q == 0)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, s), rsc,
                                                      row * orow + t.col * 4, 0, 0);
        }
    }
    // the next tile's loads overwrite the stages this one's waves still read,
    // and the maxima
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
}

template <int DT, bool kSwiglu>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void
moe_gemm_kernel(GemmArgs a)
{
    __shared__ __align__(1024) uint8_t lds[kLdsBytes];
    __shared__ float s_amax[4][256];
    __shared__ int s_part[kThreads / kWave];
    __shared__ int s_tile[4];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);

    // Row tiles of this thread's share of the groups, and where they start in
    // the list of all (group after group).
    const int share = (a.groups + kThreads - 1) / kThreads;
    const int g0 = min(a.groups, (int)threadIdx.x * share), g1 = min(a.groups, g0 + share);
    auto row_tiles = [&](int g, int* rows) {
        const int n = a.counts ? max(0, min(a.counts[g], a.cap)) : a.cap;
        *rows = n;
        return (n + 255) / 256;
    };
    int mine = 0, unused;
    for (int g = g0; g < g1; ++g)
        mine += row_tiles(g, &unused);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int u = __shfl_up(inc, o);
        if (lane >= o)
            inc += u;
    }
    if (lane == kWave - 1)
        s_part[wave] = inc;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        before += w < wave ? s_part[w] : 0;
        total += s_part[w];
    }
    total = uniform(total);

    // Tiles in rounds of the grid; in a round each of the 8 XCDs (blocks are
    // dealt to them in turn) takes consecutive tiles, which share weights and
    // rows in its L2. A group's tiles are numbered rows first.
    const int64_t tiles = (int64_t)total * a.col_tiles;
    for (int64_t t0 = 0; t0 < tiles; t0 += gridDim.x) {
        const int here = (int)min((int64_t)gridDim.x, tiles - t0);
        const int each = (here + 7) / 8;
        const int slot = (int)blockIdx.x / 8, place = ((int)blockIdx.x & 7) * each + slot;
        if (slot >= each || place >= here)
            continue;  // the whole block
        const int64_t tile = t0 + place;
        const int u = (int)(tile / a.col_tiles);
        if (u >= before && u < before + mine) {  // one thread: it holds the group
            int base = before, g = g0, rows, n = row_tiles(g, &rows);
            while (u >= base + n) {
                base += n;
                ++g;
                n = row_tiles(g, &rows);
            }
            const int at = (int)(tile - (int64_t)base * a.col_tiles);
            s_tile[0] = g;
            s_tile[1] = rows;
            s_tile[2] = at % n;
            s_tile[3] = at / n;
        }
        __syncthreads();
        Tile t;
        t.group = uniform(s_tile[0]);
        const int m = uniform(s_tile[2]);
        t.rows = min(256, uniform(s_tile[1]) - m * 256);
        t.col = uniform(s_tile[3]);
        t.row0 = (int64_t)t.group * a.cap + m * 256;
        if (t.rows > 128)
            run_tile<8, DT, kSwiglu>(a, t, lds, s_amax);
        else if (t.rows > 64)
            run_tile<4, DT, kSwiglu>(a, t, lds, s_amax);
        else
            run_tile<2, DT, kSwiglu>(a, t, lds, s_amax);
    }
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& a, int dtype, bool swiglu, int blocks, hipStream_t s)
{
    const dim3 grid(blocks), block(kThreads);
    if (swiglu)
        hipLaunchKernelGGL((moe_gemm_kernel<0, true>), grid, block, 0, s, a);
    else if (dtype == 0)
        hipLaunchKernelGGL((moe_gemm_kernel<0, false>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((moe_gemm_kernel<1, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
