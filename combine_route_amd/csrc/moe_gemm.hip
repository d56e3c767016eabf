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

#include <type_traits>

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
constexpr int kBLoads = kTileN / 64;            // 16-byte loads a lane and weight slice

// Token rows of a tile whose waves hold TS operands of 16 rows each, and its
// place in LDS: S slices of the rows, S of the weights, and two blocks of
// scales (4 steps of every row, then of the tile's two weight blocks).
constexpr int tile_rows(int ts) { return 2 * 16 * ts; }
constexpr int stages(int ts) { return ts == 8 ? 2 : 3; }
constexpr int a_bytes(int ts) { return tile_rows(ts) * kSlice; }
constexpr int kBBytes = kTileN * kSlice;
constexpr int scale_bytes(int ts) { return (tile_rows(ts) + 64) * 16; }
constexpr int lds_bytes(int ts) { return stages(ts) * (a_bytes(ts) + kBBytes) + 2 * scale_bytes(ts); }
constexpr int kLdsBytes = lds_bytes(4);
static_assert(lds_bytes(8) <= kLdsBytes && lds_bytes(2) <= kLdsBytes, "LDS of a block");

// Waits until at most N of this wave's loads are in flight, then for every
// wave: their slices have arrived, and LDS reads before here have returned.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Every wave's LDS reads before here have returned.
__device__ __forceinline__ void wait_reads()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 16 bytes a lane straight to LDS: lane i's to dst + 16 * i. NT: stream. In
// assembly because the compiler makes every LDS read after the builtin wait
// for all loads in flight (it cannot tell which slice a read is of); written
// so, the only waits are this file's own. No register is written, so nothing
// the load does later can meet the compiler's registers, and its own counted
// waits only get stricter by loads it does not know of.
// dst is an LDS address. M0 holds it; nothing else here uses M0.
template <bool NT>
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t dst, uint32_t off)
{
    const int at = uniform((int)dst);
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                     ::"s"(at), "v"(off), "s"(rsrc)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     ::"s"(at), "v"(off), "s"(rsrc)
                     : "memory");
}

// A base that every lane holds alike, and its row_rsrc, in scalar registers: a
// resource the compiler takes for a lane's own costs a loop over the lanes at
// every use.
__device__ __forceinline__ const uint8_t* uniform_ptr(const void* base)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint64_t lo = (uint32_t)uniform((int)(uint32_t)p);
    const uint64_t hi = (uint32_t)uniform((int)(uint32_t)(p >> 32));
    return reinterpret_cast<const uint8_t*>(lo | hi << 32);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, int64_t bytes)
{
    return row_rsrc(uniform_ptr(base), (uint32_t)uniform((int)bytes));
}

// The same resource as its four words.
__device__ __forceinline__ u32x4 rsrc_words(const uint8_t* base, int bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{(uint32_t)uniform((int)(uint32_t)p),
                 (uint32_t)uniform((int)(uint32_t)(p >> 32)) & 0xFFFFu, (uint32_t)uniform(bytes),
                 (uint32_t)kRsrcWord3};
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
    int rows;       // rows of the tile that exist, 1 .. 256; 0: no tile
    int col;        // column tile
};

// The loads of a tile's slices and scales. Wave w's i-th 1 KB of a slice holds
// rows 8 * (8 * i + w) .. + 7, a lane one 16-byte chunk of a row.
// kSwiglu: weight rows [0, 128) of the tile are gate rows 128 * col .., rows
// [128, 256) the up rows. Otherwise they are rows 256 * col .. .
template <int TS, bool kSwiglu>
struct Loads {
    static constexpr int S = stages(TS);
    static constexpr int kRows = tile_rows(TS);
    static constexpr int kALoads = kRows / 64;
    static constexpr int kB = S * a_bytes(TS);              // offsets in LDS
    static constexpr int kScale = kB + S * kBBytes;
    // weights of few rows are read once a call, and stream
    static constexpr bool kBStream = TS < 8;

    const uint8_t *abase, *bbase, *sbase;   // uniform, as the sizes
    int64_t bhalf;                           // from the tile's weight row 128 to row 0
    int abytes, bbytes0, bbytes1, sbytes;
    uint32_t aoff, boff, soff;
    int wave, nk;
    uint8_t* lds;                            // the block's, and its LDS address
    uint32_t lds0;

    __device__ __forceinline__ Loads(const GemmArgs& a, const Tile& t, uint8_t* block_lds,
                                     uint32_t block_lds0)
        : lds(block_lds), lds0(block_lds0)
    {
        const int lane = threadIdx.x & (kWave - 1);
        wave = uniform(threadIdx.x / kWave);
        nk = a.k / kSlice;
        const uint32_t K = (uint32_t)a.k;
        const int lr = wave * 8 + (lane >> 3);      // row of i = 0; i adds 64
        const int chunk = lane & 7;
        abase = uniform_ptr(a.a + t.row0 * K);
        abytes = uniform(t.rows * (int)K);
        aoff = (uint32_t)lr * K + (uint32_t)((chunk ^ (lr & 7)) * 16);
        // the key of a weight row: the bits in which the rows of an operand differ
        constexpr int kKeyShift = kSwiglu ? 3 : 4;
        const int key = (lr & 3) | (((lr >> kKeyShift) & 1) << 2);
        boff = (uint32_t)lr * K + (uint32_t)((chunk ^ key) * 16);
        const int64_t first = (int64_t)t.group * a.n;
        const int r0 = t.col * (kSwiglu ? 128 : kTileN);
        const int r1 = kSwiglu ? a.n / 2 + r0 : r0 + 128;
        bbase = uniform_ptr(a.b + (first + r0) * K);
        bhalf = (int64_t)(r1 - r0) * K;
        bbytes0 = uniform(min(128, a.n - r0) * (int)K);
        bbytes1 = uniform(max(0, min(128, a.n - r1)) * (int)K);
        // wave w loads the scales of rows 64 w .., the wave after the last of
        // them the two weight blocks' (lanes 0 and 1)
        const uint32_t srow = (uint32_t)nk * 4u;
        if (wave < kRows / 64) {
            sbase = uniform_ptr(a.as + (t.row0 + wave * 64) * srow);
            sbytes = uniform(max(0, min(64, t.rows - wave * 64)) * (int)srow);
            soff = (uint32_t)lane * srow;
        } else {
            const int nb = (a.n + 127) / 128;
            const int b0 = kSwiglu ? t.col : t.col * 2;
            const int b1 = kSwiglu ? nb / 2 + t.col : min(b0 + 1, nb - 1);
            const int64_t block = (int64_t)t.group * nb + b0;
            sbase = uniform_ptr(reinterpret_cast<const uint8_t*>(a.bs) + block * srow);
            sbytes = uniform((b1 - b0 + 1) * (int)srow);
            soff = (uint32_t)(lane == 0 ? 0 : lane == 1 ? b1 - b0 : b1 - b0 + 1) * srow;
        }
    }

    // First step of the 4 whose scales the block of step kb holds. The last
    // block of a row that is no multiple of 4 steps overlaps the one before.
    __device__ __forceinline__ int scale_start(int kb) const
    {
        return min(kb & ~3, max(0, nk - 4));
    }

    __device__ __forceinline__ void rows(int kb, int stage) const
    {
        if ((kb & 3) == 0 && wave <= kRows / 64) {
            const uint32_t at = kScale + ((kb >> 2) & 1) * scale_bytes(TS) + wave * 1024;
            if (nk >= 4) {
                load_to_lds<false>(rsrc_words(sbase, sbytes), lds0 + at,
                                   soff + (uint32_t)scale_start(kb) * 4u);
            } else {  // rows of 1 to 3 scales, once a tile
                const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(sbase, sbytes);
                float* own = reinterpret_cast<float*>(lds + at) + (threadIdx.x & (kWave - 1)) * 4;
                for (int c = 0; c < nk; ++c)
                    own[c] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(rs, (int)soff, c * 4, 0));
            }
        }
#pragma unroll
        for (int i = 0; i < kALoads; ++i)
            load_to_lds<false>(part(abase, abytes, i, kb),
                               lds0 + stage * a_bytes(TS) + (i * 8 + wave) * 1024, aoff);
    }

    __device__ __forceinline__ void weights(int kb, int stage) const
    {
#pragma unroll
        for (int i = 0; i < kBLoads; ++i)
            load_to_lds<kBStream>(i < 2 ? part(bbase, bbytes0, i, kb)
                                        : part(bbase + bhalf, bbytes1, i - 2, kb),
                                  lds0 + kB + stage * kBBytes + (i * 8 + wave) * 1024, boff);
    }

    // The rows from the i-th 64 on, from column kb * 128 on: a row of the tile
    // starts inside the bytes that are left and the first row past it does not.
    __device__ __forceinline__ u32x4 part(const uint8_t* base, int bytes, int i, int kb) const
    {
        const int skip = i * 64 * nk * kSlice + kb * kSlice;
        return rsrc_words(base + skip, max(0, bytes - skip));
    }

    // The first slices, in the order in which the steps ask for them: the
    // weights are one slice ahead of the rows.
    __device__ __forceinline__ void prologue() const
    {
        weights(0, 0);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) {
            if (i < nk)
                rows(i, i);
            if (i + 1 < nk)
                weights(i + 1, i + 1);
        }
    }
};

// The sums of one tile, whose first slices are on their way.
template <int TS, bool kSwiglu>
__device__ __forceinline__ void multiply(const Loads<TS, kSwiglu>& ld,
                                         f32x4 (&acc)[TS][kSubs])
{
    using L = Loads<TS, kSwiglu>;
    constexpr int S = L::S;
    const uint8_t* lds = ld.lds;
    const int lane = threadIdx.x & (kWave - 1);
    const int wm = ld.wave >> 2, wn = ld.wave & 3;
    const int q = lane >> 4, i16 = lane & 15;
    // a lane's row of each operand, its chunks q and q + 4 (exclusive-or 4)
    constexpr int kKeyShift = kSwiglu ? 3 : 4;
    const int wrow = kSwiglu ? wn * 32 + 8 * (i16 >> 2) + (i16 & 3)
                             : wn * kWaveRows + 16 * (i16 >> 2) + (i16 & 3);
    const int wkey = (wrow & 3) | (((wrow >> kKeyShift) & 1) << 2);
    const uint32_t wlo = L::kB + (uint32_t)wrow * kSlice + (uint32_t)((q ^ wkey) * 16);
    const int trow = wm * 16 * TS + i16;
    const uint32_t tlo = (uint32_t)trow * kSlice + (uint32_t)((q ^ (trow & 7)) * 16);
    auto sub_offset = [](int s) {
        return kSwiglu ? (uint32_t)((s & 1) * 4 + (s >> 1) * 128) * kSlice
                       : (uint32_t)(s * 4) * kSlice;
    };

#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            acc[j][s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int nk = ld.nk;
    int stage = 0;
    for (int kb = 0; kb < nk; ++kb) {
        // Issued after this step's rows: S - 1 slices of weights and S - 2 of
        // rows, fewer near the end.
        if (kb + S <= nk)
            wait_loads<(S - 1) * kBLoads + (S - 2) * L::kALoads>();
        else
            wait_loads<0>();
        const uint8_t* sa = lds + stage * a_bytes(TS);
        const uint8_t* sb = lds + stage * kBBytes;
        auto weights = [&](int s) {
            return operand(sb + wlo + sub_offset(s), sb + (wlo ^ 64) + sub_offset(s));
        };
        auto tokens = [&](int j) {
            return operand(sa + tlo + j * 16 * kSlice, sa + (tlo ^ 64) + j * 16 * kSlice);
        };
        if (kb + S - 1 < nk)
            ld.rows(kb + S - 1, stage == 0 ? S - 1 : stage - 1);
        i32x8 w[kSubs];
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            w[s] = weights(s);
        const float* scale = reinterpret_cast<const float*>(
                                 lds + L::kScale + ((kb >> 2) & 1) * scale_bytes(TS)) +
                             (kb - ld.scale_start(kb));
        const float wb0 = scale[(L::kRows + (kSwiglu ? 0 : wn >> 1)) * 4];
        const float wb1 = kSwiglu ? scale[(L::kRows + 1) * 4] : wb0;
        i32x8 x = tokens(0);
        // the weights' slice is in registers: its place takes the next but S - 1
        wait_reads();
        if (kb + S < nk)
            ld.weights(kb + S, stage);
        if constexpr (!kSwiglu) {
            f32x4 old[kSubs];
            float oldc = 0.0f;
#pragma unroll
            for (int j = 0; j < TS; ++j) {
                i32x8 next = x;
                if (j + 1 < TS)
                    next = tokens(j + 1);
                const float c = scale[(trow + j * 16) * 4] * wb0;
                f32x4 p[kSubs];
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    p[s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w[s], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                    if (j > 0) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[j - 1][s][r] = __builtin_fmaf(old[s][r], oldc, acc[j - 1][s][r]);
                    }
                }
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
                    old[s] = p[s];
                oldc = c;
                x = next;
            }
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[TS - 1][s][r] = __builtin_fmaf(old[s][r], oldc, acc[TS - 1][s][r]);
        } else {
            Widened v[kSubs];
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
                v[s] = widened(w[s]);
#pragma unroll
            for (int j = 0; j < TS; ++j) {
                const Widened y = widened(x);
                if (j + 1 < TS)
                    x = tokens(j + 1);
                const float sx = scale[(trow + j * 16) * 4];
                const float c0 = sx * wb0, c1 = sx * wb1;
#pragma unroll
                for (int s0 = 0; s0 < kSubs; s0 += 2) {
                    f32x4 p[2];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            p[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                v[s0 + s].v[h], y.v[h],
                                h == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : p[s], 0, 0, 0);
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[j][s0 + s][r] =
                                __builtin_fmaf(p[s][r], s0 ? c1 : c0, acc[j][s0 + s][r]);
                    }
                }
            }
        }
        stage = stage + 1 == S ? 0 : stage + 1;
    }
}

// The tile's sums to memory.
template <int TS, int DT, bool kSwiglu>
__device__ __forceinline__ void finish(const GemmArgs& a, const Tile& t, float (*s_amax)[256],
                                       f32x4 (&acc)[TS][kSubs])
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;
    const int q = lane >> 4;
    const int trow0 = wm * 16 * TS + (lane & 15);
    // ---- epilogue
    if constexpr (!kSwiglu) {
        // a lane holds 16 consecutive columns of each of its rows
        const int col = t.col * kTileN + wn * kWaveRows + q * 16;
        const __amdgpu_buffer_rsrc_t ro =
            uniform_rsrc(a.out + t.row0 * a.n * 2, (uint32_t)t.rows * (uint32_t)a.n * 2u);
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
            uniform_rsrc(a.out + t.row0 * inter, (uint32_t)t.rows * (uint32_t)inter);
        const uint32_t orow = (uint32_t)(inter / 128) * 4u;
        const __amdgpu_buffer_rsrc_t rsc =
            uniform_rsrc(a.osc + t.row0 * orow, (uint32_t)t.rows * orow);
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
}

// Operands of 16 rows a wave that a tile of this many rows needs.
__device__ __forceinline__ int tile_class(int rows) { return rows > 128 ? 8 : rows > 64 ? 4 : 2; }

template <int DT, bool kSwiglu>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void
moe_gemm_kernel(GemmArgs a)
{
    __shared__ __align__(1024) uint8_t lds[kLdsBytes];
    __shared__ float s_amax[4][256];
    __shared__ int s_part[kThreads / kWave];
    __shared__ int s_first[kThreads + 1];
    __shared__ int s_tile[2][4];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);

    // Row tiles of each thread's share of the groups, as where they start in
    // the list of all (group after group). Kept in LDS: the sums need every
    // register.
    auto rows_of = [&](int g) {
        return a.counts ? max(0, min(a.counts[g], a.cap)) : a.cap;
    };
    const int share = (a.groups + kThreads - 1) / kThreads;
    {
        const int g0 = min(a.groups, (int)threadIdx.x * share), g1 = min(a.groups, g0 + share);
        int mine = 0;
        for (int g = g0; g < g1; ++g)
            mine += (rows_of(g) + 255) / 256;
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
        s_first[threadIdx.x] = before;
        if (threadIdx.x == 0)
            s_first[kThreads] = total;
        __syncthreads();
    }
    const int64_t tiles = (int64_t)uniform(s_first[kThreads]) * a.col_tiles;

    // Tiles in rounds of the grid; in a round each of the 8 XCDs (blocks are
    // dealt to them in turn) takes consecutive tiles, which share weights and
    // rows in its L2. A group's tiles are numbered rows first. Only the last
    // round can leave a block without a tile.
    auto tile_at = [&](int64_t t0) -> int64_t {
        const int64_t left = tiles - t0;
        if (left <= 0)
            return -1;
        const int here = (int)min((int64_t)gridDim.x, left);
        const int each = (here + 7) / 8;
        const int slot = (int)blockIdx.x / 8, place = ((int)blockIdx.x & 7) * each + slot;
        return slot < each && place < here ? t0 + place : -1;
    };
    // The thread whose share holds the tile says which it is.
    auto look_up = [&](int64_t tile, int (&info)[4]) {
        const int u = (int)(tile / a.col_tiles);
        int base = s_first[threadIdx.x];
        if (u < base || u >= s_first[threadIdx.x + 1])
            return;
        int g = (int)threadIdx.x * share, rows = rows_of(g), n = (rows + 255) / 256;
        while (u >= base + n) {
            base += n;
            ++g;
            rows = rows_of(g);
            n = (rows + 255) / 256;
        }
        const int at = (int)(tile - (int64_t)base * a.col_tiles);
        info[0] = g;
        info[1] = rows;
        info[2] = at % n;
        info[3] = at / n;
    };
    auto read_tile = [&](const int (&info)[4]) {
        Tile t;
        t.group = uniform(info[0]);
        const int m = uniform(info[2]);
        t.rows = min(256, uniform(info[1]) - m * 256);
        t.col = uniform(info[3]);
        t.row0 = (int64_t)t.group * a.cap + m * 256;
        return t;
    };

    int64_t t0 = 0;
    int64_t tile = tile_at(t0);
    if (tile < 0)
        return;  // the whole block
    look_up(tile, s_tile[0]);
    __syncthreads();
    Tile t = read_tile(s_tile[0]);
    bool loading = false;  // t's first slices are on their way
    int slot = 0;
    // One tile of class TS; then t is the next one (or has no rows).
    auto run = [&](auto ts) {
        constexpr int TS = decltype(ts)::value;
        const Loads<TS, kSwiglu> ld(a, t, lds, lds0);
        if (!loading)
            ld.prologue();
        t0 += gridDim.x;
        const int64_t next = tile_at(t0);
        slot ^= 1;
        if (next >= 0)
            look_up(next, s_tile[slot]);  // read after the steps' barriers
        f32x4 acc[TS][kSubs];
        multiply<TS, kSwiglu>(ld, acc);
        wait_reads();
        const Tile done = t;
        t.rows = 0;
        loading = false;
        if (next >= 0) {
            t = read_tile(s_tile[slot]);
            if (tile_class(t.rows) == TS) {
                // the next tile's loads run under this one's stores
                const Loads<TS, kSwiglu> then(a, t, lds, lds0);
                then.prologue();
                loading = true;
            }
        }
        finish<TS, DT, kSwiglu>(a, done, s_amax, acc);
    };
    while (t.rows > 0) {
        switch (tile_class(t.rows)) {
        case 8: run(std::integral_constant<int, 8>()); break;
        case 4: run(std::integral_constant<int, 4>()); break;
        default: run(std::integral_constant<int, 2>()); break;
        }
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
