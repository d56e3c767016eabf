// gfx950 (MI355X, CDNA4) kernel of moe_grouped_gemm (include/moe.h): each
// expert's product of its expert-major FP8 rows with its FP8 weights, a scale
// per row and 128 elements on one side and per 128 x 128 block on the other,
// to bf16 / fp16 rows or, with gate and up weights, to FP8 rows of
// silu(gate) * up with their own scales.
//
// A work item is a tile of up to 224 rows of one expert by 256 weight rows.
// Row counts are on the GPU, so the launch is a fixed grid of one block a
// compute unit; each block works out every expert's tile range from the
// counts and walks its share of the tiles. An expert's last tile computes as
// few of 32 (swiglu form), 64, 128 or 224 rows as hold its rows, so that experts
// with few rows cost their weights' bytes and little else.
//
// The FP8 matrix instruction adds 8 products of neighbouring k at a time, each
// first cut toward zero to a multiple of 2^(E - 13), E the largest sum of the
// operands' exponents among the nonzero ones, a subnormal's taken as -6 (measured
// on gfx950: this gives its every result over random codes of all ranges; between
// eights nothing is cut, 200704 - 200704 + 2^-6 is 2^-6; the same in
// v_mfma_f32_16x16x32_fp8_fp8). Rows of bf16 / fp16 take it at twice the 16-bit
// rate: what is lost is under 7/512 of what half a step of the codes that set E
// makes up, and in rows of ordinary spread 1.3e-5 of a row's norm whatever k, 1/20
// of fp16's rounding and 1/150 of bf16's. The swiglu form returns its block scales
// in FP32 (off by 1.2e-5 that way), so there both operands are widened to fp16
// (exact) in registers and multiplied by v_mfma_f32_16x16x32_f16, whose sums
// of such products are FP32's (scales off by 2e-7); the matrix rate is half.
//
// Inside a tile: 8 waves, 2 along the rows x 4 along the weight rows (1 x 8 of
// 32 rows). For each 128 elements of k (a step) the block holds both operands'
// slices (128 bytes a row) in LDS, loaded there directly from memory two steps
// and more before. The matrix instruction has the weights as its rows and the
// token rows as its columns: v_mfma_f32_16x16x128_f8f6f4 takes a whole scale
// block of k, a lane then holds one token row's partial sums, so the scales'
// product is one value a lane and the partial joins the FP32 sum with a fused
// multiply-add an element, beside the next matrix instruction. 224 rows: the
// largest tile whose rows' slices fit LDS three times beside two of the
// weights' (256 rows with two of each: 1009 against 960 us at 32 experts x
// 1024 rows, k 7168, n 4096).
//
// LDS slices are 128 bytes a row without padding; the eight 16-byte chunks of
// a row are permuted by a key of the row, so the 16 rows a matrix operand
// reads together fall in different banks. Both operands take the chunks in
// the same order, so the order of k inside an instruction is the same too.
//
// Measured on MI355X (a large FP8 library product: 2.6 PFLOP/s, bf16 1.35;
// weights streamed to LDS alone: 7.0 TB/s): 32 experts x 1024 rows, n 7168, k
// 2048 520 to 590 us over cards and row counts (1.6 to 1.85 PFLOP/s), n 4096, k
// 7168 965 us (2.0); gate and up, n 4096, k 7168, 32768 rows in all 1.66 to 1.86 ms
// (1.0 to 1.16 PFLOP/s in fp16 products; without its loads 1.4 ms). No unit is full
// in large tiles (counters at the first case): matrix units busy 42% of the
// cycles, vector issue 37%, LDS 23%, at 2.0 GHz; without their loads they take 780
// us instead of 960, so what bounds them is the phases of a step that do not run
// beside each other. 256 experts x 32 rows, n 7168, k 2048 650 to 690 us (5.7 TB/s;
// 545 without its stores: 117 MB of scattered rows in a stream of reads), gate and
// up of 32 experts x 32 rows 175 us (5.3 TB/s; its loads alone 143, its products
// and conversions alone 145): bound by memory and those phases. Fewer tiles than
// compute units leave the rest idle and a step its loads' latency: 27 experts x 4
// rows, k 4608, n 256, gate and up, 35 us for 32 MB.
//   The swiglu kernel has 47 registers a lane in scratch memory (the rows kernels
// none): a loop over k touches one, on the branch of k below 512, but the code
// between tiles reloads them, and a reload waits for every load before it, the next
// tile's first slices among them. They are 21 MB of scratch memory over the grid,
// written once a call and more (counters: 23.5 MB written at 32 x 32 rows for 2.2
// MB of output).
//   Tried and no faster: widening by shifts and masks instead of conversions (221
// against 180 us), the wave halves taking turns at reading and multiplying (1108
// against 1010 us), raised wave priority, a step's loads all in its first
// products (980 against 950 us), products of 32 x 32 x 16 in the swiglu form
// (2.0 ms: a product's 32 sums run in one piece), operands a step ahead in
// tiles of few rows, streamed weights in large tiles (1027 against 972 us),
// one range of tiles an XCD (790 against 745 us with skewed rows).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_lds.h"

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
constexpr int kBLoads = kTileN / 64;            // 16-byte loads a lane and weight slice

// A tile of class TS has 32 TS token rows. Its waves lie 2 along the rows and 4
// along the weight rows; those of 32 rows 1 and 8, so that each weight row is
// read from LDS (and widened) once. A wave holds row_subs operands of 16 token
// rows and col_subs of 16 weight rows.
constexpr int kMaxTS = 7;
constexpr int row_waves(int ts) { return ts == 1 ? 1 : 2; }
constexpr int col_waves(int ts) { return ts == 1 ? 8 : 4; }
constexpr int row_subs(int ts) { return 2 * ts / row_waves(ts); }
constexpr int col_subs(int ts) { return kTileN / 16 / col_waves(ts); }
constexpr int tile_rows(int ts) { return 32 * ts; }
// Its place in LDS: kAStages slices of the rows, b_stages of the weights, and
// two blocks of scales (4 steps of every row, then of the tile's two weight
// blocks), of which the second holds the col_waves' block maxima at the end.
constexpr int kTileRows = tile_rows(kMaxTS);
constexpr int kAStages = 3;
constexpr int b_stages(int ts) { return ts == 7 ? 2 : ts == 4 ? 3 : 4; }
// Whether a step has one barrier, see multiply().
constexpr bool one_barrier(int ts, bool swiglu) { return swiglu && ts < kMaxTS; }
constexpr int a_bytes(int ts) { return tile_rows(ts) * kSlice; }
constexpr int kBBytes = kTileN * kSlice;
constexpr int scale_bytes(int ts)
{
    return ts == 1 ? col_waves(ts) * 4 * tile_rows(ts) : (tile_rows(ts) + 2) * 16;
}
constexpr int scale_at(int ts) { return kAStages * a_bytes(ts) + b_stages(ts) * kBBytes; }
constexpr int lds_bytes(int ts) { return scale_at(ts) + 2 * scale_bytes(ts); }
constexpr int kLdsBytes = lds_bytes(7);
static_assert(lds_bytes(4) <= kLdsBytes && lds_bytes(2) <= kLdsBytes && lds_bytes(1) <= kLdsBytes,
              "LDS of a block");

// As load_to_lds, for those of lanes 0 to 31 that are active; the mask is as
// before afterwards.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_half_to_lds(u32x4 rsrc, uint32_t dst, uint32_t off,
                                                 uint32_t soff)
{
    uint64_t lanes;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, exec\n\ts_mov_b32 exec_hi, 0\n\t"
                 "buffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b64 exec, %0"
                 : "=&s"(lanes)
                 : "s"(dst), "v"(off), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

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

// The same resource as its four words, and back.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(u32x4 w)
{
    const uint32_t lo = w[0], hi = w[1];
    return row_rsrc(reinterpret_cast<const void*>(lo | (uint64_t)hi << 32), w[2]);
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

// Two fp16 values of an operand of 8, pair i of operand h, from the half of the
// chunks that holds it.
__device__ __forceinline__ uint32_t widened2(const i32x4& half, int h, int i)
{
    const int word = half[(h & 1) * 2 + (i >> 1)];
    const f16x2 r = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, false);
    return __builtin_bit_cast(uint32_t, r);
}

// One tile: the group's first row, how many rows, and the column tile.
struct Tile {
    int64_t row0;   // first row (of [groups * cap])
    int group;
    int rows;       // rows of the tile that exist, 1 .. kTileRows; 0: no tile
    int col;        // column tile
};

// The loads of a tile's slices and scales. Wave w's i-th 1 KB of a slice holds
// rows 8 * (8 * i + w) .. + 7, a lane one 16-byte chunk of a row; the last 32
// of 224 rows are shared by half waves, 4 rows each. Slices past the last are
// asked for too, from beyond the resource's end (zeros, without memory
// traffic), so that a step has the same loads in flight near the end and no
// branch.
// kSwiglu: weight rows [0, 128) of the tile are gate rows 128 * col .., rows
// [128, 256) the up rows. Otherwise they are rows 256 * col .. .
template <int TS, bool kSwiglu>
struct Loads {
    static constexpr int SB = b_stages(TS);
    static constexpr bool kOneBarrier = one_barrier(TS, kSwiglu);
    static constexpr int kLead = kOneBarrier ? SB - 1 : SB;  // steps the weights are ahead
    static constexpr int kRows = tile_rows(TS);
    static constexpr int kALoads = (kRows + 63) / 64;       // loads a wave and slice of rows
    static constexpr int kAll = kALoads + kBLoads;          // and of both
    static constexpr int kB = kAStages * a_bytes(TS);       // offsets in LDS
    static constexpr int kScale = scale_at(TS);
    // weights of few rows are read once a call, and stream (a stream of
    // weights alone reaches 7.0 TB/s so, 6.2 without)
    static constexpr bool kBStream = TS < kMaxTS;

    u32x4 ra, rb0, rb1, rs;                  // rows, the two halves of the weights, scales
    int slanes;                              // lanes that load a scale
    uint32_t aoff, alast, boff, soff;
    uint32_t step64;                         // bytes of 64 rows of k
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
        step64 = 64 * K;
        ra = rsrc_words(a.a + t.row0 * K, t.rows * (int)K);
        aoff = (uint32_t)lr * K + (uint32_t)((chunk ^ (lr & 7)) * 16);
        const int hr = (kALoads - 1) * 64 + wave * 4 + (lane >> 3);
        alast = kRows % 64 ? (uint32_t)hr * K + (uint32_t)((chunk ^ (hr & 7)) * 16)
                           : aoff + (uint32_t)(kALoads - 1) * step64;
        // the key of a weight row: the bits in which the rows of an operand differ
        const int key = (lr & 3) | (((lr >> 3) & 1) << 2);
        boff = (uint32_t)lr * K + (uint32_t)((chunk ^ key) * 16);
        const int64_t first = (int64_t)t.group * a.n;
        const int r0 = t.col * (kSwiglu ? 128 : kTileN);
        const int r1 = kSwiglu ? a.n / 2 + r0 : r0 + 128;
        rb0 = rsrc_words(a.b + (first + r0) * K, min(128, a.n - r0) * (int)K);
        rb1 = rsrc_words(a.b + (first + (r1 < a.n ? r1 : r0)) * K,
                         max(0, min(128, a.n - r1)) * (int)K);
        // wave w loads the scales of rows 64 w .. (below kRows), the wave after
        // the last of them the two weight blocks' (lanes 0 and 1)
        const uint32_t srow = (uint32_t)nk * 4u;
        if (wave < kALoads) {
            rs = rsrc_words(a.as + (t.row0 + wave * 64) * srow,
                            max(0, min(64, t.rows - wave * 64)) * (int)srow);
            soff = (uint32_t)lane * srow;
            slanes = uniform(min(64, kRows - wave * 64));
        } else {
            const int nb = (a.n + 127) / 128;
            const int b0 = kSwiglu ? t.col : t.col * 2;
            const int b1 = kSwiglu ? nb / 2 + t.col : min(b0 + 1, nb - 1);
            const int64_t block = (int64_t)t.group * nb + b0;
            rs = rsrc_words(reinterpret_cast<const uint8_t*>(a.bs) + block * srow,
                            (b1 - b0 + 1) * (int)srow);
            soff = (uint32_t)(lane == 1 ? b1 - b0 : 0) * srow;
            slanes = uniform(wave == kALoads ? 2 : 0);
        }
    }

    // First step of the 4 whose scales the block of step kb holds. The last
    // block of a row that is no multiple of 4 steps overlaps the one before.
    __device__ __forceinline__ int scale_start(int kb) const
    {
        return min(kb & ~3, max(0, nk - 4));
    }

    // The scales of 4 steps, with the first of them.
    __device__ __forceinline__ void scales(int kb) const
    {
        const int lane = threadIdx.x & (kWave - 1);
        if (kb < nk && (kb & 3) == 0 && lane < slanes) {
            const int first = wave < kALoads ? wave * 64 : kRows;
            const uint32_t at = kScale + ((kb >> 2) & 1) * scale_bytes(TS) + first * 16;
            if (nk >= 4) {
                load_to_lds<false>(rs, lds0 + at, soff, (uint32_t)scale_start(kb) * 4u);
            } else {  // rows of 1 to 3 scales, once a tile
                const __amdgpu_buffer_rsrc_t r = rsrc_of(rs);
                float* own = reinterpret_cast<float*>(lds + at) + lane * 4;
                for (int c = 0; c < nk; ++c)
                    own[c] = __builtin_bit_cast(
                        float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)soff, c * 4, 0));
            }
        }
    }

    // Offset that takes a load of a slice past the last beyond any resource.
    __device__ __forceinline__ uint32_t past(int kb) const { return kb < nk ? 0u : 1u << 30; }

    // Load i of slice kb of the rows, or of the weights, to its stage.
    __device__ __forceinline__ void row_load(int i, int kb, int stage) const
    {
        const uint32_t dst = lds0 + stage * a_bytes(TS) + i * 8192;
        if (kRows % 64 && i == kALoads - 1)
            load_half_to_lds(ra, dst + wave * 512, alast + past(kb), (uint32_t)kb * kSlice);
        else
            load_to_lds<false>(ra, dst + wave * 1024, aoff + i * step64 + past(kb),
                               (uint32_t)kb * kSlice);
    }

    __device__ __forceinline__ void weight_load(int i, int kb, int stage) const
    {
        load_to_lds<kBStream>(i < 2 ? rb0 : rb1,
                              lds0 + kB + stage * kBBytes + i * 8192 + wave * 1024,
                              boff + (i & 1) * step64 + past(kb), (uint32_t)kb * kSlice);
    }

    // The first slices, in the order in which the steps ask for them.
    __device__ __forceinline__ void prologue() const
    {
        auto weights = [&](int kb) {
#pragma unroll
            for (int i = 0; i < kBLoads; ++i)
                weight_load(i, kb, kb);
        };
#pragma unroll
        for (int kb = 0; kb < kLead - 2; ++kb)
            weights(kb);
        scales(0);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int i = 0; i < kALoads; ++i)
                row_load(i, kb, kb);
            weights(kLead - 2 + kb);
        }
    }
};

// The sums of one tile, whose first slices are on their way. A step has two
// barriers. The first waits for the step's slices and ends the reads of the
// step before, so the place of the rows' slice kb - 1 is free for slice kb +
// 2. Then every wave takes its weights' operands to registers; the second
// barrier frees their place for slice kb + SB. In the swiglu form's smaller
// tiles there is none: the weights' slice kb + SB - 1 goes where slice kb - 1
// was, and a wave may read while another multiplies (27 experts x 4 rows, k
// 4608, n 256: 38 -> 34 us; 32 x 32 rows, k 7168, n 4096: 180 -> 176; in the
// other form, 256 x 32 rows, k 2048, n 7168, 684 -> 690).
// The products follow, each matrix instruction with as much other work as runs
// beside it, and the loads spread among them: issued together they hold up the
// waves, which issue in order, until the load unit has taken them.
template <int TS, bool kSwiglu>
__device__ __forceinline__ void multiply(const Loads<TS, kSwiglu>& ld,
                                         f32x4 (&acc)[row_subs(TS)][col_subs(TS)])
{
    using L = Loads<TS, kSwiglu>;
    constexpr int kRowSubs = row_subs(TS), kSubs = col_subs(TS);
    constexpr int SB = L::SB;
    const uint8_t* lds = ld.lds;
    const int lane = threadIdx.x & (kWave - 1);
    const int wm = ld.wave / col_waves(TS), wn = ld.wave % col_waves(TS);
    const int q = lane >> 4, i16 = lane & 15;
    // a lane's row of each operand, its chunks q and q + 4 (exclusive-or 4)
    // (gate rows in the swiglu form; its up rows are 128 further)
    const int wrow = (!kSwiglu     ? wn * 16 * kSubs
                      : kSubs == 4 ? wn * 32
                                   : (wn >> 1) * 32 + (wn & 1) * 4) +
                     8 * (i16 >> 2) + (i16 & 3);
    const int wkey = (wrow & 3) | (((wrow >> 3) & 1) << 2);
    const uint32_t wlo = L::kB + (uint32_t)wrow * kSlice + (uint32_t)((q ^ wkey) * 16);
    const int trow = wm * 16 * kRowSubs + i16;
    const uint32_t tlo = (uint32_t)trow * kSlice + (uint32_t)((q ^ (trow & 7)) * 16);
    auto sub_offset = [](int s) {
        return (uint32_t)(kSwiglu && kSubs == 2 ? s * 128
                                                : (s & 1) * 4 + (s >> 1) * (kSwiglu ? 128 : 32)) *
               kSlice;
    };

#pragma unroll
    for (int j = 0; j < kRowSubs; ++j)
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            acc[j][s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int nk = ld.nk;
    // Loads a wave has in flight when a step starts, of those asked for after
    // the step's rows (two steps ahead its weights come after them). Scales
    // come on top now and then, which only makes the wait stricter.
    constexpr int kLater = L::kLead > 2 ? L::kAll + kBLoads : L::kAll;

    int sta = 0, stb = 0;  // stages of step kb
    for (int kb = 0; kb < nk; ++kb) {
        const uint8_t* sa = lds + sta * a_bytes(TS);
        const uint8_t* sb = lds + stb * kBBytes;
        static_assert(kAStages == 3, "stage of step kb + 2");
        // 16 bytes of this lane's row of operand j: chunk q (half 0) or q + 4
        auto tokens = [&](int j, int half) {
            return *reinterpret_cast<const i32x4*>(sa + (half ? tlo ^ 64 : tlo) + j * 16 * kSlice);
        };
        phase_end<kLater>();
        ld.scales(kb + 2);
        const int free_a = sta == 0 ? 2 : sta - 1;
        const int free_b = !L::kOneBarrier ? stb : stb == 0 ? SB - 1 : stb - 1;
        // load `i` of the step's, rows first
        auto ask = [&](int i) {
            if (i < L::kALoads)
                ld.row_load(i, kb + 2, free_a);
            else
                ld.weight_load(i - L::kALoads, kb + L::kLead, free_b);
        };
        i32x8 w[kSubs];
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            w[s] = operand(sb + wlo + sub_offset(s), sb + (wlo ^ 64) + sub_offset(s));
        const float* scale =
            reinterpret_cast<const float*>(lds + L::kScale + ((kb >> 2) & 1) * scale_bytes(TS)) +
            (kb - ld.scale_start(kb));
        const float wb0 = scale[(L::kRows + (kSwiglu ? 0 : wn / (col_waves(TS) / 2))) * 4];
        const float wb1 = kSwiglu ? scale[(L::kRows + 1) * 4] : wb0;
        float sx = scale[trow * 4];
        i32x4 lo = tokens(0, 0), hi = tokens(0, 1);
        if constexpr (!L::kOneBarrier)
            phase_end();
        Widened v[kSwiglu ? kSubs : 1];
        u32x4 y[2];  // operands of 8 values, in turn
        if constexpr (kSwiglu) {
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
                v[s] = widened(w[s]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[0][i] = widened2(lo, 0, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        auto asks = [&](int j) {  // the loads of operand j's turn
#pragma unroll
            for (int i = 0; i < L::kAll; ++i)
                if (i * kRowSubs / L::kAll == j)
                    ask(i);
        };
        f32x4 old[kSubs];  // the products of operand j - 1
        float oldc0 = 0.0f, oldc1 = 0.0f;
        if constexpr (!kSwiglu) {
#pragma unroll
            for (int j = 0; j < kRowSubs; ++j) {
                const i32x8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                const float c = sx * wb0;
                if (j + 1 < kRowSubs) {
                    lo = tokens(j + 1, 0);
                    hi = tokens(j + 1, 1);
                    sx = scale[(trow + (j + 1) * 16) * 4];
                }
                f32x4 p[kSubs];
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    p[s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w[s], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                    if (j > 0) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[j - 1][s][r] = __builtin_fmaf(old[s][r], oldc0, acc[j - 1][s][r]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                asks(j);
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
                    old[s] = p[s];
                oldc0 = c;
            }
            oldc1 = oldc0;
        } else {
#pragma unroll
            for (int j = 0; j < kRowSubs; ++j) {
                const float c0 = sx * wb0, c1 = sx * wb1;
                f32x4 p[kSubs];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
#pragma unroll
                    for (int s = 0; s < kSubs; ++s) {
                        p[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            v[s].v[h], __builtin_bit_cast(f16x8, y[h & 1]),
                            h == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : p[s], 0, 0, 0);
                        // its share of the next operand's value pairs
#pragma unroll
                        for (int i = s * 4 / kSubs; i < (s + 1) * 4 / kSubs; ++i) {
                            if (h < 3)
                                y[(h + 1) & 1][i] = widened2(h == 0 ? lo : hi, h + 1, i);
                            else if (j + 1 < kRowSubs)
                                y[0][i] = widened2(lo, 0, i);
                        }
                        // and one sum of the products before
                        if (j > 0) {
                            const int c = (h * kSubs + s) / 4, r = (h * kSubs + s) % 4;
                            acc[j - 1][c][r] = __builtin_fmaf(
                                old[c][r], c < kSubs / 2 ? oldc0 : oldc1, acc[j - 1][c][r]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (j + 1 < kRowSubs) {  // the halves are read again as soon as they are widened
                        if (h == 0)
                            lo = tokens(j + 1, 0);
                        if (h == 2)
                            hi = tokens(j + 1, 1);
                        if (h == 3)
                            sx = scale[(trow + (j + 1) * 16) * 4];
                    }
                    if (h == 1)
                        asks(j);
                }
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
                    old[s] = p[s];
                oldc0 = c0;
                oldc1 = c1;
            }
        }
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[kRowSubs - 1][s][r] = __builtin_fmaf(
                    old[s][r], s < kSubs / 2 ? oldc0 : oldc1, acc[kRowSubs - 1][s][r]);
        sta = sta == 2 ? 0 : sta + 1;
        stb = stb + 1 == SB ? 0 : stb + 1;
    }
    phase_end();
}

// The tile's sums to memory.
template <int TS, int DT, bool kSwiglu>
__device__ __forceinline__ void finish(const GemmArgs& a, const Tile& t, float (*s_amax)[tile_rows(TS)],
                                       f32x4 (&acc)[row_subs(TS)][col_subs(TS)])
{
    constexpr int kRowSubs = row_subs(TS), kSubs = col_subs(TS);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave / col_waves(TS), wn = wave % col_waves(TS);
    const int q = lane >> 4;
    const int trow0 = wm * 16 * kRowSubs + (lane & 15);
    // ---- epilogue
    if constexpr (!kSwiglu) {
        // a lane holds runs of 8 columns of each of its rows; the 4 lanes of
        // a row write 64 bytes together. Rows few and far between are written
        // through the L2 (sc1), which the weights stream through (256 experts x
        // 32 rows, k 2048, n 7168: 716 -> 680 us).
        constexpr int kStore = TS < kMaxTS ? 16 : 0;
        const int col = t.col * kTileN + wn * 16 * kSubs + q * 8;
        const __amdgpu_buffer_rsrc_t ro =
            uniform_rsrc(a.out + t.row0 * a.n * 2, (uint32_t)t.rows * (uint32_t)a.n * 2u);
#pragma unroll
        for (int j = 0; j < kRowSubs; ++j) {
            const uint32_t at = ((uint32_t)(trow0 + j * 16) * (uint32_t)a.n + (uint32_t)col) * 2u;
#pragma unroll
            for (int h = 0; h < kSubs / 2; ++h) {
                float f[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f[r] = acc[j][2 * h][r];
                    f[4 + r] = acc[j][2 * h + 1][r];
                }
                if (col + h * 32 < a.n)  // rows past the tile's are dropped by the resource
                    bstore16<kStore>(narrow<DT>(f), ro, at + h * 64u);
            }
        }
    } else {
        // gate in the first half of the operands, up in the second: a lane holds
        // 8 (4 of 2 operands) consecutive values of each of its rows
        constexpr int kGate = kSubs / 2;
#pragma unroll
        for (int j = 0; j < kRowSubs; ++j) {
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < kGate; ++s) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float z = silu_times(acc[j][s][r], acc[j][kGate + s][r]);
                    acc[j][s][r] = z;
                    amax = __builtin_fmaxf(amax, __builtin_fabsf(z));
                }
            }
            amax = __builtin_fmaxf(amax, __shfl_xor(amax, 16));
            amax = __builtin_fmaxf(amax, __shfl_xor(amax, 32));
            if (q == 0)
                s_amax[wn][trow0 + j * 16] = amax;
        }
        phase_end();
        const int inter = a.n / 2;
        const int col =
            t.col * 128 + q * 8 + (kGate == 2 ? wn * 32 : (wn >> 1) * 32 + (wn & 1) * 4);
        const __amdgpu_buffer_rsrc_t ro =
            uniform_rsrc(a.out + t.row0 * inter, (uint32_t)t.rows * (uint32_t)inter);
        const uint32_t orow = (uint32_t)(inter / 128) * 4u;
        const __amdgpu_buffer_rsrc_t rsc =
            uniform_rsrc(a.osc + t.row0 * orow, (uint32_t)t.rows * orow);
#pragma unroll
        for (int j = 0; j < kRowSubs; ++j) {
            const int row = trow0 + j * 16;
            float amax = s_amax[0][row];
#pragma unroll
            for (int w = 1; w < col_waves(TS); ++w)
                amax = __builtin_fmaxf(amax, s_amax[w][row]);
            float s, f;
            block_scale(amax, &s, &f);
            uint32_t c[kGate];
#pragma unroll
            for (int s = 0; s < kGate; ++s)
                c[s] = e4m3x4(acc[j][s][0] * f, acc[j][s][1] * f, acc[j][s][2] * f,
                              acc[j][s][3] * f);
            if constexpr (kGate == 2)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{c[0], c[1]}, ro, row * inter + col, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(c[0], ro, row * inter + col, 0, 0);
            if (wn == 0 && q == 0)
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, s), rsc,
                                                      row * orow + t.col * 4, 0, 0);
        }
    }
}

// The class of a tile with this many rows. The class of 32 rows is the swiglu
// form's alone: what it saves is the widening (222 experts x 1 to 9 rows, k
// 6272, n 512: 149 -> 134 us; 27 x 4 rows, k 4608, n 256: 50 -> 38), and in the
// other form a change of class between tiles, whose loads then start late,
// costs more than it gains (256 experts x 16 to 48 rows: 684 -> 698 us).
template <bool kSwiglu>
__device__ __forceinline__ int tile_class(int rows)
{
    return rows > 128 ? 7 : rows > 64 ? 4 : rows > 32 || !kSwiglu ? 2 : 1;
}

template <int DT, bool kSwiglu>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void
moe_gemm_kernel(GemmArgs a)
{
    __shared__ __align__(1024) uint8_t lds[kLdsBytes];
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
            mine += (rows_of(g) + kTileRows - 1) / kTileRows;
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
        int g = (int)threadIdx.x * share, rows = rows_of(g), n = (rows + kTileRows - 1) / kTileRows;
        while (u >= base + n) {
            base += n;
            ++g;
            rows = rows_of(g);
            n = (rows + kTileRows - 1) / kTileRows;
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
        t.rows = min(kTileRows, uniform(info[1]) - m * kTileRows);
        t.col = uniform(info[3]);
        t.row0 = (int64_t)t.group * a.cap + m * kTileRows;
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
        if (!loading) {
            // a tile of another class may still use its block maxima, and its
            // loads past the end may still write
            phase_end<0>();
            ld.prologue();
        }
        t0 += gridDim.x;
        const int64_t next = tile_at(t0);
        slot ^= 1;
        if (next >= 0)
            look_up(next, s_tile[slot]);  // read after the steps' barriers
        f32x4 acc[row_subs(TS)][col_subs(TS)];
        multiply<TS, kSwiglu>(ld, acc);
        const Tile done = t;
        t.rows = 0;
        loading = false;
        if (next >= 0) {
            t = read_tile(s_tile[slot]);
            if (tile_class<kSwiglu>(t.rows) == TS) {
                // the next tile's loads run under this one's stores (in the
                // swiglu form finish() waits for them: it reloads what it
                // needs from scratch memory, and waits are in order)
                const Loads<TS, kSwiglu> then(a, t, lds, lds0);
                then.prologue();
                loading = true;
            }
        }
        // the block maxima go where the second block of scales was: the next
        // tile asks for that one after its first phases
        static_assert(scale_bytes(TS) >= (tile_rows(TS) + 2) * 16 &&
                          scale_bytes(TS) >= (int)sizeof(float) * col_waves(TS) * tile_rows(TS),
                      "scales, block maxima");
        finish<TS, DT, kSwiglu>(
            a, done,
            reinterpret_cast<float(*)[tile_rows(TS)]>(lds + scale_at(TS) + scale_bytes(TS)), acc);
    };
    while (t.rows > 0) {
        switch (tile_class<kSwiglu>(t.rows)) {
        case 7: run(std::integral_constant<int, 7>()); break;
        case 4: run(std::integral_constant<int, 4>()); break;
        case 1:
            if constexpr (kSwiglu) {
                run(std::integral_constant<int, 1>());
                break;
            }
            [[fallthrough]];  // the other form has no such tile
        default: run(std::integral_constant<int, 2>()); break;
        }
    }
    phase_end<0>();  // no load may write LDS after the block's end
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
