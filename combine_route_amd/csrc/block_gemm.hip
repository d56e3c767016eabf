// gfx950 (MI355X, CDNA4) kernel of moe_grouped_gemm_int8
// (include/moe_block.h): each expert's product of its expert-major INT8 rows
// with its INT8 weights, summed exactly in 32-bit integers and scaled once an
// element, to bf16 / fp16 rows or, with gate and up weights, to rows of
// silu(gate) * up.
//
// A work item is a tile of up to 256 rows of one expert by 256 weight rows.
// Row counts are on the GPU, so the launch is a fixed grid of one block a
// compute unit; each block works out every expert's tile range from the
// counts and walks its share of the tiles. An expert's last tile computes as
// few of 64, 128, 192 or 256 rows as hold its rows, so that experts with few
// rows cost their weights' bytes and little else.
//
// Inside a tile: 4 waves, one a SIMD, 2 along the rows x 2 along the weight
// rows, each with up to 128 x 128 sums in registers: the fewest reads of LDS a
// product (a wave of 128 x 64 would read 1.5 times as much, which with the
// loads' writes is all that LDS can do while the matrix units are busy). For
// each 128 elements of k (a step) the block holds both operands' slices in LDS,
// loaded there directly from memory a step or two before; a wave reads half a
// step's operands to registers while it multiplies the half before. One
// barrier a step. A load takes whole cache lines: with 64 elements a step, half
// a line a request, 256 experts x 32 rows (k 2048, n 7168) took 1130 us
// instead of 750.
//
// LDS slices are 128 bytes a row without padding; the 16-byte chunks of a
// row are permuted by a key of the row, so that the rows a matrix operand reads
// together fall in different banks. The matrix instruction,
// v_mfma_i32_32x32x32_i8, has the weights as its rows and the token rows as
// its columns; which weight row is which of its rows is chosen so that a lane
// ends up with runs of 8 consecutive columns of one token row.
//
// Measured on MI355X (a large INT8 library product 2.4 POP/s, FP8 2.8; weights
// streamed to LDS alone 7.0 TB/s): 32 experts, 32768 rows, n 7168, k 2048 500 to 600
// us (1.6 to 1.9 POP/s), gate and up, n 4096, k 7168 870 to 960 us (2.0 to 2.2); 256
// experts x 32 rows, n 7168, k 2048 717 us (5.4 TB/s), gate and up of 32 experts x
// 32 rows 144 us (6.5 TB/s). Large tiles: matrix units busy 45 to 63% of the cycles,
// at 1.8 GHz under this load. Without its loads gate and up takes 780 us, without
// its stores 910, without its reads of LDS as long as with them: what bounds it is
// the loads, whose requests fill the load path for half of each step, and the
// step's barrier. 256 x 32 rows without the stores: 580 us; 117 MB of scattered rows
// in a stream of reads cost the rest, whatever their cache policy (through the L2,
// streamed) and whether a store writes 32 bytes a row or whole lines (turned round
// in LDS first). Fewer tiles than compute units leave the rest idle: 8 experts x 256
// rows, n 2048, k 7168 68 us (0.9 POP/s), 27 x 4 rows, n 256, k 4608 27 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_lds.h"

namespace block {
namespace {

using namespace block::dev;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTileN = 256;   // weight rows a tile
constexpr int kSubs = 4;      // operands of 32 weight rows a wave
constexpr int kMaxTS = 4;     // a tile of class TS has 64 TS rows
constexpr int kTileRows = 64 * kMaxTS;

constexpr int kStep = 128;    // bytes of k a step: whole cache lines of a row
constexpr int kChunks = kStep / 16;
constexpr int a_bytes(int ts) { return 64 * ts * kStep; }
constexpr int stage_bytes(int ts) { return a_bytes(ts) + kTileN * kStep; }
// Slices held: as many as fit.
constexpr int stages(int ts) { return ts <= 2 ? 3 : 2; }
constexpr int kHeldGroups = 1024;  // whose row counts are kept in LDS
constexpr int kScaleBytes = (kTileRows + kTileN) * 4;
constexpr int kScales = 144 * 1024;  // their place
static_assert(stages(4) * stage_bytes(4) <= kScales && stages(3) * stage_bytes(3) <= kScales &&
                  stages(2) * stage_bytes(2) <= kScales && stages(1) * stage_bytes(1) <= kScales,
              "LDS of a block");
constexpr int kLdsBytes = kScales + 2 * kScaleBytes;

// One tile: the group's first row, how many rows, and the column tile.
struct Tile {
    int64_t row0;   // first row (of [groups * cap])
    int group;
    int rows;       // rows of the tile that exist, 1 .. kTileRows; 0: no tile
    int col;        // column tile
};

// Place of a row's 16-byte chunk in its slice: exclusive-or with this. The 16
// rows that an operand reads together (lanes 0-3, 12-15, 20-27 of 32, and the
// others) lie in different banks so, of 64 (measured: no conflicts).
__device__ __forceinline__ int key(int row) { return (row >> 1) & (kChunks - 1); }

// The loads of a tile. A wave's i-th 1 KB of a slice holds rows 8 * (4 * i +
// wave) .. of 8, a lane one 16-byte chunk of a row. Chunks past k are asked
// for too, from beyond the resource's end (zeros, without memory traffic), so
// that every step has the same loads in flight and no branch.
// kSwiglu: weight rows [0, 128) of the tile are gate rows 128 * col .., rows
// [128, 256) the up rows. Otherwise they are rows 256 * col .. .
template <int TS, bool kSwiglu>
struct Loads {
    static constexpr int kALoads = 2 * TS;
    static constexpr int kBLoads = 8;
    static constexpr int kAll = kALoads + kBLoads;  // a wave and step
    u32x4 ra, rb0, rb1;                        // rows, the two halves of the weights
    u32x4 ras, rbs;                            // the rows' scales, this wave's weight rows'
    uint32_t off;                              // of this lane's chunk of the load's first rows
    int left;                                  // bytes of k from this lane's chunk on
    uint32_t rows32;                           // bytes of 32 rows of k
    uint32_t lds0;
    int wave;

    __device__ __forceinline__ Loads(const GemmArgs& a, const Tile& t, uint32_t block_lds0)
        : lds0(block_lds0)
    {
        const int lane = threadIdx.x & (kWave - 1);
        wave = uniform(threadIdx.x / kWave);
        const uint32_t K = (uint32_t)a.k;
        const int lr = wave * 8 + lane / kChunks;  // row of i = 0; i adds 32
        rows32 = 32 * K;
        const int chunk = (lane & (kChunks - 1)) ^ key(lr);
        off = (uint32_t)lr * K + (uint32_t)chunk * 16u;
        left = a.k - chunk * 16;
        ra = rsrc_words(a.a + t.row0 * K, t.rows * (int)K);
        const int64_t first = (int64_t)t.group * a.n;
        const int half = kSwiglu ? a.n / 2 : a.n;   // rows of one projection
        const int r0 = t.col * (kSwiglu ? 128 : kTileN);
        const int r1 = kSwiglu ? half + r0 : min(r0 + 128, a.n - 1);
        const int n0 = min(128, half - r0);
        const int n1 = kSwiglu ? n0 : max(0, min(128, a.n - r0 - 128));
        rb0 = rsrc_words(a.b + (first + r0) * K, n0 * (int)K);
        rb1 = rsrc_words(a.b + (first + r1) * K, n1 * (int)K);
        ras = rsrc_words(a.as + t.row0, t.rows * 4);
        rbs = wave < 2 ? rsrc_words(a.bs + first + r0, n0 * 4)
                       : rsrc_words(a.bs + first + r1, n1 * 4);
    }

    // Load i of step h's, to its stage: the rows', then the weights'.
    __device__ __forceinline__ void load(int i, int h, int stage) const
    {
        const uint32_t at = off + (h * kStep < left ? 0u : 1u << 30);
        const uint32_t dst = lds0 + stage * stage_bytes(TS) + i * 4096 + wave * 1024;
        constexpr int kHalf = kBLoads / 2;
        if (i < kALoads)
            load_to_lds<false>(ra, dst, at + i * rows32, (uint32_t)h * kStep);
        else if (i < kALoads + kHalf)
            load_to_lds<(TS < kMaxTS)>(rb0, dst, at + (i - kALoads) * rows32, (uint32_t)h * kStep);
        else
            load_to_lds<(TS < kMaxTS)>(rb1, dst, at + (i - kALoads - kHalf) * rows32,
                                       (uint32_t)h * kStep);
    }

    // The scales (to block `which` of them) and the first slices.
    __device__ __forceinline__ void prologue(int which) const
    {
        const uint32_t lane4 = (threadIdx.x & (kWave - 1)) * 4u;
        const uint32_t at = lds0 + kScales + which * kScaleBytes + wave * 256;
        load4_to_lds(ras, at, wave * 256 + lane4);
        load4_to_lds(rbs, at + kTileRows * 4, (wave & 1) * 256 + lane4);
#pragma unroll
        for (int h = 0; h < stages(TS); ++h)
#pragma unroll
            for (int i = 0; i < kAll; ++i)
                load(i, h, h);
    }
};

// A tile's stores: of each 8 columns of a lane's rows. The first kNow are made
// at the tile's end, the others, kEach at a time, in the first kDelay steps of
// the next tile: a wave's waits are in order, so that one for a load waits for
// the stores before it too, and a whole tile's at once take long.
template <int TS, bool kSwiglu>
struct Stores {
    static constexpr int kCols = kSwiglu ? kSubs / 2 : kSubs;  // operands of columns
    static constexpr int kAll = 2 * kCols * TS;
    static constexpr int kDelay = 4;
    static constexpr int kHeld = kAll < 16 ? kAll : 16;        // (64 registers)
    static constexpr int kEach = kHeld / kDelay;
    static constexpr int kNow = kAll - kHeld;
    static_assert(kHeld % kDelay == 0, "whole steps");

    u32x4 held[kHeld];
    u32x4 words;      // of the resource over the tile's rows
    uint32_t off;     // of this lane's first column in its first row
    int left;         // columns from there to the row's end
    uint32_t rows32;  // bytes of 32 rows

    __device__ __forceinline__ Stores() : words{}, off(0), left(0), rows32(0)
    {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = u32x4{};
    }

    // Store i is of columns 16 (i / TS) and rows 32 (i % TS) from the first on.
    __device__ __forceinline__ void store(int i, const u32x4& v) const
    {
        const int col = i / TS * 16;
        const uint32_t lo = words[0], hi = words[1], at = off + i % TS * rows32 + col * 2;
        // rows past the tile's (and all without a tile) are dropped by the resource
        bstore16<0>(v, row_rsrc(reinterpret_cast<const void*>(lo | (uint64_t)hi << 32), words[2]),
                    col < left ? at : 1u << 31);
    }

    __device__ __forceinline__ void later(int i) const { store(kNow + i, held[i]); }

    __device__ __forceinline__ void rest(int from) const
    {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i >= from)
                later(i);
    }
};

// A wave's operands of half a step: 32 bytes of k, twice.
template <int TS>
struct Operands {
    i32x4 w[kSubs][2], t[TS][2];
};

// The sums of one tile, whose first slices are on their way. A step's first
// half multiplies while the second half's operands are read; then a barrier
// says that every wave has them, so that the step's place is free for the
// slice `stages` further, and that the next step's slice is there, from which
// the second half reads. fresh: no immediate stores came after the first
// slices' loads, so that none may be allowed for in the waits.
template <int TS, bool kSwiglu>
__device__ __forceinline__ void multiply(const Loads<TS, kSwiglu>& ld, const uint8_t* lds, int nk,
                                         const Stores<TS, kSwiglu>& stores, bool fresh,
                                         i32x16 (&acc)[TS][kSubs])
{
    using L = Loads<TS, kSwiglu>;
    using St = Stores<TS, kSwiglu>;
    constexpr int S = stages(TS);
    const int lane = threadIdx.x & (kWave - 1);
    const int wm = ld.wave >> 1, wn = ld.wave & 1;
    const int q = lane >> 5, i32 = lane & 31;
    // the weight row that is row i32 of an operand: runs of 8 for a lane of
    // the result, which holds rows 8 b + 4 q + t, b and t 0 .. 3
    const int b = i32 >> 3, j = (b >> 1) * 16 + ((i32 >> 2) & 1) * 8 + (b & 1) * 4 + (i32 & 3);
    const int wrow = wn * (kSwiglu ? 64 : 128) + j;
    const uint32_t wat = a_bytes(TS) + (uint32_t)wrow * kStep + (uint32_t)((q ^ key(wrow)) * 16);
    const int trow = wm * 32 * TS + i32;
    const uint32_t tat = (uint32_t)trow * kStep + (uint32_t)((q ^ key(trow)) * 16);
    auto sub = [](int s) {
        return (uint32_t)(kSwiglu ? (s >> 1) * 128 + (s & 1) * 32 : s * 32) * kStep;
    };

    Operands<TS> op[2];
    constexpr int kFetches = 2 * (kSubs + TS);
    constexpr int kProducts = 2 * kSubs * TS;
    // operand i of a half of the step in `stage`, weights, then rows
    auto fetch = [&](int half, int i, int stage) {
        const uint8_t* base = lds + stage * stage_bytes(TS);
        const int part = i / (kSubs + TS), k = i % (kSubs + TS), c = half * 64 + part * 32;
        if (k < kSubs)
            op[half].w[k][part] = *reinterpret_cast<const i32x4*>(base + (wat ^ c) + sub(k));
        else
            op[half].t[k - kSubs][part] = *reinterpret_cast<const i32x4*>(
                base + (tat ^ c) + (k - kSubs) * 32 * kStep);
    };
    // the products of a half, with `more(p)` after each
    auto products = [&](int half, auto more) {
#pragma unroll
        for (int p = 0; p < kProducts; ++p) {
            const int part = p / (kSubs * TS), m = p / kSubs % TS, s = p % kSubs;
            acc[m][s] = __builtin_amdgcn_mfma_i32_32x32x32_i8(op[half].w[s][part],
                                                              op[half].t[m][part], acc[m][s], 0, 0,
                                                              0);
            more(p);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // this product's share of the other half's operands: all of them in the
    // first half of the products
    auto fetches = [&](int p, int half, int stage) {
#pragma unroll
        for (int i = 2 * p * kFetches / kProducts;
             i < 2 * (p + 1) * kFetches / kProducts && i < kFetches; ++i)
            fetch(half, i, stage);
    };

    if (fresh)
        phase_end<(S - 1) * L::kAll>();
    else
        phase_end<(S - 1) * L::kAll + St::kNow>();
#pragma unroll
    for (int i = 0; i < kFetches; ++i)
        fetch(0, i, 0);
#pragma unroll
    for (int m = 0; m < TS; ++m)
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
            acc[m][s] = i32x16{};

    int stage = 0;
    // Step h. D: h up to kDelay, whose stores come with it. In flight at its
    // barrier at most what was asked for after the loads of step h + 1: those
    // of the steps after it, and stores: these are one or two steps' (S - 1),
    // and the last tile's immediate ones as long as the loads are older.
    auto step = [&](int h, auto d) {
        constexpr int D = decltype(d)::value;
        constexpr int kEach = D < St::kDelay ? St::kEach : 0;
        constexpr int kBefore = S > 2 && D > 0 && D <= St::kDelay ? St::kEach : 0;
        constexpr int kFirst = D < S - 1 ? St::kNow : 0;
        const int next = stage + 1 == S ? 0 : stage + 1;
        products(0, [&](int p) {
            fetches(p, 1, stage);
#pragma unroll
            for (int i = p * kEach / kProducts; i < (p + 1) * kEach / kProducts; ++i)
                stores.later(D * St::kEach + i);
        });
        if (kFirst > 0 && fresh)
            phase_end<(S - 2) * L::kAll + kEach + kBefore>();
        else
            phase_end<(S - 2) * L::kAll + kEach + kBefore + kFirst>();
        products(1, [&](int p) {
            fetches(p, 0, next);
#pragma unroll
            for (int i = p * L::kAll / kProducts; i < (p + 1) * L::kAll / kProducts; ++i)
                ld.load(i, h + S, stage);
        });
        stage = next;
    };
    static_assert(St::kDelay == 4, "the steps below");
    step(0, std::integral_constant<int, 0>());
    if (nk > 1)
        step(1, std::integral_constant<int, 1>());
    if (nk > 2)
        step(2, std::integral_constant<int, 2>());
    if (nk > 3)
        step(3, std::integral_constant<int, 3>());
    else  // (from a constant, so that the held ones stay in registers)
        nk == 3 ? stores.rest(3 * St::kEach) : nk == 2 ? stores.rest(2 * St::kEach)
                                                       : stores.rest(St::kEach);
    if (nk > 4)
        step(4, std::integral_constant<int, 4>());
    for (int h = 5; h < nk; ++h)
        step(h, std::integral_constant<int, 5>());
    phase_end();
    // the last products' results, before sum() reads them: a read may not
    // follow a product of 16 passes within 18 issue slots
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A sum, out of the accumulation registers. In assembly because the compiler
// would move all 256 to the other registers at once, and those of the next
// tile's addresses to memory.
__device__ __forceinline__ int sum(int a)
{
#ifdef __HIP_DEVICE_COMPILE__
    int v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
#else
    return a;
#endif
}

// The tile's sums to memory, or to `stores` for later.
template <int TS, int DT, bool kSwiglu>
__device__ __forceinline__ void finish(const GemmArgs& a, const Tile& t, const uint8_t* scales,
                                       i32x16 (&acc)[TS][kSubs], Stores<TS, kSwiglu>& stores)
{
    using St = Stores<TS, kSwiglu>;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave >> 1, wn = wave & 1, q = lane >> 5;
    const float* as = reinterpret_cast<const float*>(scales);
    const float* bs = as + kTileRows;
    const int width = kSwiglu ? a.n / 2 : a.n;
    const int trow = wm * 32 * TS + (lane & 31);
    const int wcol = wn * St::kCols * 32 + q * 8;       // in the tile
    const int col = t.col * (kSwiglu ? 128 : kTileN) + wcol;
    stores.words = rsrc_words(a.out + t.row0 * width * 2, t.rows * width * 2);
    stores.off = ((uint32_t)trow * (uint32_t)width + (uint32_t)col) * 2u;
    stores.left = width - col;
    stores.rows32 = 64u * (uint32_t)width;
#pragma unroll
    for (int s = 0; s < 2 * St::kCols; ++s) {  // runs of 8 columns, 16 apart
        float cs[8], us[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            cs[r] = bs[wcol + s * 16 + r];
            us[r] = kSwiglu ? bs[128 + wcol + s * 16 + r] : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < TS; ++m) {
            const float sa = as[trow + m * 32];
            float f[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                f[r] = sa * (cs[r] * (float)sum(acc[m][s / 2][s % 2 * 8 + r]));
                if constexpr (kSwiglu)
                    f[r] = silu_times(
                        f[r], sa * (us[r] * (float)sum(acc[m][s / 2 + St::kCols][s % 2 * 8 + r])));
            }
            const int i = s * TS + m;
            if (i < St::kNow)
                stores.store(i, narrow<DT>(f));
            else
                stores.held[i - St::kNow] = narrow<DT>(f);
        }
    }
}

__device__ __forceinline__ int tile_class(int rows) { return (rows + 63) / 64; }

template <int DT, bool kSwiglu>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void
block_gemm_kernel(GemmArgs a)
{
    __shared__ __align__(1024) uint8_t lds[kLdsBytes];
    __shared__ int s_part[kThreads / kWave];
    __shared__ int s_first[kThreads + 1];
    __shared__ int s_tile[2][4];
    __shared__ int s_rows[kHeldGroups];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);

    // Row tiles of each thread's share of the groups, as where they start in
    // the list of all (group after group). Row counts of the first groups are
    // kept in LDS: a look at memory between tiles would wait for every load and
    // store before it.
    auto count_of = [&](int g) {
        return a.counts ? max(0, min(a.counts[g], a.cap)) : a.cap;
    };
    auto rows_of = [&](int g) { return g < kHeldGroups ? s_rows[g] : count_of(g); };
    for (int g = threadIdx.x; g < min(a.groups, kHeldGroups); g += kThreads)
        s_rows[g] = count_of(g);
    __syncthreads();
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
    const int64_t tile = tile_at(t0);
    if (tile < 0)
        return;  // the whole block
    look_up(tile, s_tile[0]);
    __syncthreads();
    Tile t = read_tile(s_tile[0]);
    const int nk = (a.k + kStep - 1) / kStep;  // steps
    int slot = 0;  // of the tile and its scales
    // Tiles of class TS, as long as the next one is of it; then t is the next
    // one (or has no rows).
    auto run = [&](auto ts) {
        constexpr int TS = decltype(ts)::value;
        Stores<TS, kSwiglu> stores;
        // loads past the end of a tile of another class may still write
        phase_end<0>();
        Loads<TS, kSwiglu>(a, t, lds0).prologue(slot);
        bool more = true, fresh = true;
        while (more) {
            t0 += gridDim.x;
            const int64_t next = tile_at(t0);
            if (next >= 0)
                look_up(next, s_tile[slot ^ 1]);  // read after the steps' barriers
            i32x16 acc[TS][kSubs];
            multiply<TS, kSwiglu>(Loads<TS, kSwiglu>(a, t, lds0), lds, nk, stores, fresh,
                                  acc);
            fresh = false;
            const Tile done = t;
            const uint8_t* scales = lds + kScales + slot * kScaleBytes;
            slot ^= 1;
            t.rows = 0;
            if (next >= 0)
                t = read_tile(s_tile[slot]);
            more = t.rows > 0 && tile_class(t.rows) == TS;
            if (more)  // the next tile's first loads
                Loads<TS, kSwiglu>(a, t, lds0).prologue(slot);
            finish<TS, DT, kSwiglu>(a, done, scales, acc, stores);
        }
        stores.rest(0);
    };
    while (t.rows > 0) {
        switch (tile_class(t.rows)) {
        case 4: run(std::integral_constant<int, 4>()); break;
        case 3: run(std::integral_constant<int, 3>()); break;
        case 2: run(std::integral_constant<int, 2>()); break;
        default: run(std::integral_constant<int, 1>()); break;
        }
    }
    phase_end<0>();  // no load may write LDS after the block's end
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& a, int dtype, bool swiglu, int blocks, hipStream_t s)
{
    const dim3 grid(blocks), block(kThreads);
    if (swiglu) {
        if (dtype == 0)
            hipLaunchKernelGGL((block_gemm_kernel<0, true>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((block_gemm_kernel<1, true>), grid, block, 0, s, a);
    } else if (dtype == 0) {
        hipLaunchKernelGGL((block_gemm_kernel<0, false>), grid, block, 0, s, a);
    } else {
        hipLaunchKernelGGL((block_gemm_kernel<1, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace block
