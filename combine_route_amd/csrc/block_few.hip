// gfx950 (MI355X, CDNA4) kernels of moe_few_tokens (include/moe_block.h): a
// whole layer's experts for a few tokens.
//
// Such a call is its weights' bytes: 3 * inter * hidden for each expert hit,
// against which tokens, hidden rows and arithmetic are nothing. So nothing is
// gathered or packed, every weight byte is loaded once for each 16 tokens of
// its expert, and the two kernels only see to it that enough loads are in
// flight: each wave has a ring in LDS that its own loads fill ahead of it, 8
// rows' whole cache lines a load, with no barrier, as nobody else reads it.
//
// The first kernel takes gate and up: a block has one expert and 16 or 32
// hidden columns, its 4 waves a quarter of k each; the quarters are added in order
// through LDS, and silu(gate) * up goes to the workspace as a bf16 value and
// the bf16 value of its rest. The second takes down: a block has 16 or 32
// output columns for every expert hit, its 8 waves share the experts (and pieces
// of k), each (token, expert) pair's sums go to LDS, and at the end each token's
// are added in slot order with their weights. No sum's order depends on which
// other tokens are there.
//
// Weights are the matrix instruction's rows, tokens its columns (16 at a time;
// absent ones are zeros that no load touches memory for). 16 bytes of weights
// of a lane are widened to two operands of 8 values of the tokens' type, which
// is exact for E4M3 and int8 alike, so that x needs no rounding; both sides take
// k in the same permuted order. An expert with few columns has them loaded
// packed, so that a load brings more of them than zeros. FP8 weights: the sum
// of each 128 elements of k is scaled as it joins the FP32 sum.
//
// Measured on MI355X (weights streamed to LDS alone: 7.0 TB/s): experts of 2048 x
// 7168 FP8, top-8, one token 38 us for gate and up (6.2 TB/s) and 24 for down (4.8
// TB/s); 64 tokens over 256 experts 950 (6.9 TB/s) and 618 us (5.3 TB/s: one block a
// CU by its LDS, 448 blocks for 256 CUs). 4 tokens, top-4, 1024 x 4096 INT8: 24 and
// 16.5 us, of which starting, routing and the last sums are the larger part. With
// weights loaded to registers as the operands lie, 64 bytes of 16 rows a load, one
// token took 52 and 36 us. What the rules above cost: experts of more than 4 columns
// have one step in flight and are read again for every 16 (8 experts of 14336 x 4096
// FP8, top-2, 8, 16 and 64 tokens 196, 243 and 533 us: 6.3, 5.8 and 2.6 TB/s);
// pieces of inter of less than three steps let the ring run empty between experts (46
// tokens, top-2 of 63, 384 x 2944: 92 us, 1.8 TB/s); a small hidden size leaves the
// down product few blocks (22 tokens, top-3 of 29, 640 x 128: 55 us).
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "block_lds.h"

namespace block {
namespace {

using namespace block::dev;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kItemSteps = kWave;             // of an item whose scales lie in LDS
constexpr int kItemScales = 2 * kItemSteps * 4;  // bytes a wave: of two items
constexpr int kMaxWords = kFewMaxExperts / 32;
constexpr int kBlockK = 128;  // elements of k a step
constexpr uint32_t kNowhere = 1u << 31;
constexpr float kBf16Max = 0x1.FEp127f;
constexpr size_t kFewLds = 160 * 1024;  // of a compute unit

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

// What a call's routing comes to: the expert of each slot that is its token's
// first to name it (else -1), and the experts hit, each once, in any order.
//
// Of up to 64 slots a wave knows it by itself, one slot a lane, without a
// barrier: a loop over the experts hit.
struct WaveRouting {
    int id;           // of this lane's slot, if it is its token's first of its expert
    uint64_t firsts;  // lanes that are the call's first of their expert
    int hits;

    __device__ __forceinline__ explicit WaveRouting(const FewArgs& a)
    {
        const int lane = threadIdx.x & (kWave - 1), P = a.T * a.topk;
        const int raw = lane < P ? a.ids[lane] : -1;
        const bool valid = raw >= 0 && raw < a.E;
        const uint64_t below = (1ull << lane) - 1;                // lanes below this one
        const uint64_t others = (1ull << (lane - lane % a.topk)) - 1;  // of tokens before
        uint64_t left = __ballot(valid);
        id = -1;
        firsts = 0;
        hits = 0;
        while (left) {
            const int first = (int)__builtin_ctzll(left);
            const int e = __builtin_amdgcn_readlane(raw, first);
            const uint64_t m = __ballot(valid && raw == e);
            if (raw == e && valid && !(m & below & ~others))
                id = e;
            firsts |= 1ull << first;
            left &= ~m;
            ++hits;
        }
    }

    // The u-th expert: its first lane in the call is its token's first too.
    __device__ __forceinline__ int expert(int u) const
    {
        const int lane = threadIdx.x & (kWave - 1);
        const bool yes = (firsts >> lane & 1) && lanes_below(firsts) == u;
        return __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(__ballot(yes)));
    }

    // The slots of expert e that are their token's first of it, in order, to
    // list; how many.
    __device__ __forceinline__ int slots_of(const FewArgs&, int e, int* list) const
    {
        const uint64_t b = __ballot(id == e);
        if (id == e)
            list[lanes_below(b)] = threadIdx.x & (kWave - 1);
        return (int)__popcll(b);
    }
};

// Of more, a block works it out in LDS.
struct Routing {
    int id[kFewMaxSlots];
    int hit[kFewMaxSlots];
    int part[16];
    int hits;
};

// Fills s in a block of N threads; bits: kMaxWords words of LDS, for the while.
// Ends with a barrier.
template <int N>
__device__ __forceinline__ void read_routing(const FewArgs& a, Routing& s, uint32_t* bits)
{
    const int tid = threadIdx.x, P = a.T * a.topk;
    const int words = (a.E + 31) / 32;
    for (int p = tid; p < P; p += N)
        s.hit[p] = a.ids[p];  // (as they come; the list of hits is made later)
    for (int i = tid; i < words; i += N)
        bits[i] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += N) {
        const int e = s.hit[p], first = p - p % a.topk;
        bool lead = e >= 0 && e < a.E;
        for (int j = first; j < p; ++j)
            lead = lead && s.hit[j] != e;
        s.id[p] = lead ? e : -1;
        if (lead)
            atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    const int share = (words + N - 1) / N;
    const int w0 = min(words, tid * share), w1 = min(words, w0 + share);
    int mine = 0;
    for (int i = w0; i < w1; ++i)
        mine += __popc(bits[i]);
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
        for (uint32_t b = bits[i]; b; b &= b - 1)
            s.hit[at++] = i * 32 + __ffs(b) - 1;
    if (tid == 0)
        s.hits = total;
    __syncthreads();
}

struct BlockRouting {
    Routing& s;
    int hits;

    __device__ __forceinline__ int expert(int u) const { return uniform(s.hit[u]); }

    __device__ __forceinline__ int slots_of(const FewArgs& a, int e, int* list) const
    {
        const int lane = threadIdx.x & (kWave - 1), P = a.T * a.topk;
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
};

// Calls f with the routing, known to every wave: of up to 64 slots (kSmall)
// without a barrier. routing, bits: LDS for it, the latter (kMaxWords words)
// only until f is called.
template <bool kSmall, int N, class F>
__device__ __forceinline__ void with_routing(const FewArgs& a, void* routing, void* bits, F&& f)
{
    if constexpr (kSmall) {
        f(WaveRouting(a));
    } else {
        Routing& s = *static_cast<Routing*>(routing);
        read_routing<N>(a, s, static_cast<uint32_t*>(bits));
        f(BlockRouting{s, uniform(s.hits)});
    }
}

// Each lane's value of the lane N further in its row of 16.
template <int N>
__device__ __forceinline__ u32x4 rotated(const u32x4& v)
{
    constexpr int kRowRotateRight = 0x120;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int w = (int)v[i];
        r[i] = (uint32_t)__builtin_amdgcn_update_dpp(w, w, kRowRotateRight + 16 - N, 0xF, 0xF, true);
    }
    return r;
}

// One wave's sums over steps [k0, k1) of R operands of 16 weight rows with up
// to C columns, 4 or 16. The wave's own ring in LDS holds D steps' weights and
// columns, loaded straight there, so that as much is in flight as there is LDS,
// whatever the registers, and a load takes whole cache lines: 8 rows of 128
// bytes (64 bytes of 16 rows, which is how the operands lie in registers, took
// a fifth longer). Its chunks are permuted by the row, as the reads' banks want.
// Up to 4 columns lie packed: lane 4 c + i of each 16 has what column i
// multiplies with the step's operand c, one load a step instead of four, and a
// rotation of the 16 lanes by 4 c puts it in place (columns 4 and up hold what
// nobody reads).
template <int R, int C, int X, int WT, int XT, int D>
struct Sums {
    static constexpr bool kPacked = C <= 4;
    static constexpr int kColumns = kPacked ? 4 : 16;  // in turn over the lanes
    static constexpr int kXLoads = kPacked ? 1 : 4;    // a step and plane of columns
    static constexpr int kAll = 2 * R + X * kXLoads;
    static constexpr int kBytes = kAll * 1024;       // a step's

    u32x4 rw[R], rx[X];  // resources: 16 rows of K bytes each; the planes of the columns
    uint32_t lds0;       // of the ring
    const uint8_t* lds;
    uint32_t woff[2];    // this lane's chunk of the first step, in either 8 rows
    uint32_t xoff;
    int wleft[2], xleft; // elements of k from there on
    int k1;

    // column: byte offset of this lane's column (kColumns of them, in turn), or
    // kNowhere.
    __device__ __forceinline__ Sums(const uint8_t* const (&rows)[R], const int (&bytes)[R],
                                    const uint8_t* columns, uint32_t plane, uint32_t column, int K,
                                    int end, uint8_t* ring, uint32_t ring0)
        : lds0(ring0), lds(ring), k1(end)
    {
        const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
        for (int r = 0; r < R; ++r)
            rw[r] = rsrc_words(rows[r], bytes[r]);
#pragma unroll
        for (int v = 0; v < X; ++v)
            rx[v] = rsrc_words(columns + (int64_t)v * plane, (int)plane);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = half * 8 + (lane >> 3), chunk = (lane & 7) ^ key(row);
            woff[half] = (uint32_t)row * (uint32_t)K + (uint32_t)chunk * 16u;
            wleft[half] = K - chunk * 16;
        }
        const int c = kPacked ? (lane & 15) >> 2 : 0;
        const int at = c / 2 * 64 + (lane >> 4) * 16 + c % 2 * 8;
        xoff = column == kNowhere ? kNowhere : column + (uint32_t)at * 2u;
        xleft = K - at;
    }

    // Place of a row's chunk: exclusive-or with this (rows 0 to 15).
    static __device__ __forceinline__ int key(int row) { return (row >> 1) & 7; }

    // Step k's loads.
    __device__ __forceinline__ void load(int k, int slot) const
    {
        const uint32_t dst = lds0 + slot * kBytes;
        const int at = k * kBlockK;
        const bool mine = k < k1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t to = mine && at < wleft[half] ? woff[half] : kNowhere;
#pragma unroll
            for (int r = 0; r < R; ++r)
                load_to_lds<true>(rw[r], dst + (2 * r + half) * 1024, to, (uint32_t)at);
        }
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int more = i / 2 * 64 + i % 2 * 8;  // elements (packed: 0)
            const uint32_t to = mine && at + more < xleft ? xoff + more * 2u : kNowhere;
#pragma unroll
            for (int v = 0; v < X; ++v)
                load_to_lds<false>(rx[v], dst + (2 * R + v * kXLoads + i) * 1024, to,
                                   (uint32_t)at * 2u);
        }
    }

    // The sums of the step that lies at `from` in the ring, once its loads have
    // come; refill: loads into the place when it has been read. scale(r):
    // operand r's scale, of FP8 weights.
    template <class Scale, class Refill>
    static __device__ __forceinline__ void step(const uint8_t* from, Scale&& scale,
                                                Refill&& refill, f32x4 (&acc)[R])
    {
        const int lane = threadIdx.x & (kWave - 1);
        const int q = lane >> 4, i16 = lane & 15;
        const uint32_t wat = (uint32_t)i16 * 128u + (uint32_t)((q ^ key(i16)) * 16);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * kAll) : "memory");
        // taken here, so that no branch comes between the products and their
        // scaling: behind one, the compiler left out the wait states that a
        // matrix instruction's result needs (element 3 of each was wrong)
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            f[r] = WT == 0 ? scale(r) : 1.0f;
        u32x4 w[R][2], x[X][kXLoads];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int half = 0; half < 2; ++half)  // of the step: chunks q, q + 4
                w[r][half] = *reinterpret_cast<const u32x4*>(from + r * 2048 + (wat ^ half * 64));
#pragma unroll
        for (int v = 0; v < X; ++v)
#pragma unroll
            for (int i = 0; i < kXLoads; ++i)
                x[v][i] = *reinterpret_cast<const u32x4*>(
                    from + (2 * R + v * kXLoads + i) * 1024 + lane * 16);
        // read before the place is loaded again
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        refill();
        __builtin_amdgcn_sched_barrier(0);

        f32x4 sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            sum[r] = WT == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[r];
        u32x4 y[X][4];
#pragma unroll
        for (int v = 0; v < X; ++v) {
            if constexpr (kPacked) {
                y[v][0] = x[v][0];
                y[v][1] = rotated<4>(x[v][0]);
                y[v][2] = rotated<8>(x[v][0]);
                y[v][3] = rotated<12>(x[v][0]);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    y[v][c] = x[v][c % kXLoads];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const u32x4 o = widened8<WT, XT>(w[r][c >> 1][(c & 1) * 2],
                                                 w[r][c >> 1][(c & 1) * 2 + 1]);
#pragma unroll
                for (int v = 0; v < X; ++v)
                    sum[r] = product<XT>(o, y[v][c], sum[r]);
            }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (WT == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[r][i] = __builtin_fmaf(f[r], sum[r][i], acc[r][i]);
            } else {
                acc[r] = sum[r];
            }
        }
    }

    // After the last step: its products' wait states, which a loop's end is a
    // branch before; kDrain: and every load here, as loads past the end may not
    // write what comes next in LDS.
    template <bool kDrain>
    static __device__ __forceinline__ void done()
    {
        __builtin_amdgcn_sched_barrier(0);
        if (kDrain)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_nop 15" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    // Steps [k0, k1). scale(r, k): operand r's scale of step k, of FP8 weights.
    template <class Scale>
    __device__ __forceinline__ void operator()(int k0, Scale&& scale, f32x4 (&acc)[R]) const
    {
#pragma unroll
        for (int d = 0; d < D; ++d)
            load(k0 + d, d);
        int slot = 0;
        for (int k = k0; k < k1; ++k) {
            step(lds + slot * kBytes, [&](int r) { return scale(r, k); },
                 [&] { load(k + D, slot); }, acc);
            slot = slot + 1 == D ? 0 : slot + 1;
        }
        done<true>();
    }
};

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
        asm volatile("" : "+v"(v));  // here already: a wait later is for later loads too
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

// A kind of Sums as a value.
template <class S>
struct Kind {
    using type = S;
    static constexpr int kColumns = S::kColumns;
};

// Gate and up, of 8 R hidden columns a block.
template <int WT, int XT, int R, bool kSmall>
__global__ __launch_bounds__(kUpWaves * kWave) void block_few_up_kernel(FewArgs a)
{
    using Few = Sums<R, 4, 1, WT, XT, 2>;    // steps in flight: as fit kRing
    using More = Sums<R, 16, 1, WT, XT, 1>;
    constexpr int kRing = 2 * Few::kBytes;
    static_assert(More::kBytes <= kRing && sizeof(f32x4) * R * kWave <= kRing, "LDS of a wave");
    constexpr int kCols = 8 * R;
    __shared__ __align__(1024) uint8_t s_ring[kUpWaves][kRing];
    static_assert(sizeof s_ring >= 16384 + kMaxWords * 4 && sizeof(Routing) <= 16384,
                  "the routing lies in the rings, before they are used");
    __shared__ int s_list[kUpWaves][kFewMaxTokens];
    const uint32_t ring0 =
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&s_ring[0][0];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int tiles = a.I / kCols;
    const int u = (int)blockIdx.x / tiles, tile = (int)blockIdx.x % tiles;
    uint8_t* mem = s_ring[0];
    with_routing<kSmall, kUpWaves * kWave>(a, mem, mem + 16384, [&](const auto& routing) {
        if (u >= routing.hits)
            return;  // the whole block
        const int e = routing.expert(u);
        int* list = s_list[wave];  // every wave has its own
        const int n = routing.slots_of(a, e, list);
        if (!kSmall)
            __syncthreads();  // the routing has been read
        // operands: R / 2 of gate rows, then the same of up rows
        const int64_t row = (int64_t)e * 2 * a.I + tile * kCols;
        const uint8_t* rows[R];
        int bytes[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rows[r] = a.up + (row + r % (R / 2) * 16 + (r < R / 2 ? 0 : a.I)) * a.H;
            bytes[r] = a.H * 16;
        }
        const int steps = (a.H + kBlockK - 1) / kBlockK;
        const int k0 = steps * wave / kUpWaves, k1 = steps * (wave + 1) / kUpWaves;
        const int blocks = a.H / kBlockK;  // of a row's scales (FP8)
        const float* first = a.ups + (WT == 0 ? (row / 128) * blocks : 0);
        const float* second = first + (WT == 0 ? (int64_t)(a.I / 128) * blocks : 0);
        f32x4* mine = reinterpret_cast<f32x4*>(s_ring[wave]);  // its sums, when it is done

        for (int c0 = 0; c0 < n; c0 += 16) {
            auto sums = [&](auto kind) {
                using S = decltype(kind);
                const int c = c0 + (lane & (S::kColumns - 1));
                const uint32_t column =
                    c < n ? (uint32_t)(list[c] / a.topk) * (uint32_t)a.H * 2u : kNowhere;
                f32x4 acc[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                StepScales sg(first, k0, WT == 0 ? k1 : k0), su(second, k0, WT == 0 ? k1 : k0);
                typename S::type(rows, bytes, a.x, (uint32_t)a.T * (uint32_t)a.H * 2u, column, a.H,
                                 k1, s_ring[wave], ring0 + wave * kRing)(
                    k0, [&](int r, int k) { return r < R / 2 ? sg.at(k) : su.at(k); }, acc);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    mine[r * kWave + lane] = acc[r];
            };
            if (n <= 4)
                sums(Kind<Few>());
            else
                sums(Kind<More>());
            __syncthreads();
            // a lane has 4 hidden columns of one token; wave r those of gate
            // operand r
            const int c = c0 + (lane & 15);
            if (wave < R / 2 && c < n) {
                f32x4 v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = (wave + h * (R / 2)) * kWave + lane;
                    v[h] = reinterpret_cast<const f32x4*>(s_ring[0])[at];
#pragma unroll
                    for (int w = 1; w < kUpWaves; ++w) {
                        const f32x4 o = reinterpret_cast<const f32x4*>(s_ring[w])[at];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[h][i] = v[h][i] + o[i];
                    }
                }
                const int col = tile * kCols + wave * 16 + (lane >> 4) * 4;
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
                    if (__builtin_isinf(z[i]) && !__builtin_isinf(y)) {
                        // a finite value past the largest of bf16: that and a rest,
                        // held below what would make their sum 2^128
                        z[i] = __builtin_copysignf(kBf16Max, y);
                        rest[i] = __builtin_copysignf(
                            __builtin_fminf(__builtin_fabsf(y - z[i]), kBf16Max * 0x1p-8f), y);
                    }
                }
                const int64_t at = (int64_t)list[c] * a.I + col;
                const int64_t plane = (int64_t)a.T * a.topk * a.I;
                auto pair = [](float lo, float hi) {
                    return (__builtin_bit_cast(uint32_t, round_to<0>(lo)) >> 16) |
                           (__builtin_bit_cast(uint32_t, round_to<0>(hi)) & 0xFFFF0000u);
                };
                *reinterpret_cast<u32x2*>(a.act + at * 2) =
                    u32x2{pair(z[0], z[1]), pair(z[2], z[3])};
                *reinterpret_cast<u32x2*>(a.act + (plane + at) * 2) =
                    u32x2{pair(rest[0], rest[1]), pair(rest[2], rest[3])};
            }
            if (c0 + 16 < n)
                __syncthreads();  // the sums have been read
        }
    });
}

// Down and the sum over experts, of 16 R output columns a block. D: steps of
// up to 4 columns in flight.
template <int WT, int XT, int R, int D, bool kSmall>
__global__ __launch_bounds__(kDownWaves * kWave) void block_few_down_kernel(FewArgs a)
{
    using Few = Sums<R, 4, 2, WT, 0, D>;
    using More = Sums<R, 16, 2, WT, 0, 1>;
    constexpr int kRing = D * Few::kBytes > More::kBytes ? D * Few::kBytes : More::kBytes;
    // rings, scales of two items a wave, [splits][T * topk][16 R] sums
    extern __shared__ __align__(1024) uint8_t s_mem[];
    __shared__ int s_list[kDownWaves][kFewMaxTokens];
    // the routing, or (kSmall) the experts of the slots that are their token's first of it
    __shared__ int s_routing[kSmall ? kWave : (sizeof(Routing) + 3) / 4];
    const int* id = s_routing;
    static_assert(offsetof(Routing, id) == 0, "the experts of the slots come first");
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    uint8_t* ring = s_mem + wave * kRing;
    const uint32_t ring0 =
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring;
    float* s_scale = reinterpret_cast<float*>(s_mem + kDownWaves * kRing + wave * kItemScales);
    const uint32_t scale0 =
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)s_scale;
    float* s_y = reinterpret_cast<float*>(s_mem + kDownWaves * (kRing + kItemScales));
    constexpr int kCols = 16 * R;
    const int h0 = (int)blockIdx.x * kCols;
    const int P = a.T * a.topk;
    with_routing<kSmall, kDownWaves * kWave>(a, s_routing, s_mem, [&](const auto& routing) {
        if constexpr (kSmall) {
            if (wave == 0)
                s_routing[lane] = routing.id;
        }
        const int steps = (a.I + kBlockK - 1) / kBlockK;
        const int items = routing.hits * a.splits;
        int* list = s_list[wave];
        // One piece of an expert's k: what its sums need.
        struct Item {
            int n, split, k0, k1;
            const uint8_t* rows[R];
            int bytes[R];
            const float* scales;  // (a block's columns lie in one block of 128)
        };
        auto look_up = [&](int item) {
            Item it;
            const int e = routing.expert(item / a.splits);
            it.split = item % a.splits;
            it.n = routing.slots_of(a, e, list);
            it.k0 = uniform(steps * it.split / a.splits);
            it.k1 = uniform(steps * (it.split + 1) / a.splits);
            const int64_t row = (int64_t)e * a.H + h0;
#pragma unroll
            for (int r = 0; r < R; ++r) {  // (H may end inside the block)
                it.rows[r] = a.down + (row + r * 16) * a.I;
                it.bytes[r] = h0 + r * 16 < a.H ? a.I * 16 : 0;
            }
            it.scales = a.downs + (WT == 0 ? (row / 128) * (a.I / kBlockK) : 0);
            return it;
        };
        const uint32_t plane = (uint32_t)P * (uint32_t)a.I * 2u;
        auto column_of = [&](int slot) {
            return slot < 0 ? kNowhere : (uint32_t)slot * (uint32_t)a.I * 2u;
        };
        // acc: 4 output columns a lane and operand of the pair `slot`
        auto keep = [&](const f32x4 (&acc)[R], int split, int slot) {
            float* y = s_y + (split * P + slot) * kCols + (lane >> 4) * 4;
#pragma unroll
            for (int r = 0; r < R; ++r)
                *reinterpret_cast<f32x4*>(y + r * 16) = acc[r];
        };
        // Experts of up to 4 columns, one after the other, keep the ring full:
        // the next one's first steps are loaded in the last steps of one (64
        // tokens over 256 experts, inter 2048: 662 us without, 618 so). So that a wave is
        // at most one ahead, an item has D steps at least; its scales lie in LDS
        // too, as a load to a register would wait for the ring's before it.
        const bool chained =
            steps / a.splits >= D && (steps + a.splits - 1) / a.splits <= kItemSteps;
        int item = wave;  // the one that is loaded
        while (item < items) {
            Item it = look_up(item);
            if (it.n > 4 || !chained) {
                for (int c0 = 0; c0 < it.n; c0 += 16) {
                    auto sums = [&](auto kind) {
                        using S = decltype(kind);
                        const int cx = c0 + (lane & (S::kColumns - 1));
                        f32x4 acc[R];
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        StepScales sc(it.scales, it.k0, WT == 0 ? it.k1 : it.k0);
                        typename S::type(it.rows, it.bytes, a.act, plane,
                                         column_of(cx < it.n ? list[cx] : -1), a.I, it.k1, ring,
                                         ring0)(
                            it.k0, [&](int, int k) { return sc.at(k); }, acc);
                        const int c = c0 + (lane & 15);
                        if (c < it.n)
                            keep(acc, it.split, list[c]);
                    };
                    if (it.n <= 4)
                        sums(Kind<Few>());
                    else
                        sums(Kind<More>());
                }
                item += kDownWaves;
                continue;
            }
            int half = 0;  // of s_scale, the loaded item's
            // (lane & 15) < n: the pair of this lane's column
            auto open = [&](const Item& at, int& slot) {
                slot = (lane & 3) < at.n ? list[lane & 3] : -1;
                if (WT == 0)
                    load4_to_lds(rsrc_words(at.scales + at.k0, (at.k1 - at.k0) * 4),
                                 scale0 + half * kItemSteps * 4, lane * 4u);
                return Few(at.rows, at.bytes, a.act, plane, column_of(slot), a.I, at.k1, ring,
                           ring0);
            };
            int slot, next_slot = -1;
            Few from = open(it, slot);
#pragma unroll
            for (int d = 0; d < D; ++d)
                from.load(it.k0 + d, d);
            int loaded = it.k0 + D, place = 0;
            for (;;) {
                bool more = false;
                Item next = it;
                f32x4 acc[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                const float* scales = s_scale + half * kItemSteps;
                for (int k = it.k0; k < it.k1; ++k) {
                    Few::step(
                        ring + place * Few::kBytes, [&](int) { return scales[k - it.k0]; },
                        [&] {
                            if (loaded == from.k1) {  // (past it: nothing is loaded any more)
                                item += kDownWaves;
                                if (item < items) {
                                    next = look_up(item);
                                    if (next.n <= 4) {
                                        more = true;
                                        half ^= 1;
                                        from = open(next, next_slot);
                                        loaded = next.k0;
                                    }
                                }
                            }
                            from.load(loaded, place);
                            ++loaded;
                        },
                        acc);
                    place = place + 1 == D ? 0 : place + 1;
                }
                Few::template done<false>();
                if ((lane & 15) < it.n)
                    keep(acc, it.split, slot);
                if (!more)
                    break;
                it = next;
                slot = next_slot;
            }
            Few::template done<true>();
        }
    });
    __syncthreads();
    // a token's pairs in slot order, each the sum of its pieces in order
    for (int i = threadIdx.x; i < a.T * kCols; i += kDownWaves * kWave) {
        const int t = i / kCols, c = i % kCols;
        float sum = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int p = t * a.topk + j, e = id[p];
            if (e < 0 || h0 + c >= a.H)
                continue;
            float y = s_y[p * kCols + c];
            for (int k = 1; k < a.splits; ++k)
                y = y + s_y[(k * P + p) * kCols + c];
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

// (hipErrorInvalidValue for more LDS than a compute unit has)
template <int WT, int XT, int R, int D, bool kSmall>
hipError_t launch_down(const FewArgs& a, hipStream_t s)
{
    constexpr int kFew = Sums<R, 4, 2, WT, 0, D>::kBytes * D, kMore = Sums<R, 16, 2, WT, 0, 1>::kBytes;
    const size_t lds = (size_t)kDownWaves * ((kFew > kMore ? kFew : kMore) + kItemScales) +
                       (size_t)a.splits * a.T * a.topk * 16 * R * sizeof(float);
    constexpr size_t kStatic = (kSmall ? kWave * sizeof(int) : sizeof(Routing)) +
                               kDownWaves * kFewMaxTokens * sizeof(int);
    if (lds + (kStatic + 1023) / 1024 * 1024 > kFewLds)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((block_few_down_kernel<WT, XT, R, D, kSmall>),
                       dim3((a.H + 16 * R - 1) / (16 * R)), dim3(kDownWaves * kWave), lds, s, a);
    return hipGetLastError();
}

template <int WT, int XT, bool kSmall>
hipError_t few_with(const FewArgs& a, hipStream_t s)
{
    // 32 hidden columns a block where they fill the compute units twice
    const int up = a.hits * (a.I / 16);
    if (a.I % 32 == 0 && up >= 1024)
        hipLaunchKernelGGL((block_few_up_kernel<WT, XT, 4, kSmall>), dim3(up / 2),
                           dim3(kUpWaves * kWave), 0, s, a);
    else
        hipLaunchKernelGGL((block_few_up_kernel<WT, XT, 2, kSmall>), dim3(up), dim3(kUpWaves * kWave),
                           0, s, a);
    // 32 output columns a block where that leaves most compute units a block and
    // the pairs' sums leave LDS for three steps; else 16, with two steps of the
    // largest calls
    const int pairs = a.splits * a.T * a.topk;
    if constexpr (kSmall) {
        if (a.H >= 32 * 192 && pairs <= 64)
            return launch_down<WT, XT, 2, 3, kSmall>(a, s);
    }
    if (pairs <= 768)
        return launch_down<WT, XT, 1, 3, kSmall>(a, s);
    return launch_down<WT, XT, 1, 2, kSmall>(a, s);
}

template <int WT, int XT>
hipError_t few_types(const FewArgs& a, hipStream_t s)
{
    return a.T * a.topk <= kWave ? few_with<WT, XT, true>(a, s) : few_with<WT, XT, false>(a, s);
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
