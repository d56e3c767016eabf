// Host side of include/moe.h: argument checks, launch geometry and launches of
// the layer operators. As in ep_plan.cpp, every precondition is checked before
// anything is enqueued and a failed check names the argument.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "ep_plan_view.h"
#include "ep_static.h"
#include "moe_kernels.h"

namespace {

constexpr size_t kPtrAlign = 16;
// Bytes a call may move before its rows stream past the caches: the 256 MB
// last-level cache of an MI355X.
constexpr int64_t kKeepBytes = 256ll << 20;

// Blocks of a grouped product: one a compute unit of an MI355X.
constexpr int kGemmBlocks = 256;

int fail(int code, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return ep::set_error(code, buf);
}

int ok() { return ep::set_error(EP_OK, ""); }

struct Pointer {
    const void* ptr;
    const char* name;
    size_t align;
    bool required;
};

int check_pointers(const Pointer* p, int n)
{
    for (int i = 0; i < n; ++i) {
        if (!p[i].ptr) {
            if (p[i].required)
                return fail(EP_ERR_NULL, "%s is NULL", p[i].name);
            continue;
        }
        if (reinterpret_cast<uintptr_t>(p[i].ptr) % p[i].align)
            return fail(EP_ERR_ALIGN, "%s = %p is not %zu-byte aligned", p[i].name, p[i].ptr,
                        p[i].align);
    }
    return EP_OK;
}

template <int N>
int check_pointers(const Pointer (&p)[N])
{
    return check_pointers(p, N);
}

}  // namespace

extern "C" {

int moe_rms_norm(const moe_rms_norm_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    if (a->dtype != EP_BF16 && a->dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.dtype = %d: must be EP_BF16 or EP_FP16", a->dtype);
    if (a->weight_dtype != a->dtype && a->weight_dtype != MOE_FP32)
        return fail(EP_ERR_ARG, "args.weight_dtype = %d: must be args.dtype or MOE_FP32",
                    a->weight_dtype);
    if (a->rows < 0)
        return fail(EP_ERR_ARG, "args.rows = %lld: must be >= 0", (long long)a->rows);
    if (a->hidden < 8 || a->hidden % 8)
        return fail(EP_ERR_ARG, "args.hidden = %d: must be a positive multiple of 8", a->hidden);
    if (a->hidden > moe::kNormMaxHidden)
        return fail(EP_ERR_SIZE, "args.hidden = %d: must be at most %d", a->hidden,
                    moe::kNormMaxHidden);
    if (!(a->eps >= 0.0f) || std::isinf(a->eps))
        return fail(EP_ERR_ARG, "args.eps = %g: must be finite and >= 0", (double)a->eps);
    if ((a->codes == nullptr) != (a->scales == nullptr))
        return fail(EP_ERR_ARG, "args.codes and args.scales must both be set or both NULL");
    if (a->codes && a->hidden % 128)
        return fail(EP_ERR_ARG, "args.hidden = %d: codes need a multiple of 128", a->hidden);
    if ((a->residual == nullptr) != (a->residual_out == nullptr))
        return fail(EP_ERR_ARG,
                    "args.residual and args.residual_out must both be set or both NULL");
    if (a->row_counts && (a->group_rows < 1 || a->rows % a->group_rows))
        return fail(EP_ERR_ARG, "args.group_rows = %lld: must be >= 1 and divide rows = %lld",
                    (long long)a->group_rows, (long long)a->rows);
    if (a->rows == 0)
        return ok();
    if (!a->out && !a->codes)
        return fail(EP_ERR_NULL, "args.out and args.codes are both NULL");
    const Pointer ptrs[] = {{a->x, "args.x", kPtrAlign, true},
                            {a->residual, "args.residual", kPtrAlign, false},
                            {a->residual_out, "args.residual_out", kPtrAlign, false},
                            {a->weight, "args.weight", kPtrAlign, true},
                            {a->out, "args.out", kPtrAlign, false},
                            {a->codes, "args.codes", kPtrAlign, false},
                            {a->scales, "args.scales", 4, false},
                            {a->row_counts, "args.row_counts", 4, false}};
    const int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;

    moe::NormArgs na;
    na.x = static_cast<const uint8_t*>(a->x);
    na.res = static_cast<const uint8_t*>(a->residual);
    na.res_out = static_cast<uint8_t*>(a->residual_out);
    na.w = static_cast<const uint8_t*>(a->weight);
    na.out = static_cast<uint8_t*>(a->out);
    na.codes = static_cast<uint8_t*>(a->codes);
    na.scales = reinterpret_cast<uint8_t*>(a->scales);
    na.counts = a->row_counts;
    na.rows = a->rows;
    na.group_rows = a->row_counts ? a->group_rows : a->rows;
    na.H = a->hidden;
    na.eps = a->eps;
    // Waves a row: as few as hold it, doubled while the call has fewer waves
    // than the chip holds at 8 a SIMD and a wave has more than one chunk.
    const int chunks = (a->hidden + moe::kNormChunk - 1) / moe::kNormChunk;
    int waves = 1;
    while (waves * moe::kNormChunks < chunks)
        waves *= 2;
    while (waves < moe::kNormMaxWaves && waves < chunks && a->rows * waves < 8192)
        waves *= 2;
    na.row_waves = waves;
    na.chunks = (chunks + waves - 1) / waves;
    // a launch's work-items must fit in 32 bits
    if (a->rows > ((int64_t)UINT32_MAX - 1024) / (waves * ep::kWave))
        return fail(EP_ERR_SIZE, "args.rows = %lld is too large for one launch",
                    (long long)a->rows);
    const int64_t row_bytes = (int64_t)a->hidden *
                              (2 + (a->residual ? 4 : 0) + (a->out ? 2 : 0) + (a->codes ? 1 : 0));
    const bool streaming = a->rows * row_bytes > kKeepBytes;
    const hipError_t e = moe::launch_norm(na, a->dtype == EP_BF16 ? 0 : 1,
                                          a->weight_dtype == MOE_FP32 ? 2
                                          : a->dtype == EP_BF16       ? 0
                                                                      : 1,
                                          streaming, static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "rms_norm launch failed: %s", hipGetErrorString(e));
    return ok();
}

int moe_grouped_gemm(const moe_grouped_gemm_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    const bool swiglu = a->epilogue == MOE_EPILOGUE_SWIGLU;
    if (!swiglu && a->epilogue != MOE_EPILOGUE_ROWS)
        return fail(EP_ERR_ARG, "args.epilogue = %d: must be a MOE_EPILOGUE_* value", a->epilogue);
    if (swiglu ? a->out_dtype != EP_FP8_E4M3
               : a->out_dtype != EP_BF16 && a->out_dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.out_dtype = %d: must be %s", a->out_dtype,
                    swiglu ? "EP_FP8_E4M3 with MOE_EPILOGUE_SWIGLU" : "EP_BF16 or EP_FP16");
    if (a->groups < 0 || a->cap < 0)
        return fail(EP_ERR_ARG, "args.groups = %d, args.cap = %d: must be >= 0", a->groups, a->cap);
    if (a->k < 128 || a->k % 128)
        return fail(EP_ERR_ARG, "args.k = %d: must be a positive multiple of 128", a->k);
    const int step = swiglu ? 256 : 8;
    if (a->n < step || a->n % step)
        return fail(EP_ERR_ARG, "args.n = %d: must be a positive multiple of %d", a->n, step);
    if (a->n > (1 << 20) || a->k > (1 << 20) || a->groups > (1 << 20))
        return fail(EP_ERR_SIZE, "args.n = %d, args.k = %d, args.groups = %d: must be at most "
                    "2^20", a->n, a->k, a->groups);
    if ((int64_t)a->groups * a->cap > INT32_MAX)
        return fail(EP_ERR_SIZE, "args.groups * args.cap = %lld exceeds 2^31 - 1",
                    (long long)a->groups * a->cap);
    if (a->groups == 0 || a->cap == 0)
        return ok();
    if (!swiglu && a->out_scales)
        return fail(EP_ERR_ARG, "args.out_scales must be NULL with MOE_EPILOGUE_ROWS");
    const Pointer ptrs[] = {{a->a, "args.a", kPtrAlign, true},
                            {a->a_scales, "args.a_scales", 4, true},
                            {a->b, "args.b", kPtrAlign, true},
                            {a->b_scales, "args.b_scales", 4, true},
                            {a->counts, "args.counts", 4, false},
                            {a->out, "args.out", kPtrAlign, true},
                            {a->out_scales, "args.out_scales", 4, swiglu}};
    const int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    moe::GemmArgs ga;
    ga.a = static_cast<const uint8_t*>(a->a);
    ga.as = reinterpret_cast<const uint8_t*>(a->a_scales);
    ga.b = static_cast<const uint8_t*>(a->b);
    ga.bs = a->b_scales;
    ga.counts = a->counts;
    ga.out = static_cast<uint8_t*>(a->out);
    ga.osc = reinterpret_cast<uint8_t*>(a->out_scales);
    ga.groups = a->groups;
    ga.cap = a->cap;
    ga.n = a->n;
    ga.k = a->k;
    ga.col_tiles = (a->n + 255) / 256;
    const hipError_t e = moe::launch_gemm(ga, a->out_dtype == EP_FP16 ? 1 : 0, swiglu, kGemmBlocks,
                                          static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "grouped_gemm launch failed: %s", hipGetErrorString(e));
    return ok();
}

int moe_combine_backward(ep_expert_plan_t* x, const moe_combine_backward_args_t* a,
                         void* stream_ptr)
{
    if (!x)
        return fail(EP_ERR_NULL, "plan is NULL");
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    const Pointer ptrs[] = {{a->grad_out, "args.grad_out", kPtrAlign, true},
                            {a->indices, "args.indices", 4, true},
                            {a->weights, "args.weights", 4, false},
                            {a->packed_y, "args.packed_y", kPtrAlign, false},
                            {a->grad_packed_y, "args.grad_packed_y", kPtrAlign, true},
                            {a->grad_weights, "args.grad_weights", 4, false}};
    int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    if ((a->packed_y == nullptr) != (a->grad_weights == nullptr))
        return fail(EP_ERR_ARG,
                    "args.packed_y and args.grad_weights must both be set or both NULL");
    if (a->grad_weights && !a->weights)
        return fail(EP_ERR_ARG, "args.grad_weights needs args.weights");
    ep::FusedView v;
    rc = ep::fused_view(x, "combine_backward", &v);
    if (rc != EP_OK)
        return rc;
    if (v.wire != EP_WIRE_NONE)
        return fail(EP_ERR_ARG, "combine_backward needs cfg.combine_wire = EP_WIRE_NONE");
    moe::CombineBackwardArgs ca;
    ca.go = static_cast<const uint8_t*>(a->grad_out);
    ca.idx = a->indices;
    ca.w = a->weights;
    ca.py = static_cast<const uint8_t*>(a->packed_y);
    ca.fslot = v.fslot;
    ca.gy = static_cast<uint8_t*>(a->grad_packed_y);
    ca.gw = a->grad_weights;
    ca.row_vecs = v.H / 8;
    ca.M = v.M;
    ca.k = v.k;
    ca.E = v.E;
    // Waves a token from the row's length alone (the dots' order depends on
    // it): as many as give each at most kBackChunks chunks.
    const int chunks = (v.H + 511) / 512;
    int waves = 1;
    while (waves < moe::kBackMaxWaves && waves * moe::kBackChunks < chunks)
        waves *= 2;
    ca.row_waves = waves;
    ca.wave_vecs = (ca.row_vecs + waves - 1) / waves;
    // Slots a wave: all of the token's, halved while the call has fewer waves
    // than the chip holds at 2 a SIMD and a wave more than 2 slots (135 tokens
    // of top-64, 936 fp16: 38.1 -> 14.4 us; 16 of top-8, 7168 bf16: 6.9 -> 4.5.
    // A limit of 8192 waves: 17.0 us, and 1024 tokens of top-8 25.1 -> 28.0).
    const int64_t token_waves = (int64_t)v.tokens.total * waves;
    int groups = 1;
    while (token_waves * groups < 2048 && groups * 2 < v.k)
        groups *= 2;
    ca.group_slots = (v.k + groups - 1) / groups;
    if (((int64_t)v.tokens.total + 4) * std::max(waves, 4) * ep::kWave > (int64_t)UINT32_MAX)
        return fail(EP_ERR_SIZE, "combine_backward of %d tokens is too large for one launch",
                    v.tokens.total);
    hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
    const hipError_t e = moe::launch_combine_backward(ca, v.tokens, v.dtype == EP_BF16 ? 0 : 1,
                                                      v.stream, stream);
    ep::fused_launched(x, stream);
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "combine_backward launch failed: %s", hipGetErrorString(e));
    return ok();
}

int moe_dispatch_backward(ep_expert_plan_t* x, const moe_dispatch_backward_args_t* a,
                          void* stream_ptr)
{
    if (!x)
        return fail(EP_ERR_NULL, "plan is NULL");
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    const Pointer ptrs[] = {{a->grad_packed_x, "args.grad_packed_x", kPtrAlign, true},
                            {a->grad_x, "args.grad_x", kPtrAlign, true}};
    int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    ep::FusedView v;
    rc = ep::fused_view(x, "dispatch_backward", &v);
    if (rc != EP_OK)
        return rc;
    if (v.wire != EP_WIRE_NONE)
        return fail(EP_ERR_ARG, "dispatch_backward needs cfg.combine_wire = EP_WIRE_NONE");
    moe::DispatchBackwardArgs da;
    da.gp = static_cast<const uint8_t*>(a->grad_packed_x);
    da.fslot = v.fslot;
    da.gx = static_cast<uint8_t*>(a->grad_x);
    da.row_vecs = v.H / 8;
    da.pieces = (da.row_vecs + ep::kWave - 1) / ep::kWave;
    da.M = v.M;
    da.k = v.k;
    // waves a block, as the combine's (large calls: 362 us with 16, 368 with 4
    // and 373 with 8 at 8 ranks x 2048 tokens x 7168 bf16, top-8)
    const int waves = v.large ? 16 : 4;
    if (((int64_t)v.tokens.total * da.pieces + waves) * ep::kWave > (int64_t)UINT32_MAX)
        return fail(EP_ERR_SIZE, "dispatch_backward of %d tokens is too large for one launch",
                    v.tokens.total);
    hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
    const hipError_t e = moe::launch_dispatch_backward(da, v.tokens, v.dtype == EP_BF16 ? 0 : 1,
                                                       waves, v.stream, stream);
    ep::fused_launched(x, stream);
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "dispatch_backward launch failed: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"
