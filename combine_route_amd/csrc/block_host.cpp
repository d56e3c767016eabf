// Host side of include/moe_block.h: argument checks, launch geometry and
// launches of the kernels of a whole MoE block. As in ep_plan.cpp, every
// precondition is checked before anything is enqueued and a failed check names
// the argument.
#include "moe_block.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "block_kernels.h"
#include "moe_check.h"

namespace {

using namespace moe::host;

// Checks that the two norm calls share.
template <class A>
int check_norm(const A* a)
{
    if (a->dtype != EP_BF16 && a->dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.dtype = %d: must be EP_BF16 or EP_FP16", a->dtype);
    if (a->weight_dtype != a->dtype && a->weight_dtype != MOE_FP32)
        return fail(EP_ERR_ARG, "args.weight_dtype = %d: must be args.dtype or MOE_FP32",
                    a->weight_dtype);
    if (a->rows < 0)
        return fail(EP_ERR_ARG, "args.rows = %lld: must be >= 0", (long long)a->rows);
    if (a->hidden < 8 || a->hidden % 8)
        return fail(EP_ERR_ARG, "args.hidden = %d: must be a positive multiple of 8", a->hidden);
    if (a->hidden > block::kNormMaxHidden)
        return fail(EP_ERR_SIZE, "args.hidden = %d: must be at most %d", a->hidden,
                    block::kNormMaxHidden);
    if (!(a->eps >= 0.0f) || std::isinf(a->eps))
        return fail(EP_ERR_ARG, "args.eps = %g: must be finite and >= 0", (double)a->eps);
    if (!std::isfinite(a->residual_scale))
        return fail(EP_ERR_ARG, "args.residual_scale = %g: must be finite",
                    (double)a->residual_scale);
    if (a->row_counts && (a->group_rows < 1 || a->rows % a->group_rows))
        return fail(EP_ERR_ARG, "args.group_rows = %lld: must be >= 1 and divide rows = %lld",
                    (long long)a->group_rows, (long long)a->rows);
    if (a->gate && a->gate_rows != 0 && (a->gate_rows < 0 || a->rows % a->gate_rows))
        return fail(EP_ERR_ARG, "args.gate_rows = %lld: must be 0 or divide rows = %lld",
                    (long long)a->gate_rows, (long long)a->rows);
    return EP_OK;
}

int weight_type(int weight_dtype, int dtype)
{
    return weight_dtype == MOE_FP32 ? 2 : dtype == EP_BF16 ? 0 : 1;
}

// How the backward's rows lie on its blocks. most_blocks: of these rows in any
// number of groups.
struct BackwardShape {
    int chunks, row_waves, group_blocks, block_groups, blocks, most_blocks;
};

// Chunks a wave: as few as let 8 waves hold the row, at most 4 (then up to 16
// waves). Blocks: one a compute unit for rows of 5 waves and more: 8 waves of
// 2 chunks fill a unit (216 to 238 registers a lane), and of 1 chunk all but fill
// it (127 to 138, where two blocks a unit would need 128); more of shorter rows.
bool backward_shape(int64_t rows, int hidden, int64_t groups, BackwardShape* s)
{
    if (rows < 1 || groups < 1 || groups > rows || rows % groups || hidden < 8 || hidden % 8 ||
        hidden > block::kNormMaxHidden)
        return false;
    const int chunks = (hidden + block::kNormChunk - 1) / block::kNormChunk;
    s->chunks = chunks <= 8 ? 1 : chunks <= 16 ? 2 : 4;
    s->row_waves = (chunks + s->chunks - 1) / s->chunks;
    const int64_t target = 256 * std::max(1, 8 / s->row_waves);
    s->most_blocks = (int)std::min(rows, target);
    if (groups >= target) {
        s->group_blocks = 1;
        const int64_t each = (groups + target - 1) / target;
        if (each > INT32_MAX)
            return false;
        s->block_groups = (int)each;
        s->blocks = (int)((groups + each - 1) / each);
    } else {
        s->group_blocks = (int)std::min<int64_t>(rows / groups, target / groups);
        s->block_groups = 1;
        s->blocks = (int)groups * s->group_blocks;
    }
    return true;
}

// Bytes of moe_few_tokens's workspace, 0 for sizes it refuses: the hidden rows
// of every slot, as bf16 values and their rests.
size_t few_bytes(int tokens, int topk, int hidden, int inter)
{
    if (tokens < 1 || tokens > block::kFewMaxTokens || topk < 1 || topk > 64 ||
        tokens * topk > block::kFewMaxSlots || hidden < 16 || hidden > 65536 || hidden % 16 ||
        inter < 16 || inter > 65536 || inter % 16)
        return 0;
    return (size_t)4 * tokens * topk * inter;
}

}  // namespace

extern "C" {

int moe_block_norm(const moe_block_norm_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    int rc = check_norm(a);
    if (rc != EP_OK)
        return rc;
    if (a->rows == 0)  // before what is set: empty tensors have no address
        return ok();
    if ((a->codes == nullptr) != (a->scales == nullptr))
        return fail(EP_ERR_ARG, "args.codes and args.scales must both be set or both NULL");
    if (a->codes && a->codes_dtype != EP_FP8_E4M3 && a->codes_dtype != MOE_INT8)
        return fail(EP_ERR_ARG, "args.codes_dtype = %d: must be EP_FP8_E4M3 or MOE_INT8",
                    a->codes_dtype);
    const bool fp8 = a->codes && a->codes_dtype == EP_FP8_E4M3;
    if (fp8 && a->hidden % 128)
        return fail(EP_ERR_ARG, "args.hidden = %d: FP8 codes need a multiple of 128", a->hidden);
    if ((a->pre_weight == nullptr) != (!a->out && !a->codes))
        return fail(EP_ERR_ARG, "args.pre_weight must be set iff args.out or args.codes is");
    const Pointer ptrs[] = {{a->y, "args.y", kPtrAlign, true},
                            {a->residual, "args.residual", kPtrAlign, true},
                            {a->residual_out, "args.residual_out", kPtrAlign, true},
                            {a->post_weight, "args.post_weight", kPtrAlign, false},
                            {a->gate, "args.gate", kPtrAlign, false},
                            {a->pre_weight, "args.pre_weight", kPtrAlign, false},
                            {a->out, "args.out", kPtrAlign, false},
                            {a->codes, "args.codes", kPtrAlign, false},
                            {a->scales, "args.scales", 4, false},
                            {a->row_counts, "args.row_counts", 4, false}};
    rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;

    block::NormArgs na;
    na.y = static_cast<const uint8_t*>(a->y);
    na.res = static_cast<const uint8_t*>(a->residual);
    na.res_out = static_cast<uint8_t*>(a->residual_out);
    na.post = static_cast<const uint8_t*>(a->post_weight);
    na.gate = static_cast<const uint8_t*>(a->gate);
    na.pre = static_cast<const uint8_t*>(a->pre_weight);
    na.out = static_cast<uint8_t*>(a->out);
    na.codes = static_cast<uint8_t*>(a->codes);
    na.scales = reinterpret_cast<uint8_t*>(a->scales);
    na.counts = a->row_counts;
    na.rows = a->rows;
    na.group_rows = a->row_counts ? a->group_rows : a->rows;
    na.gate_rows = a->gate && a->gate_rows ? a->gate_rows : a->rows;
    na.H = a->hidden;
    na.kind = !a->codes ? block::kNoCodes : fp8 ? block::kFp8Codes : block::kInt8Codes;
    na.res_scale = a->residual_scale;
    na.eps = a->eps;
    // Waves a row: as few as hold it, doubled while the call has fewer waves
    // than the chip holds at 8 a SIMD and a wave has more than one chunk.
    const int chunks = (a->hidden + block::kNormChunk - 1) / block::kNormChunk;
    int waves = 1;
    while (waves * block::kNormChunks < chunks)
        waves *= 2;
    while (waves < block::kNormMaxWaves && waves < chunks && a->rows * waves < 8192)
        waves *= 2;
    na.row_waves = waves;
    na.chunks = (chunks + waves - 1) / waves;
    // a launch's work-items must fit in 32 bits
    if (a->rows > ((int64_t)UINT32_MAX - 1024) / (waves * ep::kWave))
        return fail(EP_ERR_SIZE, "args.rows = %lld is too large for one launch",
                    (long long)a->rows);
    const int64_t row_bytes = (int64_t)a->hidden * (6 + (a->out ? 2 : 0) + (a->codes ? 1 : 0));
    const hipError_t e = block::launch_norm(na, a->dtype == EP_BF16 ? 0 : 1,
                                            weight_type(a->weight_dtype, a->dtype),
                                            a->rows * row_bytes > kKeepBytes,
                                            static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "block_norm launch failed: %s", hipGetErrorString(e));
    return ok();
}

size_t moe_block_norm_backward_workspace_bytes(int64_t rows, int32_t hidden, int64_t groups)
{
    BackwardShape s;
    if (!backward_shape(rows, hidden, groups, &s)) {
        fail(EP_ERR_ARG,
             "rows = %lld, hidden = %d, groups = %lld: groups must divide rows and hidden be a "
             "multiple of 8 up to %d",
             (long long)rows, hidden, (long long)groups, block::kNormMaxHidden);
        return 0;
    }
    ok();
    return (size_t)3 * s.most_blocks * hidden * sizeof(float);
}

int moe_block_norm_backward(const moe_block_norm_backward_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    int rc = check_norm(a);
    if (rc != EP_OK)
        return rc;
    if (a->rows == 0)
        return ok();
    if ((a->pre_weight == nullptr) != (a->grad_out == nullptr))
        return fail(EP_ERR_ARG, "args.pre_weight and args.grad_out must both be set or both NULL");
    if (!a->grad_out && !a->grad_h)
        return fail(EP_ERR_NULL, "args.grad_h and args.grad_out are both NULL");
    if (a->grad_post_weight && !a->post_weight)
        return fail(EP_ERR_ARG, "args.grad_post_weight needs args.post_weight");
    if (a->grad_gate && !a->gate)
        return fail(EP_ERR_ARG, "args.grad_gate needs args.gate");
    if (a->grad_pre_weight && !a->pre_weight)
        return fail(EP_ERR_ARG, "args.grad_pre_weight needs args.pre_weight");
    const bool sums = a->grad_post_weight || a->grad_gate || a->grad_pre_weight;
    const Pointer ptrs[] = {{a->y, "args.y", kPtrAlign, true},
                            {a->h, "args.h", kPtrAlign, a->grad_out != nullptr},
                            {a->grad_h, "args.grad_h", kPtrAlign, false},
                            {a->grad_out, "args.grad_out", kPtrAlign, false},
                            {a->post_weight, "args.post_weight", kPtrAlign, false},
                            {a->gate, "args.gate", kPtrAlign, false},
                            {a->pre_weight, "args.pre_weight", kPtrAlign, false},
                            {a->grad_y, "args.grad_y", kPtrAlign, true},
                            {a->grad_residual, "args.grad_residual", kPtrAlign, false},
                            {a->grad_post_weight, "args.grad_post_weight", kPtrAlign, false},
                            {a->grad_gate, "args.grad_gate", kPtrAlign, false},
                            {a->grad_pre_weight, "args.grad_pre_weight", kPtrAlign, false},
                            {a->workspace, "args.workspace", kPtrAlign, sums},
                            {a->row_counts, "args.row_counts", 4, false}};
    rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    const int64_t gates = a->gate && a->gate_rows ? a->rows / a->gate_rows : 1;
    if (gates > 1 && a->row_counts && a->gate_rows != a->group_rows)
        return fail(EP_ERR_ARG, "args.gate_rows = %lld must be args.group_rows = %lld with "
                    "args.row_counts", (long long)a->gate_rows, (long long)a->group_rows);
    const int64_t groups = gates > 1 ? gates : a->row_counts ? a->rows / a->group_rows : 1;
    BackwardShape s;
    if (!backward_shape(a->rows, a->hidden, groups, &s) || gates > INT32_MAX)
        return fail(EP_ERR_SIZE, "args.rows = %lld is too large", (long long)a->rows);
    const int64_t need = (int64_t)3 * s.blocks * a->hidden * (int64_t)sizeof(float);
    if (sums && a->workspace_bytes < need)
        return fail(EP_ERR_SIZE, "args.workspace_bytes = %lld: %lld are needed",
                    (long long)a->workspace_bytes, (long long)need);

    block::NormBackwardArgs na;
    na.y = static_cast<const uint8_t*>(a->y);
    na.h = static_cast<const uint8_t*>(a->h);
    na.gh = static_cast<const uint8_t*>(a->grad_h);
    na.go = static_cast<const uint8_t*>(a->grad_out);
    na.post = static_cast<const uint8_t*>(a->post_weight);
    na.gate = static_cast<const uint8_t*>(a->gate);
    na.pre = static_cast<const uint8_t*>(a->pre_weight);
    na.gy = static_cast<uint8_t*>(a->grad_y);
    na.gres = static_cast<uint8_t*>(a->grad_residual);
    na.gpost = a->grad_post_weight;
    na.ggate = a->grad_gate;
    na.gpre = a->grad_pre_weight;
    na.part = static_cast<float*>(a->workspace);
    na.counts = a->row_counts;
    na.groups = groups;
    na.group_rows = a->rows / groups;
    na.group_blocks = s.group_blocks;
    na.block_groups = s.block_groups;
    na.blocks = s.blocks;
    na.gates = (int)gates;
    na.H = a->hidden;
    na.row_waves = s.row_waves;
    na.chunks = s.chunks;
    na.res_scale = a->residual_scale;
    na.eps = a->eps;
    const int64_t row_bytes = (int64_t)a->hidden * 12;
    const hipError_t e = block::launch_norm_backward(na, a->dtype == EP_BF16 ? 0 : 1,
                                                     weight_type(a->weight_dtype, a->dtype),
                                                     a->rows * row_bytes > kKeepBytes,
                                                     static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "block_norm_backward launch failed: %s", hipGetErrorString(e));
    return ok();
}

int moe_quantize_int8(const moe_quantize_int8_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    if (a->dtype != EP_BF16 && a->dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.dtype = %d: must be EP_BF16 or EP_FP16", a->dtype);
    if (a->n_rows < 0)
        return fail(EP_ERR_ARG, "args.n_rows = %lld: must be >= 0", (long long)a->n_rows);
    if (a->hidden < 8 || a->hidden % 8)
        return fail(EP_ERR_ARG, "args.hidden = %d: must be a positive multiple of 8", a->hidden);
    if (a->hidden > block::kQuantMaxHidden)
        return fail(EP_ERR_SIZE, "args.hidden = %d: must be at most %d", a->hidden,
                    block::kQuantMaxHidden);
    if (a->row_counts && (a->group_rows < 1 || a->n_rows % a->group_rows))
        return fail(EP_ERR_ARG, "args.group_rows = %lld: must be >= 1 and divide n_rows = %lld",
                    (long long)a->group_rows, (long long)a->n_rows);
    if (a->n_rows == 0)
        return ok();
    const Pointer ptrs[] = {{a->rows, "args.rows", kPtrAlign, true},
                            {a->codes, "args.codes", kPtrAlign, true},
                            {a->scales, "args.scales", 4, true},
                            {a->row_counts, "args.row_counts", 4, false}};
    const int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    block::QuantizeArgs qa;
    qa.rows = static_cast<const uint8_t*>(a->rows);
    qa.codes = static_cast<uint8_t*>(a->codes);
    qa.scales = a->scales;
    qa.counts = a->row_counts;
    qa.n_rows = a->n_rows;
    qa.group_rows = a->row_counts ? a->group_rows : a->n_rows;
    qa.H = a->hidden;
    // waves a row: as moe_block_norm's
    const int chunks = (a->hidden + block::kNormChunk - 1) / block::kNormChunk;
    int waves = 1;
    while (waves * block::kQuantChunks < chunks)
        waves *= 2;
    while (waves < block::kQuantMaxWaves && waves < chunks && a->n_rows * waves < 8192)
        waves *= 2;
    qa.row_waves = waves;
    qa.chunks = (chunks + waves - 1) / waves;
    // a launch's work-items must fit in 32 bits
    if (a->n_rows > ((int64_t)UINT32_MAX - 1024) / (waves * ep::kWave))
        return fail(EP_ERR_SIZE, "args.n_rows = %lld is too large for one launch",
                    (long long)a->n_rows);
    const hipError_t e =
        block::launch_quantize(qa, a->dtype == EP_BF16 ? 0 : 1,
                               a->n_rows * a->hidden * 3 > kKeepBytes,
                               static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "quantize_int8 launch failed: %s", hipGetErrorString(e));
    return ok();
}

int moe_grouped_gemm_int8(const moe_grouped_gemm_int8_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    const bool swiglu = a->epilogue == MOE_EPILOGUE_SWIGLU;
    if (!swiglu && a->epilogue != MOE_EPILOGUE_ROWS)
        return fail(EP_ERR_ARG, "args.epilogue = %d: must be a MOE_EPILOGUE_* value", a->epilogue);
    if (a->out_dtype != EP_BF16 && a->out_dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.out_dtype = %d: must be EP_BF16 or EP_FP16", a->out_dtype);
    if (a->groups < 0 || a->cap < 0)
        return fail(EP_ERR_ARG, "args.groups = %d, args.cap = %d: must be >= 0", a->groups, a->cap);
    if (a->k < 16 || a->k % 16)
        return fail(EP_ERR_ARG, "args.k = %d: must be a positive multiple of 16", a->k);
    const int step = swiglu ? 16 : 8;
    if (a->n < step || a->n % step)
        return fail(EP_ERR_ARG, "args.n = %d: must be a positive multiple of %d", a->n, step);
    if (a->n > (1 << 20) || a->k > (1 << 16) || a->groups > (1 << 20))
        return fail(EP_ERR_SIZE, "args.n = %d, args.k = %d, args.groups = %d: must be at most "
                    "2^20, 2^16 and 2^20", a->n, a->k, a->groups);
    if ((int64_t)a->groups * a->cap > INT32_MAX)
        return fail(EP_ERR_SIZE, "args.groups * args.cap = %lld exceeds 2^31 - 1",
                    (long long)a->groups * a->cap);
    if (a->groups == 0 || a->cap == 0)
        return ok();
    const Pointer ptrs[] = {{a->a, "args.a", kPtrAlign, true},
                            {a->a_scales, "args.a_scales", 4, true},
                            {a->b, "args.b", kPtrAlign, true},
                            {a->b_scales, "args.b_scales", 4, true},
                            {a->counts, "args.counts", 4, false},
                            {a->out, "args.out", kPtrAlign, true}};
    const int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    block::GemmArgs ga;
    ga.a = static_cast<const uint8_t*>(a->a);
    ga.as = a->a_scales;
    ga.b = static_cast<const uint8_t*>(a->b);
    ga.bs = a->b_scales;
    ga.counts = a->counts;
    ga.out = static_cast<uint8_t*>(a->out);
    ga.groups = a->groups;
    ga.cap = a->cap;
    ga.n = a->n;
    ga.k = a->k;
    ga.col_tiles = (a->n + 255) / 256;
    const hipError_t e = block::launch_gemm(ga, a->out_dtype == EP_FP16 ? 1 : 0, swiglu,
                                            kGemmBlocks, static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "grouped_gemm_int8 launch failed: %s", hipGetErrorString(e));
    return ok();
}

size_t moe_few_tokens_workspace_bytes(int32_t tokens, int32_t topk, int32_t hidden, int32_t inter)
{
    const size_t n = few_bytes(tokens, topk, hidden, inter);
    if (n == 0)
        fail(EP_ERR_ARG,
             "tokens = %d, topk = %d, hidden = %d, inter = %d: must be 1 to %d, 1 to 64 (at most "
             "%d slots) and multiples of 16 up to 65536",
             tokens, topk, hidden, inter, block::kFewMaxTokens, block::kFewMaxSlots);
    else
        ok();
    return n;
}

int moe_few_tokens(const moe_few_tokens_args_t* a, void* stream_ptr)
{
    if (!a)
        return fail(EP_ERR_NULL, "args is NULL");
    if (a->dtype != EP_BF16 && a->dtype != EP_FP16)
        return fail(EP_ERR_ARG, "args.dtype = %d: must be EP_BF16 or EP_FP16", a->dtype);
    if (a->weight_dtype != EP_FP8_E4M3 && a->weight_dtype != MOE_INT8)
        return fail(EP_ERR_ARG, "args.weight_dtype = %d: must be EP_FP8_E4M3 or MOE_INT8",
                    a->weight_dtype);
    const int step = a->weight_dtype == MOE_INT8 ? 16 : 128;
    if (a->hidden < step || a->hidden % step)
        return fail(EP_ERR_ARG, "args.hidden = %d: must be a positive multiple of %d", a->hidden,
                    step);
    if (a->inter < step || a->inter % step)
        return fail(EP_ERR_ARG, "args.inter = %d: must be a positive multiple of %d", a->inter,
                    step);
    if (a->tokens < 0 || a->topk < 1 || a->experts < 1)
        return fail(EP_ERR_ARG,
                    "args.tokens = %d, args.topk = %d, args.experts = %d: must be >= 0, 1 and 1",
                    a->tokens, a->topk, a->experts);
    if (a->tokens > block::kFewMaxTokens || a->topk > 64 ||
        a->tokens * a->topk > block::kFewMaxSlots || a->experts > block::kFewMaxExperts ||
        a->hidden > 65536 || a->inter > 65536)
        return fail(EP_ERR_SIZE,
                    "args.tokens = %d, args.topk = %d, args.experts = %d, args.hidden = %d, "
                    "args.inter = %d: must be at most %d, 64 (%d slots in all), %d, 65536 and "
                    "65536",
                    a->tokens, a->topk, a->experts, a->hidden, a->inter, block::kFewMaxTokens,
                    block::kFewMaxSlots, block::kFewMaxExperts);
    if (a->tokens == 0)
        return ok();
    const Pointer ptrs[] = {{a->x, "args.x", kPtrAlign, true},
                            {a->indices, "args.indices", 4, true},
                            {a->weights, "args.weights", 4, false},
                            {a->gate_up, "args.gate_up", kPtrAlign, true},
                            {a->gate_up_scales, "args.gate_up_scales", 4, true},
                            {a->down, "args.down", kPtrAlign, true},
                            {a->down_scales, "args.down_scales", 4, true},
                            {a->out, "args.out", kPtrAlign, true},
                            {a->workspace, "args.workspace", kPtrAlign, true}};
    const int rc = check_pointers(ptrs);
    if (rc != EP_OK)
        return rc;
    const int64_t need = (int64_t)few_bytes(a->tokens, a->topk, a->hidden, a->inter);
    if (a->workspace_bytes < need)
        return fail(EP_ERR_SIZE, "args.workspace_bytes = %lld: %lld are needed",
                    (long long)a->workspace_bytes, (long long)need);
    block::FewArgs fa;
    fa.x = static_cast<const uint8_t*>(a->x);
    fa.ids = a->indices;
    fa.w = a->weights;
    fa.up = static_cast<const uint8_t*>(a->gate_up);
    fa.ups = a->gate_up_scales;
    fa.down = static_cast<const uint8_t*>(a->down);
    fa.downs = a->down_scales;
    fa.out = static_cast<uint8_t*>(a->out);
    fa.act = static_cast<uint8_t*>(a->workspace);
    fa.T = a->tokens;
    fa.topk = a->topk;
    fa.E = a->experts;
    fa.H = a->hidden;
    fa.I = a->inter;
    fa.hits = std::min(a->experts, a->tokens * a->topk);
    // Pieces of inter in the down product, so that a single token's experts
    // occupy a block's waves; by topk alone, so that a token's sums are the
    // same in every call.
    fa.splits = a->topk >= 8 ? 1 : a->topk >= 4 ? 2 : 4;
    const hipError_t e = block::launch_few(fa, a->dtype == EP_BF16 ? 0 : 1,
                                           a->weight_dtype == MOE_INT8 ? 1 : 0,
                                           static_cast<hipStream_t>(stream_ptr));
    if (e != hipSuccess)
        return fail(EP_ERR_HIP, "few_tokens launch failed: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"
