"""moe_few_tokens on the GPU against the plain 64-bit layer; the bound is
block_reference.few_tokens's."""
import pytest
import torch

import block_reference as ref
import combine_route_amd as cra
from moe_reference import close_to

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def make(E, T, k, H, I, dtype, kind, seed, repeats=False, weighted=True):
    g = torch.Generator().manual_seed(seed)

    def weights(n, cols):
        if kind == "int8":
            return (torch.randint(-127, 128, (E, n, cols), generator=g).to(torch.int8).cuda(),
                    ((0.5 + torch.rand((E, n), generator=g)) * cols ** -0.5 / 73).cuda())
        c = torch.randn((E, n, cols), generator=g) * 60
        return (c.clamp(-448, 448).to(E4M3).cuda(),
                ((0.5 + torch.rand((E, n // 128, cols // 128), generator=g)) * cols ** -0.5 /
                 60).cuda())

    if repeats:
        ids = torch.randint(-2, E + 2, (T, k), generator=g)
    else:
        ids = torch.rand((T, E), generator=g).argsort(-1)[:, :k]
    s = dict(x=torch.randn((T, H), generator=g).to(dtype).cuda(), ids=ids.to(torch.int32).cuda(),
             w=torch.rand((T, k), generator=g).cuda() if weighted else None)
    s["up"], s["ups"] = weights(2 * I, H)
    s["down"], s["downs"] = weights(H, I)
    return s


def run(s, workspace=None, stream=None, rows=slice(None)):
    x, ids = s["x"][rows].contiguous(), s["ids"][rows].contiguous()
    w = None if s["w"] is None else s["w"][rows].contiguous()
    out = torch.full_like(x, 77.0)
    cra.moe_few_tokens(x, ids, w, s["up"], s["ups"], s["down"], s["downs"], out,
                       workspace=workspace, stream=stream)
    return out


def check(s, out, rows=slice(None)):
    w = None if s["w"] is None else s["w"][rows]
    want, err = ref.few_tokens(s["x"][rows], s["ids"][rows], w, ref.weights_of(s["up"], s["ups"]),
                               ref.weights_of(s["down"], s["downs"]))
    close_to(out, want, s["x"].dtype, 0.0, err)


@pytest.mark.parametrize("E,T,k,H,I", [
    (1, 1, 1, 128, 128), (4, 1, 2, 256, 128), (8, 2, 3, 128, 384), (16, 5, 4, 640, 256),
    (8, 16, 8, 384, 128), (4, 17, 2, 256, 128), (2, 33, 1, 128, 128), (3, 64, 2, 256, 256),
    (40, 64, 16, 128, 128), (1, 64, 1, 384, 128), (256, 3, 8, 128, 128), (70, 20, 37, 128, 128),
    (16, 16, 64, 128, 128), (6, 2, 6, 4224, 128), (2, 3, 2, 128, 8320)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_sizes(E, T, k, H, I, dtype, kind):
    s = make(E, T, min(k, E) if k <= E else k, H, I, dtype, kind, E + T + H, repeats=k > E)
    check(s, run(s))


@pytest.mark.parametrize("E,T,k,H,I", [
    (1, 1, 1, 16, 16), (4, 3, 2, 48, 80), (5, 20, 3, 144, 16), (3, 64, 2, 272, 112),
    (4, 2, 4, 4112, 48), (3, 5, 2, 16, 4112)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_sizes_off_128(E, T, k, H, I, dtype):
    s = make(E, T, k, H, I, dtype, "int8", E + T + H)
    check(s, run(s))


@pytest.mark.parametrize("E,T,k,I", [(3, 1, 2, 48), (8, 4, 4, 160), (20, 4, 8, 400)])
@pytest.mark.parametrize("H", [6160, 7152, 6176])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_output_columns_that_end_inside_a_block(E, T, k, I, H, dtype):
    """32 output columns a block, of which the last may have 16."""
    s = make(E, T, k, H, I, dtype, "int8", E + H)
    check(s, run(s))


@pytest.mark.parametrize("E", [300, 5000, 65536])
@pytest.mark.parametrize("T,k", [(9, 3), (64, 3), (64, 16)])
def test_many_experts(E, T, k):
    """Of few slots and of many, to the last expert there can be."""
    s = make(E, T, k, 16, 16, BF16, "int8", E + T)
    s["ids"][T - 1, 0] = E - 1
    s["ids"][0, k - 1] = E - 1
    check(s, run(s))


@pytest.mark.parametrize("E,T,k,H,I", [
    (1, 1, 1, 33280, 128), (2, 6, 1, 33280, 128), (8, 2, 8, 128, 8320), (8, 6, 8, 128, 8320),
    (8, 1, 8, 256, 16512)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_more_steps_than_scales_are_held(E, T, k, H, I, dtype, kind):
    """Over 64 steps of k a wave, in gate and up and in down, of few columns and
    of many: FP8 scales are fetched again on the way."""
    s = make(E, T, k, H, I, dtype, kind, T + H)
    check(s, run(s))


@pytest.mark.parametrize("E,T,k,H,I,kind", [
    (100, 64, 8, 128, 384, "fp8"), (100, 64, 8, 128, 512, "int8"), (60, 30, 4, 256, 1024, "fp8"),
    (60, 50, 8, 144, 400, "int8"), (40, 16, 3, 128, 2048, "int8"), (60, 8, 8, 6272, 640, "fp8"),
    (80, 64, 16, 128, 640, "fp8")])
def test_many_experts_of_few_and_many_columns(E, T, k, H, I, kind):
    """Experts of 1 to 4 columns follow each other and ones of more, in a wave;
    every eighth is named more often."""
    s = make(E, T, k, H, I, BF16, kind, E + I)
    g = torch.Generator().manual_seed(I)
    score = torch.rand((T, E), generator=g) + 0.3 * (torch.arange(E) % 8 == 3)
    s["ids"] = score.argsort(-1, descending=True)[:, :k].to(torch.int32).cuda()
    for _ in range(2):
        check(s, run(s))


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T", [1, 9, 40])
def test_repeated_and_foreign_ids(kind, weighted, T):
    s = make(3, T, 6, 256, 128, BF16, kind, T, repeats=True, weighted=weighted)
    s["ids"][0] = torch.tensor([7, -1, 3, 2 ** 31 - 1, -2 ** 31, 99])
    out = run(s)
    check(s, out)
    assert bool((out[0] == 0).all())
    s["ids"].fill_(-1)
    assert bool((run(s) == 0).all())
    s["ids"].fill_(1)   # one expert, named by every slot
    check(s, run(s))


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_only_the_experts_hit_are_read(kind):
    """Weights and scales of the others hold NaN."""
    s = make(12, 4, 2, 256, 128, FP16, kind, 3)
    s["ids"].copy_(torch.tensor([[1, 5], [5, 9], [9, 1], [5, 1]]))
    want = run(s)
    other = [e for e in range(12) if e not in (1, 5, 9)]
    for e in other:
        for n in ("ups", "downs"):
            s[n][e] = float("nan")
        if kind == "fp8":
            for n in ("up", "down"):
                s[n].view(torch.uint8)[e] = 0x7F
    assert torch.equal(run(s), want)
    check({**s, **{n: torch.nan_to_num(s[n]) for n in ("ups", "downs")},
           **({n: torch.where(s[n].view(torch.uint8) == 0x7F, 0, s[n].view(torch.uint8)).view(E4M3)
               for n in ("up", "down")} if kind == "fp8" else {})}, want)


def test_values_that_are_no_numbers_stay_in_their_token():
    s = make(4, 6, 2, 256, 128, BF16, "fp8", 5)
    want = run(s)
    s["x"][2, 100] = float("nan")
    s["x"][4, 17] = float("inf")
    out = run(s)
    for t in range(6):
        if t == 2:
            assert bool(out[t].isnan().all())
        elif t == 4:
            assert not bool(out[t].isfinite().any())
        else:
            assert torch.equal(out[t], want[t])


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [1, 7])
def test_hidden_values_between_the_largest_of_bf16_and_of_binary32(kind, dtype, T):
    """Finite hidden values that round to infinity in bf16: (2 - 2^-20) 2^127, the
    gate 2^64 (silu gives it back), down a diagonal of 2^-100."""
    n = 128
    x = torch.zeros((T, n), dtype=dtype, device="cuda")
    x[:, 0] = 1.0
    sign = torch.tensor([(1.0, -1.0, 0.0)[i % 3] for i in range(n)])
    up = torch.zeros((1, 2 * n, n))
    up[0, :n, 0] = 1.0
    up[0, n:, 0] = sign
    s = dict(x=x, ids=torch.zeros((T, 1), dtype=torch.int32, device="cuda"), w=None)
    one = (lambda t: t.to(torch.int8)) if kind == "int8" else (lambda t: t.to(E4M3))
    s["up"], s["down"] = one(up).cuda(), one(torch.eye(n)[None]).cuda()
    each = n if kind == "int8" else 1
    s["ups"] = torch.cat((torch.full((1, each), 2.0 ** 64),
                          torch.full((1, each), (2.0 - 2.0 ** -20) * 2.0 ** 63)), 1).cuda()
    s["downs"] = torch.full((1, each), 2.0 ** -100).cuda()
    if kind == "fp8":
        s["ups"], s["downs"] = s["ups"][..., None].contiguous(), s["downs"][..., None].contiguous()
    scale = 2.0 ** -15 if dtype == FP16 else 1.0  # 2^28 is no fp16 number
    s["downs"] *= scale
    out = run(s)
    check(s, out)
    want = (sign * 2.0 ** 28 * scale).to(dtype).cuda()
    assert torch.equal(out, want.expand(T, n))


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("dtype,scale", [(FP16, 2.0 ** -20), (BF16, 2.0 ** -128)])
@pytest.mark.parametrize("T", [1, 9])
def test_values_below_the_normal_range_count(kind, dtype, scale, T):
    """Rows of x that lie below the type's normal range are not taken for zero."""
    s = make(4, T, 2, 256, 128, dtype, kind, 11)
    s["x"].mul_(scale)
    assert bool((s["x"] != 0).any()) and float(s["x"].abs().max()) < torch.finfo(dtype).tiny
    s["ups"] /= scale if dtype == FP16 else 2.0 ** -100
    s["downs"] /= 1.0 if dtype == FP16 else 2.0 ** -56
    out = run(s)
    check(s, out)
    assert bool((out != 0).any())


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("k", [2, 5, 8])
def test_a_token_alone_is_the_token_in_a_batch(kind, k):
    s = make(10, 64, k, 384, 256, BF16, kind, 7)
    many = run(s)
    for rows in (slice(0, 1), slice(63, 64), slice(5, 21), slice(10, 27), slice(20, 55)):
        assert torch.equal(run(s, rows=rows), many[rows]), rows


def test_no_tokens_leading_sizes_and_workspace():
    s = make(4, 6, 2, 256, 128, BF16, "fp8", 5)
    want = run(s)
    out = torch.zeros((2, 3, 256), dtype=BF16, device="cuda")
    ws = torch.empty(cra.moe_few_tokens_workspace_bytes(6, 2, 256, 128), dtype=torch.uint8,
                     device="cuda")
    cra.moe_few_tokens(s["x"].view(2, 3, 256), s["ids"].view(2, 3, 2), s["w"].view(2, 3, 2),
                       s["up"].view(torch.uint8), s["ups"], s["down"].view(torch.uint8),
                       s["downs"], out, workspace=ws)
    assert torch.equal(out.view(6, 256), want)
    run(s, rows=slice(0, 0))
    with pytest.raises(ValueError, match="workspace holds"):
        run(s, workspace=ws[:-1])
    with pytest.raises(ValueError, match="down"):
        cra.moe_few_tokens(s["x"], s["ids"], None, s["up"], s["ups"],
                           s["down"].view(torch.int8), s["downs"], torch.empty_like(s["x"]))
    with pytest.raises(ValueError, match="indices"):
        cra.moe_few_tokens(s["x"], s["ids"].long(), None, s["up"], s["ups"], s["down"],
                           s["downs"], torch.empty_like(s["x"]))
    with pytest.raises(cra.EpError, match="tokens"):
        cra.moe_few_tokens(s["x"].repeat(11, 1), s["ids"].repeat(11, 1), None, s["up"], s["ups"],
                           s["down"], s["downs"], s["x"].repeat(11, 1))


def test_streams_and_graphs():
    s = make(8, 5, 3, 256, 128, BF16, "fp8", 31)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            out = run(s, stream=stream)
        torch.cuda.synchronize()
        check(s, out)
    ws = torch.empty(cra.moe_few_tokens_workspace_bytes(5, 3, 256, 128), dtype=torch.uint8,
                     device="cuda")
    out = torch.full_like(s["x"], 77.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cra.moe_few_tokens(s["x"], s["ids"], s["w"], s["up"], s["ups"], s["down"], s["downs"], out,
                           workspace=ws)
    for seed in range(3):
        new = make(8, 5, 3, 256, 128, BF16, "fp8", 40 + seed, repeats=seed == 1)
        for n in ("x", "ids", "w"):
            s[n].copy_(new[n])
        want = run(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        check(s, out)


def test_is_near_the_layer_of_a_dispatch():
    """The FP8 layer through dispatch, experts and combine: the same weights,
    rows quantized on the way (E4M3, half a step 2^-4 of a value at most, twice)."""
    W, M, H, I, ER, K = 2, 4, 256, 128, 4, 2
    s = make(W * ER, W * M, K, H, I, BF16, "fp8", 9)
    few = run(s)
    op = cra.EpDispatchCombineOp(cra.make_config(W, H, M, ER, K, "fp8", "bf16", scale_dim=2),
                                 with_weights=False, expert_capacity=W * M)
    codes = torch.empty((W, M, H), dtype=E4M3, device="cuda")
    scales = torch.empty((W, M, H // 128), device="cuda")
    one = torch.ones(H, device="cuda")
    # x is nearly of unit mean square: the norm changes it little, and both see its result
    n = torch.empty((W, M, H), dtype=BF16, device="cuda")
    cra.moe_rms_norm(s["x"].view(W, M, H), one, 0.0, out=n, codes=codes, scales=scales)
    s["x"].copy_(n.view(-1, H))
    few = run(s)
    ids, w = s["ids"].view(W, M, K), s["w"].view(W, M, K)
    px, count, _, _ = op.dispatch_standard_moe(codes, None, scales, ids)
    y = op.expert_mlp(px, count, s["up"], s["ups"], s["down"], s["downs"])
    out = op.combine_standard_moe(y, w, ids).view(-1, H)
    torch.cuda.synchronize()
    off = float((out.double() - few.double()).norm() / few.double().norm())
    assert off <= 4 * 2.0 ** -4, off
    op.close()
