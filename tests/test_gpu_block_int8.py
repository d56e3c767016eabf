"""The INT8 rows, the grouped INT8 product and its swiglu form on the GPU, and
an INT8 layer from the norm to the combine. The product's sums are exact, so
its bf16 rows are the definition's bit for bit: one conversion, two FP32
products, one rounding. fp16 rows take the second product and the rounding in
one: within half a step of the exact product of the row's scale and the FP32
value, which has 48 bits and is whole in 64."""
import pytest
import torch

import block_reference as ref
import combine_route_amd as cra
from moe_reference import F32 as HALF, close_to

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed), device="cuda")).to(dtype)


def codes(shape, seed, low=-127):
    return torch.randint(low, 128, shape, generator=gen(seed), device="cuda").to(torch.int8)


def counts_of(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


# ---- rows

@pytest.mark.parametrize("G,M,H", [(1, 1, 8), (2, 3, 16), (3, 5, 136), (1, 7, 520), (2, 40, 2048),
                                   (1, 9, 7168), (1, 3, 40960), (1, 2, 65536), (1, 9001, 264),
                                   (2, 9000, 4104)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantized_rows(G, M, H, dtype):
    x = rand((G, M, H), dtype, H)
    x[0, 0] = 0
    q = torch.full(x.shape, 77, dtype=torch.int8, device="cuda")
    s = torch.full((G, M), 77.0, device="cuda")
    cra.moe_quantize_int8(x, q, s)
    ref.int8_close(q, s, x.double(), 0.0)
    assert float(s[0, 0]) == 1.0 and bool((q.abs() <= 127).all())
    n = [M // 2 if g % 2 else M + 3 for g in range(G)]
    q2, s2 = torch.full_like(q, 77), torch.full_like(s, 77.0)
    cra.moe_quantize_int8(x, q2, s2, counts=counts_of(n))
    for g in range(G):
        c = min(n[g], M)
        assert torch.equal(q2[g, :c], q[g, :c]) and torch.equal(s2[g, :c], s[g, :c])
        assert bool((q2[g, c:] == 77).all() and (s2[g, c:] == 77).all())


def test_quantized_rows_without_numbers():
    x = rand((5, 1024), BF16, 1)
    x[0, 3], x[1, 1000], x[2, 5], x[2, 6] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[3] = 2.0 ** -126
    q, s = torch.full(x.shape, 77, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda")
    cra.moe_quantize_int8(x, q, s)
    assert bool((q[:4] == 0).all())
    assert bool(s[0].isnan()) and float(s[1]) == float("inf") and bool(s[2].isnan())
    assert float(s[3]) == float(torch.tensor(2.0 ** -100) / 127)
    ref.int8_close(q[4:], s[4:], x[4:].double(), 0.0)


# ---- products

def sums(a, b):
    return (a.double() @ b.double().t()).float()


def product_case(G, cap, n, k, seed, low=-127):
    return (codes((G, cap, k), seed, low), rand((G, cap), torch.float32, seed + 1).abs() * 0.01,
            codes((G, n, k), seed + 2, low), rand((G, n), torch.float32, seed + 3).abs() * 0.01)


def check_rows(case, out, n):
    a, sa, b, sb = case
    for g in range(a.shape[0]):
        m = max(0, min(a.shape[1], n[g]))
        cols = sb[g][None] * sums(a[g, :m], b[g])
        if out.dtype == BF16:
            want = (sa[g, :m, None] * cols).to(BF16)
            assert torch.equal(out[g, :m], want), (
                g, float((out[g, :m].double() - want.double()).abs().max()))
        else:
            close_to(out[g, :m], sa[g, :m, None].double() * cols.double(), FP16, 0.0)
        assert bool((out[g, m:] == 77).all()), g


def run_rows(case, n, dtype, stream=None):
    a, _, b, _ = case
    out = torch.full((a.shape[0], a.shape[1], b.shape[1]), 77.0, dtype=dtype, device="cuda")
    cra.moe_grouped_gemm_int8(*case, out, counts=counts_of(n), stream=stream)
    return out


@pytest.mark.parametrize("k", [16, 48, 64, 80, 128, 192, 272, 512, 1040, 2048])
@pytest.mark.parametrize("n", [8, 136, 264])
def test_sizes(k, n):
    case = product_case(3, 70, n, k, k + n)
    check_rows(case, run_rows(case, [70, 1, 33], BF16), [70, 1, 33])


@pytest.mark.parametrize("rows", [1, 5, 63, 64, 65, 128, 129, 192, 193, 255, 256, 257, 320, 700])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_row_counts(rows, dtype):
    case = product_case(2, 704, 520, 320, rows)
    n = [rows, rows // 3]
    check_rows(case, run_rows(case, n, dtype), n)


@pytest.mark.parametrize("n", [[0, 0, 0, 0, 0], [300, 0, -4, 7, 9999], [0, 0, 0, 0, 1]])
def test_counts(n):
    case = product_case(5, 310, 256, 256, 3)
    check_rows(case, run_rows(case, n, BF16), n)


def test_without_counts_many_groups_and_tiles():
    """More groups than threads of a block, more tiles than blocks, classes of
    every size in turn."""
    case = product_case(600, 6, 264, 64, 5)
    check_rows(case, run_rows(case, None, BF16), [6] * 600)
    case = product_case(40, 300, 1032, 448, 6)
    n = [(37 * g * g) % 301 for g in range(40)]
    check_rows(case, run_rows(case, n, FP16), n)


@pytest.mark.parametrize("counted", [False, True])
def test_more_groups_than_counts_are_held(counted):
    """Past 1024 groups the counts come from memory between tiles: of small
    groups, and of groups of several tiles and of every class."""
    for G, cap, n, k in ((1500, 5, 272, 64), (1100, 330, 272, 272)):
        case = product_case(G, cap, n, k, G)
        m = [(37 * g * g + g) % (cap + 9) - 4 for g in range(G)] if counted else None
        want = [max(0, min(cap, v)) for v in m] if counted else [cap] * G
        check_rows(case, run_rows(case, m, BF16), want)
        case = (case[0], case[1] * 8 / k ** 0.5, case[2], case[3])
        out = torch.full((G, cap, n // 2), 77.0, dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8_swiglu(*case, out, counts=counts_of(m))
        for g in [0, 1, 1023, 1024, 1025, G - 2, G - 1, *range(2, G, 61)]:
            z, err = swiglu_reference(case, want[g], g)
            close_to(out[g, :want[g]], z, BF16, 0.0, err)
            assert bool((out[g, want[g]:] == 77).all())


@pytest.mark.parametrize("G,cap,n,k,rows", [
    (8, 1100, 7168, 2048, [1100, 1000, 300, 64, 1024, 600, 700, 900]),
    (6, 800, 7168, 1024, [200, 190, 800, 130, 256, 769]),
    (64, 130, 7168, 1024, [(29 * g) % 131 for g in range(64)]),
    (8, 1100, 2048, 7168, [1024, 1100, 0, 300, 192, 512, 256, 700])])
def test_many_tiles_of_new_inputs(G, cap, n, k, rows):
    """Several tiles a block, of one class after another, over inputs that lie in
    no cache: the first slices of a tile take their time."""
    for seed in range(3):
        case = product_case(G, cap, n, k, 100 + seed)
        torch.empty(300_000_000, dtype=torch.uint8, device="cuda").fill_(seed)  # out of the caches
        check_rows(case, run_rows(case, rows, BF16), rows)


@pytest.mark.parametrize("rows", [[1100, 1000, 300, 64], [1024, 200, 700, 129]])
def test_many_tiles_of_gate_and_up(rows):
    for seed in range(3):
        case = product_case(4, 1100, 4096, 7168, 200 + seed)
        case = (case[0], case[1] * 8 / 7168 ** 0.5, case[2], case[3])
        torch.empty(300_000_000, dtype=torch.uint8, device="cuda").fill_(seed)
        out = torch.full((4, 1100, 2048), 77.0, dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8_swiglu(*case, out, counts=counts_of(rows))
        for g in range(4):
            z, err = swiglu_reference(case, rows[g], g)
            close_to(out[g, :rows[g]], z, BF16, 0.0, err)
            assert bool((out[g, rows[g]:] == 77).all())


def test_largest_sums_are_exact():
    """The longest k with the largest codes: 2^30 a sum, odd ones among them."""
    a = torch.full((1, 4, 65536), -128, dtype=torch.int8, device="cuda")
    b = torch.full((1, 8, 65536), -128, dtype=torch.int8, device="cuda")
    a[0, 1] = 127
    b[0, 3] = 127
    a[0, 2, 5] = -127
    one = torch.ones((1, 8), device="cuda")
    out = torch.zeros((1, 4, 8), dtype=BF16, device="cuda")
    case = (a, one[:, :4].contiguous(), b, one)
    cra.moe_grouped_gemm_int8(*case, out)
    check_rows(case, out, [4])
    # small sums of large products: what is left is whole
    a = codes((1, 64, 65536), 9)
    b = codes((1, 64, 65536), 10)
    a[0, :, 32768:] = -a[0, :, :32768]
    b[0, :, 32768:] = b[0, :, :32768]
    a[0, :, 7] += 1
    case = (a, torch.ones((1, 64), device="cuda"), b, torch.ones((1, 64), device="cuda"))
    out = torch.full((1, 64, 64), 77.0, dtype=FP16, device="cuda")
    cra.moe_grouped_gemm_int8(*case, out)
    check_rows(case, out, [64])


def test_scales_without_numbers_stay_in_their_row_and_column():
    case = product_case(1, 70, 264, 256, 12)
    a, sa, b, sb = case
    want = run_rows(case, None, BF16)
    sa[0, 3], sa[0, 4], sb[0, 100] = float("nan"), float("inf"), float("nan")
    out = run_rows(case, None, BF16)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 3:5] = False
    keep[0, :, 100] = False
    assert torch.equal(out[keep], want[keep])
    assert bool(out[0, 3].isnan().all() and out[0, :, 100].isnan().all())
    assert not bool(out[0, 4].isfinite().any())


def swiglu_reference(case, m, g):
    """z and a bound of its FP32 error: gate and up are each off by 3 half
    steps; silu's derivative is at most 1.1 and |g| times its logarithmic
    derivative at most 1 + |g|; the exponential and the quotient 8 more. Where
    exp(-gate) passes 2^128 it is infinite in binary32 and the formula's
    quotient 0, off by less than |gate| 2^-128."""
    a, sa, b, sb = case
    y = sa[g, :m, None].double() * sb[g][None].double() * (a[g, :m].double() @ b[g].double().t())
    gate, up = y.chunk(2, -1)
    z = gate * torch.sigmoid(gate) * up
    return z, (16 + 4 * gate.abs().clamp_max(100.0)) * HALF * z.abs() + \
        (gate * up).abs() * 2.0 ** -128


@pytest.mark.parametrize("inter", [8, 120, 128, 136, 264, 640])
@pytest.mark.parametrize("k", [16, 208, 1024])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_swiglu(inter, k, dtype):
    n = [270, 33, 0, 130]
    case = product_case(4, 272, 2 * inter, k, k + inter)
    case = (case[0], case[1] * 8 / k ** 0.5, case[2], case[3])
    out = torch.full((4, 272, inter), 77.0, dtype=dtype, device="cuda")
    cra.moe_grouped_gemm_int8_swiglu(*case, out, counts=counts_of(n))
    for g in range(4):
        z, err = swiglu_reference(case, n[g], g)
        close_to(out[g, :n[g]], z, dtype, 0.0, err)
        assert bool((out[g, n[g]:] == 77).all())


def test_swiglu_of_large_gates():
    """Gates past the exponential's range: silu is 0 or the gate itself."""
    a = torch.ones((1, 2, 16), dtype=torch.int8, device="cuda")
    b = torch.zeros((1, 16, 16), dtype=torch.int8, device="cuda")
    b[0, :, 0] = torch.tensor([1, -1, 2, -2, 100, -100, 127, -127] + [1] * 8, dtype=torch.int8)
    sa, sb = torch.tensor([[1.0, 50.0]], device="cuda"), torch.ones((1, 16), device="cuda")
    out = torch.zeros((1, 2, 8), dtype=BF16, device="cuda")
    cra.moe_grouped_gemm_int8_swiglu(a, sa, b, sb, out)
    for r, s in enumerate((1.0, 50.0)):
        g = s * b[0, :8, 0].double()
        z = g * torch.sigmoid(g) * s
        close_to(out[0, r], z, BF16, 512 * HALF, 1e-35)


def test_streams_and_graphs():
    case = product_case(4, 300, 520, 256, 31)
    n = [300, 20, 0, 129]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            out = run_rows(case, n, BF16, stream)
        torch.cuda.synchronize()
        check_rows(case, out, n)
    cnt = counts_of(n)
    out = torch.full((4, 300, 520), 77.0, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cra.moe_grouped_gemm_int8(*case, out, counts=cnt)
    for seed, n in ((1, [1, 300, 256, 0]), (2, [64, 65, 300, 300]), (3, [0, 0, 0, 5])):
        case[0].copy_(codes(case[0].shape, seed))
        cnt.copy_(counts_of(n))
        out.fill_(77.0)
        run_rows(case, n, BF16)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(case, out, n)
