"""Numerics of moe_grouped_gemm on the GPU where they can go wrong: the swiglu
quotient far from zero, and sums whose large products cancel.

The rows form's first step (include/moe.h): of 8 neighbouring products each is cut
toward zero to a multiple of 2^(E - 13), E the largest sum of exponents among
the nonzero ones. The eight's sum of 7 losses is then below 7 * 2^(E - 13); the
rest is FP32."""
import pytest
import torch

import combine_route_amd as cra
import moe_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def quotient(gate, up):
    """(codes, scales) of rows of silu(gate) * up, one pair a row and equal over
    the row: the gate is block 0 of k alone and the up projection block 1."""
    rows = len(gate)
    a = torch.zeros((1, rows, 256))
    a[0, :, 0], a[0, :, 128] = gate.sign(), up.sign()
    b = torch.zeros((1, 256, 256))
    b[0, :128, 0], b[0, 128:, 128] = 1.0, 1.0
    codes = torch.full((1, rows, 128), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, rows, 1), 7.0, device="cuda")
    cra.moe_grouped_gemm_swiglu(
        a.to(ref.E4M3).cuda(), torch.stack((gate, up), -1).abs().view(1, rows, 2).cuda(),
        b.to(ref.E4M3).cuda(), torch.ones((1, 2, 2), device="cuda"), codes, scales)
    return codes[0].cpu().view(ref.E4M3).double(), scales.view(-1).cpu().double()


# Half steps of the scale: the quotient's exponential 4 (2 of the instruction, a
# rounding of each of its two factors' product), of which the sum with 1 takes at
# most its share, the sum 1, the reciprocal 2, two products 2, the division by 448 1.
HALF_STEPS = 10


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_quotient_holds_far_from_zero(sign):
    """The error does not grow with the gate: where the exponential is normal,
    whatever its argument."""
    gate = torch.cat((torch.linspace(-87, 87, 601), torch.tensor([2.0 ** -20, -2.0 ** -20])))
    gate = gate[gate != 0]
    up = torch.full_like(gate, sign * 2.0 ** 40)
    codes, scales = quotient(gate, up)
    z = gate.double() * torch.sigmoid(gate.double()) * up.double()
    off = (scales - z.abs() / 448).abs() / (z.abs() / 448) / ref.F32
    assert float(off.max()) <= HALF_STEPS * (1 + 2.0 ** -16), (float(off.max()),
                                                              float(gate[off.argmax()]))
    assert torch.equal(codes, (448 * z.sign())[:, None].expand_as(codes))


def test_the_quotient_past_the_exponentials_range():
    """Where exp(-gate) is 0 in FP32 the quotient is the gate, and where it is
    infinite 0."""
    big = torch.tensor([89.0, 200.0, 1e30, 3e38])
    up = torch.full_like(big, 2.0 ** -30)
    codes, scales = quotient(big, up)
    want = big.double() * 2.0 ** -30 / 448
    assert bool(((scales - want).abs() <= HALF_STEPS * ref.F32 * want).all())
    assert bool((codes == 448).all())
    codes, scales = quotient(-big, up)
    assert bool((scales == 1).all()) and bool((codes == 0).all())


def rows_form(a, b, dtype=torch.bfloat16):
    """Rows of E4M3 codes a [m, k], b [n, k] with scales of 1."""
    (m, k), n = a.shape, b.shape[0]
    out = torch.full((1, m, n), 7.0, dtype=dtype, device="cuda")
    cra.moe_grouped_gemm(a.view(ref.E4M3).cuda()[None], torch.ones((1, m, k // 128), device="cuda"),
                         b.view(ref.E4M3).cuda()[None],
                         torch.ones((1, -(-n // 128), k // 128), device="cuda"), out)
    return out[0].cpu()


def exponents(codes):
    e = (codes.to(torch.int32) >> 3) & 15
    return torch.where(e == 0, -6, e - 7)


def eights(a, b):
    """(products, the cut's step of each eight [m, n, k / 8]) in 64 bits."""
    (m, k), n = a.shape, b.shape[0]
    p = a.view(ref.E4M3).double()[:, None] * b.view(ref.E4M3).double()[None]
    e = exponents(a)[:, None] + exponents(b)[None]
    e = torch.where(p != 0, e, -100).view(m, n, k // 8, 8).amax(-1)
    return p.view(m, n, k // 8, 8), 2.0 ** (e - 13).double()


def codes(shape, lo, hi, seed):
    """Random codes of magnitude code lo <= c < hi and both signs."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(lo, hi, shape, generator=g, dtype=torch.uint8)
    return c | torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7


def code(v):
    return torch.tensor(v).to(ref.E4M3).view(torch.uint8)


SPREADS = [(0, 127, 0, 127), (0, 40, 0, 127), (0, 8, 0, 127), (1, 16, 0, 60), (0, 8, 0, 8)]


@pytest.mark.parametrize("spread", SPREADS, ids=str)
def test_one_eight_is_summed_as_stated(spread):
    """Every kind of code, subnormals setting the step among them: the row is the
    cut products' sum, rounded."""
    a = torch.zeros((300, 128), dtype=torch.uint8)
    b = torch.zeros((264, 128), dtype=torch.uint8)
    a[:, 40:48] = codes((300, 8), *spread[:2], seed=1)
    b[:, 40:48] = codes((264, 8), *spread[2:], seed=2)
    p, step = eights(a, b)
    want = (torch.trunc(p / step[..., None]) * step[..., None]).sum((-1, -2))
    assert torch.equal(rows_form(a, b), want.float().bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("spread", SPREADS, ids=str)
@pytest.mark.parametrize("k", [128, 1024])
def test_rows_keep_the_stated_bound(spread, k, dtype):
    a, b = codes((100, k), *spread[:2], seed=3), codes((72, k), *spread[2:], seed=4)
    if dtype == torch.float16:  # its range
        a, b = (torch.where((v & 127) >= 0x48, v - 0x20, v) for v in (a, b))
    p, step = eights(a, b)
    # FP32: the additions' half steps of the sum of magnitudes
    tol = 7 * step.sum(-1) + (4 * k ** 0.5 + 18) * ref.F32 * p.abs().sum((-1, -2))
    ref.close_to(rows_form(a, b, dtype), p.sum((-1, -2)), dtype, 0.0, tol)


@pytest.mark.parametrize("at", [(0, 8, 16), (0, 16, 64), (7, 8, 127), (64, 3, 90)])
def test_cancelling_products_of_different_eights_leave_the_rest(at):
    a = torch.zeros((15, 128), dtype=torch.uint8)
    b = torch.zeros((8, 128), dtype=torch.uint8)
    small = [2.0 ** (i - 6) for i in range(15)]  # 24 bits below 2^17, the largest's
    a[:, at[0]] = a[:, at[1]] = b[:, at[0]] = code(448.0)
    b[:, at[1]] = code(-448.0)
    a[:, at[2]] = code(small)
    b[:, at[2]] = code(1.0)
    want = torch.tensor(small).double()[:, None].expand(15, 8)
    assert torch.equal(rows_form(a, b).double(), want)


@pytest.mark.parametrize("at", [(0, 1, 2), (8, 15, 11), (0, 8, 16), (120, 3, 126)])
def test_the_swiglu_form_keeps_every_product(at):
    """Its sums are FP32's within an eight too: 448 * 448 - 448 * 448 + s is s."""
    small = [2.0 ** (i - 6) for i in range(9)]
    a = torch.zeros((9, 128), dtype=torch.uint8)
    b = torch.zeros((256, 128), dtype=torch.uint8)
    a[:, at[0]] = a[:, at[1]] = b[:, at[0]] = code(448.0)
    b[:, at[1]] = code(-448.0)
    a[:, at[2]] = code(small)
    b[:, at[2]] = code(1.0)
    scales = torch.full((1, 9, 1), 7.0, device="cuda")
    cra.moe_grouped_gemm_swiglu(
        a.view(ref.E4M3).cuda()[None], torch.ones((1, 9, 1), device="cuda"),
        b.view(ref.E4M3).cuda()[None], torch.ones((1, 2, 1), device="cuda"),
        torch.zeros((1, 9, 128), dtype=torch.uint8, device="cuda"), scales)
    s = torch.tensor(small).double()
    want = s * torch.sigmoid(s) * s / 448
    off = (scales.view(-1).cpu().double() - want).abs()
    assert bool((off <= HALF_STEPS * ref.F32 * want).all())
