"""Numerics of moe_grouped_gemm on the GPU where they can go wrong: the swiglu
quotient far from zero."""
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
