"""The operators of include/moe_block.h on rows that lie more than 4 GiB behind
the start of their tensors: each is the same row's result in a small call, bit
for bit (a row's arithmetic does not depend on the call). Most rows are absent
by their counts, so that little is computed."""
import pytest
import torch

import combine_route_amd as cra

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
G, H, NEAR = 3, 4096, 5
M = 2 ** 32 // (2 * H * 2) + 1  # group 2 of bf16 rows begins past 4 GiB


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def rand(shape, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def far(near, rows=M):
    """near [G, NEAR, ...] as the first rows of groups of `rows` rows."""
    t = torch.zeros((G, rows) + near.shape[2:], dtype=near.dtype, device="cuda")
    t[:, :NEAR] = near
    return t


def counts():
    return torch.tensor([2, 0, NEAR], dtype=torch.int32, device="cuda")


def same(large, small):
    for g, n in enumerate([2, 0, NEAR]):
        assert torch.equal(large[g, :n], small[g, :n]), g
        assert not bool(large[g, n:n + 64].any()), g
    assert not bool(large[:, -64:].any())


def test_norm_and_its_gradient():
    y, res, go = (rand((G, NEAR, H), i) for i in range(3))
    w = rand((H,), 3)

    def forward(y, res):
        h, out = torch.zeros_like(y), torch.zeros_like(y)
        codes = torch.zeros(y.shape, dtype=torch.int8, device="cuda")
        scales = torch.zeros(y.shape[:2], device="cuda")
        cra.moe_block_norm(y, res, w, 1e-6, out=out, residual_out=h, post_weight=w, codes=codes,
                           scales=scales, counts=counts())
        return h, out, codes, scales

    def backward(y, h, go):
        gy, gr = torch.zeros_like(y), torch.zeros_like(y)
        gw, gp = torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
        cra.moe_block_norm_backward(y, h, 1e-6, gy, grad_out=go, grad_h=go, grad_residual=gr,
                                    pre_weight=w, post_weight=w, grad_pre_weight=gw,
                                    grad_post_weight=gp, counts=counts())
        return gy, gr, gw, gp

    small = forward(y, res)
    large_y = far(y)
    large = forward(large_y, far(res))
    for a, b in zip(large, small):
        same(a, b)
    small_g = backward(y, small[0], go)
    large_g = backward(large_y, large[0], far(go))
    for a, b in zip(large_g[:2], small_g[:2]):
        same(a, b)
    for a, b in zip(large_g[2:], small_g[2:]):  # sums over other blocks: by their 7 rows
        # at most 7 products of factors below 2^5 each, added in some order
        assert float((a - b).abs().max()) <= 7 * 7 * 2.0 ** -24 * 2 ** 10


def test_int8_rows_and_products():
    x = rand((G, NEAR, H), 10)
    K = H

    def quantized(x):
        codes = torch.zeros(x.shape, dtype=torch.int8, device="cuda")
        scales = torch.zeros(x.shape[:2], device="cuda")
        cra.moe_quantize_int8(x, codes, scales, counts())
        return codes, scales

    small = quantized(x)
    large = quantized(far(x, 2 * M))  # codes of one byte: twice the rows
    for a, b in zip(large, small):
        same(a, b)
    b = torch.randint(-127, 128, (G, 32, K), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(11)).to(torch.int8)
    sb = rand((G, 32), 12, torch.float32)
    for call, width in ((cra.moe_grouped_gemm_int8, 32), (cra.moe_grouped_gemm_int8_swiglu, 16)):
        outs = []
        for codes, scales in (small, large):
            out = torch.zeros(codes.shape[:2] + (width,), dtype=BF16, device="cuda")
            call(codes, scales, b, sb, out, counts())
            outs.append(out)
        same(outs[1], outs[0])


def test_product_rows_far_out():
    """Output rows past 4 GiB, of short rows of k."""
    n, k = H, 16
    a = torch.randint(-127, 128, (G, NEAR, k), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(20)).to(torch.int8)
    sa = rand((G, NEAR), 21, torch.float32)
    b = torch.randint(-127, 128, (G, n, k), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(22)).to(torch.int8)
    sb = rand((G, n), 23, torch.float32)
    outs = []
    for x, s in ((a, sa), (far(a), far(sa))):
        out = torch.zeros(x.shape[:2] + (n,), dtype=BF16, device="cuda")
        cra.moe_grouped_gemm_int8(x, s, b, sb, out, counts())
        outs.append(out)
    same(outs[1], outs[0])
