"""moe_rms_norm on the GPU against the plain 64-bit form.

Bounds: the mean of squares is a sum of H nonnegative FP32 squares, added in
chains of 8, a tree of 6 levels and a chain of H / 512 chunks, so its relative
error is at most (8 + 6 + H / 512 + 2) half steps of binary32; the square root
halves it, the roots and the division add 3, the two products 2: at most
(16 + H / 512) / 2 + 5 half steps."""
import pytest
import torch

import combine_route_amd as cra
import moe_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def rel32(H):
    return ((16 + H / 512) / 2 + 5) * ref.F32


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def outputs(x, residual, out, quant, fill=77):
    """Sentinel-filled outputs."""
    H = x.shape[-1]

    def full(shape, dtype):
        return torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(dtype) \
            if dtype == torch.uint8 else torch.full(shape, float(fill), dtype=dtype, device="cuda")

    return dict(residual_out=full(x.shape, x.dtype) if residual else None,
                out=full(x.shape, x.dtype) if out else None,
                codes=full(x.shape, torch.uint8) if quant else None,
                scales=full(x.shape[:-1] + (H // 128,), torch.float32) if quant else None)


def check(x, w, eps, residual, o, rows=slice(None)):
    h, y = ref.rms_norm(x[rows], w, eps, None if residual is None else residual[rows])
    r = rel32(x.shape[-1])
    if residual is not None:
        assert torch.equal(o["residual_out"][rows].double(), h)
    if o["out"] is not None:
        ref.close_to(o["out"][rows], y, x.dtype, r)
    if o["codes"] is not None:
        ref.quantized_close(o["codes"][rows], o["scales"][rows], y, r)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,H", [(1, 8), (3, 128), (5, 136), (2, 512), (7, 520), (33, 1024),
                                    (130, 2048), (1, 7168), (257, 7168), (3, 8192), (5, 16384),
                                    (2, 65536), (9001, 256), (2050, 4096)])
def test_sizes(dtype, rows, H):
    x = rand((rows, H), dtype, 1)
    for seed, (res, out, quant, wt) in enumerate([(True, True, H % 128 == 0, dtype),
                                                  (False, True, False, torch.float32),
                                                  (False, H % 128 != 0, H % 128 == 0, dtype)]):
        w = rand((H,), wt, 2 + seed)
        residual = rand((rows, H), dtype, 9 + seed, 3.0) if res else None
        o = outputs(x, res, out, quant)
        cra.moe_rms_norm(x, w, 1e-5, residual=residual, **o)
        check(x, w, 1e-5, residual, o)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts", [[0, 5, 17, 3], [17, -3, 40, 1]])
@pytest.mark.parametrize("H", [256, 7168])
def test_counts_leave_other_rows_alone(dtype, counts, H):
    x, w = rand((4, 17, H), dtype, 3), rand((H,), dtype, 4)
    residual = rand((4, 17, H), dtype, 5)
    o = outputs(x, True, True, True)
    cra.moe_rms_norm(x, w, 1e-6, residual=residual, counts=torch.tensor(
        counts, dtype=torch.int32, device="cuda"), **o)
    for g, c in enumerate(counts):
        n = max(0, min(17, c))
        if n:
            check(x, w, 1e-6, residual, o, (g, slice(0, n)))
        for v in o.values():
            rest = v[g, n:]
            assert bool((rest == 77).all())


def test_in_place():
    x, w, res = rand((40, 7168), BF16, 6), rand((7168,), BF16, 7), rand((40, 7168), BF16, 8)
    o = outputs(x, True, True, True)
    cra.moe_rms_norm(x, w, 1e-6, residual=res, **o)
    x2, res2 = x.clone(), res.clone()
    cra.moe_rms_norm(x2, w, 1e-6, out=x2, residual=res2)
    assert torch.equal(x2, o["out"]) and torch.equal(res2, o["residual_out"])


@pytest.mark.parametrize("H", [1024, 7168])
def test_a_row_does_not_depend_on_the_call(H):
    """The same bits alone, in a small call and in a large one."""
    big = rand((9000, H), BF16, 10)
    w = rand((H,), BF16, 11)
    o = outputs(big, False, True, True)
    cra.moe_rms_norm(big, w, 1e-6, **o)
    for lo, hi in ((0, 1), (100, 140), (5000, 6500)):
        s = outputs(big[lo:hi], False, True, True)
        cra.moe_rms_norm(big[lo:hi].contiguous(), w, 1e-6, **s)
        for k in ("out", "codes", "scales"):
            assert torch.equal(s[k], o[k][lo:hi])


def test_zero_rows_and_special_values():
    H = 512
    x = rand((6, H), BF16, 12)
    x[0] = 0
    x[2, 7] = float("nan")
    x[4, 130] = float("inf")
    w = rand((H,), BF16, 13)
    o = outputs(x, False, True, True)
    cra.moe_rms_norm(x, w, 1e-6, **o)
    assert bool((o["out"][0] == 0).all()) and bool((o["scales"][0] == 1).all())
    assert bool((o["codes"][0].view(ref.E4M3).float() == 0).all())
    assert bool(o["out"][2].isnan().all())
    assert bool((o["codes"][2] == 0x7F).all())
    assert bool(o["out"][4, 130].isnan()) and int(o["codes"][4, 130]) == 0x7F
    check(x, w, 1e-6, None, o, [1, 3, 5])


def test_tiny_blocks_keep_a_finite_factor():
    H = 256
    x = rand((3, H), BF16, 14)
    w = torch.full((H,), 2.0 ** -110, device="cuda")
    w[128:] = 2.0 ** -60
    o = outputs(x, False, False, True)
    cra.moe_rms_norm(x, w, 1e-6, **o)
    check(x, w, 1e-6, None, o)
    assert bool((o["scales"][:, 0].double() - ref.TINY / 448).abs().le(
        ref.TINY / 448 * 2.0 ** -23).all())


def test_no_rows():
    x = torch.empty((3, 0, 256), dtype=BF16, device="cuda")
    w = rand((256,), BF16, 1)
    cra.moe_rms_norm(x, w, 1e-6, out=torch.empty_like(x),
                     counts=torch.zeros(3, dtype=torch.int32, device="cuda"))


def test_binding_refuses():
    x, w = rand((4, 256), BF16, 1), rand((256,), BF16, 2)
    out = torch.empty_like(x)
    with pytest.raises(ValueError, match="contiguous"):
        cra.moe_rms_norm(x[:, :128], w[:128], 1e-6, out=out[:, :128])
    with pytest.raises(ValueError, match="weight"):
        cra.moe_rms_norm(x, w[:128], 1e-6, out=out)
    with pytest.raises(ValueError, match="weight"):
        cra.moe_rms_norm(x, w.half(), 1e-6, out=out)
    with pytest.raises(ValueError, match="out"):
        cra.moe_rms_norm(x, w, 1e-6, out=out.float())
    with pytest.raises(ValueError, match="scales"):
        cra.moe_rms_norm(x, w, 1e-6, codes=torch.empty_like(x, dtype=torch.uint8),
                         scales=torch.empty((4, 1), device="cuda"))
    with pytest.raises(ValueError, match="counts"):
        cra.moe_rms_norm(x, w, 1e-6, out=out, counts=torch.zeros(4, device="cuda"))
    with pytest.raises(cra.EpError, match="out"):
        cra.moe_rms_norm(x, w, 1e-6)
    with pytest.raises(cra.EpError, match="multiple of 8"):
        cra.moe_rms_norm(x.view(-1)[:12].clone(), w[:12].clone(), 1e-6,
                         out=out.view(-1)[:12].clone())


def test_streams_and_graph():
    x, w, res = rand((300, 2048), FP16, 1), rand((2048,), FP16, 2), rand((300, 2048), FP16, 3)
    want = outputs(x, True, True, True)
    cra.moe_rms_norm(x, w, 1e-6, residual=res, **want)
    got = [outputs(x, True, True, True) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(streams, got):
        cra.moe_rms_norm(x, w, 1e-6, residual=res, stream=s, **o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cra.moe_rms_norm(x, w, 1e-6, residual=res, **got[2])
    for _ in range(3):
        for v in got[2].values():
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(got[2][k], v)
    for o in got[:2]:
        for k, v in want.items():
            assert torch.equal(o[k], v)
