"""Gradients where more than one dispatch goes forward before the first backward:
an op a layer, or the layer's dispatch again."""
import pytest
import torch

import combine_route_amd as cra
from test_gpu_moe_backward import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cra.load()


def backward(c, dispatch_id):
    """Both gradients of a case through its op, checked against the formula."""
    c.check_combine(*c.combine_backward(dispatch_id=dispatch_id))
    gp = torch.randn(c.y.shape, generator=torch.Generator().manual_seed(3)).to(c.dt)
    gx = torch.full((c.W, c.M, c.H), 7.0, dtype=c.dt, device="cuda")
    c.op.dispatch_standard_moe_backward(gp.cuda(), grad_x=gx, dispatch_id=dispatch_id)
    c.check_dispatch(gp, gx)


SIZES = dict(W=2, M=40, H=520, k=3, E=6, cap=15, dtype="bf16")


def test_layers_with_an_op_each():
    layers = [Case(seed=s, ntok=n, **SIZES) for s, n in ((1, None), (2, [17, 40]), (3, [40, 5]))]
    after = [c.op.dispatch_id for c in layers]
    for c, a in reversed(list(zip(layers, after))):
        backward(c, a)


def test_layers_that_share_an_op():
    """The first layer's backward is refused after the second's dispatch, and
    right once its own has run again."""
    first, second = Case(seed=4, **SIZES), Case(seed=5, ntok=[9, 33], **SIZES)
    op = second.op = first.op
    after = op.dispatch_id
    op.dispatch_standard_moe(second.x, None, None, second.dev_ids, second.ntok)
    with pytest.raises(cra.EpError, match="of dispatch 1") as e:
        first.combine_backward(dispatch_id=after)
    assert e.value.code == cra.EP_ERR_STATE
    with pytest.raises(cra.EpError, match="of dispatch 1"):
        op.dispatch_standard_moe_backward(first.y.cuda(), dispatch_id=after)
    backward(second, op.dispatch_id)
    op.dispatch_standard_moe(first.x, None, None, first.dev_ids, first.ntok)
    backward(first, op.dispatch_id)
