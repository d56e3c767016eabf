"""Which dispatch a backward call is of, without a GPU: the library's calls are
stand-ins."""
from types import SimpleNamespace as Fields

import pytest
import torch

import combine_route_amd as cra


@pytest.fixture
def op(monkeypatch):
    """An op whose library calls record their names."""
    op = object.__new__(cra.EpDispatchCombineOp)
    op.cfg = cra.make_config(2, 64, 4, 2, 2)
    op.expert_capacity, op.plan, op._dev_index, op._ex = 8, None, 0, None
    op.workspace = Fields(device=torch.device("cpu"))
    op.calls = []
    op._lib = Fields(ep_dispatch_standard_moe=lambda *a: op.calls.append("dispatch") or 0)
    names = ("packed_x", "packed_scales", "packed_count", "packed_src_info",
             "packed_layout_range")
    monkeypatch.setattr(op, "_expert_state", lambda: op._ex, raising=False)
    monkeypatch.setattr(cra, "_dispatch_standard_args",
                        lambda *a: (cra.EpDispatchStandardArgs(), None))
    monkeypatch.setattr(cra, "ep_expert_plan_destroy", lambda plan: None)
    for name in ("moe_combine_backward", "moe_dispatch_backward"):
        monkeypatch.setattr(cra, name, lambda *a, name=name, **kw: op.calls.append(name))
    op.fresh = lambda: op.__dict__.update(_ex=dict.fromkeys(names, None) | {"plan": 7})
    yield op
    op._ex = None


def test_a_backward_of_an_earlier_dispatch_is_refused(op):
    x, ids = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 2),
                                                                        dtype=torch.int32)
    assert op.dispatch_id == 0
    op.fresh()
    assert op.dispatch_id == 0
    after = []
    for _ in range(2):
        op.dispatch_standard_moe(x, None, None, ids, stream=1)
        after.append(op.dispatch_id)
    assert after == [1, 2]
    op.calls.clear()

    def backward(dispatch_id):
        op.combine_standard_moe_backward(x, None, ids, grad_packed_y=x, stream=1,
                                         dispatch_id=dispatch_id)
        op.dispatch_standard_moe_backward(x, grad_x=x, stream=1, dispatch_id=dispatch_id)

    backward(2)
    backward(None)
    assert op.calls == ["moe_combine_backward", "moe_dispatch_backward"] * 2
    op.calls.clear()
    for call in (lambda: op.combine_standard_moe_backward(x, None, ids, grad_packed_y=x, stream=1,
                                                          dispatch_id=1),
                 lambda: op.dispatch_standard_moe_backward(x, grad_x=x, stream=1, dispatch_id=1)):
        with pytest.raises(cra.EpError, match="of dispatch 1: .* the map of dispatch 2") as e:
            call()
        assert e.value.code == cra.EP_ERR_STATE
    assert op.calls == []
