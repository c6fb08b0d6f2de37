"""The layers' Python binding on the CPU: tensors in host memory pass for ones
on the current device, and calls whose arguments are all valid stop at the
library's device check.  Skipped where there is a GPU, which they would reach."""
import pytest

from gemv_gemm_f32_amd import binding as bd
from test_abi import _gpu_present


@pytest.fixture
def t(monkeypatch):
    if _gpu_present():
        pytest.skip("a valid call on host memory would launch on the GPU")
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # get_device() of a CPU tensor
    monkeypatch.setattr(bd, "_stream", lambda stream, dev=None: 0)
    return torch


def reaches_the_device_check(call):
    with pytest.raises(bd.GGError) as e:
        call()
    assert e.value.status == bd.GG_ERR_NO_DEVICE, e.value


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("tw", [False, True])
def test_wanted_gradients_need_no_more_than_they_read(t, act, tw):
    dY, X, W = t.ones(4, 6), t.ones(4, 8), t.ones((6, 8) if tw else (8, 6))
    Z = t.ones(4, 6) if act != "none" else None

    def bwd(X, W, *want):
        return lambda: bd.linear_f32_bwd(dY, X, W, Z=Z, act=act, trans_w=tw, want=want)
    reaches_the_device_check(bwd(None, None, "db"))
    reaches_the_device_check(bwd(X, None, "dW", "db"))
    reaches_the_device_check(bwd(None, W, "dX", "db"))
    for call in (bwd(None, W, "dW"), bwd(X, None, "dX"), bwd(None, None, "dX", "dW")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
def test_bias_gradient_alone_equals_the_full_call(act):
    import torch
    torch.manual_seed(0)
    dY, Z, X, W = (torch.randn(s, device="cuda") for s in ((50, 70), (50, 70), (50, 30), (30, 70)))
    full = bd.linear_f32_bwd(dY, X, W, Z=Z, act=act)
    dX, dW, db = bd.linear_f32_bwd(dY, None, None, Z=Z, act=act, want=("db",))
    assert dX is None and dW is None and torch.equal(db, full[2])
