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


NOT_TENSORS = ([[1.0] * 8] * 4, 3.0, "X", object())


@pytest.mark.parametrize("bad", NOT_TENSORS, ids=["list", "float", "str", "object"])
def test_what_is_no_tensor_is_a_type_error(t, bad):
    """As in the products: every operand of every layer, None where it may not
    be absent."""
    f, u, h = (lambda *s: t.ones(*s)), (lambda *s: t.zeros(*s, dtype=t.uint8)), t.float16
    good = {
        bd.linear_f32: dict(X=f(4, 8), W=f(8, 6), bias=f(6), residual=f(4, 6), Z=f(4, 6), Y=f(4, 6)),
        bd.linear_f32_bwd: dict(dY=f(4, 6), X=f(4, 8), W=f(8, 6), Z=f(4, 6), dX=f(4, 8), dW=f(8, 6), db=f(6),
                                workspace=u(1 << 14), act="silu"),
        bd.rmsnorm_f32: dict(X=f(4, 8), gamma=f(8), residual=f(4, 8), S=f(4, 8), Y=f(4, 8), rstd=f(4)),
        bd.rmsnorm_mx8: dict(X=f(4, 8), gamma=f(8), residual=f(4, 8), S=f(4, 8), Q=u(4, 8), E=u(4, 1)),
        bd.rmsnorm_f32_bwd: dict(dY=f(4, 8), S=f(4, 8), gamma=f(8), rstd=f(4), dS=f(4, 8), dX=f(4, 8), dgamma=f(8),
                                 workspace=u(1 << 14)),
        bd.linear_q4_mx8: dict(X8=u(4, 8), XE=u(4, 1), Q=u(6, 4), S=t.ones(6, 1, dtype=h), bias=f(6),
                               residual=f(4, 6), Y=f(4, 6), Y8=u(4, 6), YE=u(4, 1), out="both"),
    }
    required = ("X", "W", "dY", "S", "rstd", "X8", "XE", "Q")
    for fn, kw in good.items():
        for name in kw:
            if name in ("act", "out"):
                continue
            with pytest.raises(TypeError):
                fn(**dict(kw, **{name: bad}))
            if name not in required or (fn is bd.linear_f32_bwd and name != "dY") or \
                    (fn in (bd.rmsnorm_f32, bd.rmsnorm_mx8) and name != "X"):
                continue
            with pytest.raises((TypeError, ValueError, bd.GGError)) as e:
                fn(**dict(kw, **{name: None}))
            assert getattr(e.value, "status", None) != bd.GG_ERR_NO_DEVICE


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
def test_bias_gradient_alone_equals_the_full_call(act):
    import torch
    torch.manual_seed(0)
    dY, Z, X, W = (torch.randn(s, device="cuda") for s in ((50, 70), (50, 70), (50, 30), (30, 70)))
    full = bd.linear_f32_bwd(dY, X, W, Z=Z, act=act)
    dX, dW, db = bd.linear_f32_bwd(dY, None, None, Z=Z, act=act, want=("db",))
    assert dX is None and dW is None and torch.equal(db, full[2])
