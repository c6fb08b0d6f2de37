"""GPU parity of linear_f32 and linear_f32_bwd against 64-bit references,
through the C ABI, with tolerances counted in fp32 roundings (layer_refs)."""
import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu


def _layer(rng, M, N, K, tw, bias=True, residual=True):
    X = inputs.normal(rng, (M, K))
    W = inputs.normal(rng, (N, K) if tw else (K, N), max(K, 1) ** -0.5)
    b = inputs.normal(rng, (N,)) if bias else None
    R = inputs.normal(rng, (M, N)) if residual else None
    return X, W, b, R


def _d(a):
    return None if a is None else dev(a)


def _check(M, N, K, tw, act, bias=True, residual=True, keep=True, seed=0):
    rng = np.random.default_rng([seed, M, N, K, tw])
    X, W, b, R = _layer(rng, M, N, K, tw, bias, residual)
    Z = torch().full((M, N), 7.0, device="cuda") if keep else None
    Y = bd.linear_f32(dev(X), dev(W), bias=_d(b), act=act, residual=_d(R), Z=Z, trans_w=bool(tw))
    z, y, ez, ey = lr.linear(X, W, b, R, act, tw)
    what = "%dx%dx%d tw%d %s" % (M, N, K, tw, act)
    if keep:
        lr.within(host(Z), z, ez, what + " Z")
    lr.within(host(Y), y, ey, what + " Y")


SHAPES = [(1, 1, 1), (1, 96, 64), (2, 33, 5), (3, 2304, 768), (5, 1000, 333), (7, 64, 2048),
          (8, 100, 100), (9, 128, 64), (16, 257, 129), (33, 65, 31), (64, 64, 64), (129, 67, 33),
          (346, 768, 768), (500, 500, 200), (1024, 48, 100), (1, 5000, 7), (4, 31, 4100)]


@pytest.mark.parametrize("tw", [0, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, tw):
    _check(M, N, K, tw, "gelu_tanh")


@pytest.mark.parametrize("tw", [0, 1])
@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 260, 132), (40, 100, 52), (700, 520, 96), (2100, 1030, 40)])
def test_activations(act, tw, M, N, K):
    _check(M, N, K, tw, act)


@pytest.mark.parametrize("M", [1, 6, 70])
@pytest.mark.parametrize("bias,residual,keep", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)])
def test_absent_operands(M, bias, residual, keep):
    for tw in (0, 1):
        _check(M, 90, 70, tw, "silu", bias, residual, keep)


@pytest.mark.parametrize("M", [1, 4, 50])
def test_without_epilogue_equals_the_product(M):
    """No bias, activation or residual: within roundings of gemm_f32."""
    rng = np.random.default_rng(M)
    X, W, _, _ = _layer(rng, M, 200, 300, 0)
    _, y, _, ey = lr.linear(X, W, None, None, "none", 0)
    lr.within(host(bd.gemm_f32(dev(X), dev(W))), y, ey)
    lr.within(host(bd.linear_f32(dev(X), dev(W))), y, ey)


@pytest.mark.parametrize("M", [1, 3, 70])
@pytest.mark.parametrize("tw", [0, 1])
def test_k_zero_is_the_bias(M, tw):
    t = torch()
    X = t.empty((M, 0), device="cuda")
    W = t.empty((40, 0) if tw else (0, 40), device="cuda")
    b = inputs.normal(np.random.default_rng(1), (40,))
    Y = host(bd.linear_f32(X, W, bias=dev(b), act="relu", trans_w=bool(tw)))
    assert np.array_equal(Y, np.tile(np.maximum(b, 0), (M, 1)))


@pytest.mark.parametrize("M", [1, 2, 8, 40])
@pytest.mark.parametrize("tw", [0, 1])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_offsets_and_what_lies_around(M, tw, shift):
    """Every operand a view with padded rows, off 16-byte alignment when
    shift; nothing outside the outputs is written, and NaN around the inputs
    is not read into results."""
    t = torch()
    rng = np.random.default_rng(8)
    N, K = 75, 133
    X, W, b, R = _layer(rng, M, N, K, tw)

    def view(a, fill=float("nan")):
        a2 = a if a.ndim == 2 else a[None]
        buf = t.full((a2.shape[0], a2.shape[1] + 4 + shift), fill, device="cuda")
        v = buf[:, 1 + shift:1 + shift + a2.shape[1]]
        v.copy_(dev(a2))
        return v if a.ndim == 2 else v[0]
    buf, _ = guarded(M, N + 7)
    Y = buf[64:64 + M * (N + 7)].view(M, N + 7)[:, :N]
    bufz, _ = guarded(M, N + 5)
    Z = bufz[64:64 + M * (N + 5)].view(M, N + 5)[:, :N]
    bd.linear_f32(view(X), view(W), bias=view(b), act="gelu_erf", residual=view(R), Z=Z, Y=Y,
                  trans_w=bool(tw))
    z, y, ez, ey = lr.linear(X, W, b, R, "gelu_erf", tw)
    lr.within(host(Z), z, ez)
    lr.within(host(Y), y, ey)
    for whole, w in ((buf, N + 7), (bufz, N + 5)):
        assert canaries_intact(whole)
        assert np.all(host(whole)[64:64 + M * w].reshape(M, w)[:, N:] == np.float32(1.2345e9))


@pytest.mark.parametrize("M", [1, 5, 300])
def test_residual_updated_in_place(M):
    rng = np.random.default_rng(2)
    X, W, b, R = _layer(rng, M, 260, 128, 1)
    dR = dev(R)
    out = bd.linear_f32(dev(X), dev(W), bias=dev(b), residual=dR, Y=dR, trans_w=True)
    fresh = bd.linear_f32(dev(X), dev(W), bias=dev(b), residual=dev(R), trans_w=True)
    assert out.data_ptr() == dR.data_ptr() and np.array_equal(host(dR), host(fresh))


@pytest.mark.parametrize("M", [1, 4, 64])
@pytest.mark.parametrize("act", lr.ACTS)
def test_nonfinite(M, act):
    """A NaN in X reaches its own row only; +inf pre-activations stay +inf,
    -inf follows the formula (0 for ReLU, -inf without activation, NaN
    otherwise)."""
    X = np.ones((M, 8), np.float32)
    W = np.zeros((8, 3), np.float32)
    W[0] = [1, -1, 0.5]
    X[M // 2, 0] = np.inf
    W[1:, :] = 0
    Y = host(bd.linear_f32(dev(X), dev(W), act=act))
    row = Y[M // 2]
    assert row[0] == np.inf
    if act == "relu":
        assert row[1] == 0
    elif act == "none":
        assert row[1] == -np.inf
    else:
        assert np.isnan(row[1])
    X[M // 2, 0] = np.nan
    Y = host(bd.linear_f32(dev(X), dev(W), act=act))
    assert np.isnan(Y[M // 2]).all() and np.isfinite(np.delete(Y, M // 2, 0)).all()


@pytest.mark.parametrize("act", lr.ACTS)
def test_activation_over_its_range(act):
    """X.W = z exactly (K = 1, W = 1): the activation alone, over tails and
    the neighbourhood of zero."""
    z = np.concatenate([np.linspace(-120, 120, 4001), np.linspace(-12, 12, 4001),
                        [0.0, 1e-30, -1e-30, 1e30, -1e30, 3e38, -3e38]]).astype(np.float32)
    Y = host(bd.linear_f32(dev(z[:, None]), dev(np.ones((1, 1), np.float32)), act=act))[:, 0]
    with np.errstate(over="ignore", invalid="ignore"):
        ref = np.where(np.abs(z) > 1e20, np.where(z > 0, z.astype(np.float64), 0.0),
                       lr.act(np.where(np.abs(z) > 1e20, 0.0, z.astype(np.float64)), act))
    if act == "none":
        ref = z.astype(np.float64)
    bound = 0 if act in ("none", "relu") else lr.ACT_ERR * np.abs(z.astype(np.float64)) + 1e-44
    # far in the left tail p underflows: |z p| is below 1e-36 there
    bound = bound + (0 if act in ("none", "relu") else np.where(z < -80, 1e-30, 0) * np.minimum(np.abs(z), 1e3))
    small = np.abs(z) < 1e30
    lr.within(Y[small], ref[small], (np.zeros_like(ref) + bound)[small], act)
    big = ~small & (z > 0)
    assert np.array_equal(Y[big], z[big])


# -------------------------------------------------------------- backward --

def _grads(dY, Z, X, W, act, tw):
    """dX, dW, db and the bounds of their errors."""
    s = lr.slope(Z, act)
    dY, X = dY.astype(np.float64), X.astype(np.float64)
    dZ = dY * s
    edz = (np.abs(dY) * lr.SLOPE_ERR if act not in ("none", "relu") else 0 * dY) + lr.U * np.abs(dZ)
    Wk = (W.T if tw else W).astype(np.float64)                  # K x N
    M, N = dY.shape
    dX = dZ @ Wk.T
    ex = edz @ np.abs(Wk.T) + (N + 1) * lr.U * ((np.abs(dZ) + edz) @ np.abs(Wk.T)) + 1e-38
    dW = X.T @ dZ
    ew = np.abs(X.T) @ edz + (M + 1) * lr.U * (np.abs(X.T) @ (np.abs(dZ) + edz)) + 1e-38
    db = dZ.sum(0)
    eb = edz.sum(0) + (M + 1) * lr.U * (np.abs(dZ) + edz).sum(0) + 1e-38
    return (dX, dW.T if tw else dW, db), (ex, ew.T if tw else ew, eb)


def _bwd_inputs(rng, M, N, K, tw):
    X, W, _, _ = _layer(rng, M, N, K, tw)
    return inputs.normal(rng, (M, N)), inputs.normal(rng, (M, N), 2.0), X, W


def _assert_grads(got, ref, bound, what=""):
    for g, r, e, n in zip(got, ref, bound, ("dX", "dW", "db")):
        lr.within(host(g), r, e, "%s %s" % (what, n))


@pytest.mark.parametrize("tw", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 70, 40), (3, 5, 9), (17, 64, 33), (65, 66, 67),
                                   (346, 768, 256), (1000, 129, 60), (1100, 36, 48), (2000, 7, 200)])
def test_gradients(M, N, K, tw):
    rng = np.random.default_rng([3, M, N, K])
    dY, Z, X, W = _bwd_inputs(rng, M, N, K, tw)
    got = bd.linear_f32_bwd(dev(dY), dev(X), dev(W), Z=dev(Z), act="gelu_tanh", trans_w=bool(tw))
    _assert_grads(got, *_grads(dY, Z, X, W, "gelu_tanh", tw), "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("tw", [0, 1])
@pytest.mark.parametrize("act", lr.ACTS)
def test_gradients_of_activations(act, tw):
    rng = np.random.default_rng(4)
    dY, Z, X, W = _bwd_inputs(rng, 150, 90, 70, tw)
    got = bd.linear_f32_bwd(dev(dY), dev(X), dev(W), Z=dev(Z), act=act, trans_w=bool(tw))
    _assert_grads(got, *_grads(dY, Z, X, W, act, tw), act)


@pytest.mark.parametrize("act", lr.ACTS)
def test_slope_over_its_range(act):
    """dY = 1, K = 1, X = 1 with one row per z: dX is the slope times W = 1;
    the limits hold out to infinity, NaN stays NaN, ReLU's slope at 0 is 0."""
    z = np.concatenate([np.linspace(-130, 130, 4001), np.linspace(-10, 10, 4001),
                        [0.0, 1e-30, 1e20, -1e20, 3e38, -3e38]]).astype(np.float32)
    one = np.ones((z.size, 1), np.float32)
    dX, _, _ = bd.linear_f32_bwd(dev(one), dev(one), dev(one[:1]), Z=dev(z[:, None]), act=act,
                                 want=("dX",))
    with np.errstate(over="ignore", invalid="ignore"):
        far = np.abs(z) > 1e10
        ref = np.where(far, (z > 0) * 1.0, lr.slope(np.where(far, 0, z), act)) if act != "none" else one[:, 0]
    lr.within(host(dX)[:, 0], ref, lr.SLOPE_ERR + 0 * ref, act)
    z = np.array([[np.inf], [-np.inf], [np.nan]], np.float32)
    dX, _, _ = bd.linear_f32_bwd(dev(one[:3]), dev(one[:3]), dev(one[:1]), Z=dev(z), act=act,
                                 want=("dX",))
    got = host(dX)[:, 0]
    if act == "none":
        assert np.array_equal(got, [1, 1, 1])
    else:
        assert got[0] == 1 and got[1] == 0 and np.isnan(got[2])


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu_erf", "silu"])
def test_gradients_against_differences(act):
    """sum(dY * Y) differentiated numerically, Y from linear_f32 itself: the
    central difference over a step h is off by h^2 |Y'''| / 6 and by the
    rounding of two sums over h, both far below the 2% allowed at h = 1/8
    for sums of this size."""
    rng = np.random.default_rng(5)
    M, N, K = 12, 20, 16
    X, W, b, _ = _layer(rng, M, N, K, 0)
    dY = inputs.normal(rng, (M, N))
    Z = torch().empty((M, N), device="cuda")

    def loss(X_, W_, b_):
        return (host(bd.linear_f32(dev(X_), dev(W_), bias=dev(b_), act=act)).astype(np.float64) * dY).sum()
    bd.linear_f32(dev(X), dev(W), bias=dev(b), act=act, Z=Z)
    grads = [host(g).astype(np.float64) for g in
             bd.linear_f32_bwd(dev(dY), dev(X), dev(W), Z=Z, act=act)]
    for k, (p, g) in enumerate(zip((X, W, b), grads)):
        d = rng.standard_normal(p.shape)
        d /= np.linalg.norm(d)
        h = 1 / 8
        args = [X, W, b]
        up, down = list(args), list(args)
        up[k] = (p + h * d).astype(np.float32)
        down[k] = (p - h * d).astype(np.float32)
        num = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(num - (g * d).sum()) <= 0.02 * np.linalg.norm(g), (k, num, (g * d).sum())


@pytest.mark.parametrize("want", [("dX",), ("dW",), ("db",), ("dX", "db"), ("dW", "db")])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_wanted_gradients_alone(want, act):
    rng = np.random.default_rng(6)
    dY, Z, X, W = _bwd_inputs(rng, 90, 70, 50, 1)
    full = bd.linear_f32_bwd(dev(dY), dev(X), dev(W), Z=dev(Z), act=act, trans_w=True)
    part = bd.linear_f32_bwd(dev(dY), dev(X) if "dW" in want else None,
                             dev(W) if ("dX" in want or "dW" not in want) else None, Z=dev(Z),
                             act=act, trans_w=True, want=want)
    for n, f, p in zip(("dX", "dW", "db"), full, part):
        assert (p is None) == (n not in want)
        if p is not None:
            assert np.array_equal(host(p), host(f)), n


@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("tw", [0, 1])
def test_accumulation_over_micro_batches(act, tw):
    """Two halves accumulated against the whole batch; dX is overwritten."""
    rng = np.random.default_rng(7)
    dY, Z, X, W = _bwd_inputs(rng, 300, 90, 70, tw)
    dW, db = dev(np.zeros_like(W)), dev(np.zeros(90, np.float32))
    for part in (slice(0, 140), slice(140, 300)):
        dX = torch().full((Z[part].shape[0], 70), float("nan"), device="cuda")
        bd.linear_f32_bwd(dev(dY[part]), dev(X[part]), dev(W), Z=dev(Z[part]), act=act,
                          trans_w=bool(tw), dX=dX, dW=dW, db=db, accumulate=True)
        assert np.isfinite(host(dX)).all()
    ref, bound = _grads(dY, Z, X, W, act, tw)
    lr.within(host(dW), ref[1], bound[1] + 2 * lr.U * np.abs(ref[1]))
    lr.within(host(db), ref[2], bound[2] + 2 * lr.U * np.abs(ref[2]))


def test_empty_batch():
    t = torch()
    e = t.empty((0, 40), device="cuda")
    X, W = t.empty((0, 30), device="cuda"), t.ones((30, 40), device="cuda")
    dX, dW, db = bd.linear_f32_bwd(e, X, W, Z=e, act="relu")
    assert dX.shape == (0, 30) and not host(dW).any() and not host(db).any()
    dW = t.ones((30, 40), device="cuda")
    db = t.ones(40, device="cuda")
    bd.linear_f32_bwd(e, X, W, Z=e, act="relu", dW=dW, db=db, accumulate=True)
    assert np.all(host(dW) == 1) and np.all(host(db) == 1)


@pytest.mark.parametrize("act", ["none", "gelu_erf"])
def test_backward_strides_and_what_lies_around(act):
    t = torch()
    rng = np.random.default_rng(9)
    M, N, K = 77, 45, 51
    dY, Z, X, W = _bwd_inputs(rng, M, N, K, 0)

    def view(a):
        buf = t.full((a.shape[0], a.shape[1] + 6), float("nan"), device="cuda")
        buf[:, 3:3 + a.shape[1]].copy_(dev(a))
        return buf[:, 3:3 + a.shape[1]]
    outs = []
    for rows, cols in ((M, K), (K, N), (1, N)):
        buf, _ = guarded(rows, cols + 3)
        outs.append((buf, buf[64:64 + rows * (cols + 3)].view(rows, cols + 3)[:, :cols]))
    need = bd.linear_f32_bwd_ws_size(act, M, N)
    ws = t.full((need + 64,), 0x55, dtype=t.uint8, device="cuda")
    bd.linear_f32_bwd(view(dY), view(X), view(W), Z=view(Z), act=act, dX=outs[0][1],
                      dW=outs[1][1], db=outs[2][1][0], workspace=ws[:need])
    _assert_grads([o[1] if o[1].shape[0] > 1 else o[1][0] for o in outs],
                  *_grads(dY, Z, X, W, act, 0))
    for (buf, v) in outs:
        assert canaries_intact(buf)
        r, c = v.shape
        assert np.all(host(buf)[64:64 + r * (c + 3)].reshape(r, c + 3)[:, c:] == np.float32(1.2345e9))
    assert np.all(host(ws)[need:] == 0x55), "wrote past the workspace"


def test_binding_refusals():
    t = torch()
    X, W = t.ones((4, 8), device="cuda"), t.ones((8, 6), device="cuda")
    with pytest.raises(ValueError):
        bd.linear_f32(X, W, act="tanh")
    with pytest.raises(ValueError):
        bd.linear_f32(X, W, trans_w=True)
    with pytest.raises(TypeError):
        bd.linear_f32(X.half(), W)
    with pytest.raises(ValueError):
        bd.linear_f32(X, W, bias=t.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        bd.linear_f32(X, W.cpu())
    with pytest.raises(ValueError):
        bd.linear_f32(X, t.ones((6, 8), device="cuda").t())
    with pytest.raises(bd.GGError):
        bd.linear_f32(X, t.ones((8, 8), device="cuda"), Y=X)
    dY = t.ones((4, 6), device="cuda")
    with pytest.raises(ValueError):
        bd.linear_f32_bwd(dY, X, W, act="silu")
    with pytest.raises(ValueError):
        bd.linear_f32_bwd(dY, None, W)
    with pytest.raises(ValueError):
        bd.linear_f32_bwd(dY, X, W, accumulate=True)
    with pytest.raises(bd.GGError):
        bd.linear_f32_bwd(dY, X, W, workspace=t.empty(16, dtype=t.uint8, device="cuda"))
