"""GPU parity of rmsnorm_f32, rmsnorm_mx8 and rmsnorm_f32_bwd against 64-bit
references, through the C ABI."""
import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
# columns around every border of the row kernels: 512, 2,048, 8,192, 32,768
SHAPES = [(1, 1), (1, 1536), (2, 31), (3, 32), (5, 33), (7, 64), (4, 100), (9, 511), (6, 512),
          (3, 513), (346, 768), (5, 2047), (4, 2048), (3, 2052), (2, 4099), (3, 8192), (2, 8196),
          (2, 10001), (1, 32768), (2, 32771), (2, 40000), (1000, 36), (1100, 12), (2500, 260)]


def _terms(K):
    """Additions that one term of a row sum can pass through: at most 32 (or
    K/1,024 in the longest rows) in a thread, then a tree over lanes and
    waves."""
    return max(32, -(-K // 1024)) + 24


def _ref(X, R, gamma, eps=EPS):
    """S (exactly rounded), y, rstd and the relative error allowed for them:
    half the sum's relative error, the quotient by K, eps, the root and the
    reciprocal, then one rounding per factor."""
    S = X if R is None else X + R                  # fp32: one rounding, as the kernel
    s = S.astype(np.float64)
    K = X.shape[1]
    rstd = 1 / np.sqrt((s * s).sum(1) / K + eps)
    rel = (_terms(K) / 2 + 4) * lr.U
    y = s * rstd[:, None] * (1 if gamma is None else gamma.astype(np.float64))
    return S, y, rstd, rel


def _inputs(M, K, residual=True, seed=0):
    rng = np.random.default_rng([seed, M, K])
    X = inputs.normal(rng, (M, K))
    R = inputs.normal(rng, (M, K), 3.0) if residual else None
    g = (1 + inputs.normal(rng, (K,), 0.3)).astype(np.float32)
    return X, R, g


def _d(a):
    return None if a is None else dev(a)


@pytest.mark.parametrize("residual", [0, 1])
@pytest.mark.parametrize("M,K", SHAPES)
def test_f32(M, K, residual):
    X, R, g = _inputs(M, K, residual)
    Y, S, rstd = bd.rmsnorm_f32(dev(X), dev(g), EPS, residual=_d(R))
    s, y, r, rel = _ref(X, R, g)
    assert np.array_equal(host(S), s)
    lr.within(host(rstd), r, rel * r)
    lr.within(host(Y), y, (rel + 2 * lr.U) * np.abs(y) + 1e-44)


@pytest.mark.parametrize("residual", [0, 1])
@pytest.mark.parametrize("M,K", SHAPES)
def test_mx8(M, K, residual):
    X, R, g = _inputs(M, K, residual)
    Q, E, S = bd.rmsnorm_mx8(dev(X), dev(g), EPS, residual=_d(R))
    s, y, r, rel = _ref(X, R, g)
    assert np.array_equal(host(S), s)
    lr.check_mx8(host(Q), host(E), y, (rel + 2 * lr.U) * np.abs(y))


@pytest.mark.parametrize("K", [96, 768, 777, 3000, 9000, 33000])
def test_both_outputs_hold_the_same_values(K):
    """The bytes are those of the fp32 output itself, exactly."""
    X, R, g = _inputs(4, K)
    Y, _, _ = bd.rmsnorm_f32(dev(X), dev(g), EPS, residual=dev(R))
    Q, E, _ = bd.rmsnorm_mx8(dev(X), dev(g), EPS, residual=dev(R))
    q, e = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(host(E), e) and np.array_equal(host(Q), q)


def test_every_e4m3_border_rounds_to_nearest_even():
    """Values that lie on e4m3 numbers, halfway between them and next to
    halfway: a row of mean square 1 would rescale them, so gamma carries the
    values and S is all ones (rstd = 1 exactly with eps = 0)."""
    table = lr.e4m3_values()[:127]
    mids = (table[1:] + table[:-1]) / 2
    rest = np.concatenate([table, mids, np.nextafter(mids.astype(np.float32), 0), -table, -mids,
                           np.nextafter(mids.astype(np.float32), 1000)]).astype(np.float32)
    v = np.where(np.arange(32 * (rest.size // 31 + 1)) % 32 == 0, 448, 0).astype(np.float32)
    v[[i for i in range(v.size) if i % 32][:rest.size]] = rest
    Q, E, _ = bd.rmsnorm_mx8(dev(np.ones((1, v.size), np.float32)), dev(v), 0.0)
    q, e = lr.to_mx8(v.astype(np.float64)[None])
    assert np.array_equal(host(E), e)
    got, want = lr.from_mx8(host(Q), host(E)), lr.from_mx8(q, e)
    assert np.array_equal(got, want)


def test_block_scales_at_their_borders():
    """Largest magnitudes at, just below and just above 448 * 2^n, tiny ones
    and zeros: the power of two is the smallest that fits, and at least
    2^-126."""
    tops = []
    for n in (-130, -126, -60, -9, -1, 0, 1, 5, 60, 110):
        t = np.float32(448 * 2.0 ** n)
        tops += [t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(np.inf))]
    tops += [np.float32(0), np.float32(1e-45), np.float32(1.2e-38)]
    v = np.zeros((len(tops), 32), np.float32)
    v[np.arange(len(tops)), np.arange(len(tops)) % 32] = tops
    v = v.reshape(1, -1)
    Q, E, _ = bd.rmsnorm_mx8(dev(np.ones(v.shape, np.float32)), dev(v[0]), 0.0)
    q, e = lr.to_mx8(v.astype(np.float64))
    assert np.array_equal(host(E)[0], np.maximum(e[0], 1))
    assert np.array_equal(lr.from_mx8(host(Q), host(E)), lr.from_mx8(q, e))


@pytest.mark.parametrize("K", [64, 100, 700, 2100, 9000, 33000])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_nonfinite_stays_in_its_row(K, bad):
    X, R, g = _inputs(6, K)
    X[3, K // 2] = bad
    Y, S, rstd = (host(a) for a in bd.rmsnorm_f32(dev(X), dev(g), EPS, residual=dev(R)))
    others = [0, 1, 2, 4, 5]
    assert np.isfinite(Y[others]).all() and np.isfinite(rstd[others]).all()
    assert np.isnan(Y[3, K // 2])
    assert np.isnan(rstd[3]) if np.isnan(bad) else rstd[3] == 0
    Q, E, _ = bd.rmsnorm_mx8(dev(X), dev(g), EPS, residual=dev(R))
    Q, E = host(Q), host(E)
    assert np.all(E[others] != 255) and E[3, K // 2 // 32] == 255
    b = K // 2 // 32 * 32
    assert np.all(Q[3, b:min(b + 32, K)] == 0x7f)


def test_zeros_and_extremes():
    t = torch()
    for K in (40, 2050):
        Z = np.zeros((2, K), np.float32)
        Y, _, rstd = bd.rmsnorm_f32(dev(Z), None, 0.25)
        assert not host(Y).any() and np.all(host(rstd) == 2)
        Q, E, _ = bd.rmsnorm_mx8(dev(Z), None, 0.25)
        assert not host(Q).any() and np.all(host(E) == 1)
        Y, _, _ = bd.rmsnorm_f32(dev(Z), None, 0.0)
        assert np.isnan(host(Y)).all()
        big = np.full((1, K), 1e25, np.float32)                 # squares past fp32
        Y, _, rstd = bd.rmsnorm_f32(dev(big), None, EPS)
        assert host(rstd)[0] == 0 and not host(Y).any()
        small = np.full((1, K), 1e-30, np.float32)              # squares vanish: eps alone
        Y, _, rstd = bd.rmsnorm_f32(dev(small), None, EPS)
        assert abs(host(rstd)[0] - EPS ** -0.5) < 1e-3
    empty = bd.rmsnorm_f32(t.empty((0, 64), device="cuda"), None)
    assert empty[0].shape == (0, 64)


@pytest.mark.parametrize("K", [96, 99, 1000, 2100, 33000])
@pytest.mark.parametrize("onto", ["X", "R"])
def test_residual_stream_in_place(K, onto):
    X, R, g = _inputs(5, K)
    ref = [host(a) for a in bd.rmsnorm_f32(dev(X), dev(g), EPS, residual=dev(R))]
    x, r = dev(X), dev(R)
    Y, S, _ = bd.rmsnorm_f32(x, dev(g), EPS, residual=r, S=x if onto == "X" else r)
    assert np.array_equal(host(Y), ref[0]) and np.array_equal(host(S), ref[1])
    x, r = dev(X), dev(R)
    q0 = bd.rmsnorm_mx8(dev(X), dev(g), EPS, residual=dev(R))
    q1 = bd.rmsnorm_mx8(x, dev(g), EPS, residual=r, S=x if onto == "X" else r)
    for a, b in zip(q0, q1):
        assert np.array_equal(host(a), host(b))


@pytest.mark.parametrize("M,K", [(5, 60), (5, 61), (4, 1000), (3, 2500), (2, 33001)])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_strides_offsets_and_what_lies_around(M, K, shift):
    t = torch()
    X, R, g = _inputs(M, K)

    def view(a):
        a2 = np.atleast_2d(a)
        buf = t.full((a2.shape[0], a2.shape[1] + 8), float("nan"), device="cuda")
        v = buf[:, shift:shift + a2.shape[1]]
        v.copy_(dev(a2))
        return v if a.ndim == 2 else v[0]
    bufs = [guarded(M, K + 4)[0] for _ in range(2)]
    S, Y = (b[64:64 + M * (K + 4)].view(M, K + 4)[:, :K] for b in bufs)
    s, y, r, rel = _ref(X, R, g)
    bd.rmsnorm_f32(view(X), view(g), EPS, residual=view(R), S=S, Y=Y)
    assert np.array_equal(host(S), s)
    lr.within(host(Y), y, (rel + 2 * lr.U) * np.abs(y))
    nb = -(-K // 32)
    Q8 = t.full((M + 2, K + 5), 0xAA, dtype=t.uint8, device="cuda")
    E8 = t.full((M + 2, nb + 3), 0xAA, dtype=t.uint8, device="cuda")
    bd.rmsnorm_mx8(view(X), view(g), EPS, residual=view(R), S=S, Q=Q8[1:M + 1, 2:K + 2],
                   E=E8[1:M + 1, 1:nb + 1])
    q, e = host(Q8), host(E8)
    lr.check_mx8(q[1:M + 1, 2:K + 2], e[1:M + 1, 1:nb + 1], y, (rel + 2 * lr.U) * np.abs(y))
    q[1:M + 1, 2:K + 2] = 0xAA
    e[1:M + 1, 1:nb + 1] = 0xAA
    assert np.all(q == 0xAA) and np.all(e == 0xAA), "wrote around the outputs"
    for b in bufs:
        assert canaries_intact(b)
        assert np.all(host(b)[64:64 + M * (K + 4)].reshape(M, K + 4)[:, K:] == np.float32(1.2345e9))


def test_rows_past_32_bit_offsets():
    """Rows whose offsets pass 2^31 elements, by a wide leading dimension."""
    t = torch()
    M, K, ld = 5, 64, 1 << 29
    buf = t.zeros((M - 1) * ld + K, device="cuda")
    X = buf.as_strided((M, K), (ld, 1))
    x = inputs.normal(np.random.default_rng(0), (M, K))
    X.copy_(dev(x))
    Y, S, rstd = bd.rmsnorm_f32(X, None, EPS)
    _, y, _, rel = _ref(x, None, None)
    lr.within(host(Y), y, (rel + 2 * lr.U) * np.abs(y))
    dx, _ = bd.rmsnorm_f32_bwd(X, X, None, rstd)
    d2, _ = bd.rmsnorm_f32_bwd(dev(x), dev(x), None, rstd)
    assert np.array_equal(host(dx), host(d2))
    Z = bd.linear_f32(X, dev(np.eye(K, dtype=np.float32)))
    assert np.array_equal(host(Z), x)


# -------------------------------------------------------------- backward --

def _bwd_ref(dY, S, g, rstd, dS):
    """dX, dgamma and the bounds of their errors: the row sum's error is
    relative to the sum of magnitudes."""
    K = S.shape[1]
    dY, S, r = dY.astype(np.float64), S.astype(np.float64), rstd.astype(np.float64)[:, None]
    gam = np.ones(K) if g is None else g.astype(np.float64)
    xh, gd = S * r, dY * gam
    dot = (gd * xh).mean(1, keepdims=True)
    edot = (_terms(K) + 4) * lr.U * np.abs(gd * xh).mean(1, keepdims=True)
    dX = (gd - xh * dot) * r
    e = r * (np.abs(xh) * edot + 5 * lr.U * (np.abs(gd) + np.abs(xh * dot)))
    if dS is not None:
        dX = dX + dS.astype(np.float64)
        e = e + lr.U * np.abs(dX)
    dg = (dY * xh).sum(0)
    eg = (S.shape[0] + 4) * lr.U * np.abs(dY * xh).sum(0)
    return dX, dg, e * 1.01 + 1e-44, eg + 1e-44


def _bwd_inputs(M, K, carried=True):
    rng = np.random.default_rng([5, M, K])
    S, dY = inputs.normal(rng, (M, K)), inputs.normal(rng, (M, K))
    g = (1 + inputs.normal(rng, (K,), 0.3)).astype(np.float32)
    rstd = (1 / np.sqrt((S.astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    return dY, S, g, rstd, inputs.normal(rng, (M, K)) if carried else None


@pytest.mark.parametrize("carried", [0, 1])
@pytest.mark.parametrize("M,K", SHAPES)
def test_gradients(M, K, carried):
    dY, S, g, rstd, dS = _bwd_inputs(M, K, carried)
    dX, dg = bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), dS=_d(dS))
    x, gg, ex, eg = _bwd_ref(dY, S, g, rstd, dS)
    lr.within(host(dX), x, ex, "dX")
    lr.within(host(dg), gg, eg, "dgamma")


@pytest.mark.parametrize("M,K", [(600, 40), (40, 2500), (3, 33000)])
def test_gradients_alone_accumulated_and_in_place(M, K):
    dY, S, g, rstd, dS = _bwd_inputs(M, K)
    full = [host(a) for a in bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), dS=dev(dS))]
    dX, none = bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), dS=dev(dS), want=("dX",))
    assert none is None and np.array_equal(host(dX), full[0])
    none, dg = bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), want=("dgamma",))
    assert none is None and np.array_equal(host(dg), full[1])
    d = dev(dS)
    dX, _ = bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), dS=d, dX=d)
    assert np.array_equal(host(d), full[0])
    acc = dev(np.full(K, 2.0, np.float32))
    bd.rmsnorm_f32_bwd(dev(dY), dev(S), dev(g), dev(rstd), dgamma=acc, accumulate=True)
    assert np.array_equal(host(acc), np.float32(2) + full[1])
    x, gg, ex, eg = _bwd_ref(dY, S, None, rstd, None)
    dX, dg = bd.rmsnorm_f32_bwd(dev(dY), dev(S), None, dev(rstd))
    lr.within(host(dX), x, ex)
    lr.within(host(dg), gg, eg)


def test_gradients_against_differences():
    """sum(dY * Y + dS * S) differentiated numerically through rmsnorm_f32:
    curvature and rounding of the difference at h = 1/16 are far below the 2%
    of the gradient's length that is allowed."""
    rng = np.random.default_rng(6)
    X, R, g = _inputs(6, 48)
    dY, dS = inputs.normal(rng, X.shape), inputs.normal(rng, X.shape)

    def loss(x, gam):
        Y, S, _ = bd.rmsnorm_f32(dev(x), dev(gam), EPS, residual=dev(R))
        return (host(Y).astype(np.float64) * dY + host(S).astype(np.float64) * dS).sum()
    Y, S, rstd = bd.rmsnorm_f32(dev(X), dev(g), EPS, residual=dev(R))
    dX, dg = bd.rmsnorm_f32_bwd(dev(dY), S, dev(g), rstd, dS=dev(dS))
    for k, (p, gr) in enumerate(((X, host(dX)), (g, host(dg)))):
        d = rng.standard_normal(p.shape)
        d /= np.linalg.norm(d)
        h = 1 / 16
        a, b = (p + h * d).astype(np.float32), (p - h * d).astype(np.float32)
        num = ((loss(a, g) - loss(b, g)) if k == 0 else (loss(X, a) - loss(X, b))) / (2 * h)
        assert abs(num - (gr.astype(np.float64) * d).sum()) <= 0.02 * np.linalg.norm(gr)


def test_empty_batch_backward():
    t = torch()
    e, r = t.empty((0, 64), device="cuda"), t.empty(0, device="cuda")
    dX, dg = bd.rmsnorm_f32_bwd(e, e, None, r)
    assert dX.shape == (0, 64) and not host(dg).any()


@pytest.mark.parametrize("M,K,shift", [(5, 61, 1), (700, 60, 4), (4, 2500, 1), (2, 33001, 0)])
def test_backward_strides_and_what_lies_around(M, K, shift):
    t = torch()
    dY, S, g, rstd, dS = _bwd_inputs(M, K)

    def view(a):
        a2 = np.atleast_2d(a)
        buf = t.full((a2.shape[0], a2.shape[1] + 8), float("nan"), device="cuda")
        v = buf[:, shift:shift + a2.shape[1]]
        v.copy_(dev(a2))
        return v if a.ndim == 2 else v[0]
    buf, _ = guarded(M, K + 4)
    dX = buf[64:64 + M * (K + 4)].view(M, K + 4)[:, :K]
    bg, _ = guarded(1, K)
    need = bd.rmsnorm_f32_bwd_ws_size(M, K)
    ws = t.full((need + 64,), 0x55, dtype=t.uint8, device="cuda")
    bd.rmsnorm_f32_bwd(view(dY), view(S), view(g), view(rstd), dS=view(dS), dX=dX,
                       dgamma=bg[64:64 + K], workspace=ws[:need])
    x, gg, ex, eg = _bwd_ref(dY, S, g, rstd, dS)
    lr.within(host(dX), x, ex)
    lr.within(host(bg)[64:64 + K], gg, eg)
    assert canaries_intact(buf) and canaries_intact(bg)
    assert np.all(host(buf)[64:64 + M * (K + 4)].reshape(M, K + 4)[:, K:] == np.float32(1.2345e9))
    assert np.all(host(ws)[need:] == 0x55)


def test_binding_refusals():
    t = torch()
    X = t.ones((4, 64), device="cuda")
    with pytest.raises(bd.GGError):
        bd.rmsnorm_f32(X, None, -1.0)
    with pytest.raises(bd.GGError):
        bd.rmsnorm_f32(X, None, Y=X)
    with pytest.raises(TypeError):
        bd.rmsnorm_f32(X.double())
    with pytest.raises(ValueError):
        bd.rmsnorm_f32(X, t.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        bd.rmsnorm_mx8(X, E=t.empty((4, 1), dtype=t.uint8, device="cuda"))
    with pytest.raises(ValueError):
        bd.rmsnorm_f32_bwd(X, X, None, t.ones(4, device="cuda"), accumulate=True)
