"""GPU parity of block_norm_f32, block_norm_mx8 and block_norm_f32_bwd against
64-bit references, through the C ABI."""
import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
# columns around every border of the row kernels: 4, 64 and its doubles up to
# 16,384, 12,288
SHAPES = [(5, 255), (5, 256), (70, 257), (3, 1023), (4, 1024), (9, 1025), (2, 4096), (3, 4097), (2, 12288), (3, 12289),
          (2, 16384), (2, 16385), (700, 1000), (1, 1), (3, 2), (2, 3), (1, 4), (2, 5), (1, 1536), (2, 31), (3, 32), (5, 33), (4, 100), (9, 511),
          (6, 512), (3, 513), (346, 768), (5, 2047), (4, 2048), (3, 2052), (2, 4099), (3, 8192), (2, 8193),
          (2, 8196), (2, 40001), (1000, 36), (1100, 13), (2500, 260), (37, 64), (19, 65), (9001, 63), (11, 127), (8, 128),
          (4100, 128), (7, 129), (9001, 2)]
GATES = ("none", "columns", "rows")


def _inputs(M, K, gate="columns", seed=0):
    rng = np.random.default_rng([seed, M, K])
    n = lambda *s, scale=1.0: inputs.normal(rng, s, scale)   # noqa: E731
    return dict(U=n(M, K, scale=2.0), X=n(M, K, scale=3.0), gu=(1 + n(K, scale=0.3)).astype(np.float32),
                gs=(1 + n(K, scale=0.3)).astype(np.float32),
                gate={"none": None, "columns": n(K), "rows": n(M, K)}[gate], dY=n(M, K), dS=n(M, K))


def _d(a):
    return None if a is None else dev(a)


def _check_forward(d, alpha, Y, S, ru, rs, eps=EPS):
    s, es, r, rel = er.block_norm_S(d["U"], d["X"], d["gu"], d["gate"], alpha, eps)
    lr.within(host(S), s, es, "S")
    lr.within(host(ru), r, rel * r, "rstd_u")
    y, ey, r, rel = er.block_norm_Y(host(S), d["gs"], eps)
    lr.within(host(rs), r, rel * r, "rstd_s")
    lr.within(host(Y), y, ey, "Y")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("M,K", SHAPES)
def test_f32(M, K, gate):
    d = _inputs(M, K, gate)
    Y, S, ru, rs = bd.block_norm_f32(dev(d["U"]), dev(d["X"]), dev(d["gu"]), dev(d["gs"]), EPS,
                                     gate=_d(d["gate"]), alpha=0.7)
    _check_forward(d, np.float32(0.7).astype(np.float64), Y, S, ru, rs)


@pytest.mark.parametrize("M,K", [(1, 1), (4, 3), (3, 96), (2, 777), (5, 2050), (1, 1536), (3, 8192), (2, 9001)])
def test_mx8_holds_the_same_values(M, K):
    """S and the bytes are those of the fp32 call, exactly."""
    d = _inputs(M, K)
    a = [dev(d[n]) for n in ("U", "X", "gu", "gs")]
    Y, S, _, _ = bd.block_norm_f32(*a, EPS, gate=_d(d["gate"]), alpha=-0.5)
    Q, E, S8 = bd.block_norm_mx8(*a, EPS, gate=_d(d["gate"]), alpha=-0.5)
    assert np.array_equal(host(S8), host(S))
    q, e = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(host(E), e) and np.array_equal(host(Q), q)


def test_absent_vectors_are_ones_and_alpha_zero():
    d = _inputs(7, 300, "none")
    ones = dict(d, gu=None, gs=None)
    Y, S, ru, rs = bd.block_norm_f32(dev(d["U"]), dev(d["X"]), None, None, EPS)
    _check_forward(ones, 1.0, Y, S, ru, rs)
    Y, S, ru, rs = bd.block_norm_f32(dev(d["U"]), dev(d["X"]), None, None, EPS, alpha=0.0)
    _check_forward(ones, 0.0, Y, S, ru, rs)
    empty = bd.block_norm_f32(torch().empty((0, 64), device="cuda"), torch().empty((0, 64), device="cuda"))
    assert empty[0].shape == (0, 64)


@pytest.mark.parametrize("K", [3, 96, 99, 1000, 2100, 8200])
def test_residual_stream_in_place(K):
    d = _inputs(5, K)
    a = [dev(d[n]) for n in ("U", "X", "gu", "gs")]
    ref = bd.block_norm_f32(*a, EPS, gate=_d(d["gate"]), alpha=0.5)
    x = dev(d["X"])
    got = bd.block_norm_f32(a[0], x, *a[2:], EPS, gate=_d(d["gate"]), alpha=0.5, S=x)
    for p, q in zip(got, ref):
        assert np.array_equal(host(p), host(q))
    x = dev(d["X"])
    q8 = bd.block_norm_mx8(*a, EPS, gate=_d(d["gate"]), alpha=0.5)
    p8 = bd.block_norm_mx8(a[0], x, *a[2:], EPS, gate=_d(d["gate"]), alpha=0.5, S=x)
    for p, q in zip(p8, q8):
        assert np.array_equal(host(p), host(q))


@pytest.mark.parametrize("K", [64, 101, 700, 2100, 9000])
@pytest.mark.parametrize("at", ["U", "X"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nonfinite_stays_in_its_row(K, at, bad):
    d = _inputs(6, K)
    d[at][3, K // 2] = bad
    a = [dev(d[n]) for n in ("U", "X", "gu", "gs")]
    Y, S, ru, rs = (host(v) for v in bd.block_norm_f32(*a, EPS, gate=_d(d["gate"])))
    others = [0, 1, 2, 4, 5]
    assert np.isfinite(Y[others]).all() and np.isfinite(S[others]).all()
    assert np.isnan(Y[3, K // 2]) and not np.isfinite(S[3, K // 2])
    Q, E, _ = bd.block_norm_mx8(*a, EPS, gate=_d(d["gate"]))
    E = host(E)
    assert np.all(E[others] != 255) and E[3, K // 2 // 32] == 255


def test_zeros_and_extremes():
    for K in (40, 2050, 8200):
        z = np.zeros((2, K), np.float32)
        Y, S, ru, rs = bd.block_norm_f32(dev(z), dev(z), None, None, 0.25)
        assert not host(Y).any() and not host(S).any() and np.all(host(ru) == 2) and np.all(host(rs) == 2)
        big = np.full((1, K), 1e25, np.float32)                 # squares past fp32
        x = np.ones((1, K), np.float32)
        Y, S, ru, rs = bd.block_norm_f32(dev(big), dev(x), None, None, 0.0)
        assert host(ru)[0] == 0 and np.all(host(S) == 1)
        assert np.all(np.abs(host(Y) - 1) <= 64 * lr.U)


@pytest.mark.parametrize("M,K", [(5, 60), (5, 61), (4, 1000), (3, 2501), (2, 8201)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strides_offsets_and_what_lies_around(M, K, shift):
    t = torch()
    d = _inputs(M, K, "rows")

    def view(a):
        a2 = np.atleast_2d(a)
        buf = t.full((a2.shape[0], a2.shape[1] + 8), float("nan"), device="cuda")
        v = buf[:, shift:shift + a2.shape[1]]
        v.copy_(dev(a2))
        return v if a.ndim == 2 else v[0]
    bufs = [guarded(M, K + 5)[0] for _ in range(5)]
    S, Y, dU, dX, dG = (b[64:64 + M * (K + 5)].view(M, K + 5)[:, :K] for b in bufs)
    v = {n: view(a) for n, a in d.items()}
    _, _, ru, rs = bd.block_norm_f32(v["U"], v["X"], v["gu"], v["gs"], EPS, gate=v["gate"], S=S, Y=Y)
    _check_forward(d, 1.0, Y, S, ru, rs)
    got = dict(zip(("dU", "dX", "dgamma_u", "dgamma_s", "dgate"),
                   bd.block_norm_f32_bwd(v["dY"], v["U"], S, v["gu"], v["gs"], ru, rs, gate=v["gate"], dS=v["dS"],
                                         dU=dU, dX=dX, dgate=dG)))
    ref = er.block_norm_bwd(d["dY"], d["U"], host(S), d["gu"], d["gs"], host(ru), host(rs), d["gate"], 1.0, d["dS"])
    for n, (r, e) in ref.items():
        lr.within(host(got[n]), r, e, n)
    nb = -(-K // 32)
    Q8 = t.full((M + 2, K + 5), 0xAA, dtype=t.uint8, device="cuda")
    E8 = t.full((M + 2, nb + 3), 0xAA, dtype=t.uint8, device="cuda")
    bd.block_norm_mx8(v["U"], v["X"], v["gu"], v["gs"], EPS, gate=v["gate"], S=S, Q=Q8[1:M + 1, 2:K + 2],
                      E=E8[1:M + 1, 1:nb + 1])
    q, e = host(Q8), host(E8)
    q0, e0 = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(q[1:M + 1, 2:K + 2], q0) and np.array_equal(e[1:M + 1, 1:nb + 1], e0)
    q[1:M + 1, 2:K + 2] = 0xAA
    e[1:M + 1, 1:nb + 1] = 0xAA
    assert np.all(q == 0xAA) and np.all(e == 0xAA), "wrote around the outputs"
    for b in bufs:
        assert canaries_intact(b)
        assert np.all(host(b)[64:64 + M * (K + 5)].reshape(M, K + 5)[:, K:] == np.float32(1.2345e9))


def test_rows_past_32_bit_offsets():
    t = torch()
    M, K, ld = 5, 64, 1 << 29
    buf = t.zeros((M - 1) * ld + K, device="cuda")
    far = buf.as_strided((M, K), (ld, 1))
    d = _inputs(M, K)
    far.copy_(dev(d["U"]))
    Y, S, ru, rs = bd.block_norm_f32(far, dev(d["X"]), dev(d["gu"]), dev(d["gs"]), EPS, gate=_d(d["gate"]))
    _check_forward(d, 1.0, Y, S, ru, rs)
    a = (dev(d["dY"]), S, dev(d["gu"]), dev(d["gs"]), ru, rs)
    one = bd.block_norm_f32_bwd(a[0], far, *a[1:], gate=_d(d["gate"]))
    two = bd.block_norm_f32_bwd(a[0], dev(d["U"]), *a[1:], gate=_d(d["gate"]))
    for p, q in zip(one, two):
        assert np.array_equal(host(p), host(q))


# -------------------------------------------------------------- backward --

def _bwd_inputs(M, K, gate, seed=0):
    d = _inputs(M, K, gate, seed)
    rng = np.random.default_rng([seed, M, K, 1])
    d["S"] = inputs.normal(rng, (M, K), 2.0)
    d["ru"] = (1 / np.sqrt((d["U"].astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    d["rs"] = (1 / np.sqrt((d["S"].astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    return d


NAMES = ("dU", "dX", "dgamma_u", "dgamma_s", "dgate")


def _bwd(d, alpha=0.6, carried=True, **kw):
    a = [dev(d[n]) for n in ("dY", "U", "S", "gu", "gs", "ru", "rs")]
    out = bd.block_norm_f32_bwd(*a, gate=_d(d["gate"]), alpha=alpha, dS=_d(d["dS"]) if carried else None, **kw)
    return dict(zip(NAMES, out))


def _bwd_ref(d, alpha=0.6, carried=True):
    return er.block_norm_bwd(d["dY"], d["U"], d["S"], d["gu"], d["gs"], d["ru"], d["rs"], d["gate"],
                             float(np.float32(alpha)), d["dS"] if carried else None)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("M,K", SHAPES)
def test_bwd(M, K, carried, gate):
    d = _bwd_inputs(M, K, gate)
    got = _bwd(d, carried=carried)
    for n, (r, e) in _bwd_ref(d, carried=carried).items():
        lr.within(host(got[n]), r, e, n)
    if gate == "none":
        assert got["dgate"] is None


@pytest.mark.parametrize("K", [40, 100, 200, 700])
def test_bwd_infinity_in_the_last_row_counts_once(K):
    """An infinite gate in the last row makes one entry of dgamma_u infinite, not
    NaN, however many rows a workgroup could hold."""
    d = _bwd_inputs(3, K, "rows")
    ref = _bwd_ref(d)["dgamma_u"]
    d["gate"][2, 5] = np.inf
    got = host(_bwd(d, want=("dgamma_u",))["dgamma_u"])
    rest = np.arange(K) != 5
    assert np.isinf(got[5])
    lr.within(got[rest], ref[0][rest], ref[1][rest])


@pytest.mark.parametrize("K", [40, 700, 2100, 8200])
@pytest.mark.parametrize("gate", GATES)
def test_bwd_of_what_is_wanted(K, gate):
    """Each gradient alone equals the full call's; absent vectors are ones."""
    d = _bwd_inputs(70, K, gate)
    full = _bwd(d)
    for n in NAMES:
        got = _bwd(d, want=(n,))
        assert all(got[o] is None for o in NAMES if o != n)
        if full[n] is not None:
            assert np.array_equal(host(got[n]), host(full[n])), n
    bare = dict(d, gu=None, gs=None)
    a = [_d(bare[n]) for n in ("dY", "U", "S", "gu", "gs", "ru", "rs")]
    got = dict(zip(NAMES, bd.block_norm_f32_bwd(*a, gate=_d(d["gate"]))))
    for n, (r, e) in _bwd_ref(bare, alpha=1.0, carried=False).items():
        lr.within(host(got[n]), r, e, n)


@pytest.mark.parametrize("M,K", [(1, 50), (70, 700), (5, 8200)])
def test_bwd_in_place_and_accumulating(M, K):
    d = _bwd_inputs(M, K, "columns")
    ref = _bwd(d)
    a = [dev(d[n]) for n in ("dY", "U", "S", "gu", "gs", "ru", "rs")]
    ds = dev(d["dS"])
    acc = [torch().full((K,), 3.0, device="cuda") for _ in range(3)]
    got = dict(zip(NAMES, bd.block_norm_f32_bwd(*a, gate=dev(d["gate"]), alpha=0.6, dS=ds, dX=ds, dgamma_u=acc[0],
                                                dgamma_s=acc[1], dgate=acc[2], accumulate=True)))
    for n in ("dU", "dX"):
        assert np.array_equal(host(got[n]), host(ref[n]))
    for n in ("dgamma_u", "dgamma_s", "dgate"):
        want = host(ref[n]).astype(np.float64)          # the last product may be fused with the addition
        lr.within(host(got[n]), want + 3, 2 * lr.U * (np.abs(want) + 3), n)


def test_bwd_of_no_rows():
    t = torch()
    e = t.empty((0, 30), device="cuda")
    v, r = t.ones(30, device="cuda"), t.empty(0, device="cuda")
    out = bd.block_norm_f32_bwd(e, e, e, v, v, r, r, gate=v)
    assert out[0].shape == (0, 30) and all(not host(o).any() and o.shape == (30,) for o in out[2:])


def test_gradients_against_differences():
    """The kernels' gradients along random directions against central
    differences of the forward pass in 64 bits."""
    M, K, alpha = 12, 90, 0.8
    for gate in ("columns", "rows"):
        d = _inputs(M, K, gate, seed=4)
        a = {n: dev(d[n]) for n in ("U", "X", "gu", "gs", "gate")}
        Y, S, ru, rs = bd.block_norm_f32(a["U"], a["X"], a["gu"], a["gs"], EPS, gate=a["gate"], alpha=alpha)
        g = dict(zip(("U", "X", "gu", "gs", "gate"), bd.block_norm_f32_bwd(
            dev(d["dY"]), a["U"], S, a["gu"], a["gs"], ru, rs, gate=a["gate"], alpha=alpha, dS=dev(d["dS"]))))

        def loss(p):
            al = float(np.float32(alpha))
            V = p["U"] / np.sqrt((p["U"] ** 2).mean(1, keepdims=True) + EPS) * p["gu"]
            s = al * p["X"] + p["gate"] * V
            y = s / np.sqrt((s ** 2).mean(1, keepdims=True) + EPS) * p["gs"]
            return (y * d["dY"]).sum() + (s * d["dS"]).sum()
        p = {n: d[n].astype(np.float64) for n in g}
        rng = np.random.default_rng(9)
        for n in g:
            v = rng.standard_normal(p[n].shape)
            h = 1e-5
            diff = (loss(dict(p, **{n: p[n] + h * v})) - loss(dict(p, **{n: p[n] - h * v}))) / (2 * h)
            got = (host(g[n]).astype(np.float64) * v).sum()
            # differences: O(h^2) terms of a loss of some 10^3, and 1e-16 / h of it
            assert abs(got - diff) <= 1e-5 * np.abs(host(g[n]) * v).sum() + 1e-6, (gate, n)
