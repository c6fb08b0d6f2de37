"""GPU parity of linear_f32_grouped and linear_f32_grouped_bwd against 64-bit
references, through the C ABI."""
import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu


def _sizes(kind, E, M, rng):
    """Sizes of E groups that M rows fall into."""
    if kind == "even":
        return [M // E + (e < M % E) for e in range(E)]
    if kind == "one":
        s = [0] * E
        s[E // 2] = M
        return s
    return np.bincount(rng.choice(E, M, p=rng.dirichlet(np.full(E, 0.4))), minlength=E).tolist()


def _inputs(M, N, K, E, trans_w, gather, kind="ragged", seed=0):
    rng = np.random.default_rng([seed, M, N, K, E, trans_w])
    n = lambda *s, scale=1.0: inputs.normal(rng, s, scale)   # noqa: E731
    T = max(1, M // 2)
    return dict(X=n(T if gather else M, K), W=n(*((E, N, K) if trans_w else (E, K, N)), scale=max(K, 1) ** -0.5),
                b=n(E, N), rows=rng.integers(0, T, M).astype(np.int32) if gather else None,
                offsets=er.sizes_to_offsets(_sizes(kind, E, M, rng)), dY=n(M, N), Z=n(M, N, scale=1.5))


def _d(a):
    return None if a is None else dev(a)


def _forward(d, act="none", trans_w=False, **kw):
    M = d["dY"].shape[0]
    Z = torch().full((M, d["dY"].shape[1]), 7.0, device="cuda")
    Y = bd.linear_f32_grouped(dev(d["X"]), dev(d["W"]), dev(d["offsets"]), rows=_d(d["rows"]), bias=_d(d["b"]),
                              act=act, Z=Z, trans_w=trans_w, **kw)
    return Y, Z


def _check(d, Y, Z, act, trans_w):
    z, y, ez, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], d["rows"], d["b"], act, trans_w)
    live = slice(int(d["offsets"][0]), int(d["offsets"][-1]))
    lr.within(host(Z)[live], z[live], ez[live], "Z")
    lr.within(host(Y)[live], y[live], ey[live], "Y")


# rows, outputs, inputs, experts: around tiles of 4 to 64 rows and 32 to 64
# columns, slabs of 32, more experts than lanes
SHAPES = [(1, 1, 1, 1), (1, 33, 5, 3), (2, 64, 32, 8), (7, 70, 31, 2), (8, 2304, 768, 8), (16, 100, 64, 5),
          (40, 65, 100, 3), (64, 64, 64, 1), (65, 130, 33, 4), (100, 48, 200, 70), (129, 31, 96, 2), (300, 200, 150, 7),
          (200, 96, 64, 200), (777, 260, 129, 16), (1500, 64, 1000, 6), (1000, 513, 40, 9), (64, 20, 48, 1000)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M,N,K,E", SHAPES)
def test_forward(M, N, K, E, trans_w, gather):
    for kind in ("ragged", "even", "one"):
        d = _inputs(M, N, K, E, trans_w, gather, kind)
        Y, Z = _forward(d, trans_w=trans_w)
        _check(d, Y, Z, "none", trans_w)


# one for each way the tiles are laid out: one and two rows per group with 16 and 8
# runs of k, and 32 rows by 32 columns with k in 8 parts and by 64 in 4, 2 and 1
WAYS = [(5, 90, 130, 9), (5, 300, 700, 10), (11, 1300, 100, 12), (8, 70, 131, 5), (14, 1200, 100, 8), (70, 300, 270, 2), (40, 1100, 260, 9),
        (40, 1100, 263, 9), (40, 263, 1100, 9), (700, 4200, 140, 4), (700, 4200, 670, 4), (600, 2900, 141, 4), (600, 140, 2900, 4)]


@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M,N,K,E", WAYS)
def test_ways(M, N, K, E, trans_w):
    for gather, kind in ((False, "ragged"), (True, "even")):
        d = _inputs(M, N, K, E, trans_w, gather, kind)
        Y, Z = _forward(d, "relu", trans_w)
        _check(d, Y, Z, "relu", trans_w)
        _check_bwd(d, _bwd(d, "relu", trans_w), "relu", trans_w)


@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("M,E", [(5, 4), (150, 3)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_activations(act, M, E, trans_w):
    d = _inputs(M, 90, 70, E, trans_w, True)
    Y, Z = _forward(d, act, trans_w)
    _check(d, Y, Z, act, trans_w)
    Y = bd.linear_f32_grouped(dev(d["X"]), dev(d["W"]), dev(d["offsets"]), rows=dev(d["rows"]), act=act,
                              trans_w=trans_w)
    _, y, _, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], d["rows"], None, act, trans_w)
    lr.within(host(Y), y, ey, "without bias")


def test_one_expert_equals_the_dense_layer():
    """Within the bounds of both, on the same rows."""
    d = _inputs(200, 150, 100, 1, True, False)
    Y, Z = _forward(d, "silu", True)
    dense = bd.linear_f32(dev(d["X"]), dev(d["W"][0]), bias=dev(d["b"][0]), act="silu", trans_w=True)
    _, _, _, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], None, d["b"], "silu", True)
    lr.within(host(Y), host(dense).astype(np.float64), 2 * ey)


def test_no_inputs_leave_the_bias():
    d = _inputs(20, 40, 0, 3, False, False)
    Y, Z = _forward(d, "relu")
    _check(d, Y, Z, "relu", False)
    assert bd.linear_f32_grouped(dev(d["X"][:0]), dev(d["W"]), dev(d["offsets"] * 0)).shape == (0, 40)


@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M,E", [(30, 6), (400, 5)])
def test_rows_outside_of_the_groups_are_left(M, E, trans_w):
    """Groups that start past row 0 and end before M: other rows of outputs stay
    as they were, and what other rows of inputs hold does not matter."""
    d = _inputs(M, 70, 50, E, trans_w, True)
    rng = np.random.default_rng(3)
    d["offsets"] = er.sizes_to_offsets(_sizes("ragged", E, M - 11, rng), 4)
    d["rows"][:4] = d["rows"][-7:] = 2 ** 31 - 1
    d["dY"][:4] = d["dY"][-7:] = d["Z"][:4] = d["Z"][-7:] = np.nan
    Y = torch().full((M, 70), 5.0, device="cuda")
    _, Z = _forward(d, "silu", trans_w, Y=Y)
    _check(d, Y, Z, "silu", trans_w)
    out = np.r_[0:4, M - 7:M]
    assert np.all(host(Y)[out] == 5) and np.all(host(Z)[out] == 7)
    dX = torch().full((M, 50), 5.0, device="cuda")
    got = _bwd(d, "silu", trans_w, dX=dX)
    _check_bwd(d, got, "silu", trans_w)
    assert np.all(host(dX)[out] == 5)


@pytest.mark.parametrize("offsets", [[0, 9, 4, 20, 30], [-5, 3, 3, 2 ** 31 - 1, 40], [-2 ** 31, 10, 2 ** 31 - 1, 5, -7],
                                     [40, 30, 20, 10, 0], [7, 7, 7, 7, 7]])
@pytest.mark.parametrize("M", [30, 300])
def test_offsets_out_of_order_stay_inside(M, offsets):
    """Whatever offsets and rows hold, nothing around the outputs is written,
    and groups that are in order hold what they should."""
    t = torch()
    d = _inputs(M, 70, 50, 4, False, True)
    d["offsets"] = np.array(offsets, np.int32)
    d["rows"][::3] = np.array([-1, 2 ** 31 - 1, -2 ** 31, 15], np.int32)[np.arange(d["rows"][::3].size) % 4]
    buf, Y = guarded(M, 70)
    bufx, dX = guarded(M, 50)
    bd.linear_f32_grouped(dev(d["X"]), dev(d["W"]), dev(d["offsets"]), rows=dev(d["rows"]), Y=Y)
    _bwd(d, "relu", False, dX=dX)
    t.cuda.synchronize()
    assert canaries_intact(buf) and canaries_intact(bufx)


@pytest.mark.parametrize("M,E", [(9, 3), (90, 2)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_strides_offsets_and_what_lies_around(M, E, trans_w):
    t = torch()
    N, K = 45, 67
    d = _inputs(M, N, K, E, trans_w, True)

    def view(a, pad=3):
        buf = t.full(a.shape[:-1] + (a.shape[-1] + pad,), float("nan"), device="cuda")
        v = buf[..., 1:a.shape[-1] + 1]
        v.copy_(dev(a))
        return v
    big = t.full((E, d["W"].shape[1] + 5, d["W"].shape[2] + 3), float("nan"), device="cuda")
    W = big[:, 2:-3, 1:-2]
    W.copy_(dev(d["W"]))
    bufs = [guarded(M, N + 4)[0] for _ in range(2)]
    Y, Z = (b[64:64 + M * (N + 4)].view(M, N + 4)[:, :N] for b in bufs)
    bd.linear_f32_grouped(view(d["X"]), W, dev(d["offsets"]), rows=dev(d["rows"]), bias=view(d["b"]), act="silu", Z=Z,
                          Y=Y, trans_w=trans_w)
    _check(d, Y, Z, "silu", trans_w)
    for b in bufs:
        assert canaries_intact(b)
        assert np.all(host(b)[64:64 + M * (N + 4)].reshape(M, N + 4)[:, N:] == np.float32(1.2345e9))
    dbig = t.full(big.shape, 9.0, device="cuda")
    dwide = t.full((E, N + 2), 9.0, device="cuda")
    buf, _ = guarded(M, K + 4)
    dX = buf[64:64 + M * (K + 4)].view(M, K + 4)[:, :K]
    got = bd.linear_f32_grouped_bwd(view(d["dY"]), view(d["X"]), W, dev(d["offsets"]), rows=dev(d["rows"]),
                                    Z=view(d["Z"]), act="silu", trans_w=trans_w, dX=dX, dW=dbig[:, 2:-3, 1:-2],
                                    db=dwide[:, 1:-1])
    _check_bwd(d, got, "silu", trans_w)
    dbig[:, 2:-3, 1:-2] = 9
    dwide[:, 1:-1] = 9
    assert np.all(host(dbig) == 9) and np.all(host(dwide) == 9) and canaries_intact(buf)
    assert np.all(host(buf)[64:64 + M * (K + 4)].reshape(M, K + 4)[:, K:] == np.float32(1.2345e9))


def test_shared_weights():
    """Experts that are views of one matrix (stride 0)."""
    d = _inputs(50, 40, 30, 4, False, False)
    d["W"] = np.repeat(d["W"][:1], 4, 0)
    Y = bd.linear_f32_grouped(dev(d["X"]), dev(d["W"][:1]).expand(4, 30, 40), dev(d["offsets"]), bias=dev(d["b"]))
    _, y, _, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], None, d["b"], "none", False)
    lr.within(host(Y), y, ey)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nonfinite_stays_in_its_row_and_expert(bad):
    d = _inputs(150, 70, 50, 3, False, False, "even")
    clean, _ = _forward(d)
    d["X"][7, 20] = bad
    d["W"][2, 3, 5] = np.nan
    Y = host(_forward(d)[0])
    want = host(clean).copy()
    third = int(d["offsets"][2])
    assert not np.isfinite(Y[7]).any() and np.isnan(Y[third:, 5]).all()
    Y[7] = want[7]
    Y[third:, 5] = want[third:, 5]
    assert np.array_equal(Y, want)


# -------------------------------------------------------------- backward --

def _bwd(d, act, trans_w, **kw):
    return bd.linear_f32_grouped_bwd(dev(d["dY"]), dev(d["X"]), dev(d["W"]), dev(d["offsets"]), rows=_d(d["rows"]),
                                     Z=dev(d["Z"]), act=act, trans_w=trans_w, **kw)


def _check_bwd(d, got, act, trans_w):
    live = slice(int(d["offsets"][0]), int(d["offsets"][-1]))
    ref = er.linear_grouped_bwd(d["dY"], d["X"], d["W"], d["offsets"], d["rows"], d["Z"], act, trans_w)
    for (n, (r, e)), g in zip(ref.items(), got):
        g = host(g)
        if n == "dX":
            r, e, g = r[live], e[live], g[live]
        lr.within(g, r, e, n)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M,N,K,E", SHAPES)
def test_bwd(M, N, K, E, trans_w, gather):
    for kind, act in (("ragged", "gelu_tanh"), ("even", "none"), ("one", "silu")):
        d = _inputs(M, N, K, E, trans_w, gather, kind)
        _check_bwd(d, _bwd(d, act, trans_w), act, trans_w)


def _lopsided(M, E, rng):
    """Sizes from none to many times the mean, in no order."""
    s = np.bincount(rng.choice(E, M, p=rng.dirichlet(np.full(E, 0.15))), minlength=E)
    assert E < 8 or (s == 0).any() and s.max() >= 4 * M // E
    return s.tolist()


# groups of unlike size, whose gradients of the weights start with the largest:
# few, as many as lanes, more; far walks of one or two tiles per CU
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("M,N,K,E", [(300, 70, 40, 2), (2000, 65, 130, 9), (8192, 40, 33, 64), (9000, 33, 20, 70),
                                     (25700, 20, 24, 200), (2100, 70, 40, 2), (4200, 1100, 1000, 1)])
def test_bwd_of_groups_of_unlike_size(M, N, K, E, gather):
    for trans_w in (False, True):
        d = _inputs(M, N, K, E, trans_w, gather)
        d["offsets"] = er.sizes_to_offsets(_lopsided(M, E, np.random.default_rng([3, M, E])))
        got = _bwd(d, "none", trans_w)
        _check_bwd(d, got, "none", trans_w)
        dW = torch().full(tuple(got[1].shape), 2.0, device="cuda")
        _bwd(d, "none", trans_w, dW=dW, want=("dW",), accumulate=True)
        assert np.array_equal(host(dW), host(got[1]) + np.float32(2))


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("trans_w", [False, True])
def test_bwd_of_what_is_wanted_and_accumulated(act, trans_w):
    d = _inputs(170, 60, 50, 5, trans_w, True)
    full = _bwd(d, act, trans_w)
    for i, n in enumerate(("dX", "dW", "db")):
        got = _bwd(d, act, trans_w, want=(n,))
        assert all(g is None for j, g in enumerate(got) if j != i)
        assert np.array_equal(host(got[i]), host(full[i])), n
    t = torch()
    dW, db = t.full(tuple(full[1].shape), 2.0, device="cuda"), t.full(tuple(full[2].shape), 2.0, device="cuda")
    _bwd(d, act, trans_w, dW=dW, db=db, accumulate=True)
    assert np.array_equal(host(dW), host(full[1]) + np.float32(2))
    assert np.array_equal(host(db), host(full[2]) + np.float32(2))


def test_bwd_of_no_rows_is_zero():
    t = torch()
    o = t.zeros(4, dtype=t.int32, device="cuda")
    W = t.ones((3, 20, 30), device="cuda")
    dX, dW, db = bd.linear_f32_grouped_bwd(t.empty((0, 30), device="cuda"), t.empty((0, 20), device="cuda"), W, o)
    assert dX.shape == (0, 20) and not host(dW).any() and not host(db).any() and dW.shape == W.shape
    # rows, but none of them in a group
    dX, dW, db = bd.linear_f32_grouped_bwd(t.ones((9, 30), device="cuda"), t.ones((9, 20), device="cuda"), W, o)
    assert not host(dW).any() and not host(db).any()


def test_gradients_against_differences():
    M, N, K, E = 40, 30, 25, 4
    for trans_w in (False, True):
        d = _inputs(M, N, K, E, trans_w, True, seed=2)
        _, Z = _forward(d, "gelu_tanh", trans_w)
        dX, dW, db = bd.linear_f32_grouped_bwd(dev(d["dY"]), dev(d["X"]), dev(d["W"]), dev(d["offsets"]),
                                               rows=dev(d["rows"]), Z=Z, act="gelu_tanh", trans_w=trans_w)
        # a token's gradient is the sum of its rows'
        dXt = np.zeros(d["X"].shape)
        np.add.at(dXt, d["rows"], host(dX).astype(np.float64))
        g = {"X": dXt, "W": host(dW), "b": host(db)}

        def loss(p):
            out = 0.0
            for e, a, b in er.spans(d["offsets"]):
                z = p["X"][d["rows"][a:b]] @ (p["W"][e].T if trans_w else p["W"][e]) + p["b"][e]
                out += (lr.act(z, "gelu_tanh") * d["dY"][a:b]).sum()
            return out
        p = {n: d[n].astype(np.float64) for n in g}
        rng = np.random.default_rng(1)
        for n in g:
            v = rng.standard_normal(p[n].shape)
            h = 1e-5
            diff = (loss(dict(p, **{n: p[n] + h * v})) - loss(dict(p, **{n: p[n] - h * v}))) / (2 * h)
            assert abs((g[n] * v).sum() - diff) <= 1e-5 * np.abs(g[n] * v).sum() + 1e-6, (n, trans_w)


# ------------------------------------------------------------ large places --

def test_offsets_that_count_rows_too_often():
    """Groups out of order whose tiles, counted together, pass 2^31: nothing
    outside of the operands is read for their sums, and offsets in order give
    theirs afterwards."""
    t = torch()
    M, E = 2 ** 29 + 128, 1024
    dY = t.zeros((M, 1), device="cuda")
    dY[5], dY[M - 1] = 3.0, 4.0
    X, W = t.empty((M, 0), device="cuda"), t.empty((E, 0, 1), device="cuda")
    ws = t.empty(bd.linear_f32_grouped_bwd_ws_size("none", M, 1, E), dtype=t.uint8, device="cuda")
    o = t.tensor([0, M] * (E // 2) + [0], dtype=t.int32, device="cuda")
    bd.linear_f32_grouped_bwd(dY, X, W, o, want=("db",), workspace=ws)
    o = t.tensor([0] + [6] * (E - 1) + [M], dtype=t.int32, device="cuda")
    db = bd.linear_f32_grouped_bwd(dY, X, W, o, want=("db",), workspace=ws)[2]
    assert db[0, 0] == 3 and db[E - 1, 0] == 4 and not host(db)[1:-1].any()


def test_places_past_32_bit_offsets():
    """Experts 2^31 floats apart, rows at the widest leading dimension, and
    outputs whose rows lie past 2^31 floats."""
    t = torch()
    M, N, K, E = 70, 40, 30, 3
    d = _inputs(M, N, K, E, False, False)
    base = t.zeros(2 * (1 << 31) + K * N, device="cuda")
    W = base.as_strided((E, K, N), (1 << 31, N, 1))
    W.copy_(dev(d["W"]))
    ld = 1 << 22
    X = t.zeros((M - 1) * ld + K, device="cuda").as_strided((M, K), (ld, 1))
    X.copy_(dev(d["X"]))
    far = t.zeros((M - 1) * (1 << 25) + N, device="cuda").as_strided((M, N), (1 << 25, 1))
    bd.linear_f32_grouped(X, W, dev(d["offsets"]), bias=dev(d["b"]), Y=far)
    _, y, _, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], None, d["b"], "none", False)
    lr.within(host(far), y, ey)
    del far
    t.cuda.empty_cache()
    dW = t.zeros(2 * (1 << 31) + K * N, device="cuda").as_strided((E, K, N), (1 << 31, N, 1))
    got = bd.linear_f32_grouped_bwd(dev(d["dY"]), X, W, dev(d["offsets"]), Z=dev(d["Z"]), act="silu", dW=dW)
    _check_bwd(d, got, "silu", False)


@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("ld", [1 << 22, (1 << 22) + 5])
def test_outputs_with_rows_far_apart(ld, trans_w):
    """At the widest leading dimension whose tiles are 32-bit offsets, and past it."""
    t = torch()
    M, N, K, E = 70, 40, 30, 2
    d = _inputs(M, N, K, E, trans_w, True)
    far = lambda rows, cols: t.full((rows * ld,), 7.0, device="cuda").as_strided((rows, cols), (ld, 1))   # noqa: E731
    Y, Z = far(M, N), far(M, N)
    bd.linear_f32_grouped(dev(d["X"]), dev(d["W"]), dev(d["offsets"]), rows=dev(d["rows"]), bias=dev(d["b"]), act="silu",
                          Z=Z, Y=Y, trans_w=trans_w)
    _check(d, Y, Z, "silu", trans_w)
    assert (Y.as_strided((M, 9), (ld, 1), N) == 7).all() and (Z.as_strided((M, 9), (ld, 1), N) == 7).all()
    del Y, Z
    r, c = d["W"].shape[1:]
    dX, dW = far(M, K), far(E * r, c).as_strided((E, r, c), (r * ld, ld, 1))
    got = _bwd(d, "silu", trans_w, dX=dX, dW=dW)
    _check_bwd(d, got, "silu", trans_w)
    assert (dX.as_strided((M, 9), (ld, 1), K) == 7).all() and (dW.as_strided((E * r, 9), (ld, 1), c) == 7).all()
    once = host(dW)
    _bwd(d, "silu", trans_w, dX=dX, dW=dW, want=("dW",), accumulate=True)
    assert np.array_equal(host(dW), once + once)


def test_picked_rows_up_to_2_gib():
    """The last of the rows that may be picked ends just below 2^31 bytes."""
    t = torch()
    ld, K, N, E = 1 << 22, 24, 40, 2
    T = 128
    M = 90
    d = _inputs(M, N, K, E, True, True)
    X = t.zeros((T - 1) * ld + K, device="cuda").as_strided((T, K), (ld, 1))
    rng = np.random.default_rng(0)
    d["X"] = inputs.normal(rng, (T, K))
    X.copy_(dev(d["X"]))
    d["rows"] = rng.integers(0, T, M).astype(np.int32)
    d["rows"][:2] = T - 1, 0
    Y = bd.linear_f32_grouped(X, dev(d["W"]), dev(d["offsets"]), rows=dev(d["rows"]), bias=dev(d["b"]), trans_w=True)
    _, y, _, ey = er.linear_grouped(d["X"], d["W"], d["offsets"], d["rows"], d["b"], "none", True)
    lr.within(host(Y), y, ey)
    got = bd.linear_f32_grouped_bwd(dev(d["dY"]), X, dev(d["W"]), dev(d["offsets"]), rows=dev(d["rows"]),
                                    Z=dev(d["Z"]), act="silu", trans_w=True)
    _check_bwd(d, got, "silu", True)
