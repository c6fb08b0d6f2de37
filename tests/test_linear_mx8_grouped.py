"""GPU parity of linear_q2_mx8_grouped and linear_q4_mx8_grouped against 64-bit
references, through the C ABI: as the packed layers, an addition is allowed a
whole step, 2 U."""
import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch
from test_linear_grouped import _sizes

pytestmark = pytest.mark.gpu

FN = {2: bd.linear_q2_mx8_grouped, 4: bd.linear_q4_mx8_grouped}


def _inputs(bits, M, N, K, E, gather=True, kind="ragged", seed=0):
    rng = np.random.default_rng([seed, bits, M, N, K, E])
    T = max(1, M // 2) if gather else M
    X8, XE = lr.to_mx8(inputs.normal(rng, (T, K)).astype(np.float64))
    return dict(X8=X8, XE=XE, Q=rng.integers(0, 256, (E, N, -(-K * bits // 8)), dtype=np.uint8),
                S=rng.uniform(-0.05, 0.05, (E, N, -(-K // 64))).astype(np.float16).view(np.int16),
                offsets=er.sizes_to_offsets(_sizes(kind, E, M, rng)), b=inputs.normal(rng, (E, N)),
                rows=rng.integers(0, T, M).astype(np.int32) if gather else None)


def _ref(bits, d, act="none"):
    K, N = d["X8"].shape[1], d["Q"].shape[1]
    x = lr.from_mx8(d["X8"], d["XE"])
    M = x.shape[0] if d["rows"] is None else d["rows"].size
    y, e = np.full((M, N), np.nan), np.full((M, N), np.nan)
    for i, a, b in er.spans(d["offsets"]):
        w = lr.weights(d["Q"][i], d["S"][i], bits, K)
        xe = x[a:b] if d["rows"] is None else x[d["rows"][a:b]]
        z = xe @ w.T
        ez = 2 * (K + 8) * lr.U * (np.abs(xe) @ np.abs(w.T)) + 1e-38
        if d["b"] is not None:
            z = z + d["b"][i].astype(np.float64)
            ez = ez + lr.U * np.abs(z)
        y[a:b] = lr.act(z, act)
        e[a:b] = lr.STEEP * ez + (lr.ACT_ERR * np.abs(z) if act not in ("none", "relu") else 0)
    return y, e


def _args(d):
    return [dev(d[n]) for n in ("X8", "XE", "Q", "S", "offsets")]


def _d(a):
    return None if a is None else dev(a)


# around tiles of 16, 32 and 64 rows and groups of columns of 64 and 128
SHAPES = [(1, 1, 1, 1), (1, 32, 64, 3), (8, 100, 1536, 64), (5, 70, 100, 2), (16, 96, 640, 16), (17, 33, 65, 1),
          (40, 129, 333, 4), (64, 64, 128, 2), (100, 260, 1000, 70), (129, 130, 96, 3), (300, 513, 200, 5),
          (513, 300, 130, 8), (600, 1100, 256, 4), (200, 48, 31, 300), (8, 1536, 12288, 8)]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("M,N,K,E", SHAPES)
def test_shapes(bits, M, N, K, E, gather):
    for kind in ("ragged", "even", "one"):
        d = _inputs(bits, M, N, K, E, gather, kind)
        Y = FN[bits](*_args(d), rows=_d(d["rows"]), bias=dev(d["b"]))
        y, e = _ref(bits, d)
        lr.within(host(Y), y, e, kind)


# one for each way the tiles are laid out: few rows with their k in 1, 4 and 16 (2, 4
# and 8) parts, cells of 32 x 32, and 32 to 128 rows by 128 or 256 columns
WAYS = [(30, 1200, 200, 30), (9, 210, 700, 3), (3, 300, 4200, 2), (100, 130, 1600, 3), (90, 100, 4170, 2),
        (60, 300, 130, 2), (700, 2100, 130, 40), (2100, 7000, 96, 8)]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("M,N,K,E", WAYS)
def test_ways(bits, M, N, K, E, gather):
    for kind in ("ragged", "even"):
        d = _inputs(bits, M, N, K, E, gather, kind)
        kw = dict(rows=_d(d["rows"]), bias=dev(d["b"]), act="relu")
        Y = FN[bits](*_args(d), **kw)
        y, e = _ref(bits, d, "relu")
        lr.within(host(Y), y, e, kind)
        Y, Y8, YE = FN[bits](*_args(d), **kw, out="both")
        lr.within(host(Y), y, e, kind)
        q, ee = lr.to_mx8(host(Y).astype(np.float64))
        assert np.array_equal(host(YE), ee) and np.array_equal(host(Y8), q), "bytes of Y itself"


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("M", [4, 60, 300])
def test_activations_and_8_bit_output(bits, act, M):
    d = _inputs(bits, M, 160, 320, 4)
    kw = dict(rows=dev(d["rows"]), bias=dev(d["b"]), act=act)
    Y, Y8, YE = FN[bits](*_args(d), **kw, out="both")
    y, e = _ref(bits, d, act)
    lr.within(host(Y), y, e, act)
    q, ee = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(host(YE), ee) and np.array_equal(host(Y8), q), "bytes of Y itself"
    p8, pe = FN[bits](*_args(d), **kw, out="mx8")
    assert np.array_equal(host(p8), q) and np.array_equal(host(pe), ee)
    alone = FN[bits](*_args(d), rows=dev(d["rows"]), act=act)
    y, e = _ref(bits, dict(d, b=None), act)
    lr.within(host(alone), y, e, "without bias")


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [30, 400])
def test_rows_outside_of_the_groups_are_left(bits, M):
    t = torch()
    d = _inputs(bits, M, 70, 200, 5)
    d["offsets"] = er.sizes_to_offsets(_sizes("ragged", 5, M - 11, np.random.default_rng(0)), 4)
    d["rows"][:4] = d["rows"][-7:] = -3
    Y = t.full((M, 70), 5.0, device="cuda")
    Y8 = t.full((M, 70), 0xAA, dtype=t.uint8, device="cuda")
    YE = t.full((M, 3), 0xAA, dtype=t.uint8, device="cuda")
    FN[bits](*_args(d), rows=dev(d["rows"]), bias=dev(d["b"]), Y=Y, Y8=Y8, YE=YE, out="both")
    y, e = _ref(bits, d)
    live, out = slice(4, M - 7), np.r_[0:4, M - 7:M]
    lr.within(host(Y)[live], y[live], e[live])
    assert np.all(host(Y)[out] == 5) and np.all(host(Y8)[out] == 0xAA) and np.all(host(YE)[out] == 0xAA)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("offsets", [[0, 9, 4, 20, 30], [-2 ** 31, 10, 2 ** 31 - 1, 5, -7], [40, 30, 20, 10, 0]])
@pytest.mark.parametrize("M", [12, 90, 500])
def test_offsets_out_of_order_stay_inside(bits, M, offsets):
    d = _inputs(bits, M, 70, 130, 4)
    d["offsets"] = np.array(offsets, np.int32)
    d["rows"][::2] = np.array([-1, 2 ** 31 - 1, -2 ** 31], np.int32)[np.arange(d["rows"][::2].size) % 3]
    buf, Y = guarded(M, 70)
    FN[bits](*_args(d), rows=dev(d["rows"]), Y=Y)
    assert canaries_intact(buf)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [6, 80, 400])
def test_strides_and_what_lies_around(bits, M):
    t = torch()
    N, K, E = 70, 150, 3
    d = _inputs(bits, M, N, K, E)

    def view(a, *pad):
        a = dev(a)
        buf = t.full([n + p for n, p in zip(a.shape, pad)], 0x7f, dtype=a.dtype, device="cuda")
        v = buf[tuple(slice(p // 2, p // 2 + n) for n, p in zip(a.shape, pad))]
        v.copy_(a)
        return v
    buf, _ = guarded(M, N + 5)
    Y = buf[64:64 + M * (N + 5)].view(M, N + 5)[:, :N]
    Y8 = t.full((M + 2, N + 5), 0xAA, dtype=t.uint8, device="cuda")
    YE = t.full((M + 2, 6), 0xAA, dtype=t.uint8, device="cuda")
    FN[bits](view(d["X8"], 0, 3), view(d["XE"], 0, 3), view(d["Q"], 0, 3, 5), view(d["S"], 0, 2, 3), dev(d["offsets"]),
             rows=dev(d["rows"]), bias=view(d["b"], 0, 3), Y=Y, Y8=Y8[1:M + 1, 2:N + 2], YE=YE[1:M + 1, 1:4], out="both")
    y, e = _ref(bits, d)
    lr.within(host(Y), y, e)
    q, ee = lr.to_mx8(host(Y).astype(np.float64))
    g, ge = host(Y8), host(YE)
    assert np.array_equal(g[1:M + 1, 2:N + 2], q) and np.array_equal(ge[1:M + 1, 1:4], ee)
    g[1:M + 1, 2:N + 2] = 0xAA
    ge[1:M + 1, 1:4] = 0xAA
    assert np.all(g == 0xAA) and np.all(ge == 0xAA) and canaries_intact(buf)
    assert np.all(host(buf)[64:64 + M * (N + 5)].reshape(M, N + 5)[:, N:] == np.float32(1.2345e9))


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [9, 60, 300])
def test_nan_stays_in_its_row_and_column(bits, M):
    d = _inputs(bits, M, 70, 200, 3, gather=False, kind="even")
    clean = host(FN[bits](*_args(d), bias=dev(d["b"]))).copy()
    d["X8"][1, 5] = 0x7f
    s = d["S"].view(np.float16)
    s[2, 9, 1] = np.nan
    Y = host(FN[bits](*_args(d), bias=dev(d["b"]))).copy()
    third = int(d["offsets"][2])
    assert np.isnan(Y[1]).all() and np.isnan(Y[third:, 9]).all()
    Y[1] = clean[1]
    Y[third:, 9] = clean[third:, 9]
    assert np.array_equal(Y, clean)


@pytest.mark.parametrize("bits", [2, 4])
def test_no_inputs_and_no_rows(bits):
    d = _inputs(bits, 20, 40, 0, 3, gather=False)
    Y = FN[bits](*_args(d), bias=dev(d["b"]))
    y, e = _ref(bits, d)
    lr.within(host(Y), y, e)
    d = _inputs(bits, 0, 40, 64, 3, gather=False)
    assert FN[bits](*_args(d)).shape == (0, 40)


def test_places_past_32_bit_offsets():
    """Experts 2^32 bytes apart, and rows 2^30 bytes apart."""
    t = torch()
    d = _inputs(4, 6, 40, 128, 3, gather=False)
    Q = t.zeros(2 * (1 << 32) + 40 * 64, dtype=t.uint8, device="cuda").as_strided((3, 40, 64), (1 << 32, 64, 1))
    Q.copy_(dev(d["Q"]))
    X = t.zeros(5 * (1 << 30) + 128, dtype=t.uint8, device="cuda").as_strided((6, 128), (1 << 30, 1))
    X.copy_(dev(d["X8"]))
    a = _args(d)
    Y = bd.linear_q4_mx8_grouped(X, a[1], Q, a[3], a[4], bias=dev(d["b"]))
    y, e = _ref(4, d)
    lr.within(host(Y), y, e)
