"""GPU parity of expert_groups, expert_combine and expert_combine_bwd, through
the C ABI."""
import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu


def _ids(T, k, E, seed=0, missing=0.0):
    rng = np.random.default_rng([seed, T, k, E])
    ids = rng.integers(0, max(E, 1), (T, k)).astype(np.int32)
    if missing:
        bad = rng.choice(np.array([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1]), (T, k))
        ids = np.where(rng.random((T, k)) < missing, bad, ids).astype(np.int32)
    return ids


# pairs around a wave, its rounds, one workgroup's share and many; experts
# around a wave, a round of the scan and the largest number
GROUPS = [(1, 1, 1), (1, 8, 64), (3, 2, 7), (64, 1, 8), (65, 1, 8), (128, 4, 16), (171, 3, 63), (512, 1, 64),
          (513, 1, 65), (300, 2, 100), (1000, 8, 128), (4097, 2, 255), (2000, 6, 1000), (1000, 1, 1023),
          (5000, 3, 1024), (16384, 4, 8), (40000, 8, 64)]


@pytest.mark.parametrize("missing", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("T,k,E", GROUPS)
def test_groups(T, k, E, missing):
    ids = _ids(T, k, E, missing=missing)
    got = bd.expert_groups(dev(ids), E)
    for g, w in zip(got, er.groups(ids, E)):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (3, 0, 5), (0, 0, 0), (6, 2, 0)])
def test_groups_of_nothing(T, k, E):
    ids = _ids(T, k, E)
    offsets, rows, pos = (host(a) for a in bd.expert_groups(dev(ids), E))
    assert offsets.shape == (E + 1,) and not offsets.any() and rows.shape == (T * k,) and pos.shape == (T, k)
    assert np.all(pos == -1) if E == 0 else pos.size == 0


@pytest.mark.parametrize("one", [0, 5, 11])
@pytest.mark.parametrize("T", [100, 5000])
def test_groups_of_one_expert(T, one):
    ids = np.full((T, 2), one, np.int32)
    offsets, rows, pos = (host(a) for a in bd.expert_groups(dev(ids), 12))
    assert np.array_equal(offsets, np.where(np.arange(13) > one, 2 * T, 0))
    assert np.array_equal(rows, np.arange(2 * T) // 2) and np.array_equal(pos.reshape(-1), np.arange(2 * T))


# either side of where more waves and more workgroups take over
@pytest.mark.parametrize("T,k,E", [(767, 1, 64), (768, 1, 64), (769, 1, 64), (8191, 1, 7), (8192, 1, 7), (8193, 1, 1000), (9000, 1, 511),
                                   (9000, 1, 512), (81919, 1, 40), (81920, 1, 40),
                                   (65536, 2, 256), (131072, 4, 64), (131073, 5, 3), (262147, 4, 1024)])
def test_groups_by_workgroups(T, k, E):
    test_groups(T, k, E, 0.1)


@pytest.mark.parametrize("T,k", [(9, 3), (700, 5)])
def test_groups_strides_and_what_lies_around(T, k):
    t = torch()
    ids = _ids(T, k, 20, missing=0.1)
    wide = t.full((T, k + 3), 4, dtype=t.int32, device="cuda")
    wide[:, 1:k + 1] = dev(ids)
    P = t.full((T + 2, k + 4), -77, dtype=t.int32, device="cuda")
    flat = t.full((21 + T * k + 30,), -77, dtype=t.int32, device="cuda")
    bd.expert_groups(wide[:, 1:k + 1], 20, offsets=flat[5:26], rows=flat[30:30 + T * k], pos=P[1:T + 1, 2:k + 2])
    o, r, p = er.groups(ids, 20)
    f, P = host(flat), host(P)
    assert np.array_equal(f[5:26], o) and np.array_equal(f[30:30 + T * k], r) and np.array_equal(P[1:T + 1, 2:k + 2], p)
    f[5:26] = f[30:30 + T * k] = -77
    P[1:T + 1, 2:k + 2] = -77
    assert np.all(f == -77) and np.all(P == -77)


# --------------------------------------------------------------- combine --

COMBINE = [(1, 1, 1), (1, 8, 768), (3, 2, 255), (2, 3, 256), (5, 4, 257), (346, 2, 768), (70, 5, 1000),
           (33, 9, 1025), (600, 3, 2048), (9, 1, 4099), (2000, 2, 36), (1200, 4, 1031), (40, 8, 64), (17, 5, 65),
           (9, 3, 128), (8, 4, 129), (1100, 7, 101), (3, 9, 3), (2, 1, 64)]


def _combine_inputs(T, k, K, seed=0, missing=0.0):
    rng = np.random.default_rng([seed, T, k, K])
    _, _, pos = er.groups(_ids(T, k, 16, seed, missing), 16)
    n = lambda *s: inputs.normal(rng, s)   # noqa: E731
    return n(T * k, K), pos, n(T, k), n(T, K), n(T, K)


@pytest.mark.parametrize("missing", [0.0, 0.3])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,k,K", COMBINE)
def test_combine(T, k, K, residual, weighted, missing):
    Y, pos, w, R, _ = _combine_inputs(T, k, K, missing=missing)
    w, R = (w if weighted else None), (R if residual else None)
    out = bd.expert_combine(dev(Y), dev(pos), weights=None if w is None else dev(w),
                            residual=None if R is None else dev(R))
    ref, e = er.combine(Y, pos, w, R)
    lr.within(host(out), ref, e)


def test_combine_edges():
    t = torch()
    Y, pos, w, R, _ = _combine_inputs(50, 3, 300)
    # no pairs, no rows, no tokens
    z = t.empty((50, 0), dtype=t.int32, device="cuda")
    assert np.array_equal(host(bd.expert_combine(dev(Y), z, residual=dev(R))), R)
    assert not host(bd.expert_combine(dev(Y), z)).any()
    none = t.empty((0, 300), device="cuda")
    assert np.array_equal(host(bd.expert_combine(none, dev(pos), residual=dev(R))), R)
    assert bd.expert_combine(dev(Y), z[:0]).shape == (0, 300)
    # entries past the end add nothing, and one row may be named by many
    far = pos.copy()
    far[::2] = 2 ** 31 - 1
    far[1::4] = 7
    lr.within(host(bd.expert_combine(dev(Y), dev(far), weights=dev(w))), *er.combine(Y, far, w, None))
    # rows that nothing names may hold anything
    Y2 = np.concatenate([Y, np.full((4, 300), np.nan, np.float32)])
    assert np.array_equal(host(bd.expert_combine(dev(Y2), dev(pos), weights=dev(w))),
                          host(bd.expert_combine(dev(Y), dev(pos), weights=dev(w))))
    # the residual updated in place
    r = dev(R)
    want = host(bd.expert_combine(dev(Y), dev(pos), weights=dev(w), residual=dev(R)))
    assert np.array_equal(host(bd.expert_combine(dev(Y), dev(pos), weights=dev(w), residual=r, out=r)), want)


@pytest.mark.parametrize("T,k,K", [(7, 3, 130), (2, 2, 1029), (300, 2, 2049)])
def test_combine_strides_and_what_lies_around(T, k, K):
    t = torch()
    Y, pos, w, R, dO = _combine_inputs(T, k, K)

    def view(a, pad, fill):
        buf = t.full((a.shape[0], a.shape[1] + pad), fill, dtype=t.int32 if a.dtype == np.int32 else t.float32,
                     device="cuda")
        v = buf[:, 1:a.shape[1] + 1]
        v.copy_(dev(a))
        return v
    a = [view(Y, 3, float("nan")), view(pos, 2, 5), view(w, 4, float("nan")), view(R, 2, float("nan"))]
    buf, _ = guarded(T, K + 3)
    out = buf[64:64 + T * (K + 3)].view(T, K + 3)[:, :K]
    bd.expert_combine(a[0], a[1], weights=a[2], residual=a[3], out=out)
    lr.within(host(out), *er.combine(Y, pos, w, R))
    assert canaries_intact(buf)
    assert np.all(host(buf)[64:64 + T * (K + 3)].reshape(T, K + 3)[:, K:] == np.float32(1.2345e9))
    buf, _ = guarded(T * k, K + 3)
    dY = buf[64:64 + T * k * (K + 3)].view(T * k, K + 3)[:, :K]
    wide = t.full((T, k + 2), 9.0, device="cuda")
    bd.expert_combine_bwd(view(dO, 1, float("nan")), a[1], Y=a[0], weights=a[2], dY=dY, dw=wide[:, 1:k + 1])
    _check_bwd(host(dY), host(wide)[:, 1:k + 1], Y, pos, w, dO)
    assert np.all(host(wide)[:, [0, k + 1]] == 9) and canaries_intact(buf)
    assert np.all(host(buf)[64:64 + T * k * (K + 3)].reshape(T * k, K + 3)[:, K:] == np.float32(1.2345e9))


def _check_bwd(dY, dw, Y, pos, w, dO):
    """dY is one product, exactly rounded; dw a sum of K products over at most
    K/64 additions in a lane and a tree."""
    T, k = pos.shape
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if p < 0:
                assert dw is None or dw[t, j] == 0
                continue
            if dY is not None:
                assert np.array_equal(dY[p], dO[t] if w is None else w[t, j] * dO[t])
            if dw is not None:
                m = dO[t].astype(np.float64) * Y[p]
                assert abs(dw[t, j] - m.sum()) <= (Y.shape[1] / 64 + 20) * lr.U * np.abs(m).sum() + 1e-44


@pytest.mark.parametrize("missing", [0.0, 0.3])
@pytest.mark.parametrize("T,k,K", [c for c in COMBINE if c[0] * c[1] < 2000])
def test_combine_bwd(T, k, K, missing):
    Y, pos, w, _, dO = _combine_inputs(T, k, K, missing=missing)
    full = torch().full((T * k, K), 7.0, device="cuda")
    dY, dw = bd.expert_combine_bwd(dev(dO), dev(pos), Y=dev(Y), weights=dev(w), dY=full)
    _check_bwd(host(dY), host(dw), Y, pos, w, dO)
    unnamed = np.setdiff1d(np.arange(T * k), pos[pos >= 0])
    assert np.all(host(dY)[unnamed] == 7)
    only, none = bd.expert_combine_bwd(dev(dO), dev(pos), want=("dY",))
    assert none is None
    _check_bwd(host(only), None, Y, pos, None, dO)
    none, dw2 = bd.expert_combine_bwd(dev(dO), dev(pos), Y=dev(Y), weights=dev(w), want=("dw",))
    assert none is None and np.array_equal(host(dw2), host(dw))


def test_rows_past_32_bit_offsets():
    t = torch()
    T, k, K, ld = 2, 2, 64, 1 << 30
    Y, pos, w, _, dO = _combine_inputs(T, k, K)
    buf = t.zeros((T * k - 1) * ld + K, device="cuda")
    far = buf.as_strided((T * k, K), (ld, 1))
    far.copy_(dev(Y))
    lr.within(host(bd.expert_combine(far, dev(pos), weights=dev(w))), *er.combine(Y, pos, w, None))
    dY, dw = bd.expert_combine_bwd(dev(dO), dev(pos), Y=far, weights=dev(w))
    _check_bwd(host(dY), host(dw), Y, pos, w, dO)
    bd.expert_combine_bwd(dev(dO), dev(pos), weights=dev(w), dY=far, want=("dY",))
    _check_bwd(host(far), None, Y, pos, w, dO)
