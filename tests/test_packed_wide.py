"""The packed layers' kernel for many rows and columns in each of its three
shapes (on 256 CUs): what the smaller shapes are tested for elsewhere, on rows
picked from the whole."""
import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gpu_util import dev, host, torch
from test_linear_mx8 import FN, _inputs, _ref

pytestmark = pytest.mark.gpu

WIDE = [(520, 4100), (1000, 6200), (2047, 4095)]


def _rows(M):
    return np.unique(np.r_[0, 31, 32, 63, 64, 127, 128, M // 2, M - 33, M - 1])


def _f16(v):
    return np.array([v], np.float16).view(np.int16)[0]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N", WIDE)
@pytest.mark.parametrize("K", [384, 330])
def test_nonfinite(bits, M, N, K):
    """A NaN in a byte, a power of two or a scale, in the first span of 128
    columns, a later one and the last (cut short or not), reaches its own row or
    column and no other cell."""
    t = torch()
    X8, XE, Q, S, _, _ = _inputs(bits, M, N, K)
    args = [dev(v) for v in (X8, XE, Q, S)]
    clean = FN[bits](*args)
    assert bool(t.isfinite(clean).all())

    def differs(Y, row=None, col=None):
        other = (Y != clean) & ~(t.isnan(Y) & t.isnan(clean))
        if row is not None:
            assert bool(t.isnan(Y[row]).all())
            other[row] = False
        else:
            assert bool(t.isnan(Y[:, col]).all())
            other[:, col] = False
        return bool(other.any())
    for m, k in ((0, 5), (M // 2, 200), (M - 1, K - 1), (33, 127), (70, 256)):
        x8, xe = args[0].clone(), args[1].clone()
        x8[m, k] = 0xff if m & 1 else 0x7f
        assert not differs(FN[bits](x8, args[1], *args[2:]), row=m)
        xe[m, k // 32] = 255
        Y, Y8, YE = FN[bits](args[0], xe, *args[2:], out="both")
        assert not differs(Y, row=m)
        assert bool((YE[m] == 255).all()) and bool((Y8[m] == 0x7f).all())
    for n, k in ((0, 0), (N - 1, K - 1), (N // 2, 130), (40, 64), (255, 320)):
        s = args[3].clone()
        s[n, k // 64] = int(_f16(np.nan))
        assert not differs(FN[bits](*args[:3], s), col=n)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N", WIDE)
def test_k_zero(bits, M, N):
    t = torch()
    u8 = dict(dtype=t.uint8, device="cuda")
    Y, Y8, YE = FN[bits](t.empty((M, 0), **u8), t.empty((M, 0), **u8), t.empty((N, 0), **u8),
                         t.empty((N, 0), dtype=t.float16, device="cuda"), bias=t.full((N,), -2.0, device="cuda"),
                         act="relu", residual=t.full((M, N), 448.0, device="cuda"), out="both")
    assert bool((Y == 448).all()) and bool((Y8 == 0x7e).all()) and bool((YE == 127).all())


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N", WIDE)
@pytest.mark.parametrize("K", [100, 256, 300])
def test_residual_in_place(bits, M, N, K):
    a = _inputs(bits, M, N, K)
    args = [dev(v) for v in a[:4]]
    r = dev(a[5])
    fresh = FN[bits](*args, bias=dev(a[4]), act="silu", residual=dev(a[5]))
    FN[bits](*args, bias=dev(a[4]), act="silu", residual=r, Y=r)
    assert torch().equal(r, fresh)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N", WIDE)
def test_every_byte_of_x(bits, M, N):
    """All 254 finite e4m3 bytes over powers of two from the smallest whose
    values bf16 holds exactly to the largest that fp32 sums hold."""
    K = 256
    b = np.arange(256, dtype=np.uint8)
    b[[0x7f, 0xff]] = 0
    X8 = np.stack([np.roll(b, 7 * m) for m in range(M)])
    X8[:, 32:64][(X8[:, 32:64] & 0x7f) >= 0x7f] = 0
    XE = np.tile(np.array([127, 3, 247 - 20, 100, 140, 127, 60, 30], np.uint8), (M, 1))
    Q = np.random.default_rng(3).integers(0, 256, (N, K * bits // 8), dtype=np.uint8)
    S = np.ones((N, K // 64), np.float16).view(np.int16)
    Y = FN[bits](dev(X8), dev(XE), dev(Q), dev(S))
    rows = _rows(M)
    y, e = _ref(bits, X8[rows], XE[rows], Q, S, None, None, "none")
    lr.within(host(Y[dev(rows)]), y, e)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("M,N", WIDE)
def test_activations_and_8_bit_output(bits, act, M, N):
    X8, XE, Q, S, b, R = _inputs(bits, M, N, 320)
    args = [dev(v) for v in (X8, XE, Q, S)]
    kw = dict(bias=dev(b), residual=dev(R), act=act)
    Y, Y8, YE = FN[bits](*args, **kw, out="both")
    rows = _rows(M)
    y, e = _ref(bits, X8[rows], XE[rows], Q, S, b, R[rows], act)
    got = host(Y[dev(rows)])
    lr.within(got, y, e, act)
    q, ee = lr.to_mx8(got.astype(np.float64))
    assert np.array_equal(host(YE)[rows], ee) and np.array_equal(host(Y8)[rows], q), "bytes of Y itself"
    q8, qe = FN[bits](*args, **kw, out="mx8")
    assert torch().equal(q8, Y8) and torch().equal(qe, YE)
    assert torch().equal(FN[bits](*args, **kw), Y)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (1, 64, 200), (9, 40, 160), (40, 96, 300), (150, 200, 256), (520, 4100, 140)])
@pytest.mark.parametrize("e", [0, 1, 2, 3, 4, 10])
def test_smallest_powers_of_two(bits, M, N, K, e):
    """Blocks at the lower end of the powers of two.  A value below 2^-133, the
    smallest step of bf16, is rounded to such a step (2^-134 off at most); all
    others, and products and sums as far as fp32's own subnormal steps (2^-149
    each), are as anywhere."""
    rng = np.random.default_rng([4, M, K])
    X8 = rng.integers(0, 256, (M, K), dtype=np.uint8)
    X8[(X8 & 0x7f) == 0x7f] = 0
    XE = np.full((M, -(-K // 32)), e, np.uint8)
    Q = rng.integers(0, 256, (N, -(-K * bits // 8)), dtype=np.uint8)
    S = np.full((N, -(-K // 64)), 1024.0, np.float16).view(np.int16)
    rows = np.arange(M) if M < 500 else _rows(M)
    w, x = np.abs(lr.weights(Q, S, bits, K)), lr.from_mx8(X8[rows], XE[rows])
    step = 2.0 ** -134 * (np.abs(x) < 2.0 ** -126)
    y, bound = _ref(bits, X8[rows], XE[rows], Q, S, None, None, "none")
    bound = bound - 1e-38 + step @ w.T + K * 2.0 ** -149 * 1024
    Y = FN[bits](dev(X8), dev(XE), dev(Q), dev(S))
    lr.within(host(Y[dev(rows)]), y, bound, "%d bits e %d" % (bits, e))
