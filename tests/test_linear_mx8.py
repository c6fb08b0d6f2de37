"""GPU parity of linear_q2_mx8 and linear_q4_mx8 against 64-bit references,
through the C ABI: codes and 8-bit values enter exactly, so the only errors
are those of fp32 sums.  A matrix instruction's adder may cut instead of
round, so an addition is allowed a whole step, 2 U."""
import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import canaries_intact, dev, guarded, host, torch

pytestmark = pytest.mark.gpu

FN = {2: bd.linear_q2_mx8, 4: bd.linear_q4_mx8}


def _inputs(bits, M, N, K, seed=0, spread=0):
    rng = np.random.default_rng([seed, bits, M, N, K])
    x = inputs.normal(rng, (M, K)).astype(np.float64)
    if spread:
        x = x * 2.0 ** rng.integers(-spread, spread + 1, (M, K))
    X8, XE = lr.to_mx8(x)
    Q = rng.integers(0, 256, (N, -(-K * bits // 8)), dtype=np.uint8)
    S = rng.uniform(-0.05, 0.05, (N, -(-K // 64))).astype(np.float16).view(np.int16)
    return X8, XE, Q, S, inputs.normal(rng, (N,)), inputs.normal(rng, (M, N))


def _ref(bits, X8, XE, Q, S, b, R, act):
    K = X8.shape[1]
    w, x = lr.weights(Q, S, bits, K), lr.from_mx8(X8, XE)
    z = x @ w.T
    e = 2 * (K + 8) * lr.U * (np.abs(x) @ np.abs(w.T)) + 1e-38
    if b is not None:
        z = z + b.astype(np.float64)
        e = e + lr.U * np.abs(z)
    y = lr.act(z, act)
    e = lr.STEEP * e + (lr.ACT_ERR * np.abs(z) if act not in ("none", "relu") else 0)
    if R is not None:
        y = y + R.astype(np.float64)
        e = e * 1.01 + lr.U * np.abs(y)
    return y, e


def _d(a):
    return None if a is None else dev(a)


SHAPES = [(1, 1, 1), (1, 32, 64), (1, 100, 1536), (2, 33, 65), (3, 64, 31), (5, 70, 100),
          (8, 31, 200), (16, 96, 640), (31, 65, 127), (32, 32, 128), (33, 200, 64), (40, 129, 333),
          (64, 64, 512), (100, 260, 1000), (129, 130, 96), (200, 513, 1536), (513, 300, 200),
          (1, 12288, 1536), (7, 1536, 12288), (300, 1536, 2050)]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(bits, M, N, K):
    a = _inputs(bits, M, N, K)
    Y = FN[bits](*(dev(v) for v in a[:4]), bias=dev(a[4]), residual=dev(a[5]))
    y, e = _ref(bits, *a, "none")
    lr.within(host(Y), y, e, "%d bits %dx%dx%d" % (bits, M, N, K))


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (3, 97, 70), (70, 300, 192), (150, 260, 200)])
def test_integers_exactly(bits, M, N, K):
    """Small integers and scales of 1/2: every product and sum is exact, so a
    wrong order of columns, code map or power of two shows in full."""
    rng = np.random.default_rng([1, M])
    x = rng.integers(-15, 16, (M, K)).astype(np.float64) * 2.0 ** rng.integers(-3, 4, (M, -(-K // 32))).repeat(32, 1)[:, :K]
    X8, XE = lr.to_mx8(x)
    assert np.array_equal(lr.from_mx8(X8, XE), x)
    Q = rng.integers(0, 256, (N, -(-K * bits // 8)), dtype=np.uint8)
    S = np.where(rng.random((N, -(-K // 64))) < 0.5, 0.5, -2.0).astype(np.float16).view(np.int16)
    Y = host(FN[bits](dev(X8), dev(XE), dev(Q), dev(S)))
    assert np.array_equal(Y.astype(np.float64), x @ lr.weights(Q, S, bits, K).T)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [1, 150])
def test_every_byte_of_x(bits, M):
    """All 254 finite e4m3 bytes against one code at a time, over the whole
    range of powers of two that fp32 sums hold."""
    K = 256
    b = np.arange(256, dtype=np.uint8)
    b[[0x7f, 0xff]] = 0
    X8 = np.tile(b, (M, 1))
    XE = np.tile(np.array([127, 1, 247 - 20, 100, 140, 127, 60, 30], np.uint8), (M, 1))
    Q = np.zeros((K, K * bits // 8), np.uint8)
    rng = np.random.default_rng(3)
    Q[:] = rng.integers(0, 256, Q.shape)
    S = np.ones((K, K // 64), np.float16).view(np.int16)
    Y = FN[bits](dev(X8), dev(XE), dev(Q), dev(S))
    y, e = _ref(bits, X8, XE, Q, S, None, None, "none")
    lr.within(host(Y), y, e)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("M", [1, 40, 140])
def test_activations_and_8_bit_output(bits, act, M):
    a = _inputs(bits, M, 160, 320)
    args = [dev(v) for v in a[:4]]
    kw = dict(bias=dev(a[4]), residual=dev(a[5]), act=act)
    y, e = _ref(bits, *a, act)
    Y, Y8, YE = FN[bits](*args, **kw, out="both")
    lr.within(host(Y), y, e, act)
    q, ee = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(host(YE), ee) and np.array_equal(host(Y8), q), "bytes of Y itself"
    assert np.array_equal(host(FN[bits](*args, **kw)), host(Y))
    q8, qe = FN[bits](*args, **kw, out="mx8")
    assert np.array_equal(host(q8), host(Y8)) and np.array_equal(host(qe), host(YE))


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("N", [1, 31, 33, 65, 100, 191])
@pytest.mark.parametrize("M", [1, 34, 130])
def test_8_bit_output_of_ragged_width(bits, N, M):
    a = _inputs(bits, M, N, 96)
    Y, Y8, YE = FN[bits](*(dev(v) for v in a[:4]), bias=dev(a[4]), out="both")
    q, e = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(host(YE), e) and np.array_equal(host(Y8), q)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [1, 33, 140])
@pytest.mark.parametrize("K", [96, 100, 190])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_offsets_and_what_lies_around(bits, M, K, shift):
    """Padded, misaligned rows; bits of codes past K, scales and bytes past
    the row are poisoned (NaN where a byte can hold one)."""
    t = torch()
    N = 75
    X8, XE, Q, S, b, R = _inputs(bits, M, N, K)

    def view(a, poison, step=1):
        pad = 32 if not shift else 7
        buf = t.full((a.shape[0], a.shape[1] + pad), poison, dtype=t.from_numpy(a[:0]).dtype, device="cuda")
        off = shift * step
        buf[:, off:off + a.shape[1]].copy_(dev(a))
        return buf[:, off:off + a.shape[1]]
    Qp = Q.copy()
    extra = K * bits % 8
    if extra:
        Qp[:, -1] |= (0xFF << extra) & 0xFF
    buf, _ = guarded(M, N + 7)
    Y = buf[64:64 + M * (N + 7)].view(M, N + 7)[:, :N]
    nb = -(-N // 32)
    Y8 = t.full((M + 2, N + 5), 0xAA, dtype=t.uint8, device="cuda")
    YE = t.full((M + 2, nb + 3), 0xAA, dtype=t.uint8, device="cuda")
    FN[bits](view(X8, 0x7f), view(XE, 255), view(Qp, 0xFF), view(S, 0x7e00), bias=dev(b),
             residual=dev(R), Y=Y, Y8=Y8[1:M + 1, 2:N + 2], YE=YE[1:M + 1, 1:nb + 1], out="both")
    y, e = _ref(bits, X8, XE, Q, S, b, R, "none")
    lr.within(host(Y), y, e)
    assert canaries_intact(buf)
    assert np.all(host(buf)[64:64 + M * (N + 7)].reshape(M, N + 7)[:, N:] == np.float32(1.2345e9))
    q, ee = host(Y8), host(YE)
    want = lr.to_mx8(host(Y).astype(np.float64))
    assert np.array_equal(q[1:M + 1, 2:N + 2], want[0]) and np.array_equal(ee[1:M + 1, 1:nb + 1], want[1])
    q[1:M + 1, 2:N + 2] = 0xAA
    ee[1:M + 1, 1:nb + 1] = 0xAA
    assert np.all(q == 0xAA) and np.all(ee == 0xAA)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [1, 6, 140])
def test_nonfinite(bits, M):
    X8, XE, Q, S, b, R = _inputs(bits, M, 96, 192)
    m = M // 2
    clean = host(FN[bits](dev(X8), dev(XE), dev(Q), dev(S)))
    for how in ("byte", "scale"):
        x8, xe = X8.copy(), XE.copy()
        if how == "byte":
            x8[m, 70] = 0x7f
        else:
            xe[m, 3] = 255
        Y, Y8, YE = (host(a) for a in FN[bits](dev(x8), dev(xe), dev(Q), dev(S), out="both"))
        assert np.isnan(Y[m]).all(), how
        assert np.array_equal(np.delete(Y, m, 0), np.delete(clean, m, 0))
        assert np.all(YE[m] == 255) and np.all(Y8[m] == 0x7f)
    s = S.copy()
    s[40, 1] = np.array([np.nan], np.float16).view(np.int16)[0]
    Y = host(FN[bits](dev(X8), dev(XE), dev(Q), dev(s)))
    assert np.isnan(Y[:, 40]).all() and np.array_equal(np.delete(Y, 40, 1), np.delete(clean, 40, 1))


@pytest.mark.parametrize("bits", [2, 4])
def test_wide_range_of_magnitudes(bits):
    a = _inputs(bits, 40, 64, 640, spread=12)
    Y = FN[bits](*(dev(v) for v in a[:4]))
    y, e = _ref(bits, *a[:4], None, None, "none")
    lr.within(host(Y), y, e)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M", [1, 150])
def test_k_zero_and_in_place(bits, M):
    t = torch()
    u8 = dict(dtype=t.uint8, device="cuda")
    Y = FN[bits](t.empty((M, 0), **u8), t.empty((M, 0), **u8), t.empty((40, 0), **u8),
                 t.empty((40, 0), dtype=t.float16, device="cuda"), bias=t.full((40,), -2.0, device="cuda"))
    assert np.all(host(Y) == -2)
    a = _inputs(bits, M, 96, 128)
    args = [dev(v) for v in a[:4]]
    r = dev(a[5])
    fresh = FN[bits](*args, residual=dev(a[5]))
    FN[bits](*args, residual=r, Y=r)
    assert np.array_equal(host(r), host(fresh))


def _poisoned(a, poison, pad=7):
    """a as the middle of a wider tensor whose other columns hold `poison`."""
    t = torch()
    buf = t.full((a.shape[0], a.shape[1] + pad), poison, dtype=t.from_numpy(a[:0]).dtype, device="cuda")
    buf[:, 1:1 + a.shape[1]].copy_(dev(a))
    return buf[:, 1:1 + a.shape[1]]


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("K", [5, 120, 128, 256, 333, 640])
@pytest.mark.parametrize("M,N", [(520, 4100), (1000, 6200), (2047, 4095)])
def test_many_rows(bits, M, N, K):
    """Enough rows and columns for a wave per 32 columns, in each of its three
    shapes; misaligned rows between NaN bytes."""
    X8, XE, Q, S, b, R = _inputs(bits, M, N, K)
    y, e = _ref(bits, X8, XE, Q, S, b, R, "none")
    Y, Y8, YE = FN[bits](_poisoned(X8, 0x7f), _poisoned(XE, 255), _poisoned(Q, 0xFF), _poisoned(S, 0x7e00),
                         bias=dev(b), residual=dev(R), out="both")
    Y = host(Y)
    lr.within(Y, y, e, "%d bits %dx%dx%d" % (bits, M, N, K))
    rows = np.r_[0:40, M - 40:M]
    q, ee = lr.to_mx8(Y[rows].astype(np.float64))
    assert np.array_equal(host(YE)[rows], ee) and np.array_equal(host(Y8)[rows], q)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N,K", [(17, 33, 5), (20, 40, 77), (33, 70, 129), (33, 70, 4099), (20, 97, 5000),
                                   (64, 500, 4096), (90, 300, 8225), (400, 700, 450)])
def test_runs_of_k(bits, M, N, K):
    """A wave per run of k: fewer pairs than runs, ragged last pairs, eight
    runs; misaligned rows between NaN bytes."""
    X8, XE, Q, S, b, R = _inputs(bits, M, N, K)
    y, e = _ref(bits, X8, XE, Q, S, b, None, "none")
    Y = FN[bits](_poisoned(X8, 0x7f), _poisoned(XE, 255), _poisoned(Q, 0xFF), _poisoned(S, 0x7e00), bias=dev(b))
    lr.within(host(Y), y, e, "%d bits %dx%dx%d" % (bits, M, N, K))


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("K", [130, 143, 144, 145, 159, 160, 161, 190, 191, 193, 255])
@pytest.mark.parametrize("M,N", [(1, 40), (9, 40), (40, 40), (1000, 6200)])
def test_ragged_rows_exactly(bits, M, N, K):
    """Rows cut at every kind of place: integers, so that a byte too many or
    too few shows in full.  (Sums stay below 2^24 halves.)"""
    rng = np.random.default_rng([2, K])
    x = rng.integers(-15, 16, (M, K)).astype(np.float64)
    X8, XE = lr.to_mx8(x)
    Q = rng.integers(0, 256, (N, -(-K * bits // 8)), dtype=np.uint8)
    S = np.ones((N, -(-K // 64)), np.float16).view(np.int16)
    Y = host(FN[bits](_poisoned(X8, 0x7f), _poisoned(XE, 255), _poisoned(Q, 0xFF), _poisoned(S, 0x7e00)))
    assert np.array_equal(Y.astype(np.float64), x @ lr.weights(Q, S, bits, K).T)


def test_against_the_packed_gemv():
    """One row whose 8-bit values are exact: the same sums as gemv_q2 and
    gemv_q4 on fp32 x, within both accuracy bounds."""
    for bits, gemv in ((2, bd.gemv_q2), (4, bd.gemv_q4)):
        X8, XE, Q, S, _, _ = _inputs(bits, 1, 500, 1536)
        x = lr.from_mx8(X8, XE)[0].astype(np.float32)
        y, e = _ref(bits, X8, XE, Q, S, None, None, "none")
        bound = 1e-4 * (np.abs(x.astype(np.float64)) @ np.abs(lr.weights(Q, S, bits, 1536).T))
        lr.within(host(gemv(dev(Q), dev(S), dev(x))), y[0], bound)
        lr.within(host(FN[bits](dev(X8), dev(XE), dev(Q), dev(S)))[0], y[0], e[0])


def test_binding_refusals():
    t = torch()
    X8, XE, Q, S, b, R = (dev(v) for v in _inputs(4, 4, 64, 96))
    with pytest.raises(ValueError):
        bd.linear_q4_mx8(X8, XE, Q, S, out="bf16")
    with pytest.raises(ValueError):
        bd.linear_q4_mx8(X8, XE[:, :2], Q, S)
    with pytest.raises(ValueError):
        bd.linear_q4_mx8(X8, XE, Q[:, :47], S)
    with pytest.raises(TypeError):
        bd.linear_q4_mx8(X8, XE, Q, S.to(t.int32))
    with pytest.raises(ValueError):
        bd.linear_q4_mx8(X8, XE, Q, S, act="swish")
    f8 = bd.linear_q4_mx8(X8.view(t.float8_e4m3fn), XE.view(t.float8_e8m0fnu), Q, S)
    assert np.array_equal(host(f8), host(bd.linear_q4_mx8(X8, XE, Q, S)))
