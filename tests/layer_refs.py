"""Plain 64-bit references of the dense layers and the norm, shared by their
tests: activations and slopes, the 8-bit row format, packed weights, and the
error terms that tolerances are built from."""
import math

import numpy as np

U = 2.0 ** -24                       # half a step of fp32, relative
ACTS = ("none", "relu", "gelu_tanh", "gelu_erf", "silu")
C = math.sqrt(2 / math.pi)
_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])

# |act'| <= 1.13 for all of them (GELU's steepest slope is 1.129)
STEEP = 1.13
# An activation's own error relative to |z|: the weight p(z) in [0, 1] that
# multiplies z is made of an exponential (or an error function, whose rational
# form is within 1.5e-7 < 2^-22 of 1), a sum and a quotient: a few units in the
# last place of 1 each, at most 16 of them (2^-19) together.
ACT_ERR = 2.0 ** -19
# A slope's own error, absolute: p (1 - p) has an absolute error of a few
# steps of 1 and is multiplied by at most 20 before it vanishes.
SLOPE_ERR = 2.0 ** -18


def act(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu_tanh":
        return z / (1 + np.exp(np.minimum(-2 * C * (z + 0.044715 * z ** 3), 700)))
    if name == "gelu_erf":
        return 0.5 * z * _erfc(-z / math.sqrt(2))
    if name == "silu":
        return z / (1 + np.exp(np.minimum(-z, 700)))
    return z


def slope(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu_tanh":
        p = 1 / (1 + np.exp(np.minimum(-2 * C * (z + 0.044715 * z ** 3), 700)))
        return p + p * (1 - p) * 2 * C * (z + 3 * 0.044715 * z ** 3)
    if name == "gelu_erf":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        p = 1 / (1 + np.exp(np.minimum(-z, 700)))
        return p + z * p * (1 - p)
    return np.ones_like(z)


def linear(X, W, bias, residual, name, trans_w):
    """(Z, Y, bound of Z's error, bound of Y's error) in 64 bits.  A product
    of K terms summed in fp32 in any order is off by at most K U sum |x w|."""
    Wk = (W.T if trans_w else W).astype(np.float64)
    X = X.astype(np.float64)
    K = X.shape[1]
    Z = X @ Wk
    ez = (K + 1) * U * (np.abs(X) @ np.abs(Wk))
    if bias is not None:
        Z = Z + bias.astype(np.float64)
        ez = ez + U * np.abs(Z) * 1.01
    ez = ez + 1e-38
    Y = act(Z, name)
    ey = (1.0 if name in ("none", "relu") else STEEP) * ez
    if name not in ("none", "relu"):
        ey = ey + ACT_ERR * np.abs(Z)
    if residual is not None:
        Y = Y + residual.astype(np.float64)
        ey = ey * 1.01 + U * np.abs(Y)
    return Z, Y, ez, ey


# ------------------------------------------------------------ 8-bit rows --

def e4m3_values():
    """The value of every e4m3 byte (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where(b & 128, -v, v)
    v[[0x7f, 0xff]] = np.nan
    return v


def from_mx8(Q, E):
    """The values that e4m3 and e8m0 bytes stand for."""
    K = Q.shape[1]
    s = np.where(E == 255, np.nan, 2.0 ** (E.astype(np.float64) - 127))
    return e4m3_values()[Q] * np.repeat(s, 32, axis=1)[:, :K]


def to_mx8(v):
    """64-bit values as (Q, E): nearest e4m3, ties to even."""
    M, K = v.shape
    n = -(-K // 32)
    full = np.zeros((M, n * 32))
    full[:, :K] = v
    top = np.abs(full).reshape(M, n, 32).max(2)
    with np.errstate(divide="ignore"):
        E = np.clip(np.ceil(np.log2(top / 448)), -126, 127).astype(int)
    x = v / np.repeat(2.0 ** E, 32, axis=1)[:, :K]
    a = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    r = np.rint(a / step) * step                        # rint: ties to even
    table = e4m3_values()[:127]
    q = np.searchsorted(table, r).astype(np.uint8)
    assert np.array_equal(table[q], r)
    return q | np.where(np.signbit(x), 128, 0).astype(np.uint8), (E + 127).astype(np.uint8)


def check_mx8(Q, E, v, err, what=""):
    """Whether (Q, E) is the 8-bit form of values within `err` of v.  The
    power of two is the smallest that holds the block's largest magnitude
    within 448, for some value that close; each byte is then the nearest
    e4m3 value: within half a step of it, plus err."""
    M, K = v.shape
    n = -(-K // 32)
    pad = lambda a: np.pad(a, ((0, 0), (0, n * 32 - K))).reshape(M, n, 32)   # noqa: E731
    hi = (np.abs(pad(v)) + pad(err)).max(2)
    lo = np.maximum(np.abs(pad(v)) - pad(err), 0).max(2)
    e = E.astype(int) - 127
    exp = lambda a: np.maximum(np.ceil(np.log2(np.maximum(a, 1e-300) / 448)), -126)   # noqa: E731
    assert np.all((e <= exp(hi)) & (e >= exp(lo))), "%s: wrong power of two" % what
    s = np.repeat(2.0 ** e, 32, axis=1)[:, :K]
    got = from_mx8(Q, E)
    half = np.maximum(np.abs(v) + err, s * 2.0 ** -6) * 2.0 ** -4
    bad = np.abs(got - v) > half + err
    assert not bad.any(), "%s: %d bytes off, first at %s" % (what, bad.sum(), np.argwhere(bad)[0])


def weights(Q, S, bits, K):
    """The N x K weights of codes and binary16 scales, in 64 bits."""
    per = 8 // bits
    col = np.arange(K)
    code = (Q[:, col // per] >> (bits * (col % per))) & (2 ** bits - 1)
    s = S.view(np.float16).astype(np.float64)
    return (code - (2 ** bits - 1) / 2) * s[:, col // 64]


def within(got, ref, bound, what=""):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d off, first at %s: got %r, ref %r, bound %r" % (
            what, bad.sum(), bad.size, i, got[i], np.asarray(ref)[i], np.asarray(bound)[i]))
