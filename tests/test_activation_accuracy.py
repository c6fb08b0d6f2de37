"""The activations' own errors on the GPU, against 64 bits, as close as the
kernels state them: z reaches the activation exactly (K = 1, W = 1).

With u = 2^-24, half a step of fp32: the logistic forms make e = exp(-t) within
(2 + 1.5 |t|) u (the hardware's 2^x is good to one step; its argument is rounded
after a rounded constant), t itself within 2.6 u in the tanh form, then p = 1 / (1
+ e) with one rounding and a reciprocal good to one step.  An error of e counts
for 1 - p in p's relative one: p is off by at most 4 u absolutely, and by (1 - p)
(2 + 1.5 |t| + 2.6 |t|) u + 3 u relatively.  The erf form: beyond 1.25 the tail has
2 u of the reciprocal, 1 of its argument, 2 of the polynomial, 1 + 1 of products,
(2 + 1.5 z^2) u of the exponential and 1 u of the fit, so p >= 0.89 is off by at
most 0.106 x 13.5 u + 0.5 u < 2 u; nearer by less.  The product with z adds u."""
import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

U = lr.U
P_ERR = {"gelu_tanh": 4 * U, "silu": 4 * U, "gelu_erf": 2 * U}


def _points(lo, hi):
    rng = np.random.default_rng(24)
    return np.concatenate([np.linspace(lo, hi, 60001), rng.uniform(-3, 3, 60000), -2.0 ** rng.uniform(-30, 0, 4000),
                           [1.25, -1.25, np.nextafter(np.float32(1.25), 0)]]).astype(np.float32)


def _value(z, act):
    return host(bd.linear_f32(dev(z[:, None]), dev(np.ones((1, 1), np.float32)), act=act))[:, 0]


@pytest.mark.parametrize("act", sorted(P_ERR))
def test_value(act):
    z = _points(-30, 30)
    ref = lr.act(z, act)
    lr.within(_value(z, act), ref, P_ERR[act] * np.abs(z.astype(np.float64)) + U * np.abs(ref) + 2.0 ** -126, act)


@pytest.mark.parametrize("act,lo", [("gelu_tanh", -9.0), ("silu", -80.0), ("gelu_erf", -13.0)])
def test_left_tail_keeps_its_digits(act, lo):
    """Where p is small its relative error is bounded too."""
    z = _points(lo, 0)
    z = z[(z < 0) & (z >= lo)]
    zd = z.astype(np.float64)
    t = np.abs(2 * lr.C * (zd + 0.044715 * zd ** 3))
    units = {"gelu_tanh": 8 + 6 * t, "silu": 8 + 2 * np.abs(zd), "gelu_erf": 12 + 2 * zd ** 2}[act]
    ref = lr.act(z, act)
    lr.within(_value(z, act), ref, units * U * np.abs(ref), act)


def test_slope_of_the_erf_form():
    """p and z exp(-z^2 / 2) / sqrt(2 pi) <= 0.242: 2 u of the first, 0.242 x (4 +
    1.5 z^2) u < 1.5 u of the second, u of their sum."""
    z = _points(-30, 30)
    one = np.ones((z.size, 1), np.float32)
    dX, _, _ = bd.linear_f32_bwd(dev(one), dev(one), dev(one[:1]), Z=dev(z[:, None]), act="gelu_erf", want=("dX",))
    lr.within(host(dX)[:, 0], lr.slope(z, "gelu_erf"), 5 * U + 0 * z.astype(np.float64))
