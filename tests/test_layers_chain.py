"""GPU: the layers together as a transformer block uses them, under captured
graphs, on other streams and from several threads.

  training   norm -> layer (GELU) -> layer (residual) forward, and back
  serving    norm to 8 bits -> packed layer to 8 bits -> packed layer onto the
             residual stream
"""
import threading

import numpy as np
import pytest

import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
M, D, H = 70, 192, 320


def _block(seed=0):
    rng = np.random.default_rng(seed)
    n = lambda *s, scale=1.0: inputs.normal(rng, s, scale)   # noqa: E731
    return dict(X=n(M, D), R=n(M, D), g=(1 + n(D, scale=0.1)).astype(np.float32),
                W1=n(D, H, scale=D ** -0.5), b1=n(H, scale=0.1), W2=n(D, H, scale=H ** -0.5),
                b2=n(D, scale=0.1), dY=n(M, D))


def _forward(d):
    """Y = S + gelu(norm(S) W1 + b1) W2^T + b2, S = X + R."""
    h0, S, rstd = bd.rmsnorm_f32(d["X"], d["g"], EPS, residual=d["R"])
    Z = torch().empty((M, H), device="cuda")
    h1 = bd.linear_f32(h0, d["W1"], bias=d["b1"], act="gelu_tanh", Z=Z)
    Y = bd.linear_f32(h1, d["W2"], bias=d["b2"], residual=S, trans_w=True)
    return Y, (h0, S, rstd, Z, h1)


def _backward(d, kept, dY):
    h0, S, rstd, Z, h1 = kept
    dh1, dW2, db2 = bd.linear_f32_bwd(dY, h1, d["W2"], trans_w=True)
    dh0, dW1, db1 = bd.linear_f32_bwd(dh1, h0, d["W1"], Z=Z, act="gelu_tanh")
    dX, dg = bd.rmsnorm_f32_bwd(dh0, S, d["g"], rstd, dS=dY)
    return dict(X=dX, R=dX, g=dg, W1=dW1, b1=db1, W2=dW2, b2=db2)


def _reference(d):
    """The block and its gradients in 64 bits, by the formulas."""
    d = {k: v.astype(np.float64) for k, v in d.items()}
    S = d["X"] + d["R"]
    r = 1 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    h0 = S * r * d["g"]
    Z = h0 @ d["W1"] + d["b1"]
    h1 = lr.act(Z, "gelu_tanh")
    Y = S + h1 @ d["W2"].T + d["b2"]
    dY = d["dY"]
    dh1 = dY @ d["W2"]
    dZ = dh1 * lr.slope(Z, "gelu_tanh")
    dh0 = dZ @ d["W1"].T
    gd, xh = dh0 * d["g"], S * r
    dX = r * (gd - xh * (gd * xh).mean(1, keepdims=True)) + dY
    return Y, dict(X=dX, R=dX, g=(dh0 * xh).sum(0), W1=h0.T @ dZ, b1=dZ.sum(0), W2=dY.T @ h1,
                   b2=dY.sum(0))


def _near(got, ref, what):
    """Within 2^-16 of the result's length: each step's sums of up to 320
    terms are off by at most 320 roundings of 2^-24 of their magnitudes, about
    2^-16 in the worst case and far less in length, as errors differ in
    sign."""
    got, ref = host(got).astype(np.float64), np.asarray(ref)
    assert np.linalg.norm(got - ref) <= 2.0 ** -16 * np.linalg.norm(ref), what


def test_training_block():
    d = _block()
    t = {k: dev(v) for k, v in d.items()}
    Y, kept = _forward(t)
    grads = _backward(t, kept, t["dY"])
    y, ref = _reference(d)
    _near(Y, y, "Y")
    for k, g in grads.items():
        _near(g, ref[k], "d" + k)


def test_gradients_accumulate_over_micro_batches():
    """Two micro-batches accumulated equal their separate gradients' sum."""
    parts = [{k: dev(v) for k, v in _block(s).items()} for s in (1, 2)]
    for k in ("W1", "b1", "W2", "b2", "g"):
        parts[1][k] = parts[0][k]
    single = []
    for p in parts:
        _, kept = _forward(p)
        single.append(_backward(p, kept, p["dY"]))
    t = torch()
    acc = {k: t.zeros_like(parts[0][k]) for k in ("W1", "b1", "W2", "b2", "g")}
    for p in parts:
        _, (h0, S, rstd, Z, h1) = _forward(p)
        dh1, _, _ = bd.linear_f32_bwd(p["dY"], h1, p["W2"], trans_w=True, dW=acc["W2"], db=acc["b2"],
                                      accumulate=True)
        dh0, _, _ = bd.linear_f32_bwd(dh1, h0, p["W1"], Z=Z, act="gelu_tanh", dW=acc["W1"],
                                      db=acc["b1"], accumulate=True)
        bd.rmsnorm_f32_bwd(dh0, S, p["g"], rstd, dS=p["dY"], dgamma=acc["g"], accumulate=True)
    for k, a in acc.items():
        _near(a, host(single[0][k]).astype(np.float64) + host(single[1][k]), k)


def _serving(bits, m, seed=3):
    rng = np.random.default_rng([seed, bits, m])
    d, h = 384, 640

    def packed(n, k):
        return (rng.integers(0, 256, (n, k * bits // 8), dtype=np.uint8),
                rng.uniform(0.005, 0.02, (n, k // 64)).astype(np.float16).view(np.int16))
    return dict(X=inputs.normal(rng, (m, d)), R=inputs.normal(rng, (m, d)),
                g=(1 + inputs.normal(rng, (d,), 0.1)).astype(np.float32), up=packed(h, d),
                down=packed(d, h), b=inputs.normal(rng, (h,), 0.1))


def _serve(bits, t, stream_S, out):
    f = bd.linear_q2_mx8 if bits == 2 else bd.linear_q4_mx8
    Q, E, S = bd.rmsnorm_mx8(t["X"], t["g"], EPS, residual=t["R"], S=stream_S)
    h8, he = f(Q, E, *t["up"], bias=t["b"], act="silu", out="mx8")
    f(h8, he, *t["down"], residual=S, Y=out)
    return Q, E, h8, he, out


def _to_dev(d):
    return {k: tuple(dev(x) for x in v) if isinstance(v, tuple) else dev(v) for k, v in d.items()}


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("m", [1, 9, 60, 300])
def test_serving_block(bits, m):
    """Each step checked from the bytes of the step before it, so that the
    8-bit roundings in between do not blur the comparison."""
    d = _serving(bits, m)
    t = _to_dev(d)
    S = torch().empty((m, 384), device="cuda")
    Q, E, h8, he, Y = (host(a) for a in _serve(bits, t, S, torch().empty((m, 384), device="cuda")))
    s = (d["X"] + d["R"]).astype(np.float64)
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + EPS) * d["g"]
    lr.check_mx8(Q, E, y, 64 * lr.U * np.abs(y), "norm")
    x, w = lr.from_mx8(Q, E), lr.weights(*d["up"], bits, 384)
    z = x @ w.T + d["b"]
    e = 2 * (384 + 8) * lr.U * (np.abs(x) @ np.abs(w.T)) * lr.STEEP + 2 * lr.ACT_ERR * np.abs(z) + 1e-12
    lr.check_mx8(h8, he, lr.act(z, "silu"), e, "up")
    h, w = lr.from_mx8(h8, he), lr.weights(*d["down"], bits, 640)
    lr.within(Y, s + h @ w.T, 2 * (640 + 8) * lr.U * (np.abs(h) @ np.abs(w.T)) + 4 * lr.U * (np.abs(s) + np.abs(Y)),
              "down")


def test_capture_and_replay():
    """Training and serving steps in two graphs with workspaces of their own,
    replayed in turn with eager calls in between; every replay redoes exactly
    what the eager calls do."""
    t = torch()
    d = _block(5)
    tr = {k: dev(v) for k, v in d.items()}
    sv = [(b, m, _to_dev(_serving(b, m))) for b in (2, 4) for m in (1, 40, 200)]
    ws = {n: t.empty(bd.linear_f32_bwd_ws_size(a, M, n), dtype=t.uint8, device="cuda")
          for n, a in ((D, "none"), (H, "gelu_tanh"))}
    wn = t.empty(bd.rmsnorm_f32_bwd_ws_size(M, D), dtype=t.uint8, device="cuda")

    def train(o, st):
        bd.rmsnorm_f32(tr["X"], tr["g"], EPS, residual=tr["R"], S=o["S"], Y=o["h0"], rstd=o["r"], stream=st)
        bd.linear_f32(o["h0"], tr["W1"], bias=tr["b1"], act="gelu_tanh", Z=o["Z"], Y=o["h1"], stream=st)
        bd.linear_f32(o["h1"], tr["W2"], bias=tr["b2"], residual=o["S"], Y=o["Y"], trans_w=True, stream=st)
        bd.linear_f32(o["h1"][:3], tr["W2"], bias=tr["b2"], Y=o["few"], trans_w=True, stream=st)
        bd.linear_f32_bwd(tr["dY"], o["h1"], tr["W2"], trans_w=True, dX=o["dh1"], dW=o["dW2"],
                          db=o["db2"], workspace=ws[D], stream=st)
        bd.linear_f32_bwd(o["dh1"], o["h0"], tr["W1"], Z=o["Z"], act="gelu_tanh", dX=o["dh0"],
                          dW=o["dW1"], db=o["db1"], accumulate=True, workspace=ws[H], stream=st)
        bd.rmsnorm_f32_bwd(o["dh0"], o["S"], tr["g"], o["r"], dS=tr["dY"], dX=o["dX"], dgamma=o["dg"],
                           workspace=wn, stream=st)

    def outputs():
        z = lambda *s: t.zeros(s, device="cuda")   # noqa: E731
        return dict(S=z(M, D), h0=z(M, D), r=z(M), Z=z(M, H), h1=z(M, H), Y=z(M, D), few=z(3, D),
                    dh1=z(M, H), dW2=z(D, H), db2=z(D), dh0=z(M, D), dW1=z(D, H), db1=z(H),
                    dX=z(M, D), dg=z(D))

    def serve(o, st):
        for (b, m, x), (S, Q, E, h8, he, Y) in zip(sv, o):
            f = bd.linear_q2_mx8 if b == 2 else bd.linear_q4_mx8
            bd.rmsnorm_mx8(x["X"], x["g"], EPS, residual=x["R"], S=S, Q=Q, E=E, stream=st)
            f(Q, E, *x["up"], bias=x["b"], act="silu", Y8=h8, YE=he, out="mx8", stream=st)
            f(h8, he, *x["down"], residual=S, Y=Y, stream=st)

    def serve_outputs():
        u8 = dict(dtype=t.uint8, device="cuda")
        return [(t.zeros((m, 384), device="cuda"), t.zeros((m, 384), **u8), t.zeros((m, 12), **u8),
                 t.zeros((m, 640), **u8), t.zeros((m, 20), **u8), t.zeros((m, 384), device="cuda"))
                for _, m, _ in sv]
    eager_t, eager_s = outputs(), serve_outputs()
    train(eager_t, None)
    serve(eager_s, None)
    t.cuda.synchronize()
    want_t = {k: host(v) for k, v in eager_t.items()}
    want_s = [[host(v) for v in o] for o in eager_s]
    one = want_t["dW1"].copy()

    got_t, got_s = outputs(), serve_outputs()
    graphs = []
    side = t.cuda.Stream()
    for f, o in ((train, got_t), (serve, got_s)):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            f(o, side)
        graphs.append(g)
    for k in range(4):
        for g in graphs:
            g.replay()
        t.cuda.synchronize()
        for n, w in want_t.items():
            if n in ("dW1", "db1"):
                continue
            assert np.array_equal(host(got_t[n]), w), (k, n)
        lr.within(host(got_t["dW1"]), (k + 1.0) * one, 4 * (k + 2) * lr.U * np.abs(one) * (k + 1) + 1e-30)
        for o, w in zip(got_s, want_s):
            for a, b in zip(o, w):
                assert np.array_equal(host(a), b), k
        # eager work between the replays, on neighbours and with torch
        _forward(tr)
        serve(serve_outputs(), None)
        (tr["X"] @ tr["W1"]).sum().item()


def test_another_stream():
    """Calls on a stream that is not the current one: outputs and workspaces
    that the binding allocates belong to that stream, so what the current
    stream does meanwhile with freed memory cannot disturb them."""
    t = torch()
    d = {k: dev(v) for k, v in _block(7).items()}
    Y, kept = _forward(d)
    ref = _backward(d, kept, d["dY"])
    t.cuda.synchronize()
    side = t.cuda.Stream()
    for handle in (side, side.cuda_stream):
        side.wait_stream(t.cuda.current_stream())
        h0, S, rstd = bd.rmsnorm_f32(d["X"], d["g"], EPS, residual=d["R"], stream=handle)
        with t.cuda.stream(side):
            Z = t.empty((M, H), device="cuda")
        h1 = bd.linear_f32(h0, d["W1"], bias=d["b1"], act="gelu_tanh", Z=Z, stream=handle)
        y = bd.linear_f32(h1, d["W2"], bias=d["b2"], residual=S, trans_w=True, stream=handle)
        dh1, dW2, db2 = bd.linear_f32_bwd(d["dY"], h1, d["W2"], trans_w=True, stream=handle)
        dh0, dW1, db1 = bd.linear_f32_bwd(dh1, h0, d["W1"], Z=Z, act="gelu_tanh", stream=handle)
        dX, dg = bd.rmsnorm_f32_bwd(dh0, S, d["g"], rstd, dS=d["dY"], stream=handle)
        for _ in range(8):
            t.full((M, H), 3.0, device="cuda")            # the current stream's own work
        t.cuda.synchronize()
        assert np.array_equal(host(y), host(Y))
        for k, g in dict(X=dX, g=dg, W1=dW1, b1=db1, W2=dW2, b2=db2).items():
            assert np.array_equal(host(g), host(ref[k])), k


def test_threads():
    """Several host threads, each with its own stream and outputs, run both
    blocks at once; every result equals the same call made alone."""
    t = torch()
    d = {k: dev(v) for k, v in _block(8).items()}
    sv = _to_dev(_serving(4, 20))
    Y, kept = _forward(d)
    ref = [host(Y)] + [host(g) for g in _backward(d, kept, d["dY"]).values()]
    sref = [host(a) for a in _serve(4, sv, t.empty((20, 384), device="cuda"), t.empty((20, 384), device="cuda"))]
    t.cuda.synchronize()
    bad = []

    def work():
        try:
            with t.cuda.stream(t.cuda.Stream()):
                for _ in range(4):
                    y, kp = _forward(d)
                    got = [y] + list(_backward(d, kp, d["dY"]).values())
                    s = _serve(4, sv, t.empty((20, 384), device="cuda"), t.empty((20, 384), device="cuda"))
                    t.cuda.current_stream().synchronize()
                    if not all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, ref)):
                        bad.append("training")
                    if not all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(s, sref)):
                        bad.append("serving")
        except Exception as e:                             # noqa: BLE001
            bad.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad, bad


def test_results_are_reproducible():
    d = {k: dev(v) for k, v in _block(9).items()}
    first = None
    for _ in range(3):
        Y, kept = _forward(d)
        got = [host(Y)] + [host(g) for g in _backward(d, kept, d["dY"]).values()]
        first = first or got
        assert all(np.array_equal(a, b) for a, b in zip(got, first))
