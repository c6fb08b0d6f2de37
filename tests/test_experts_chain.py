"""GPU: a transformer layer with experts as it is used, under captured graphs, on
other streams and from several threads.

  training   groups -> grouped layer (GELU) -> grouped layer -> joined, the norms
             around the block, and back
  serving    norms to 8 bits -> groups -> packed grouped layer to 8 bits -> packed
             grouped layer -> joined
"""
import threading

import numpy as np
import pytest

import expert_refs as er
import layer_refs as lr
from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd import inputs
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu

EPS, ALPHA = 1e-5, 0.75
T, KE, E, D, H = 90, 2, 6, 96, 160


def _layer(seed=0):
    rng = np.random.default_rng(seed)
    n = lambda *s, scale=1.0: inputs.normal(rng, s, scale)   # noqa: E731
    ids = np.stack([rng.choice(E - 1, KE, replace=False) for _ in range(T)]).astype(np.int32)   # the last gets none
    ids[-5:] = -1                                            # padding
    w = rng.random((T, KE)).astype(np.float32)
    return dict(X=n(T, D), R=n(T, D), ids=ids, w=(w / w.sum(1, keepdims=True)).astype(np.float32),
                W1=n(E, D, H, scale=D ** -0.5), b1=n(E, H, scale=0.1), W2=n(E, D, H, scale=H ** -0.5), b2=n(E, D, scale=0.1),
                gu=(1 + n(D, scale=0.1)).astype(np.float32), gs=(1 + n(D, scale=0.1)).astype(np.float32),
                gate=n(D, scale=0.5), dY=n(T, D), dS=n(T, D))


def _forward(d, stream=None):
    """R's next value S = alpha R + gate norm(experts(X)) and Y = norm(S)."""
    kw = dict(stream=stream)
    offsets, rows, pos = bd.expert_groups(d["ids"], E, **kw)
    Z = torch().empty((T * KE, H), device="cuda")
    h = bd.linear_f32_grouped(d["X"], d["W1"], offsets, rows=rows, bias=d["b1"], act="gelu_tanh", Z=Z, **kw)
    y = bd.linear_f32_grouped(h, d["W2"], offsets, bias=d["b2"], trans_w=True, **kw)
    u = bd.expert_combine(y, pos, weights=d["w"], **kw)
    Y, S, ru, rs = bd.block_norm_f32(u, d["R"], d["gu"], d["gs"], EPS, gate=d["gate"], alpha=ALPHA, **kw)
    return Y, S, (offsets, rows, pos, Z, h, y, u, ru, rs)


def _backward(d, kept, S, stream=None):
    kw = dict(stream=stream)
    offsets, rows, pos, Z, h, y, u, ru, rs = kept
    du, dR, dgu, dgs, dgate = bd.block_norm_f32_bwd(d["dY"], u, S, d["gu"], d["gs"], ru, rs, gate=d["gate"], alpha=ALPHA,
                                                    dS=d["dS"], **kw)
    dy, dw = bd.expert_combine_bwd(du, pos, Y=y, weights=d["w"], **kw)
    dh, dW2, db2 = bd.linear_f32_grouped_bwd(dy, h, d["W2"], offsets, trans_w=True, **kw)
    dx, dW1, db1 = bd.linear_f32_grouped_bwd(dh, d["X"], d["W1"], offsets, rows=rows, Z=Z, act="gelu_tanh", **kw)
    return dict(X=bd.expert_combine(dx, pos, **kw), R=dR, w=dw, W1=dW1, b1=db1, W2=dW2, b2=db2, gu=dgu, gs=dgs,
                gate=dgate)


def _reference(d):
    """Forward by the formulas in 64 bits, token by token: (Y, S)."""
    u = np.zeros((T, D))
    for j in range(KE):
        e = d["ids"][:, j]
        live = np.flatnonzero(e >= 0)
        z = np.einsum("td,tdh->th", d["X"][live], d["W1"][e[live]]) + d["b1"][e[live]]
        y = np.einsum("th,tdh->td", lr.act(z, "gelu_tanh"), d["W2"][e[live]]) + d["b2"][e[live]]
        u[live] += d["w"][live, j:j + 1] * y
    V = u / np.sqrt((u * u).mean(1, keepdims=True) + EPS) * d["gu"]
    S = ALPHA * d["R"] + d["gate"] * V
    return S / np.sqrt((S * S).mean(1, keepdims=True) + EPS) * d["gs"], S


def _near(got, ref, what):
    """Within 2^-16 of the result's length: each step's sums of up to 160
    terms are off by at most 160 roundings of 2^-24 of their magnitudes, about
    2^-17 in the worst case and far less in length, as errors differ in
    sign."""
    got, ref = host(got).astype(np.float64), np.asarray(ref)
    assert np.linalg.norm(got - ref) <= 2.0 ** -16 * np.linalg.norm(ref), what


def test_training_layer():
    """Outputs against the formulas, gradients against differences of them."""
    d = _layer()
    t = {k: dev(v) for k, v in d.items()}
    Y, S, kept = _forward(t)
    p = {k: v.astype(np.float64) if v.dtype == np.float32 else v for k, v in d.items()}
    y, s = _reference(p)
    _near(Y, y, "Y")
    _near(S, s, "S")
    grads = _backward(t, kept, S)

    def loss(q):
        y, s = _reference(q)
        return (y * p["dY"]).sum() + (s * p["dS"]).sum()
    rng = np.random.default_rng(7)
    for k, g in grads.items():
        g = host(g).astype(np.float64)
        v = rng.standard_normal(p[k].shape)
        if k == "w":
            v[p["ids"] < 0] = 0
        h = 1e-5
        diff = (loss(dict(p, **{k: p[k] + h * v})) - loss(dict(p, **{k: p[k] - h * v}))) / (2 * h)
        # as in _near, of the terms' length; differences of a loss of some 10^3 to 1e-16 / h of it
        assert abs((g * v).sum() - diff) <= 2.0 ** -14 * np.linalg.norm(g * v) + 1e-7, k
    # an expert that no token chose, and tokens that chose none
    assert not host(grads["W1"])[E - 1].any() and not host(grads["b2"])[E - 1].any()
    assert not host(grads["X"])[-5:].any() and not host(grads["w"])[-5:].any()


def _serving(bits, t, seed=3):
    rng = np.random.default_rng([seed, bits, t])
    d, h, e, k = 192, 320, 8, 3

    def packed(n, m):
        return (rng.integers(0, 256, (e, n, m * bits // 8), dtype=np.uint8),
                rng.uniform(0.005, 0.02, (e, n, m // 64)).astype(np.float16).view(np.int16))
    ids = np.stack([rng.choice(e, k, replace=False) for _ in range(t)]).astype(np.int32)
    w = rng.random((t, k)).astype(np.float32)
    return dict(U=inputs.normal(rng, (t, d)), X=inputs.normal(rng, (t, d)), gu=(1 + inputs.normal(rng, (d,), 0.1)),
                gs=(1 + inputs.normal(rng, (d,), 0.1)), up=packed(h, d), down=packed(d, h), ids=ids, w=w,
                b=inputs.normal(rng, (e, h), 0.1))


def _serve(bits, d, stream=None):
    f = bd.linear_q2_mx8_grouped if bits == 2 else bd.linear_q4_mx8_grouped
    kw = dict(stream=stream)
    Q, S8, S = bd.block_norm_mx8(d["U"], d["X"], d["gu"], d["gs"], EPS, alpha=ALPHA, **kw)
    offsets, rows, pos = bd.expert_groups(d["ids"], 8, **kw)
    h8, he = f(Q, S8, *d["up"], offsets, rows=rows, bias=d["b"], act="silu", out="mx8", **kw)
    y = f(h8, he, *d["down"], offsets, **kw)
    out = bd.expert_combine(y, pos, weights=d["w"], residual=S, **kw)
    return Q, S8, S, offsets, rows, pos, h8, he, y, out


def _to_dev(d):
    return {k: tuple(dev(x) for x in v) if isinstance(v, tuple) else dev(v.astype(np.float32) if v.dtype == np.float64 else v)
            for k, v in d.items()}


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("t", [1, 9, 60, 300])
def test_serving_layer(bits, t):
    """Each step checked from the bytes of the step before it, so that the
    8-bit roundings in between do not blur the comparison."""
    d = _serving(bits, t)
    d = {k: v.astype(np.float32) if isinstance(v, np.ndarray) and v.dtype == np.float64 else v for k, v in d.items()}
    got = [host(a) for a in _serve(bits, _to_dev(d))]
    Q, S8, S, offsets, rows, pos, h8, he, y, out = got
    s, es, _, _ = er.block_norm_S(d["U"], d["X"], d["gu"], None, ALPHA, EPS)
    lr.within(S, s, es, "S")
    n, en, _, _ = er.block_norm_Y(S, d["gs"], EPS)
    lr.check_mx8(Q, S8, n, en, "norm")
    for g, w in zip((offsets, rows, pos), er.groups(d["ids"], 8)):
        assert np.array_equal(g, w)
    x = lr.from_mx8(Q, S8)[rows]
    z, ez = np.zeros((t * 3, 320)), np.zeros((t * 3, 320))
    for e, a, b in er.spans(offsets):
        w = lr.weights(d["up"][0][e], d["up"][1][e], bits, 192)
        z[a:b] = x[a:b] @ w.T + d["b"][e]
        ez[a:b] = 2 * (192 + 8) * lr.U * (np.abs(x[a:b]) @ np.abs(w.T)) * lr.STEEP
    lr.check_mx8(h8, he, lr.act(z, "silu"), ez + 2 * lr.ACT_ERR * np.abs(z) + 1e-12, "up")
    h = lr.from_mx8(h8, he)
    for e, a, b in er.spans(offsets):
        w = lr.weights(d["down"][0][e], d["down"][1][e], bits, 320)
        lr.within(y[a:b], h[a:b] @ w.T, 2 * (320 + 8) * lr.U * (np.abs(h[a:b]) @ np.abs(w.T)) + 1e-38, "down")
    lr.within(out, *er.combine(y, pos, d["w"], S), "joined")


def test_capture_and_replay_with_new_choices():
    """Training and serving steps in two graphs with workspaces of their own.
    Before each replay other experts are chosen, in place; every replay equals
    the eager calls on the same choice, with eager work in between."""
    t = torch()
    d = _layer(5)
    tr = {k: dev(v) for k, v in d.items()}
    bits, toks = 4, 40
    sv = _to_dev(_serving(bits, toks))
    z = lambda *s, dtype=t.float32: t.zeros(s, dtype=dtype, device="cuda")   # noqa: E731
    i32, u8 = t.int32, t.uint8
    M = T * KE
    ws1 = z(bd.linear_f32_grouped_bwd_ws_size("gelu_tanh", M, H, E), dtype=u8)
    ws2 = z(bd.linear_f32_grouped_bwd_ws_size("none", M, D, E), dtype=u8)
    wsn = z(bd.block_norm_f32_bwd_ws_size(T, D), dtype=u8)

    def train(st):
        o = dict(offsets=z(E + 1, dtype=i32), rows=z(M, dtype=i32), pos=z(T, KE, dtype=i32), Z=z(M, H), h=z(M, H), y=z(M, D),
                 u=z(T, D), S=z(T, D), Y=z(T, D), ru=z(T), rs=z(T), du=z(T, D), dR=z(T, D), dgu=z(D), dgs=z(D), dg=z(D),
                 dy=z(M, D), dw=z(T, KE), dh=z(M, H), dW2=z(E, D, H), db2=z(E, D), dx=z(M, D), dW1=z(E, D, H), db1=z(E, H),
                 dX=z(T, D))

        def run():
            bd.expert_groups(tr["ids"], E, offsets=o["offsets"], rows=o["rows"], pos=o["pos"], stream=st)
            bd.linear_f32_grouped(tr["X"], tr["W1"], o["offsets"], rows=o["rows"], bias=tr["b1"], act="gelu_tanh", Z=o["Z"],
                                  Y=o["h"], stream=st)
            bd.linear_f32_grouped(o["h"], tr["W2"], o["offsets"], bias=tr["b2"], trans_w=True, Y=o["y"], stream=st)
            bd.expert_combine(o["y"], o["pos"], weights=tr["w"], out=o["u"], stream=st)
            bd.block_norm_f32(o["u"], tr["R"], tr["gu"], tr["gs"], EPS, gate=tr["gate"], alpha=ALPHA, S=o["S"], Y=o["Y"],
                              rstd_u=o["ru"], rstd_s=o["rs"], stream=st)
            bd.block_norm_f32_bwd(tr["dY"], o["u"], o["S"], tr["gu"], tr["gs"], o["ru"], o["rs"], gate=tr["gate"],
                                  alpha=ALPHA, dS=tr["dS"], dU=o["du"], dX=o["dR"], dgamma_u=o["dgu"], dgamma_s=o["dgs"],
                                  dgate=o["dg"], workspace=wsn, stream=st)
            bd.expert_combine_bwd(o["du"], o["pos"], Y=o["y"], weights=tr["w"], dY=o["dy"], dw=o["dw"], stream=st)
            bd.linear_f32_grouped_bwd(o["dy"], o["h"], tr["W2"], o["offsets"], trans_w=True, dX=o["dh"], dW=o["dW2"],
                                      db=o["db2"], workspace=ws2, stream=st)
            bd.linear_f32_grouped_bwd(o["dh"], tr["X"], tr["W1"], o["offsets"], rows=o["rows"], Z=o["Z"], act="gelu_tanh",
                                      dX=o["dx"], dW=o["dW1"], db=o["db1"], workspace=ws1, stream=st)
            bd.expert_combine(o["dx"], o["pos"], out=o["dX"], stream=st)
        return o, run

    d_, h_, e_ = 192, 320, 8
    m = toks * 3

    def serve(st):
        o = dict(Q=z(toks, d_, dtype=u8), E8=z(toks, 6, dtype=u8), S=z(toks, d_), offsets=z(e_ + 1, dtype=i32),
                 rows=z(m, dtype=i32), pos=z(toks, 3, dtype=i32), h8=z(m, h_, dtype=u8), he=z(m, 10, dtype=u8), y=z(m, d_),
                 out=z(toks, d_))

        def run():
            bd.block_norm_mx8(sv["U"], sv["X"], sv["gu"], sv["gs"], EPS, alpha=ALPHA, S=o["S"], Q=o["Q"], E=o["E8"],
                              stream=st)
            bd.expert_groups(sv["ids"], e_, offsets=o["offsets"], rows=o["rows"], pos=o["pos"], stream=st)
            bd.linear_q4_mx8_grouped(o["Q"], o["E8"], *sv["up"], o["offsets"], rows=o["rows"], bias=sv["b"], act="silu",
                                     Y8=o["h8"], YE=o["he"], out="mx8", stream=st)
            bd.linear_q4_mx8_grouped(o["h8"], o["he"], *sv["down"], o["offsets"], Y=o["y"], stream=st)
            bd.expert_combine(o["y"], o["pos"], weights=sv["w"], residual=o["S"], out=o["out"], stream=st)
        return o, run
    side = t.cuda.Stream()
    graphs = []
    for make in (train, serve):
        o, run = make(side)
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            run()
        graphs.append((g, o))
    eager = [train(None), serve(None)]
    rng = np.random.default_rng(0)
    for k in range(4):
        ids = np.stack([rng.choice(E, KE, replace=False) for _ in range(T)]).astype(np.int32)
        ids[:3 * k] = -1
        tr["ids"].copy_(dev(ids))
        sv["ids"].copy_(dev(np.stack([rng.choice(8, 3, replace=False) for _ in range(toks)]).astype(np.int32)))
        t.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        t.cuda.synchronize()
        got = [{n: host(v).copy() for n, v in o.items()} for _, o in graphs]
        for (o, run), g in zip(eager, got):
            run()
            t.cuda.synchronize()
            live = int(host(o["offsets"])[-1])
            for n, v in o.items():
                a, b = g[n], host(v)
                if n in ("Z", "h", "y", "dy", "dh", "dx", "h8", "he"):       # rows of no group keep older values
                    a, b = a[:live], b[:live]
                assert np.array_equal(a, b), (k, n)
        (tr["X"] @ tr["W1"][0]).sum().item()


def test_another_stream():
    t = torch()
    d = {k: dev(v) for k, v in _layer(7).items()}
    sv = _to_dev(_serving(2, 20))
    Y, S, kept = _forward(d)
    ref = [host(Y), host(S)] + [host(g) for g in _backward(d, kept, S).values()]
    sref = [host(a) for a in _serve(2, sv)]
    t.cuda.synchronize()
    side = t.cuda.Stream()
    for handle in (side, side.cuda_stream):
        side.wait_stream(t.cuda.current_stream())
        y, s, kp = _forward(d, handle)
        got = [y, s] + list(_backward(d, kp, s, handle).values())
        served = _serve(2, sv, handle)
        for _ in range(8):
            t.full((T * KE, H), 3.0, device="cuda")       # the current stream's own work
        t.cuda.synchronize()
        assert all(np.array_equal(host(a), b) for a, b in zip(got, ref))
        assert all(np.array_equal(host(a), b) for a, b in zip(served, sref))


def test_threads():
    """Several host threads, each with its own stream and outputs, run both
    layers at once; every result equals the same call made alone."""
    t = torch()
    d = {k: dev(v) for k, v in _layer(8).items()}
    sv = _to_dev(_serving(4, 20))
    Y, S, kept = _forward(d)
    ref = [host(Y)] + [host(g) for g in _backward(d, kept, S).values()]
    sref = [host(a) for a in _serve(4, sv)]
    t.cuda.synchronize()
    bad = []

    def work():
        try:
            with t.cuda.stream(t.cuda.Stream()):
                for _ in range(4):
                    y, s, kp = _forward(d)
                    got = [y] + list(_backward(d, kp, s).values())
                    served = _serve(4, sv)
                    t.cuda.current_stream().synchronize()
                    if not all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, ref)):
                        bad.append("training")
                    if not all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(served, sref)):
                        bad.append("serving")
        except Exception as e:                             # noqa: BLE001
            bad.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad, bad


def test_gradients_accumulate_over_micro_batches():
    parts = [{k: dev(v) for k, v in _layer(s).items()} for s in (1, 2)]
    names = ("W1", "b1", "W2", "b2", "gu", "gs", "gate")
    for k in names:
        parts[1][k] = parts[0][k]
    single = []
    for p in parts:
        _, S, kept = _forward(p)
        single.append(_backward(p, kept, S))
    t = torch()
    acc = {k: t.zeros_like(parts[0][k]) for k in names}
    for p in parts:
        _, S, (offsets, rows, pos, Z, h, y, u, ru, rs) = _forward(p)
        du, _, _, _, _ = bd.block_norm_f32_bwd(p["dY"], u, S, p["gu"], p["gs"], ru, rs, gate=p["gate"], alpha=ALPHA,
                                               dS=p["dS"], dgamma_u=acc["gu"], dgamma_s=acc["gs"], dgate=acc["gate"],
                                               accumulate=True)
        dy, _ = bd.expert_combine_bwd(du, pos, Y=y, weights=p["w"])
        dh, _, _ = bd.linear_f32_grouped_bwd(dy, h, p["W2"], offsets, trans_w=True, dW=acc["W2"], db=acc["b2"],
                                             accumulate=True)
        bd.linear_f32_grouped_bwd(dh, p["X"], p["W1"], offsets, rows=rows, Z=Z, act="gelu_tanh", dW=acc["W1"], db=acc["b1"],
                                  accumulate=True)
    for k, a in acc.items():
        _near(a, host(single[0][k]).astype(np.float64) + host(single[1][k]), k)


def test_results_are_reproducible():
    d = {k: dev(v) for k, v in _layer(9).items()}
    first = None
    for _ in range(3):
        Y, S, kept = _forward(d)
        got = [host(Y)] + [host(g) for g in _backward(d, kept, S).values()]
        first = first or got
        assert all(np.array_equal(a, b) for a, b in zip(got, first))
