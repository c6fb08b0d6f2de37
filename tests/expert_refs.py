"""Plain 64-bit references of the layers with experts and of the norms around a
block, with the bounds of fp32's errors, shared by their tests."""
import numpy as np

import layer_refs as lr

U = lr.U


def groups(ids, E):
    """(offsets, rows, pos) by a stable sort."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    pos[key == E] = -1
    return offsets.astype(np.int32), (order // max(k, 1)).astype(np.int32), pos.astype(np.int32).reshape(T, k)


def sizes_to_offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def spans(offsets):
    """(expert, first, end) of the groups that hold rows."""
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(offsets, offsets[1:])) if a < b]


def combine(Y, pos, w, R):
    """out and the bound of its error: k additions and products."""
    Y64 = Y.astype(np.float64)
    live = (pos >= 0) & (pos < Y.shape[0])
    y = Y64[np.where(live, pos, 0)] if Y.shape[0] else np.zeros(pos.shape + (Y.shape[1],))
    y = y * live[:, :, None] * (1.0 if w is None else w.astype(np.float64)[:, :, None])
    out, mag = y.sum(1), np.abs(y).sum(1)
    if R is not None:
        out, mag = out + R.astype(np.float64), mag + np.abs(R)
    return out, (pos.shape[1] + 1) * U * mag + 1e-44


def linear_grouped(X, W, offsets, rows, bias, act, trans_w):
    """(Z, Y, bound of Z's error, bound of Y's error); NaN in rows of no group."""
    M = X.shape[0] if rows is None else rows.size
    N = W.shape[1] if trans_w else W.shape[2]
    Z, Y, ez, ey = (np.full((M, N), np.nan) for _ in range(4))
    for e, a, b in spans(offsets):
        x = X[a:b] if rows is None else X[rows[a:b]]
        Z[a:b], Y[a:b], ez[a:b], ey[a:b] = lr.linear(x, W[e], None if bias is None else bias[e], None, act, trans_w)
    return Z, Y, ez, ey


def linear_grouped_bwd(dY, X, W, offsets, rows, Z, act, trans_w):
    """{name: (gradient, bound of its error)}; NaN in rows of dX of no group."""
    dY, X, W = (a.astype(np.float64) for a in (dY, X, W))
    M, K, (E, N) = dY.shape[0], X.shape[1], (W.shape[0], dY.shape[1])
    s = np.ones_like(dY) if act == "none" else lr.slope(Z, act)
    dZ = dY * s
    ez = U * np.abs(dZ) + (0 if act in ("none", "relu") else lr.SLOPE_ERR * np.abs(dY))
    if act == "none":
        ez = ez * 0
    dX, ex = (np.full((M, K), np.nan) for _ in range(2))
    dW, ew, db, eb = np.zeros(W.shape), np.zeros(W.shape), np.zeros((E, N)), np.zeros((E, N))
    for e, a, b in spans(offsets):
        x = X[a:b] if rows is None else X[rows[a:b]]
        w = W[e] if trans_w else W[e].T                       # N x K
        z, az = dZ[a:b], np.abs(dZ[a:b])
        dX[a:b] = z @ w
        ex[a:b] = (N + 1) * U * (az @ np.abs(w)) * 1.01 + ez[a:b] @ np.abs(w) + 1e-38
        g, eg = z.T @ x, (b - a + 1) * U * (az.T @ np.abs(x)) * 1.01 + ez[a:b].T @ np.abs(x) + 1e-38
        dW[e], ew[e] = (g, eg) if trans_w else (g.T, eg.T)
        db[e], eb[e] = z.sum(0), (b - a + 1) * U * az.sum(0) * 1.01 + ez[a:b].sum(0) + 1e-38
    return {"dX": (dX, ex), "dW": (dW, ew), "db": (db, eb)}


# -------------------------------------------------- norms around a block --

def terms(K):
    """Additions that one term of a row sum can pass through: at most 32 (or
    K/1,024 in the longest rows) in a thread, then a tree over lanes and
    waves."""
    return max(32, -(-K // 1024)) + 24


def rstd(v, eps):
    """1 / sqrt(mean v^2 + eps) and its relative error: half the sum's, the
    product with 1/K (itself rounded), eps, the root and the reciprocal."""
    v = v.astype(np.float64)
    return 1 / np.sqrt((v * v).mean(1) + eps), (terms(v.shape[1]) / 2 + 5) * U


def _ones(v, shape=1.0):
    return shape if v is None else v.astype(np.float64)


def block_norm_S(U_, X, gu, gate, alpha, eps):
    """(S, bound of its error, rstd_u, its relative error)."""
    r, rel = rstd(U_, eps)
    V = U_.astype(np.float64) * r[:, None] * _ones(gu) * _ones(gate)
    S = alpha * X.astype(np.float64) + V
    return S, (rel + 3 * U) * np.abs(V) + U * np.abs(S) + 1e-44, r, rel


def block_norm_Y(S, gs, eps):
    """From S as it was stored: (Y, its bound, rstd_s, its relative error)."""
    r, rel = rstd(S, eps)
    Y = S.astype(np.float64) * r[:, None] * _ones(gs)
    return Y, (rel + 2 * U) * np.abs(Y) + 1e-44, r, rel


def block_norm_bwd(dY, U_, S, gu, gs, ru, rs, gate, alpha, dS):
    """{name: (gradient, bound of its error)}.  A row's sums are off by
    terms(K) roundings of their magnitudes, a sum over M rows by one per row
    that a workgroup adds, one per partial sum and run, and its terms' errors."""
    M, K = dY.shape
    n = (terms(K) + 4) * U
    dY, Um, S = (a.astype(np.float64) for a in (dY, U_, S))
    ru, rs = ru.astype(np.float64)[:, None], rs.astype(np.float64)[:, None]
    gu_, gs_, gt = _ones(gu, np.ones(K)), _ones(gs, np.ones(K)), _ones(gate, np.ones(K))
    xs, xu, a = S * rs, Um * ru, np.abs
    g = gs_ * dY
    dot = (g * xs).mean(1, keepdims=True)
    edot = n * a(g * xs).mean(1, keepdims=True)
    G0 = rs * (g - xs * dot)
    G = G0 + (0 if dS is None else dS.astype(np.float64))
    eG = rs * (4 * U * (a(g) + a(xs * dot)) + a(xs) * edot) + 2 * U * (a(G0) + a(G))
    H = gt * G
    eH = a(gt) * eG + U * a(H)
    h, eh = gu_ * H, a(gu_) * eH + U * a(gu_ * H)
    dot = (h * xu).mean(1, keepdims=True)
    edot = (eh * a(xu)).mean(1, keepdims=True) + n * a(h * xu).mean(1, keepdims=True)
    dU = ru * (h - xu * dot)
    eU = ru * (eh + a(xu) * edot + 4 * U * (a(h) + a(xu * dot))) + U * a(dU)
    rows = -(-M // 256) + 100

    def over_rows(t, et):
        return t.sum(0), (rows * U * a(t).sum(0) + et.sum(0)) * 1.01 + 1e-40
    out = {"dU": (dU, eU + 1e-40), "dX": (alpha * G, abs(alpha) * eG + U * a(alpha * G) + 1e-40),
           "dgamma_s": over_rows(dY * xs, 3 * U * a(dY * xs)),
           "dgamma_u": over_rows(H * xu, eH * a(xu) + 4 * U * a(H * xu))}
    if gate is not None:
        t = gu_ * xu * G
        et = a(gu_ * xu) * eG + 4 * U * a(t)
        out["dgate"] = over_rows(t, et) if gate.ndim == 1 else (t, et + 1e-40)
    return out
