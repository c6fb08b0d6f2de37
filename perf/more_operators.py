"""Cases of a transformer layer with experts, from the router's choice to the norm before the next
block: inputs, plain forms in elementary torch operations, calls of this package's entry points, and
the operators' definitions in 64 bits.

    groups        the (token, expert) pairs of a router's choice in the order of their experts  (int32)
    combine       out_t = R_t + sum_j w_tj Y[pos_tj], tokens' expert results joined             (fp32)
    combine_bwd   dY and dw of that sum from the gradient of out                                (fp32)
    grouped       Y_i = act(X[rows_i] . W_e + b_e), rows grouped by expert e in ragged sizes    (fp32)
    grouped_bwd   dX (in grouped order), dW and db of every expert from dY                      (fp32)
    packed        the same layer on 2-bit or 4-bit weights and 8-bit rows, to fp32 or 8 bits    (mx8)
    block_norm    S = alpha X + gate . norm(U) gamma_u, Y = norm(S) gamma_s, in fp32 or 8 bits
    block_norm_bwd  dU, dX, dgamma_u, dgamma_s and dgate of that, with the gradient that reaches S

8 bits (mx8): e4m3 values with one power of two (e8m0) per 32 columns of a row, the smallest that
keeps the block's largest magnitude within 448.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu_tanh", "gelu_erf", "silu")
EPS = 1e-5


def listed():
    return [
        # one generated token's eight of 64 experts: latency alone
        dict(name="groups token", op="groups", T=1, k=8, E=64, padded=False),
        # a training batch with padding behind its sequences, whose choices are dropped
        dict(name="groups training", op="groups", T=8192, k=8, E=128, padded=True),
        # a prompt of 346 tokens back into the residual stream
        dict(name="combine prompt", op="combine", T=346, k=2, K=768, residual=True, weights=True, padded=False),
        # the gradients of the same sum over a training batch
        dict(name="combine_bwd training", op="combine_bwd", T=8192, k=2, K=2048),
        # four sequences' next tokens through fp32 experts, bound by the chosen experts' weights
        dict(name="grouped token", op="grouped", T=4, k=2, E=8, N=2304, K=768, trans_w=False, act="gelu_tanh",
             gather=True, keep=False),
        # a training batch through the experts' widening layer, its pre-activations kept
        dict(name="grouped training", op="grouped", T=4096, k=2, E=8, N=2048, K=1024, trans_w=True, act="silu",
             gather=True, keep=True),
        # and that layer's gradients over a shorter batch
        dict(name="grouped_bwd training", op="grouped_bwd", T=2048, k=2, E=8, N=2048, K=1024, trans_w=True,
             act="gelu_tanh", gather=True),
        # one token through eight of 64 experts in 4 bits, its activations in 8 bits for the next layer
        dict(name="packed token q4", op="packed", bits=4, T=1, k=8, E=64, N=1536, K=1536, act="silu", out="mx8"),
        # a prompt of 500 tokens through experts in 2 bits
        dict(name="packed prompt q2", op="packed", bits=2, T=500, k=2, E=16, N=12288, K=1536, act="none", out="f32"),
        # one token between two blocks, in 8 bits for the packed layer behind the norm
        dict(name="block_norm token mx8", op="block_norm", M=1, K=1536, gate="columns", out="mx8"),
        # a training batch between two blocks, more data than the caches hold, and its gradients
        dict(name="block_norm training", op="block_norm", M=16384, K=2048, gate="columns", out="f32"),
        dict(name="block_norm_bwd training", op="block_norm_bwd", M=16384, K=2048, gate="columns", carried=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("groups", "combine", "combine_bwd", "grouped", "grouped", "grouped_bwd", "packed", "packed",
                     "block_norm", "block_norm", "block_norm_bwd"))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op == "groups":
        while True:
            T, k, E = _log(rng, 1, 16384), rng.randint(1, 8), rng.randint(8, 256)
            if T * k <= 65536:
                return dict(op=op, T=T, k=k, E=E, padded=coin())
    if op in ("combine", "combine_bwd"):
        while True:
            T, k, K = _log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 33, 8192)
            if T * k * K <= 8192 * 2 * 2048:
                break
        if op == "combine_bwd":
            return dict(op=op, T=T, k=k, K=K)
        return dict(op=op, T=T, k=k, K=K, residual=coin(), weights=coin(), padded=coin())
    if op in ("grouped", "grouped_bwd"):
        while True:
            T, k, E = _log(rng, 1, 4096), rng.randint(1, 4), rng.choice((4, 7, 8, 16, 32))
            N, K = _log(rng, 48, 2304), _log(rng, 48, 2304)
            if T * k * N * K <= 8192 * 2048 * 1024 / (1 if op == "grouped" else 2) and E * N * K <= 1 << 26:
                break
        case = dict(op=op, T=T, k=k, E=E, N=N, K=K, trans_w=coin(), act=rng.choice(ACTS), gather=coin())
        return dict(case, keep=coin()) if op == "grouped" else case
    if op == "packed":
        while True:
            T, k, E = _log(rng, 1, 512), rng.randint(1, 8), rng.choice((8, 13, 16, 32, 64))
            N, K = _log(rng, 64, 12288), _log(rng, 64, 12288)
            if T * k * N * K <= 1000 * 12288 * 1536 and E * N * K <= 16 * 12288 * 1536 and N * K <= 12288 * 1536:
                break
        return dict(op=op, bits=rng.choice((2, 4)), T=T, k=k, E=E, N=N, K=K, act=rng.choice(ACTS),
                    out=rng.choice(("f32", "mx8")))
    while True:
        M, K = _log(rng, 1, 16384), _log(rng, 33, 16384)
        if M * K <= 16384 * 2048:
            break
    case = dict(op=op, M=M, K=K, gate=rng.choice(("none", "columns", "rows")))
    return dict(case, carried=coin()) if op == "block_norm_bwd" else dict(case, out=rng.choice(("f32", "mx8")))


# ---------------------------------------------------------------- inputs --

def _choice(g, T, k, E):
    """k different experts of E for each of T tokens: some experts are more popular than others."""
    popular = torch.randn(E, generator=g, device="cuda") * 0.7
    logits = popular + torch.randn(T, E, generator=g, device="cuda")
    top, ids = logits.topk(k, 1)
    return torch.softmax(top, 1), ids.to(torch.int32)


def _grouped(ids, E):
    """(offsets, rows, pos) of a choice whose experts all exist."""
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(flat.numel(), device="cuda")
    return offsets, (order // ids.shape[1]).to(torch.int32), pos.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    s, op = dict(case), case["op"]
    if op == "groups":
        _, s["ids"] = _choice(g, case["T"], case["k"], case["E"])
        if case["padded"]:
            s["ids"][case["T"] - case["T"] // 8:] = -1
    elif op in ("combine", "combine_bwd"):
        T, k, K = case["T"], case["k"], case["K"]
        s["w"], ids = _choice(g, T, k, max(16, k))
        _, _, s["pos"] = _grouped(ids, max(16, k))
        s["Y"] = normal(T * k, K)
        if op == "combine":
            s["R"] = normal(T, K) if case["residual"] else None
            s["w"] = s["w"] if case["weights"] else None
            if case["padded"]:
                s["pos"][T - T // 8:] = -1
        else:
            s["dO"] = normal(T, K)
    elif op in ("grouped", "grouped_bwd", "packed"):
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        k = s["k"] = min(k, E)
        _, ids = _choice(g, T, k, E)
        s["offsets"], s["rows"], _ = _grouped(ids, E)
        s["ends"] = s["offsets"].tolist()               # the plain form's loop runs on the host
        if op == "packed":
            bits = case["bits"]
            s["X8"], s["XE"] = _to_mx8(normal(T, K))
            s["Q"] = torch.randint(0, 256, (E, N, -(-K * bits // 8)), generator=g, device="cuda", dtype=torch.uint8)
            s["S"] = (0.01 + 0.04 * torch.rand(E, N, -(-K // 64), generator=g, device="cuda")).half()
            s["b"] = normal(E, N, scale=0.5)
        else:
            s["X"] = normal(T if case["gather"] else T * k, K)
            s["rows"] = s["rows"] if case["gather"] else None
            s["W"] = normal(*((E, N, K) if case["trans_w"] else (E, K, N)), scale=K ** -0.5)
            if op == "grouped":
                s["b"] = normal(E, N, scale=0.5)
            else:
                s["dY"] = normal(T * k, N)
                s["Z"] = normal(T * k, N, scale=1.5)
    else:
        M, K = case["M"], case["K"]
        # a residual stream has a few channels far larger than the rest
        s["U"] = normal(M, K, scale=2.0)
        s["gu"] = 1 + normal(K, scale=0.2)
        s["gs"] = 1 + normal(K, scale=0.2)
        s["gate"] = None
        if case["gate"] == "columns":
            s["gate"] = 0.5 + normal(K, scale=0.2)
        elif case["gate"] == "rows":
            s["gate"] = torch.sigmoid(normal(M, K))
        s["alpha"] = 0.75
        big = 1 + 20 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        if op == "block_norm":
            s["X"] = normal(M, K) * big
        else:
            s["S"] = normal(M, K) * big
            s["ru"] = 1 / torch.sqrt((s["U"] * s["U"]).mean(1) + EPS)
            s["rs"] = 1 / torch.sqrt((s["S"] * s["S"]).mean(1) + EPS)
            s["dY"] = normal(M, K)
            s["dS"] = normal(M, K) if case["carried"] else None
    return s


# ----------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "gelu_erf":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _to_mx8(v):
    """v (M x K) as e4m3 bytes and e8m0 bytes, blocks of 32 columns."""
    M, K = v.shape
    pad = -K % 32
    if pad:
        v = torch.cat([v, v.new_zeros(M, pad)], 1)
    blocks = v.float().reshape(M, -1, 32)
    frac, exp = torch.frexp(blocks.abs().amax(2))        # amax = frac * 2^exp, frac in [1/2, 1)
    e = (exp - 9 + (frac > 0.875).to(exp.dtype)).clamp(min=-126)
    q = torch.ldexp(blocks, -e[..., None]).to(torch.float8_e4m3fn).reshape(M, -1)[:, :K]
    return q.contiguous().view(torch.uint8), (e + 127).to(torch.uint8)


def _from_mx8(q, e, dtype):
    """The values that e4m3 and e8m0 bytes stand for."""
    K = q.shape[1]
    scale = torch.ldexp(torch.ones(e.shape, dtype=dtype, device=e.device), e.to(torch.int32) - 127)
    return q.view(torch.float8_e4m3fn).to(dtype) * scale.repeat_interleave(32, 1)[:, :K]


def _weights(Q, S, bits, K, dtype):
    """The values that 2-bit or 4-bit codes with one scale per 64 columns stand for."""
    shifts = torch.arange(0, 8, bits, device=Q.device, dtype=torch.uint8)
    codes = (Q[:, :, None] >> shifts & (2 ** bits - 1)).reshape(Q.shape[0], -1)[:, :K]
    return (codes.to(dtype) - (2 ** bits - 1) / 2) * S.to(dtype).repeat_interleave(64, 1)[:, :K]


def _mx8_out(q, e):
    return {"q": q.view(torch.float8_e4m3fn), "e": e.view(torch.float8_e8m0fnu)}


def _groups_of(s):
    """(expert, first row, end) of the groups that hold any."""
    e = s["ends"]
    return [(i, a, b) for i, (a, b) in enumerate(zip(e, e[1:])) if a < b]


def _norm(v, gamma):
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r * gamma, r[:, 0]


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "groups":
        T, k, E = s["T"], s["k"], s["E"]
        flat = s["ids"].flatten().long()
        there = (flat >= 0) & (flat < E)
        key = torch.where(there, flat, torch.full_like(flat, E))
        order = torch.argsort(key, stable=True)
        sizes = torch.zeros(E + 1, dtype=torch.int64, device=key.device).index_add_(0, key, torch.ones_like(key))
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=key.device)
        offsets[1:] = torch.cumsum(sizes[:E], 0)
        pos = torch.empty_like(key)
        pos[order] = torch.arange(T * k, device=key.device)
        pos = torch.where(there, pos, torch.full_like(pos, -1))
        return {"offsets": offsets, "rows": (order // k).to(torch.int32), "pos": pos.to(torch.int32).view(T, k)}
    if op == "combine":
        pos = s["pos"].long()
        y = s["Y"][pos.clamp(min=0)] * (pos >= 0)[:, :, None]
        if s["w"] is not None:
            y = y * s["w"][:, :, None]
        out = y.sum(1)
        return {"out": out if s["R"] is None else out + s["R"]}
    if op == "combine_bwd":
        pos = s["pos"].long()
        dy = torch.empty_like(s["Y"])
        dy[pos] = s["w"][:, :, None] * s["dO"][:, None, :]
        return {"dy": dy, "dw": (s["Y"][pos] * s["dO"][:, None, :]).sum(2)}
    if op == "grouped":
        x = s["X"] if s["rows"] is None else s["X"][s["rows"].long()]
        z = torch.empty(x.shape[0], s["N"], device=x.device)
        for e, a, b in _groups_of(s):
            z[a:b] = x[a:b] @ (s["W"][e].t() if s["trans_w"] else s["W"][e]) + s["b"][e]
        y = _act(z, s["act"])
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    if op == "grouped_bwd":
        x = s["X"] if s["rows"] is None else s["X"][s["rows"].long()]
        dz = s["dY"] * _act_grad(s["Z"], s["act"])
        dx, dw = torch.empty_like(x), torch.zeros_like(s["W"])
        db = torch.zeros(s["E"], s["N"], device=x.device)
        for e, a, b in _groups_of(s):
            dx[a:b] = dz[a:b] @ (s["W"][e] if s["trans_w"] else s["W"][e].t())
            dw[e] = dz[a:b].t() @ x[a:b] if s["trans_w"] else x[a:b].t() @ dz[a:b]
            db[e] = dz[a:b].sum(0)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "packed":
        x = _from_mx8(s["X8"], s["XE"], torch.float32)[s["rows"].long()]
        y = torch.empty(x.shape[0], s["N"], device=x.device)
        for e, a, b in _groups_of(s):
            y[a:b] = x[a:b] @ _weights(s["Q"][e], s["S"][e], s["bits"], s["K"], torch.float32).t() + s["b"][e]
        y = _act(y, s["act"])
        return {"y": y} if s["out"] == "f32" else _mx8_out(*_to_mx8(y))
    gate = s["gate"]
    if op == "block_norm":
        v, ru = _norm(s["U"], s["gu"])
        S = s["alpha"] * s["X"] + (v if gate is None else gate * v)
        y, rs = _norm(S, s["gs"])
        if s["out"] == "f32":
            return {"s": S, "y": y, "ru": ru, "rs": rs}
        return {"s": S, **_mx8_out(*_to_mx8(y))}
    xs, xu = s["S"] * s["rs"][:, None], s["U"] * s["ru"][:, None]
    g = s["dY"] * s["gs"]
    ds = (g - xs * (g * xs).mean(1, keepdim=True)) * s["rs"][:, None]
    if s["dS"] is not None:
        ds = ds + s["dS"]
    dv = ds if gate is None else ds * gate
    g = dv * s["gu"]
    du = (g - xu * (g * xu).mean(1, keepdim=True)) * s["ru"][:, None]
    out = {"du": du, "dx": s["alpha"] * ds, "dgu": (dv * xu).sum(0), "dgs": (s["dY"] * xs).sum(0)}
    if gate is not None:
        dg = ds * (xu * s["gu"])
        out["dgate"] = dg.sum(0) if gate.dim() == 1 else dg
    return out


def _run_own(s):
    from gemv_gemm_f32_amd import binding as bd
    op = s["op"]
    if op == "groups":
        offsets, rows, pos = bd.expert_groups(s["ids"], s["E"])
        return {"offsets": offsets, "rows": rows, "pos": pos}
    if op == "combine":
        return {"out": bd.expert_combine(s["Y"], s["pos"], weights=s["w"], residual=s["R"])}
    if op == "combine_bwd":
        dy, dw = bd.expert_combine_bwd(s["dO"], s["pos"], Y=s["Y"], weights=s["w"])
        return {"dy": dy, "dw": dw}
    if op == "grouped":
        z = torch.empty((s["T"] * s["k"], s["N"]), device="cuda") if s["keep"] else None
        y = bd.linear_f32_grouped(s["X"], s["W"], s["offsets"], rows=s["rows"], bias=s["b"], act=s["act"], Z=z,
                                  trans_w=s["trans_w"])
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    if op == "grouped_bwd":
        dx, dw, db = bd.linear_f32_grouped_bwd(s["dY"], s["X"], s["W"], s["offsets"], rows=s["rows"], Z=s["Z"],
                                               act=s["act"], trans_w=s["trans_w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "packed":
        f = bd.linear_q2_mx8_grouped if s["bits"] == 2 else bd.linear_q4_mx8_grouped
        y = f(s["X8"], s["XE"], s["Q"], s["S"], s["offsets"], rows=s["rows"], bias=s["b"], act=s["act"], out=s["out"])
        return {"y": y} if s["out"] == "f32" else _mx8_out(*y)
    if op == "block_norm":
        if s["out"] == "f32":
            y, S, ru, rs = bd.block_norm_f32(s["U"], s["X"], s["gu"], s["gs"], EPS, gate=s["gate"], alpha=s["alpha"])
            return {"s": S, "y": y, "ru": ru, "rs": rs}
        q, e, S = bd.block_norm_mx8(s["U"], s["X"], s["gu"], s["gs"], EPS, gate=s["gate"], alpha=s["alpha"])
        return {"s": S, **_mx8_out(q, e)}
    du, dx, dgu, dgs, dgate = bd.block_norm_f32_bwd(s["dY"], s["U"], s["S"], s["gu"], s["gs"], s["ru"], s["rs"],
                                                    gate=s["gate"], alpha=s["alpha"], dS=s["dS"])
    out = {"du": du, "dx": dx, "dgu": dgu, "dgs": dgs}
    return out if s["gate"] is None else {**out, "dgate": dgate}


# ----------------------------------------------------------------- costs --

def work(case):
    op = case["op"]
    if op == "groups":
        n = case["T"] * case["k"]
        return {"bytes": 4 * (3 * n + case["E"] + 1), "flops": n}
    if op in ("combine", "combine_bwd"):
        T, k, K = case["T"], case["k"], case["K"]
        if op == "combine":
            words = T * k * (K + 1 + case["weights"]) + T * K * (1 + case["residual"])
            return {"bytes": 4 * words, "flops": 2 * T * k * K}
        return {"bytes": 4 * (2 * T * k * K + T * K + 3 * T * k), "flops": 3 * T * k * K}
    if op in ("grouped", "grouped_bwd", "packed"):
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        k = min(k, E)
        M, met = T * k, E * (1 - (1 - k / E) ** T)      # experts that some token chooses, on average
        if op == "grouped":
            words = K * min(M, T if case["gather"] else M) + met * (N * K + N) + M * N * (1 + case["keep"])
            return {"bytes": 4 * words, "flops": 2 * M * N * K}
        if op == "grouped_bwd":
            words = M * N * (1 + (case["act"] != "none")) + K * (T if case["gather"] else M) + M * K
            return {"bytes": 4 * (words + met * N * K + E * (N * K + N)), "flops": 4 * M * N * K}
        row = lambda n: n + -(-n // 32)  # noqa: E731
        w = N * (-(-K * case["bits"] // 8) + 2 * -(-K // 64) + 4)
        y = 4 * M * N if case["out"] == "f32" else M * row(N)
        return {"bytes": T * row(K) + met * w + y + 4 * M, "flops": 2 * M * N * K}
    M, K = case["M"], case["K"]
    gate = {"none": 0, "columns": K, "rows": M * K}[case["gate"]]
    if op == "block_norm":
        y = 4 * (M * K + 2 * M) if case["out"] == "f32" else M * (K + -(-K // 32))
        return {"bytes": 4 * (3 * M * K + 2 * K + gate) + y, "flops": 11 * M * K}
    return {"bytes": 4 * (M * K * (5 + case["carried"]) + 4 * K + 2 * M + 2 * gate), "flops": 22 * M * K}


# ------------------------------------------------------- definitions, fp64 --

def _parts(z, act):
    """The activation and its derivative in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu_erf":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    return z * p, p + 2 * c * z * p * (1 - p) * (1 + 0.134145 * z ** 2)


def _mx8_exact(v):
    """What the 8-bit values of v stand for before their rounding; no value for the powers of two,
    which jump where a block's largest magnitude crosses a border."""
    M, K = v.shape
    n = -(-K // 32)
    full = torch.zeros(M, n * 32, dtype=torch.float64, device=v.device)
    full[:, :K] = v
    top = full.view(M, n, 32).abs().amax(2)
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-126)
    return {"q": v / torch.exp2(e).repeat_interleave(32, 1)[:, :K], "e": None}


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.dtype == torch.float32 else v for k, v in s.items()}
    op, act = case["op"], case.get("act")
    if op == "groups":
        # by counting: an entry's place is the number of entries of lower experts and of earlier
        # ones of its own
        ids = s["ids"].flatten().cpu().tolist()
        E, k = case["E"], case["k"]
        lists = [[] for _ in range(E + 1)]
        for i, e in enumerate(ids):
            lists[e if 0 <= e < E else E].append(i)
        rows, pos, offsets = [], [-1] * len(ids), [0]
        for e, of in enumerate(lists):
            for i in of:
                if e < E:
                    pos[i] = len(rows)
                rows.append(i // k)
            if e < E:
                offsets.append(len(rows))
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"offsets": whole(offsets), "rows": whole(rows), "pos": whole(pos).view(case["T"], k)}
    if op == "combine":
        out = torch.zeros(case["T"], case["K"], dtype=torch.float64, device="cuda") if d["R"] is None else d["R"].clone()
        for j in range(case["k"]):
            p = d["pos"][:, j].long()
            live = torch.nonzero(p >= 0).flatten()
            y = d["Y"].index_select(0, p[live])
            out[live] += y if d["w"] is None else y * d["w"][live, j].unsqueeze(1)
        return {"out": out}
    if op == "combine_bwd":
        dy, dw = torch.zeros_like(d["Y"]), torch.zeros_like(d["w"])
        for j in range(case["k"]):
            p = d["pos"][:, j].long()
            dy.index_copy_(0, p, d["dO"] * d["w"][:, j].unsqueeze(1))
            dw[:, j] = (d["Y"].index_select(0, p) * d["dO"]).sum(1)
        return {"dy": dy, "dw": dw}
    if op in ("grouped", "grouped_bwd", "packed"):
        T, E, N, K = (case[n] for n in ("T", "E", "N", "K"))
        M = T * s["k"]
        off = [int(v) for v in s["offsets"].cpu()]
        take = (lambda x, a, b: x[a:b]) if s["rows"] is None else (lambda x, a, b: x.index_select(0, s["rows"][a:b]))
        zeros = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")  # noqa: E731
        if op == "grouped_bwd":
            dz = d["dY"] * _parts(d["Z"], act)[1]
            dx, dw, db = zeros(M, K), zeros(*d["W"].shape), zeros(E, N)
            for e in range(E):
                a, b = off[e], off[e + 1]
                w = d["W"][e] if case["trans_w"] else d["W"][e].T.contiguous()      # N x K
                dx[a:b] = torch.matmul(dz[a:b], w)
                g = torch.matmul(dz[a:b].T.contiguous(), take(d["X"], a, b))        # N x K
                dw[e] = g if case["trans_w"] else g.T
                db[e] = dz[a:b].sum(0)
            return {"dx": dx, "dw": dw, "db": db}
        z = zeros(M, N)
        if op == "packed":
            bits, col = case["bits"], torch.arange(K, device="cuda")
            per = 8 // bits
            x = s["X8"].view(torch.float8_e4m3fn).double() * torch.exp2(s["XE"].double() - 127)[:, col // 32]
        for e in range(E):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            if op == "packed":
                code = (s["Q"][e].long()[:, col // per] >> (bits * (col % per))) & (2 ** bits - 1)
                w = (code.double() - (1.5 if bits == 2 else 7.5)) * s["S"][e].double()[:, col // 64]
                z[a:b] = torch.matmul(take(x, a, b), w.T.contiguous()) + d["b"][e]
            else:
                w = d["W"][e].T.contiguous() if case["trans_w"] else d["W"][e]
                z[a:b] = torch.matmul(take(d["X"], a, b), w) + d["b"][e]
        y = _parts(z, act)[0]
        if op == "packed":
            return {"y": y} if case["out"] == "f32" else _mx8_exact(y)
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    K = case["K"]
    gate = 1.0 if d["gate"] is None else d["gate"]
    if op == "block_norm":
        ru = torch.rsqrt(d["U"].pow(2).sum(1) / K + EPS)
        S = d["alpha"] * d["X"] + gate * (d["gu"] * d["U"] * ru.unsqueeze(1))
        rs = torch.rsqrt(S.pow(2).sum(1) / K + EPS)
        y = d["gs"] * S * rs.unsqueeze(1)
        return {"s": S, "y": y, "ru": ru, "rs": rs} if case["out"] == "f32" else {"s": S, **_mx8_exact(y)}
    ru, rs = d["ru"].unsqueeze(1), d["rs"].unsqueeze(1)
    h = d["dY"] * d["gs"]
    ds = rs * h - d["S"] * rs ** 3 * (h * d["S"]).sum(1, keepdim=True) / K
    ds = ds if d["dS"] is None else ds + d["dS"]
    h = ds * gate * d["gu"]
    du = ru * h - d["U"] * ru ** 3 * (h * d["U"]).sum(1, keepdim=True) / K
    out = {"du": du, "dx": d["alpha"] * ds, "dgu": (ds * gate * d["U"] * ru).sum(0), "dgs": (d["dY"] * d["S"] * rs).sum(0)}
    if d["gate"] is not None:
        dg = ds * d["gu"] * d["U"] * ru
        out["dgate"] = dg if case["gate"] == "rows" else dg.sum(0)
    return out
