"""Cases of the dense layer with its epilogue, its backward pass, the root-mean-square norm and the
packed products of 8-bit rows: inputs, plain forms in elementary torch operations, calls of this
package's entry points, and the operators' definitions in 64 bits.

    linear        Y = act(X.W + b) + R, the pre-activation kept on request        (fp32)
    linear_bwd    dX, dW and db of that layer from dY                             (fp32)
    rmsnorm       S = X + R, Y = S * rstd * gamma, in fp32 or in 8 bits           (fp32 / mx8)
    rmsnorm_bwd   dX and dgamma of the norm, with the gradient that reaches S     (fp32)
    packed        Y = act(X8.W^T + b) + R, W in 2-bit or 4-bit codes, Y in fp32 or in 8 bits

8 bits (mx8): e4m3 values with one power of two (e8m0) per 32 columns of a row, the smallest that
keeps the block's largest magnitude within 448.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu_tanh", "gelu_erf", "silu")
SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token through a layer whose weights are stored output by output
        dict(name="linear token", op="linear", M=1, N=2304, K=768, trans_w=True, act="gelu_tanh", bias=True, residual=False, keep=False),
        # a prompt of 346 tokens through a projection back into the residual stream
        dict(name="linear prompt", op="linear", M=346, N=768, K=768, trans_w=False, act="none", bias=True, residual=True, keep=False),
        # a training batch through a wide layer, its pre-activations kept for the backward pass
        dict(name="linear training", op="linear", M=2048, N=2048, K=2048, trans_w=True, act="silu", bias=True, residual=True, keep=True),
        # the gradients of a small layer over a short batch
        dict(name="linear_bwd short", op="linear_bwd", M=346, N=768, K=768, trans_w=False, act="gelu_tanh"),
        # the gradients of a widening layer over a training batch
        dict(name="linear_bwd training", op="linear_bwd", M=1024, N=4096, K=1024, trans_w=True, act="gelu_erf"),
        # a prompt's norm before a projection
        dict(name="rmsnorm prompt", op="rmsnorm", M=346, K=768, residual=True, out="f32"),
        # a training batch's norm, more data than the caches hold
        dict(name="rmsnorm training", op="rmsnorm", M=16384, K=2048, residual=True, out="f32"),
        # one token's norm before a packed product
        dict(name="rmsnorm token mx8", op="rmsnorm", M=1, K=1536, residual=True, out="mx8"),
        dict(name="rmsnorm_bwd short", op="rmsnorm_bwd", M=346, K=768, carried=False),
        dict(name="rmsnorm_bwd training", op="rmsnorm_bwd", M=16384, K=2048, carried=True),
        # one token through a 4-bit matrix, its activations in 8 bits for the next one
        dict(name="packed token q4", op="packed", bits=4, M=1, N=12288, K=1536, act="gelu_tanh", bias=True, residual=False, out="mx8"),
        # a prompt of 500 tokens through a 2-bit matrix
        dict(name="packed prompt q2", op="packed", bits=2, M=500, N=12288, K=1536, act="none", bias=True, residual=True, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "rmsnorm", "rmsnorm_bwd", "packed", "packed"))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("linear", "linear_bwd"):
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 48, 4096), _log(rng, 48, 4096)
            if M * N * K <= 2048 ** 3 // 2:
                break
        if op == "linear_bwd":
            return dict(op=op, M=M, N=N, K=K, trans_w=coin(), act=rng.choice(ACTS))
        return dict(op=op, M=M, N=N, K=K, trans_w=coin(), act=rng.choice(ACTS), bias=coin(), residual=coin(), keep=coin())
    if op in ("rmsnorm", "rmsnorm_bwd"):
        while True:
            M, K = _log(rng, 1, 16384), _log(rng, 33, 16384)
            if M * K <= 16384 * 2048:
                break
        if op == "rmsnorm_bwd":
            return dict(op=op, M=M, K=K, carried=coin())
        return dict(op=op, M=M, K=K, residual=coin(), out=rng.choice(("f32", "mx8")))
    while True:
        M, N, K = _log(rng, 1, 512), _log(rng, 64, 12288), _log(rng, 64, 12288)
        if N * K <= 12288 * 1536 and M * N * K <= 500 * 12288 * 1536:
            break
    return dict(op=op, bits=rng.choice((2, 4)), M=M, N=N, K=K, act=rng.choice(ACTS), bias=coin(), residual=coin(), out=rng.choice(("f32", "mx8")))


# ---------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    s, op, M, K = dict(case), case["op"], case["M"], case["K"]
    if op in ("linear", "linear_bwd"):
        N = case["N"]
        s["X"] = normal(M, K)
        s["W"] = normal(N, K, scale=K ** -0.5) if case["trans_w"] else normal(K, N, scale=K ** -0.5)
        if op == "linear":
            s["b"] = normal(N, scale=0.5) if case["bias"] else None
            s["R"] = normal(M, N) if case["residual"] else None
        else:
            s["dY"] = normal(M, N)
            s["Z"] = normal(M, N, scale=1.5)
    elif op == "rmsnorm":
        # a residual stream has a few channels far larger than the rest
        s["X"] = normal(M, K)
        s["R"] = normal(M, K) * (1 + 20 * (torch.rand(K, generator=g, device="cuda") < 0.01)) if case["residual"] else None
        s["gamma"] = 1 + normal(K, scale=0.2)
    elif op == "rmsnorm_bwd":
        s["S"] = normal(M, K)
        s["gamma"] = 1 + normal(K, scale=0.2)
        s["rstd"] = 1 / torch.sqrt((s["S"] * s["S"]).mean(1) + 1e-5)
        s["dY"] = normal(M, K)
        s["dS"] = normal(M, K) if case["carried"] else None
    else:
        N, bits = case["N"], case["bits"]
        s["X8"], s["XE"] = _to_mx8(normal(M, K))
        s["Q"] = torch.randint(0, 256, (N, -(-K * bits // 8)), generator=g, device="cuda", dtype=torch.uint8)
        s["S"] = (0.01 + 0.04 * torch.rand(N, -(-K // 64), generator=g, device="cuda")).half()
        s["b"] = normal(N, scale=0.5) if case["bias"] else None
        s["R"] = normal(M, N) if case["residual"] else None
    return s


# ----------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(SQRT_2_OVER_PI * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_tanh":
        t = torch.tanh(SQRT_2_OVER_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * SQRT_2_OVER_PI * (1 + 3 * 0.044715 * z * z)
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
    M, K = q.shape
    scale = torch.ldexp(torch.ones(e.shape, dtype=dtype, device=e.device), e.to(torch.int32) - 127)
    return q.view(torch.float8_e4m3fn).to(dtype) * scale.repeat_interleave(32, 1)[:, :K]


def _weights(Q, S, bits, K, dtype):
    """The values that 2-bit or 4-bit codes with one scale per 64 columns stand for."""
    shifts = torch.arange(0, 8, bits, device=Q.device, dtype=torch.uint8)
    codes = (Q[:, :, None] >> shifts & (2 ** bits - 1)).reshape(Q.shape[0], -1)[:, :K]
    return (codes.to(dtype) - (2 ** bits - 1) / 2) * S.to(dtype).repeat_interleave(64, 1)[:, :K]


def _mx8_out(q, e):
    return {"q": q.view(torch.float8_e4m3fn), "e": e.view(torch.float8_e8m0fnu)}


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "linear":
        z = s["X"] @ (s["W"].t() if s["trans_w"] else s["W"])
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["R"] is not None:
            y = y + s["R"]
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    if op == "linear_bwd":
        dz = s["dY"] * _act_grad(s["Z"], s["act"])
        dx = dz @ (s["W"] if s["trans_w"] else s["W"].t())
        dw = dz.t() @ s["X"] if s["trans_w"] else s["X"].t() @ dz
        return {"dx": dx, "dw": dw, "db": dz.sum(0)}
    if op == "rmsnorm":
        v = s["X"] if s["R"] is None else s["X"] + s["R"]
        rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5)
        y = v * rstd * s["gamma"]
        out = {} if s["R"] is None else {"s": v}
        if s["out"] == "f32":
            return {**out, "y": y, "rstd": rstd[:, 0]}
        return {**out, **_mx8_out(*_to_mx8(y))}
    if op == "rmsnorm_bwd":
        xhat = s["S"] * s["rstd"][:, None]
        gdy = s["dY"] * s["gamma"]
        dx = (gdy - xhat * (gdy * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["dS"] is not None:
            dx = dx + s["dS"]
        return {"dx": dx, "dgamma": (s["dY"] * xhat).sum(0)}
    w = _weights(s["Q"], s["S"], s["bits"], s["K"], torch.float32)
    y = _from_mx8(s["X8"], s["XE"], torch.float32) @ w.t()
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    if s["R"] is not None:
        y = y + s["R"]
    return {"y": y} if s["out"] == "f32" else _mx8_out(*_to_mx8(y))


def _run_own(s):
    from gemv_gemm_f32_amd import binding as bd
    op = s["op"]
    if op == "linear":
        z = torch.empty((s["M"], s["N"]), device="cuda") if s["keep"] else None
        y = bd.linear_f32(s["X"], s["W"], bias=s["b"], act=s["act"], residual=s["R"], Z=z, trans_w=s["trans_w"])
        return {"y": y, "z": z} if s["keep"] else {"y": y}
    if op == "linear_bwd":
        dx, dw, db = bd.linear_f32_bwd(s["dY"], s["X"], s["W"], Z=s["Z"], act=s["act"], trans_w=s["trans_w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "rmsnorm":
        if s["out"] == "f32":
            y, v, rstd = bd.rmsnorm_f32(s["X"], s["gamma"], 1e-5, residual=s["R"])
            return {"y": y, "rstd": rstd} if s["R"] is None else {"s": v, "y": y, "rstd": rstd}
        q, e, v = bd.rmsnorm_mx8(s["X"], s["gamma"], 1e-5, residual=s["R"])
        return _mx8_out(q, e) if s["R"] is None else {"s": v, **_mx8_out(q, e)}
    if op == "rmsnorm_bwd":
        dx, dgamma = bd.rmsnorm_f32_bwd(s["dY"], s["S"], s["gamma"], s["rstd"], dS=s["dS"])
        return {"dx": dx, "dgamma": dgamma}
    f = bd.linear_q2_mx8 if s["bits"] == 2 else bd.linear_q4_mx8
    y = f(s["X8"], s["XE"], s["Q"], s["S"], bias=s["b"], act=s["act"], residual=s["R"], out=s["out"])
    return {"y": y} if s["out"] == "f32" else _mx8_out(*y)


# ----------------------------------------------------------------- costs --

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "linear":
        N = case["N"]
        words = M * K + K * N + M * N * (1 + case["residual"] + case["keep"]) + N * case["bias"]
        return {"bytes": 4 * words, "flops": 2 * M * N * K}
    if op == "linear_bwd":
        N = case["N"]
        words = M * N * (1 + (case["act"] != "none")) + 2 * M * K + 2 * N * K + N
        return {"bytes": 4 * words, "flops": 4 * M * N * K}
    if op == "rmsnorm":
        read = M * K * (1 + case["residual"]) + K
        y = 4 * (M * K + M) if case["out"] == "f32" else M * (K + -(-K // 32))
        return {"bytes": 4 * (read + M * K * case["residual"]) + y, "flops": 6 * M * K}
    if op == "rmsnorm_bwd":
        return {"bytes": 4 * (M * K * (3 + case["carried"]) + 2 * K + M), "flops": 10 * M * K}
    N, bits = case["N"], case["bits"]
    rows = lambda n: n + -(-n // 32)  # noqa: E731
    w = N * (-(-K * bits // 8) + 2 * -(-K // 64))
    y = 4 * M * N if case["out"] == "f32" else M * rows(N)
    return {"bytes": M * rows(K) + w + y + 4 * (M * N * case["residual"] + N * case["bias"]), "flops": 2 * M * N * K}


# ------------------------------------------------------- definitions, fp64 --

def _gelu_parts(z, act):
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
    if op == "linear":
        z = torch.matmul(d["X"], d["W"].T.contiguous() if case["trans_w"] else d["W"])
        z = z if d["b"] is None else z + d["b"]
        y = _gelu_parts(z, act)[0]
        y = y if d["R"] is None else y + d["R"]
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if op == "linear_bwd":
        dz = d["dY"] * _gelu_parts(d["Z"], act)[1]
        w = d["W"] if case["trans_w"] else d["W"].T.contiguous()      # N x K
        dw = torch.matmul(dz.T.contiguous(), d["X"])                  # N x K
        return {"dx": torch.matmul(dz, w), "dw": dw if case["trans_w"] else dw.T.contiguous(), "db": dz.sum(0)}
    if op == "rmsnorm":
        v = d["X"] if d["R"] is None else d["X"] + d["R"]
        r = torch.rsqrt(v.pow(2).sum(1) / case["K"] + 1e-5)
        y = d["gamma"] * v * r.unsqueeze(1)
        out = {} if d["R"] is None else {"s": v}
        return {**out, "y": y, "rstd": r} if case["out"] == "f32" else {**out, **_mx8_exact(y)}
    if op == "rmsnorm_bwd":
        r = d["rstd"].unsqueeze(1)
        g = d["dY"] * d["gamma"]
        dx = r * g - d["S"] * r ** 3 * (g * d["S"]).sum(1, keepdim=True) / case["K"]
        return {"dx": dx if d["dS"] is None else dx + d["dS"], "dgamma": (d["dY"] * d["S"] * r).sum(0)}
    K, bits = case["K"], case["bits"]
    col = torch.arange(K, device="cuda")
    per = 8 // bits
    code = (s["Q"].long()[:, col // per] >> (bits * (col % per))) & (2 ** bits - 1)
    w = (code.double() - (1.5 if bits == 2 else 7.5)) * s["S"].double()[:, col // 64]
    x = s["X8"].view(torch.float8_e4m3fn).double() * torch.exp2(s["XE"].double() - 127)[:, col // 32]
    y = torch.matmul(x, w.T.contiguous())
    y = y if d["b"] is None else y + d["b"]
    y = _gelu_parts(y, act)[0]
    y = y if d["R"] is None else y + d["R"]
    return {"y": y} if case["out"] == "f32" else _mx8_exact(y)
