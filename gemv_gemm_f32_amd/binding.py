"""ctypes binding of libgemvgemm.so: the C entry points on torch tensors.

Argument marshalling only: every step of every product runs in the HIP
kernels behind the C ABI (include/gemvgemm.h).  torch supplies device memory
and the current stream.  If the library has not been built this module
raises; there is no fallback of any kind.

Each tensor function has the name of its C entry point and takes row-major
2-D tensors whose last dimension is contiguous; the row stride is passed as
the leading dimension.  The output is written in place (allocated when not
given) and returned.  A non-zero status raises ``GGError``.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgemvgemm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gemvgemm.h")

GG_OK = 0
GG_ERR_INVALID_ARG = -1
GG_ERR_ALIAS = -2
GG_ERR_NO_DEVICE = -3
GG_ERR_LAUNCH = -4
GG_ERR_SCRATCH = -5

ENTRY_POINTS = ("gemm_f32", "gemm_f32_tn", "gemm_f32_nt", "gemm_f32_ex", "gemv_f32",
                "gemv_f32_batched", "gemv_q2", "gemv_q2_batched", "gemv_q2_batched_ws",
                "gemv_q2_batched_ws_size", "gemv_q2_batched_noalloc", "gemv_q4",
                "gemv_q4_batched", "linear_f32", "linear_f32_bwd", "linear_f32_bwd_ws_size",
                "rmsnorm_f32", "rmsnorm_mx8", "rmsnorm_f32_bwd", "rmsnorm_f32_bwd_ws_size",
                "linear_q2_mx8", "linear_q4_mx8", "gg_strerror")

# enum gg_act by name
ACTIVATIONS = {"none": 0, "relu": 1, "gelu_tanh": 2, "gelu_erf": 3, "silu": 4}

_lib = None


class GGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, strerror(status), status))


def load(path: str = LIB_PATH):
    """Open the library (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    # torch ships its own HIP runtime (soname libamdhip64.so.7).  Importing it
    # first makes this library's libamdhip64.so.7 dependency resolve to that
    # already-loaded copy, so torch's streams and allocations and these
    # kernels live in one runtime.  (Loaded first on its own, the library
    # would pull in a second runtime, and torch's stream handles would be
    # meaningless to it.)
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(path):
        raise RuntimeError(
            "libgemvgemm.so is not built (%s); run `python -m gemv_gemm_f32_amd.build`"
            % path)
    lib = ctypes.CDLL(path)
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    for name in ("gemm_f32", "gemm_f32_tn", "gemm_f32_nt"):
        f = getattr(lib, name)
        f.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        f.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.gemm_f32_ex.argtypes = [ctypes.c_int, ctypes.c_int, i64, i64, i64, f32, vp, i64,
                                vp, i64, f32, vp, i64, vp]
    lib.gemm_f32_ex.restype = ctypes.c_int
    lib.gemv_f32.argtypes = [i64, i64, vp, i64, vp, vp, vp]
    lib.gemv_f32.restype = ctypes.c_int
    pp = ctypes.POINTER(ctypes.c_void_p)
    lib.gemv_f32_batched.argtypes = [i64, i64, i64, pp, i64, pp, pp, vp]
    lib.gemv_f32_batched.restype = ctypes.c_int
    for name in ("gemv_q2", "gemv_q4"):
        f = getattr(lib, name)
        f.argtypes = [i64, i64, vp, i64, vp, i64, vp, vp, vp]
        f.restype = ctypes.c_int
        f = getattr(lib, name + "_batched")
        f.argtypes = [i64, i64, i64, pp, i64, pp, i64, pp, pp, vp]
        f.restype = ctypes.c_int
    lib.gemv_q2_batched_ws.argtypes = [i64, i64, i64, pp, i64, pp, i64, pp, pp, vp, i64, vp]
    lib.gemv_q2_batched_ws.restype = ctypes.c_int
    lib.gemv_q2_batched_noalloc.argtypes = [i64, i64, i64, pp, i64, pp, i64, pp, pp, vp]
    lib.gemv_q2_batched_noalloc.restype = ctypes.c_int
    lib.gemv_q2_batched_ws_size.argtypes = [i64, i64, i64]
    lib.gemv_q2_batched_ws_size.restype = i64
    i32 = ctypes.c_int
    lib.linear_f32.argtypes = [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64,
                               vp, i64, vp]
    lib.linear_f32.restype = i32
    lib.linear_f32_bwd.argtypes = [i32, i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp,
                                   i64, vp, i64, vp, i64, vp, vp, i64, vp]
    lib.linear_f32_bwd.restype = i32
    lib.linear_f32_bwd_ws_size.argtypes = [i32, i64, i64]
    lib.linear_f32_bwd_ws_size.restype = i64
    lib.rmsnorm_f32.argtypes = [i64, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, vp]
    lib.rmsnorm_f32.restype = i32
    lib.rmsnorm_mx8.argtypes = [i64, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, i64, vp, i64, vp]
    lib.rmsnorm_mx8.restype = i32
    lib.rmsnorm_f32_bwd.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp,
                                    vp, i64, vp]
    lib.rmsnorm_f32_bwd.restype = i32
    lib.rmsnorm_f32_bwd_ws_size.argtypes = [i64, i64]
    lib.rmsnorm_f32_bwd_ws_size.restype = i64
    for name in ("linear_q2_mx8", "linear_q4_mx8"):
        f = getattr(lib, name)
        f.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp,
                      i64, vp, i64, vp, i64, vp]
        f.restype = i32
    lib.gg_strerror.argtypes = [ctypes.c_int]
    lib.gg_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


def strerror(status: int) -> str:
    return load().gg_strerror(int(status)).decode()


def header_functions(path: str = HEADER):
    """Names of the functions declared in the public header."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


# ------------------------------------------------------------ tensor side --

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream, dev=None):
    torch = _torch()
    if stream is None:
        # the handle alone: building a Stream object takes longer than the
        # rest of a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _mat(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU device" % name)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)
    return t.data_ptr(), ld


def _vec(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device.type != "cuda":
        raise TypeError("%s must be a %s GPU tensor" % (name, dtype))
    if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector" % name)
    return t.data_ptr()


def _check(status, where):
    if status != GG_OK:
        raise GGError(status, where)


def _gemm(name, A, B, C, M, N, K, stream):
    torch = _torch()
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be %d x %d" % (M, N))
    pa, lda = _mat(A, torch.float32, "A")
    pb, ldb = _mat(B, torch.float32, "B")
    pc, ldc = _mat(C, torch.float32, "C")
    _check(getattr(load(), name)(M, N, K, pa, lda, pb, ldb, pc, ldc, _stream(stream)), name)
    return C


def gemm_f32(A, B, C=None, stream=None):
    """C = A.B with A (M x K) and B (K x N)."""
    M, K = A.shape
    if B.shape[0] != K:
        raise ValueError("inner dimensions differ")
    return _gemm("gemm_f32", A, B, C, M, B.shape[1], K, stream)


def gemm_f32_tn(A, B, C=None, stream=None):
    """C = A^T.B with A stored K x M and B (K x N)."""
    K, M = A.shape
    if B.shape[0] != K:
        raise ValueError("inner dimensions differ")
    return _gemm("gemm_f32_tn", A, B, C, M, B.shape[1], K, stream)


def gemm_f32_nt(A, B, C=None, stream=None):
    """C = A.B^T with A (M x K) and B stored N x K."""
    M, K = A.shape
    if B.shape[1] != K:
        raise ValueError("inner dimensions differ")
    return _gemm("gemm_f32_nt", A, B, C, M, B.shape[0], K, stream)


def gemm_f32_ex(A, B, C=None, alpha=1.0, beta=0.0, trans_a=False, trans_b=False,
                stream=None):
    """C = alpha * op(A).op(B) + beta * C in place (C is not read when beta
    == 0; a new C is allocated when None, which needs beta == 0).  op(A) =
    A^T when trans_a (A stored K x M), op(B) = B^T when trans_b."""
    torch = _torch()
    M = A.shape[1] if trans_a else A.shape[0]
    K = A.shape[0] if trans_a else A.shape[1]
    Kb = B.shape[1] if trans_b else B.shape[0]
    N = B.shape[0] if trans_b else B.shape[1]
    if K != Kb:
        raise ValueError("inner dimensions differ")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError("C must be M x N")
    pa, lda = _mat(A, torch.float32, "A")
    pb, ldb = _mat(B, torch.float32, "B")
    pc, ldc = _mat(C, torch.float32, "C")
    _check(load().gemm_f32_ex(int(bool(trans_a)), int(bool(trans_b)), M, N, K, float(alpha),
                              pa, lda, pb, ldb, float(beta), pc, ldc, _stream(stream)),
           "gemm_f32_ex")
    return C


def gemv_f32(W, x, y=None, stream=None):
    """y = W.x with W (M x K) fp32 and x (K,) fp32."""
    torch = _torch()
    M, K = W.shape
    if x.shape != (K,):
        raise ValueError("x must have K entries")
    if y is None:
        y = torch.empty(M, dtype=torch.float32, device=W.device)
    if y.shape != (M,):
        raise ValueError("y must have M entries")
    pw, ldw = _mat(W, torch.float32, "W")
    _check(load().gemv_f32(M, K, pw, ldw, _vec(x, torch.float32, "x"),
                           _vec(y, torch.float32, "y"), _stream(stream)), "gemv_f32")
    return y


def gemv_f32_batched(Ws, xs, ys=None, stream=None):
    """y_b = W_b.x_b for every b: lists of W (fp32 M x K, one shape and
    leading dimension for all) and x (K,) fp32.  Returns the list of
    outputs."""
    torch = _torch()
    n = len(Ws)
    if len(xs) != n:
        raise ValueError("Ws and xs must have the same length")
    if n == 0:
        return []
    M, K = Ws[0].shape
    if ys is None:
        ys = [torch.empty(M, dtype=torch.float32, device=Ws[0].device) for _ in range(n)]
    wp, xp, yp, ldw = [], [], [], None
    for W, x, y in zip(Ws, xs, ys):
        if tuple(W.shape) != (M, K) or x.shape != (K,) or y.shape != (M,):
            raise ValueError("every product must have the same M and K")
        pw, lw = _mat(W, torch.float32, "W")
        if ldw is None:
            ldw = lw
        elif lw != ldw:
            raise ValueError("every W must have the same leading dimension")
        wp.append(pw)
        xp.append(_vec(x, torch.float32, "x"))
        yp.append(_vec(y, torch.float32, "y"))
    _check(load().gemv_f32_batched(n, M, K, _ptr_array(wp), ldw, _ptr_array(xp),
                                   _ptr_array(yp), _stream(stream)), "gemv_f32_batched")
    return ys


def _packed(name, Q, S, x, y, stream):
    torch = _torch()
    M = Q.shape[0]
    K = x.shape[0]
    if S.shape[0] != M:
        raise ValueError("Q and S must have the same number of rows")
    if S.dtype in (torch.float16, torch.int16):
        S = S.view(torch.float16)
    else:
        raise TypeError("S must hold binary16 bit patterns (float16 or int16)")
    if y is None:
        y = torch.empty(M, dtype=torch.float32, device=Q.device)
    if y.shape != (M,):
        raise ValueError("y must have M entries")
    pq, ldq = _mat(Q, torch.uint8, "Q")
    ps, lds = _mat(S, torch.float16, "S")
    _check(getattr(load(), name)(M, K, pq, ldq, ps, lds, _vec(x, torch.float32, "x"),
                                 _vec(y, torch.float32, "y"), _stream(stream)), name)
    return y


def gemv_q2(Q, S, x, y=None, stream=None):
    """y = W.x with W as 2-bit codes Q (uint8, M x >= ceil(K/4)) and binary16
    scales S (float16 or int16 bit patterns, M x >= ceil(K/64)); x (K,) fp32."""
    return _packed("gemv_q2", Q, S, x, y, stream)


def gemv_q4(Q, S, x, y=None, stream=None):
    """y = W.x with W as 4-bit codes Q (uint8, M x >= ceil(K/2)) and binary16
    scales S (float16 or int16 bit patterns, M x >= ceil(K/64)); x (K,) fp32."""
    return _packed("gemv_q4", Q, S, x, y, stream)


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(len(ptrs), 1))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


def _packed_batched(name, Qs, Ss, xs, ys, stream, ws=None):
    torch = _torch()
    n = len(Qs)
    if len(Ss) != n or len(xs) != n:
        raise ValueError("Qs, Ss and xs must have the same length")
    if n == 0:
        return []
    M, K = Qs[0].shape[0], xs[0].shape[0]
    if ys is None:
        ys = [torch.empty(M, dtype=torch.float32, device=Qs[0].device) for _ in range(n)]
    qp, sp, xp, yp, ldq, lds = [], [], [], [], None, None
    for Q, S, x, y in zip(Qs, Ss, xs, ys):
        if Q.shape[0] != M or S.shape[0] != M or x.shape != (K,) or y.shape != (M,):
            raise ValueError("every product must have the same M and K")
        if S.dtype not in (torch.float16, torch.int16):
            raise TypeError("S must hold binary16 bit patterns (float16 or int16)")
        pq, lq = _mat(Q, torch.uint8, "Q")
        ps, ls = _mat(S.view(torch.float16), torch.float16, "S")
        if ldq is None:
            ldq, lds = lq, ls
        elif (lq, ls) != (ldq, lds):
            raise ValueError("every Q (and every S) must have the same leading dimension")
        qp.append(pq)
        sp.append(ps)
        xp.append(_vec(x, torch.float32, "x"))
        yp.append(_vec(y, torch.float32, "y"))
    args = [n, M, K, _ptr_array(qp), ldq, _ptr_array(sp), lds, _ptr_array(xp), _ptr_array(yp)]
    if ws is not None:
        if ws.numel() and (ws.device.type != "cuda" or not ws.is_contiguous()):
            raise ValueError("the workspace must be a contiguous GPU tensor")
        args += [ws.data_ptr() if ws.numel() else None, ws.numel() * ws.element_size()]
    _check(getattr(load(), name)(*args, _stream(stream)), name)
    return ys


def gemv_q2_batched(Qs, Ss, xs, ys=None, stream=None):
    """y_b = W_b.x_b for every b: lists of Q (uint8 M x >= ceil(K/4)), S
    (float16/int16 M x >= ceil(K/64)), x (K,) fp32; all Q share one shape and
    leading dimension, as do all S.  Returns the list of outputs."""
    return _packed_batched("gemv_q2_batched", Qs, Ss, xs, ys, stream)


def gemv_q2_batched_ws_size(count, M, K):
    """Bytes of workspace gemv_q2_batched_ws needs for count products of M x K."""
    n = load().gemv_q2_batched_ws_size(count, M, K)
    if n < 0:
        raise GGError(n, "gemv_q2_batched_ws_size")
    return n


def gemv_q2_batched_ws(Qs, Ss, xs, ys=None, workspace=None, stream=None):
    """gemv_q2_batched with a workspace (a contiguous GPU tensor of at least
    gemv_q2_batched_ws_size bytes; allocated here as uint8 when None)."""
    torch = _torch()
    if workspace is None:
        n = gemv_q2_batched_ws_size(len(Qs), Qs[0].shape[0] if Qs else 0,
                                    xs[0].shape[0] if xs else 0)
        workspace = torch.empty(n, dtype=torch.uint8, device=Qs[0].device if Qs else "cuda")
    return _packed_batched("gemv_q2_batched_ws", Qs, Ss, xs, ys, stream, ws=workspace)


def gemv_q2_batched_noalloc(Qs, Ss, xs, ys=None, stream=None):
    """gemv_q2_batched_ws on the library's fixed per-GPU scratch buffer
    instead of a workspace (outputs are allocated here when ys is None)."""
    return _packed_batched("gemv_q2_batched_noalloc", Qs, Ss, xs, ys, stream)


def gemv_q4_batched(Qs, Ss, xs, ys=None, stream=None):
    """As gemv_q2_batched for 4-bit codes (Q uint8 M x >= ceil(K/2))."""
    return _packed_batched("gemv_q4_batched", Qs, Ss, xs, ys, stream)


# ----------------------------------------------------- dense layers, norm --

def _arg(t, shape, dtype, name, dev):
    """(address, leading dimension) of a row-major tensor (or vector) of this
    shape and type on device number `dev`; (None, 0) for None."""
    if t is None:
        return None, 0
    if getattr(t, "dtype", None) is not dtype:
        raise _type_error(t, dtype, name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on the current GPU device" % name)
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    if len(shape) == 1:
        return t.data_ptr(), shape[0]
    return t.data_ptr(), st[0] if shape[0] > 1 else shape[1] or 1


def _type_error(t, dtype, name):
    return TypeError("%s must be a torch tensor of %s, got %s" % (name, dtype, getattr(t, "dtype", type(t).__name__)))


def _wide(t, rows, cols, dtype, name, dev):
    """As _arg for rows of at least `cols` entries."""
    if getattr(t, "dtype", None) is not dtype:
        raise _type_error(t, dtype, name)
    shape = t.shape
    if len(shape) != 2 or shape[1] < cols:
        raise ValueError("%s must be 2-D with at least %d columns" % (name, cols))
    return _arg(t, (rows, shape[1]), dtype, name, dev)


def _out(t, shape, dtype, name, dev, like, stream):
    """An output and its (address, leading dimension): the one given, checked,
    or a new one."""
    if t is None:
        t = _new(shape, dtype, like, stream)
        return t, t.data_ptr(), shape[-1] or 1
    return (t, *_arg(t, shape, dtype, name, dev))


def _new(shape, dtype, like, stream):
    """A new tensor that belongs to the stream the call runs on, so that its
    memory is neither taken from nor given back to work of another stream."""
    torch = _torch()
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _matrix(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return tuple(t.shape)


def _activation(act):
    try:
        return ACTIVATIONS[act]
    except KeyError:
        raise ValueError("act must be one of %s" % ", ".join(ACTIVATIONS)) from None


def _workspace(ws, need, dev, like, stream):
    torch = _torch()
    if ws is None:
        ws = _new((need,), torch.uint8, like, stream)
    elif not isinstance(ws, torch.Tensor):
        raise TypeError("the workspace must be a torch tensor")
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the current GPU device")
    n = ws.numel() * ws.element_size()
    return ws, ws.data_ptr() if n else None, n


def _ws_size(name, *sizes):
    n = getattr(load(), name)(*sizes)
    if n < 0:
        raise GGError(n, name)
    return n


def linear_f32(X, W, bias=None, act="none", residual=None, Z=None, Y=None, trans_w=False,
               stream=None):
    """Y = act(X.op(W) + bias) + residual, fp32: X (M x K), W (K x N, or N x K
    when trans_w), bias (N,), residual and Y (M x N).  act is a name of
    ACTIVATIONS.  Z (M x N), when given, receives the pre-activation that
    linear_f32_bwd takes.  Y may be the residual itself."""
    torch = _torch()
    f32, dev = torch.float32, torch.cuda.current_device()
    M, K = _matrix(X, "X")
    wshape = _matrix(W, "W")
    N = wshape[0] if trans_w else wshape[1]
    px, ldx = _arg(X, (M, K), f32, "X", dev)
    pw, ldw = _arg(W, (N, K) if trans_w else (K, N), f32, "W", dev)
    pb, _ = _arg(bias, (N,), f32, "bias", dev)
    pr, ldr = _arg(residual, (M, N), f32, "residual", dev)
    pz, ldz = _arg(Z, (M, N), f32, "Z", dev)
    Y, py, ldy = _out(Y, (M, N), f32, "Y", dev, X, stream)
    _check(load().linear_f32(int(bool(trans_w)), _activation(act), M, N, K, px, ldx, pw, ldw, pb,
                             pr, ldr, pz, ldz, py, ldy, _stream(stream, dev)), "linear_f32")
    return Y


def linear_f32_bwd_ws_size(act, M, N):
    """Bytes of workspace linear_f32_bwd needs for an M x N output."""
    return _ws_size("linear_f32_bwd_ws_size", _activation(act), M, N)


def linear_f32_bwd(dY, X, W, Z=None, act="none", trans_w=False, dX=None, dW=None, db=None,
                   want=("dX", "dW", "db"), accumulate=False, workspace=None, stream=None):
    """Gradients (dX, dW, db) of linear_f32 from dY (M x N) and the kept
    pre-activation Z (not needed for act "none"); the residual's gradient is
    dY itself.  X is needed for dW alone and W for dX; either may be None
    otherwise.  Gradients not named in `want` are not computed and returned
    as None; outputs not given are allocated.  accumulate: dW and db, which
    must then be given, are added to."""
    torch = _torch()
    f32, dev = torch.float32, torch.cuda.current_device()
    M, N = _matrix(dY, "dY")
    wx, ww, wb = (n in want for n in ("dX", "dW", "db"))
    if (wx and W is None) or (ww and X is None):
        raise ValueError("dX needs W and dW needs X")
    # db alone needs neither, and no K
    K = _matrix(X, "X")[1] if X is not None else _matrix(W, "W")[1 if trans_w else 0] if W is not None else 0
    wshape = (N, K) if trans_w else (K, N)
    a = _activation(act)
    if a and Z is None:
        raise ValueError("act %r needs Z" % act)
    if accumulate and ((ww and dW is None) or (wb and db is None)):
        raise ValueError("accumulate needs the gradients to add to")
    pd, lddy = _arg(dY, (M, N), f32, "dY", dev)
    pz, ldz = _arg(Z if a else None, (M, N), f32, "Z", dev)
    px, ldx = _arg(X, (M, K), f32, "X", dev)
    pw, ldw = _arg(W, wshape, f32, "W", dev)
    none = (None, None, 0)
    dX, pdx, lddx = _out(dX, (M, K), f32, "dX", dev, dY, stream) if wx else none
    dW, pdw, lddw = _out(dW, wshape, f32, "dW", dev, dY, stream) if ww else none
    db, pdb, _ = _out(db, (N,), f32, "db", dev, dY, stream) if wb else none
    need = _ws_size("linear_f32_bwd_ws_size", a, M, N)
    keep, pws, nws = _workspace(workspace, need, dev, dY, stream)
    _check(load().linear_f32_bwd(int(bool(trans_w)), a, int(bool(accumulate)), M, N, K, pd, lddy,
                                 pz, ldz, px, ldx, pw, ldw, pdx, lddx, pdw, lddw, pdb, pws, nws,
                                 _stream(stream, dev)), "linear_f32_bwd")
    return dX, dW, db


def rmsnorm_f32(X, gamma=None, eps=1e-5, residual=None, S=None, Y=None, rstd=None, stream=None):
    """(Y, S, rstd) with S = X + residual, rstd = 1 / sqrt(mean of S^2 over a
    row + eps) and Y = S * rstd * gamma, fp32, rows of X (M x K).  Without a
    residual (and with no S given) S is X itself and nothing is written for
    it.  S may be given as X or the residual itself, to update it in place."""
    torch = _torch()
    f32, dev = torch.float32, torch.cuda.current_device()
    M, K = _matrix(X, "X")
    px, ldx = _arg(X, (M, K), f32, "X", dev)
    pr, ldr = _arg(residual, (M, K), f32, "residual", dev)
    pg, _ = _arg(gamma, (K,), f32, "gamma", dev)
    ps = lds = 0
    if S is not None or residual is not None:
        S, ps, lds = _out(S, (M, K), f32, "S", dev, X, stream)
    Y, py, ldy = _out(Y, (M, K), f32, "Y", dev, X, stream)
    rstd, pt, _ = _out(rstd, (M,), f32, "rstd", dev, X, stream)
    _check(load().rmsnorm_f32(M, K, px, ldx, pr, ldr, pg, float(eps), ps, lds, py, ldy, pt,
                              _stream(stream, dev)), "rmsnorm_f32")
    return Y, X if S is None else S, rstd


def _bytes(t):
    """A float8 tensor as its bytes; a uint8 tensor as it is."""
    torch = _torch()
    if getattr(t, "dtype", None) in (torch.float8_e4m3fn, torch.float8_e8m0fnu):
        return t.view(torch.uint8)
    return t


def rmsnorm_mx8(X, gamma=None, eps=1e-5, residual=None, S=None, Q=None, E=None, stream=None):
    """(Q, E, S): the norm of rmsnorm_f32 with its output in 8 bits, Q (M x K)
    e4m3 bytes and E (M x ceil(K/32)) powers of two, as uint8 (view them as
    torch.float8_e4m3fn and torch.float8_e8m0fnu for their values)."""
    torch = _torch()
    f32, u8, dev = torch.float32, torch.uint8, torch.cuda.current_device()
    M, K = _matrix(X, "X")
    px, ldx = _arg(X, (M, K), f32, "X", dev)
    pr, ldr = _arg(residual, (M, K), f32, "residual", dev)
    pg, _ = _arg(gamma, (K,), f32, "gamma", dev)
    ps = lds = 0
    if S is not None or residual is not None:
        S, ps, lds = _out(S, (M, K), f32, "S", dev, X, stream)
    Q, pq, ldq = _out(_bytes(Q), (M, K), u8, "Q", dev, X, stream)
    E, pe, lde = _out(_bytes(E), (M, -(-K // 32)), u8, "E", dev, X, stream)
    _check(load().rmsnorm_mx8(M, K, px, ldx, pr, ldr, pg, float(eps), ps, lds, pq, ldq, pe, lde,
                              _stream(stream, dev)), "rmsnorm_mx8")
    return Q, E, X if S is None else S


def rmsnorm_f32_bwd_ws_size(M, K):
    """Bytes of workspace rmsnorm_f32_bwd needs for dgamma."""
    return _ws_size("rmsnorm_f32_bwd_ws_size", M, K)


def rmsnorm_f32_bwd(dY, S, gamma, rstd, dS=None, dX=None, dgamma=None, want=("dX", "dgamma"),
                    accumulate=False, workspace=None, stream=None):
    """Gradients (dX, dgamma) of rmsnorm_f32 from dY (M x K), with the S and
    rstd that it returned; dX is the gradient of X and of the residual alike.
    dS: the gradient that reaches S past the norm; dX may be dS itself.
    Gradients not named in `want` are returned as None.  accumulate: dgamma,
    which must then be given, is added to."""
    torch = _torch()
    f32, dev = torch.float32, torch.cuda.current_device()
    M, K = _matrix(dY, "dY")
    wx, wg = "dX" in want, "dgamma" in want
    if accumulate and wg and dgamma is None:
        raise ValueError("accumulate needs the gradient to add to")
    pd, lddy = _arg(dY, (M, K), f32, "dY", dev)
    ps, lds = _arg(S, (M, K), f32, "S", dev)
    pg, _ = _arg(gamma, (K,), f32, "gamma", dev)
    pt, _ = _arg(rstd, (M,), f32, "rstd", dev)
    pds, ldds = _arg(dS, (M, K), f32, "dS", dev)
    none = (None, None, 0)
    dX, pdx, lddx = _out(dX, (M, K), f32, "dX", dev, dY, stream) if wx else none
    dgamma, pdg, _ = _out(dgamma, (K,), f32, "dgamma", dev, dY, stream) if wg else none
    need = _ws_size("rmsnorm_f32_bwd_ws_size", M, K) if wg else 0
    keep, pws, nws = _workspace(workspace, need, dev, dY, stream)
    _check(load().rmsnorm_f32_bwd(int(bool(accumulate)), M, K, pd, lddy, ps, lds, pg, pt, pds,
                                  ldds, pdx, lddx, pdg, pws, nws, _stream(stream, dev)),
           "rmsnorm_f32_bwd")
    return dX, dgamma


def _packed_linear(name, bits, X8, XE, Q, S, bias, act, residual, Y, Y8, YE, out, stream):
    torch = _torch()
    f32, u8, dev = torch.float32, torch.uint8, torch.cuda.current_device()
    if out not in ("f32", "mx8", "both"):
        raise ValueError("out must be f32, mx8 or both")
    X8, XE = _bytes(X8), _bytes(XE)
    M, K = _matrix(X8, "X8")
    N = _matrix(Q, "Q")[0]
    if getattr(S, "dtype", None) is torch.int16:
        S = S.view(torch.float16)
    px, ldx = _arg(X8, (M, K), u8, "X8", dev)
    pe, ldxe = _arg(XE, (M, -(-K // 32)), u8, "XE", dev)
    pq, ldq = _wide(Q, N, -(-K * bits // 8), u8, "Q", dev)
    ps, lds = _wide(S, N, -(-K // 64), torch.float16, "S", dev)
    pb, _ = _arg(bias, (N,), f32, "bias", dev)
    pr, ldr = _arg(residual, (M, N), f32, "residual", dev)
    py = ldy = p8 = ldy8 = pye = ldye = 0
    if out != "mx8":
        Y, py, ldy = _out(Y, (M, N), f32, "Y", dev, X8, stream)
    if out != "f32":
        Y8, p8, ldy8 = _out(_bytes(Y8), (M, N), u8, "Y8", dev, X8, stream)
        YE, pye, ldye = _out(_bytes(YE), (M, -(-N // 32)), u8, "YE", dev, X8, stream)
    _check(getattr(load(), name)(_activation(act), M, N, K, px, ldx, pe, ldxe, pq, ldq, ps, lds,
                                 pb, pr, ldr, py, ldy, p8, ldy8, pye, ldye, _stream(stream, dev)), name)
    return Y if out == "f32" else (Y8, YE) if out == "mx8" else (Y, Y8, YE)


def linear_q2_mx8(X8, XE, Q, S, bias=None, act="none", residual=None, Y=None, Y8=None, YE=None,
                  out="f32", stream=None):
    """Y = act(X.W^T + bias) + residual with X in 8 bits (X8 (M x K), XE (M x
    ceil(K/32)), as rmsnorm_mx8 returns them) and W (N x K) as gemv_q2's codes
    Q (N x >= ceil(K/4)) and scales S (N x >= ceil(K/64)).  out: "f32" returns Y,
    "mx8" the result in 8 bits (Y8, YE) for a following layer, "both" (Y, Y8,
    YE).  Y may be the residual itself."""
    return _packed_linear("linear_q2_mx8", 2, X8, XE, Q, S, bias, act, residual, Y, Y8, YE, out,
                          stream)


def linear_q4_mx8(X8, XE, Q, S, bias=None, act="none", residual=None, Y=None, Y8=None, YE=None,
                  out="f32", stream=None):
    """As linear_q2_mx8 for gemv_q4's codes, Q (N x >= ceil(K/2))."""
    return _packed_linear("linear_q4_mx8", 4, X8, XE, Q, S, bias, act, residual, Y, Y8, YE, out,
                          stream)
