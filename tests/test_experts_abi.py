"""Refusals of the layers with experts and of the norms around a block, through
the C ABI and the binding, on the CPU: arguments are checked before any HIP
call, with made-up addresses that are never dereferenced.  Calls that pass
every check stop at the device check and are made only without a GPU."""
import math

import pytest

from gemv_gemm_f32_amd import binding as bd
from test_abi import _gpu_present, passes_checks

lib = bd.load()
BAD, ALIAS, OK = bd.GG_ERR_INVALID_ARG, bd.GG_ERR_ALIAS, bd.GG_OK
BIG = (1 << 31) - 1

# addresses 256 MiB apart
A = [0x10000000 * i for i in range(1, 16)]
X, W, B, R, Z, Y, DX, DW, DB, WS, E, Q, S, P, O = A


def groups(T=6, k=2, E=8, ids=X, ldi=2, off=O, rows=R, pos=P, ldp=2):
    return lib.expert_groups(T, k, E, ids, ldi, off, rows, pos, ldp, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=-1), dict(E=-1), dict(E=1025), dict(T=1 << 31), dict(T=1 << 16, k=1 << 15, ldi=1 << 15, ldp=1 << 15),
    dict(ids=None), dict(off=None), dict(rows=None), dict(pos=None), dict(ids=X + 2), dict(off=O + 1),
    dict(rows=R + 2), dict(pos=P + 3), dict(ldi=1), dict(ldp=1), dict(ids=(1 << 64) - 16)])
def test_groups_refuses(kw):
    assert groups(**kw) == BAD


def test_groups_alias_and_passes():
    assert groups(off=X) == ALIAS and groups(rows=P) == ALIAS and groups(pos=X) == ALIAS
    assert groups(off=R + 44) == ALIAS                  # the last of 12 rows
    passes_checks(groups)
    passes_checks(lambda: groups(off=R + 48))
    passes_checks(lambda: groups(T=0, ids=None, rows=None, pos=None))
    passes_checks(lambda: groups(E=0))
    passes_checks(lambda: groups(E=1024))


def combine(T=6, k=2, M=12, K=20, y=Y, ldy=20, pos=P, ldp=2, w=W, ldw=2, r=None, ldr=0, out=O, ldo=20):
    return lib.expert_combine(T, k, M, K, y, ldy, pos, ldp, w, ldw, r, ldr, out, ldo, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=-1), dict(M=-1), dict(K=-1), dict(K=1 << 31), dict(y=None), dict(pos=None), dict(out=None),
    dict(ldy=19), dict(ldp=1), dict(ldw=1), dict(ldo=19), dict(r=R, ldr=19), dict(y=Y + 2), dict(pos=P + 2),
    dict(w=W + 1), dict(out=O + 2), dict(out=(1 << 64) - 64)])
def test_combine_refuses(kw):
    assert combine(**kw) == BAD


def test_combine_alias_and_passes():
    assert combine(out=Y) == ALIAS and combine(out=P) == ALIAS and combine(out=W) == ALIAS
    assert combine(r=O, ldr=21) == ALIAS and combine(r=O + 4, ldr=20) == ALIAS
    assert combine(T=0, y=None) == OK and combine(K=0, y=None) == OK
    passes_checks(lambda: combine(r=O, ldr=20))
    passes_checks(lambda: combine(w=None, ldw=-3, ldr=-3))
    passes_checks(lambda: combine(M=0, y=None))
    passes_checks(lambda: combine(k=0, pos=None, w=None))


def cbwd(T=6, k=2, M=12, K=20, do=X, lddo=20, y=Y, ldy=20, pos=P, ldp=2, w=W, ldw=2, dy=DX, lddy=20, dw=DW, lddw=2):
    return lib.expert_combine_bwd(T, k, M, K, do, lddo, y, ldy, pos, ldp, w, ldw, dy, lddy, dw, lddw, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=1 << 31), dict(M=-1), dict(K=-1), dict(do=None), dict(y=None), dict(pos=None), dict(lddo=19),
    dict(ldy=19), dict(ldp=1), dict(ldw=1), dict(lddy=19), dict(lddw=1), dict(dy=DX + 2), dict(dw=DW + 2)])
def test_combine_bwd_refuses(kw):
    assert cbwd(**kw) == BAD


def test_combine_bwd_alias_and_passes():
    assert cbwd(dy=X) == ALIAS and cbwd(dy=Y) == ALIAS and cbwd(dw=W) == ALIAS and cbwd(dw=DX) == ALIAS
    assert cbwd(dy=None, dw=None, do=None) == OK and cbwd(T=0, do=None) == OK and cbwd(k=0, do=None) == OK
    passes_checks(lambda: cbwd(dw=None, y=None))
    passes_checks(lambda: cbwd(dy=None))
    passes_checks(lambda: cbwd(M=0, y=None, dy=None))
    passes_checks(lambda: cbwd(K=0, do=None, y=None))


def grouped(tw=0, act=0, M=12, N=6, K=5, n=4, T=7, x=X, ldx=5, rows=R, off=O, w=W, ldw=6, sw=30, b=None, ldb=6, z=None,
            ldz=6, y=Y, ldy=6):
    return lib.linear_f32_grouped(tw, act, M, N, K, n, T, x, ldx, rows, off, w, ldw, sw, b, ldb, z, ldz, y, ldy, None)


@pytest.mark.parametrize("kw", [
    dict(tw=2), dict(act=5), dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(n=-1), dict(n=1025), dict(T=-1), dict(T=0),
    dict(T=1 << 31), dict(x=None), dict(rows=R + 2), dict(off=None), dict(off=O + 2), dict(w=None), dict(y=None),
    dict(x=X + 2), dict(ldx=4), dict(ldw=5), dict(tw=1, ldw=4), dict(sw=-1), dict(b=B, ldb=5), dict(z=Z, ldz=5),
    dict(ldy=5), dict(ldx=(1 << 22) + 1), dict(ldw=(1 << 22) + 1), dict(T=129, ldx=1 << 22),
    dict(T=1 << 20, ldx=513), dict(M=BIG, N=1100), dict(M=BIG, N=BIG, ldy=BIG), dict(sw=1 << 62),
    dict(x=(1 << 64) - 16)])
def test_grouped_refuses(kw):
    assert grouped(**kw) == BAD


def test_grouped_alias_and_passes():
    assert grouped(y=X) == ALIAS and grouped(y=R) == ALIAS and grouped(y=O) == ALIAS and grouped(y=B, b=B) == ALIAS
    assert grouped(y=W + 4 * 119) == ALIAS               # the last weight of the last expert
    assert grouped(z=Y) == ALIAS and grouped(z=X) == ALIAS
    assert grouped(M=0, x=None) == OK and grouped(N=0, x=None) == OK and grouped(n=0, x=None) == OK
    passes_checks(lambda: grouped(y=W + 4 * 120))
    passes_checks(lambda: grouped(rows=None, T=-5))
    passes_checks(lambda: grouped(sw=0))                 # experts may share their weights
    passes_checks(lambda: grouped(n=1, sw=-7))           # the stride of one expert does not matter
    passes_checks(lambda: grouped(K=0, x=None, w=None, b=B))
    passes_checks(lambda: grouped(T=128, x=1 << 40, ldx=1 << 22, z=Z, act=3))
    passes_checks(lambda: grouped(M=BIG, N=1, x=1 << 40, ldx=8, rows=None, K=1, y=1 << 45))


def gbwd(tw=0, act=2, acc=0, M=12, N=6, K=5, n=4, T=7, dy=Y, lddy=6, z=Z, ldz=6, x=X, ldx=5, rows=R, off=O, w=W, ldw=6,
         sw=30, dx=DX, lddx=5, dw=DW, lddw=6, sdw=30, db=DB, lddb=6, ws=WS, wsb=1 << 20):
    return lib.linear_f32_grouped_bwd(tw, act, acc, M, N, K, n, T, dy, lddy, z, ldz, x, ldx, rows, off, w, ldw, sw, dx,
                                      lddx, dw, lddw, sdw, db, lddb, ws, wsb, None)


NEED = 4 * (12 * 8 + 4 * 6)          # dZ at a stride of 8, and up to 4 tiles' sums


@pytest.mark.parametrize("kw", [
    dict(tw=2), dict(act=-1), dict(acc=2), dict(M=-1), dict(n=1025), dict(T=0), dict(dy=None), dict(z=None), dict(x=None),
    dict(off=None), dict(w=None), dict(lddy=5), dict(ldz=5), dict(ldx=4), dict(ldw=5), dict(lddx=4), dict(lddw=5),
    dict(sdw=28), dict(sdw=0), dict(sw=-1), dict(lddb=5), dict(ws=None), dict(ws=WS + 4), dict(wsb=NEED - 1), dict(wsb=-1),
    dict(ldx=(1 << 22) + 1), dict(lddy=(1 << 22) + 1), dict(T=1 << 29), dict(db=DB + 2)])
def test_grouped_bwd_refuses(kw):
    assert gbwd(**kw) == BAD


def test_grouped_bwd_alias_and_passes():
    assert gbwd(dx=Y) == ALIAS and gbwd(dw=W) == ALIAS and gbwd(dw=DX) == ALIAS and gbwd(db=DX) == ALIAS
    assert gbwd(ws=Z) == ALIAS and gbwd(dx=O) == ALIAS and gbwd(db=R) == ALIAS and gbwd(ws=DB) == ALIAS
    assert gbwd(dx=None, dw=None, db=None, dy=None) == OK and gbwd(n=0, dy=None) == OK
    passes_checks(lambda: gbwd(wsb=NEED, sdw=29 + 1))
    passes_checks(lambda: gbwd(dx=None, w=None))
    passes_checks(lambda: gbwd(dw=None, x=None, rows=None))
    passes_checks(lambda: gbwd(act=0, z=None, wsb=4 * 4 * 6))
    passes_checks(lambda: gbwd(M=0, dy=None, z=None, x=None, rows=None, w=None, ws=None, wsb=0))
    passes_checks(lambda: gbwd(n=1, sdw=-1, sw=-1))


def test_grouped_bwd_workspace_size():
    f = lib.linear_f32_grouped_bwd_ws_size
    assert f(2, 12, 6, 4) == NEED and f(0, 12, 6, 4) == 4 * 4 * 6
    assert f(0, 3, 6, 4) == 4 * 3 * 6                    # no more tiles than rows
    assert f(0, 12800, 6, 1) == 4 * 100 * 6
    assert f(1, 0, 6, 4) == 0 and f(1, 6, 0, 4) == 0 and f(1, 6, 6, 0) == 0
    for bad in ((5, 8, 6, 1), (0, -1, 6, 1), (0, 8, 1 << 31, 1), (0, 8, 6, 1025), (0, 8, 6, -1), (1, BIG, BIG, 1)):
        assert f(*bad) == BAD


def packed(bits, act=0, M=12, N=64, K=100, n=4, T=7, x=X, ldx=100, xe=E, ldxe=4, rows=R, off=O, q=Q, ldq=50, sq=3200, s=S,
           lds=2, ss=128, b=None, ldb=64, y=Y, ldy=64, y8=None, ldy8=0, ye=None, ldye=0):
    f = lib.linear_q2_mx8_grouped if bits == 2 else lib.linear_q4_mx8_grouped
    return f(act, M, N, K, n, T, x, ldx, xe, ldxe, rows, off, q, ldq, sq, s, lds, ss, b, ldb, y, ldy, y8, ldy8, ye, ldye,
             None)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("kw", [
    dict(act=5), dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(n=-1), dict(n=1025), dict(T=0), dict(T=-1), dict(x=None),
    dict(xe=None), dict(off=None), dict(q=None), dict(s=None), dict(s=S + 1), dict(rows=R + 2), dict(ldx=99), dict(ldxe=3),
    dict(lds=1), dict(sq=-1), dict(ss=-1), dict(b=B + 2), dict(b=B, ldb=63), dict(ldy=63), dict(y=None), dict(y8=P, ldy8=64),
    dict(ye=P, ldye=2), dict(y8=P, ldy8=63, ye=WS, ldye=2), dict(y8=P, ldy8=64, ye=WS, ldye=1), dict(M=BIG, N=4000, ldy=4000)])
def test_packed_refuses(bits, kw):
    assert packed(bits, **kw) == BAD


@pytest.mark.parametrize("bits", [2, 4])
def test_packed_alias_and_passes(bits):
    for at in (X, E, R, O, Q, S):
        assert packed(bits, y=at) == ALIAS
    assert packed(bits, y=B, b=B) == ALIAS and packed(bits, y8=Y, ldy8=64, ye=WS, ldye=2) == ALIAS
    assert packed(bits, M=0, x=None) == OK and packed(bits, n=0, x=None) == OK
    passes_checks(lambda: packed(bits, rows=None, T=-3))
    passes_checks(lambda: packed(bits, y=None, y8=P + 1, ldy8=64, ye=WS + 3, ldye=2, b=B))
    passes_checks(lambda: packed(bits, K=0, x=None, xe=None, q=None, s=None))
    passes_checks(lambda: packed(bits, sq=0, ss=0))
    assert packed(4, ldq=49) == BAD and packed(2, ldq=24) == BAD


def norm(M=8, K=96, u=X, ldu=96, x=R, ldx=96, gu=B, gate=None, ldg=0, alpha=1.0, gs=W, eps=1e-5, s=S, lds=96, y=Y, ldy=96,
         ru=None, rs=None):
    return lib.block_norm_f32(M, K, u, ldu, x, ldx, gu, gate, ldg, alpha, gs, eps, s, lds, y, ldy, ru, rs, None)


def norm8(M=8, K=96, u=X, ldu=96, x=R, ldx=96, gu=B, gate=None, ldg=0, alpha=1.0, gs=W, eps=1e-5, s=S, lds=96, q=Q, ldq=96,
          e=E, lde=3):
    return lib.block_norm_mx8(M, K, u, ldu, x, ldx, gu, gate, ldg, alpha, gs, eps, s, lds, q, ldq, e, lde, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(K=1 << 31), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf), dict(alpha=math.nan),
    dict(alpha=math.inf), dict(u=None), dict(x=None), dict(s=None), dict(u=X + 2), dict(ldu=95), dict(ldx=95), dict(lds=95),
    dict(gu=B + 2), dict(gs=W + 1), dict(gate=Z + 2), dict(gate=Z, ldg=95), dict(gate=Z, ldg=-1)])
def test_norm_refuses(kw):
    assert norm(**kw) == BAD and norm8(**kw) == BAD


def test_norm_alias_and_passes():
    assert norm(y=None) == BAD and norm(ldy=95) == BAD and norm(ru=P + 2) == BAD
    assert norm8(q=None) == BAD and norm8(ldq=95) == BAD and norm8(lde=2) == BAD
    assert norm(s=X) == ALIAS and norm(y=X) == ALIAS and norm(y=R) == ALIAS and norm(s=Y) == ALIAS
    assert norm(s=R, lds=97) == ALIAS and norm(s=R + 4) == ALIAS and norm(gate=S) == ALIAS and norm(ru=P, rs=P) == ALIAS
    assert norm(u=R, x=R, s=R) == ALIAS                  # X may be replaced, U may not
    assert norm8(q=X) == ALIAS and norm8(e=Q) == ALIAS
    assert norm(M=0, u=None) == OK and norm8(K=0, u=None) == OK
    passes_checks(lambda: norm(s=R))
    passes_checks(lambda: norm(gu=None, gs=None, gate=Z, ldg=96, ru=P, rs=E, eps=0.0, alpha=0.0))
    passes_checks(lambda: norm8(gate=Z, q=Q + 3, e=E + 1, ldq=99))
    passes_checks(lambda: norm(ldg=-5))                  # an absent gate's


def nbwd(acc=0, M=8, K=96, dy=Y, lddy=96, u=X, ldu=96, s=S, lds=96, gu=B, gate=None, ldg=0, alpha=1.0, gs=W, ru=P, rs=E,
         ds=None, ldds=0, du=DW, lddu=96, dx=DX, lddx=96, dgu=DB, dgs=DB + 4096, dgt=None, lddg=0, ws=WS, wsb=8 * 96 * 8):
    return lib.block_norm_f32_bwd(acc, M, K, dy, lddy, u, ldu, s, lds, gu, gate, ldg, alpha, gs, ru, rs, ds, ldds, du, lddu,
                                  dx, lddx, dgu, dgs, dgt, lddg, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(acc=2), dict(M=-1), dict(K=-1), dict(alpha=math.inf), dict(dy=None), dict(u=None), dict(s=None), dict(ru=None),
    dict(rs=None), dict(ru=P + 1), dict(lddy=95), dict(ldu=95), dict(lds=95), dict(lddu=95), dict(lddx=95),
    dict(ds=R, ldds=95), dict(dgt=O), dict(gate=Z, ldg=96, dgt=O, lddg=95), dict(ws=None), dict(ws=WS + 8),
    dict(wsb=8 * 96 * 8 - 1), dict(dgu=DB + 2)])
def test_norm_bwd_refuses(kw):
    assert nbwd(**kw) == BAD


def test_norm_bwd_alias_and_passes():
    assert nbwd(dx=Y) == ALIAS and nbwd(du=X) == ALIAS and nbwd(du=DX) == ALIAS and nbwd(dgs=DB) == ALIAS
    assert nbwd(ds=DX, ldds=97) == ALIAS and nbwd(ds=DW, ldds=96) == ALIAS and nbwd(gate=Z, dgt=Z) == ALIAS
    assert nbwd(du=None, dx=None, dgu=None, dgs=None) == OK and nbwd(K=0) == OK
    passes_checks(lambda: nbwd(ds=DX, ldds=96))
    passes_checks(lambda: nbwd(dgu=None, dgs=None, ws=None, wsb=0))
    passes_checks(lambda: nbwd(dgu=None, dgs=None, ws=None, wsb=0, gate=Z, ldg=96, dgt=O, lddg=96))
    passes_checks(lambda: nbwd(gate=Z, dgt=O))
    passes_checks(lambda: nbwd(M=0, dy=None, u=None, s=None, ru=None, rs=None, ws=None, wsb=0))
    f = lib.block_norm_f32_bwd_ws_size
    assert f(8, 96) == 8 * 96 * 8 and f(0, 96) == 0 and f(1 << 20, 96) == 512 * 96 * 8
    assert f(-1, 96) == BAD and f(8, 1 << 31) == BAD


NAMES = ["expert_groups", "expert_combine", "expert_combine_bwd", "linear_f32_grouped", "linear_f32_grouped_bwd",
         "linear_q2_mx8_grouped", "linear_q4_mx8_grouped", "block_norm_f32", "block_norm_mx8", "block_norm_f32_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_package_names(name):
    import gemv_gemm_f32_amd
    assert getattr(gemv_gemm_f32_amd, name) is getattr(bd, name)


# ---------------------------------------------------------------- binding --

@pytest.fixture
def t(monkeypatch):
    """Tensors in host memory pass for ones on the current device."""
    if _gpu_present():
        pytest.skip("a valid call on host memory would launch on the GPU")
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # get_device() of a CPU tensor
    monkeypatch.setattr(bd, "_stream", lambda stream, dev=None: 0)
    return torch


def _good(t):
    f = lambda *s: t.ones(*s)                                # noqa: E731
    i = lambda *s: t.zeros(*s, dtype=t.int32)                # noqa: E731
    u = lambda *s: t.zeros(*s, dtype=t.uint8)                # noqa: E731
    h = lambda *s: t.ones(*s, dtype=t.float16)               # noqa: E731
    return {
        bd.expert_groups: dict(ids=i(4, 2), E=3, offsets=i(4), rows=i(8), pos=i(4, 2)),
        bd.expert_combine: dict(Y=f(8, 6), pos=i(4, 2), weights=f(4, 2), residual=f(4, 6), out=f(4, 6)),
        bd.expert_combine_bwd: dict(dO=f(4, 6), pos=i(4, 2), Y=f(8, 6), weights=f(4, 2), dY=f(8, 6), dw=f(4, 2)),
        bd.linear_f32_grouped: dict(X=f(4, 5), W=f(3, 5, 6), offsets=i(4), rows=i(8), bias=f(3, 6), Z=f(8, 6), Y=f(8, 6)),
        bd.linear_f32_grouped_bwd: dict(dY=f(8, 6), X=f(4, 5), W=f(3, 5, 6), offsets=i(4), rows=i(8), Z=f(8, 6), act="silu",
                                        dX=f(8, 5), dW=f(3, 5, 6), db=f(3, 6), workspace=u(1 << 14)),
        bd.linear_q4_mx8_grouped: dict(X8=u(4, 8), XE=u(4, 1), Q=u(3, 6, 4), S=h(3, 6, 1), offsets=i(4), rows=i(8),
                                       bias=f(3, 6), Y=f(8, 6), Y8=u(8, 6), YE=u(8, 1), out="both"),
        bd.linear_q2_mx8_grouped: dict(X8=u(4, 8), XE=u(4, 1), Q=u(3, 6, 2), S=h(3, 6, 1), offsets=i(4), rows=i(8),
                                       bias=f(3, 6), Y=f(8, 6), Y8=u(8, 6), YE=u(8, 1), out="both"),
        bd.block_norm_f32: dict(U=f(4, 8), X=f(4, 8), gamma_u=f(8), gamma_s=f(8), gate=f(4, 8), S=f(4, 8), Y=f(4, 8),
                                rstd_u=f(4), rstd_s=f(4)),
        bd.block_norm_mx8: dict(U=f(4, 8), X=f(4, 8), gamma_u=f(8), gamma_s=f(8), gate=f(8), S=f(4, 8), Q=u(4, 8), E=u(4, 1)),
        bd.block_norm_f32_bwd: dict(dY=f(4, 8), U=f(4, 8), S=f(4, 8), gamma_u=f(8), gamma_s=f(8), rstd_u=f(4), rstd_s=f(4),
                                    gate=f(8), dS=f(4, 8), dU=f(4, 8), dX=f(4, 8), dgamma_u=f(8), dgamma_s=f(8), dgate=f(8),
                                    workspace=u(1 << 14)),
    }


def test_good_calls_reach_the_device_check(t):
    for fn, kw in _good(t).items():
        with pytest.raises(bd.GGError) as e:
            fn(**kw)
        assert e.value.status == bd.GG_ERR_NO_DEVICE, (fn, e.value)


@pytest.mark.parametrize("bad", ([[1.0] * 8] * 4, 3.0, "X", object()), ids=["list", "float", "str", "object"])
def test_what_is_no_tensor_is_a_type_error(t, bad):
    for fn, kw in _good(t).items():
        for name in kw:
            if name in ("act", "out", "E") and not t.is_tensor(kw[name]):
                continue
            with pytest.raises(TypeError):
                fn(**dict(kw, **{name: bad}))


@pytest.mark.parametrize("change", ["type", "shape", "stride", "dimensions"])
def test_tensors_of_another_form_are_refused(t, change):
    for fn, kw in _good(t).items():
        for name, v in kw.items():
            if not t.is_tensor(v) or name == "workspace":
                continue
            if change == "type":
                w = v.to(t.float64)
            elif change == "shape":
                # one more in the last dimension: codes and scales may have spare columns
                if name in ("Q", "S") and v.dim() == 3:
                    continue
                w = t.zeros(*v.shape[:-1], v.shape[-1] + 1, dtype=v.dtype)
            elif change == "stride":
                if v.shape[-1] < 2:
                    continue
                w = t.zeros(*v.shape[:-1], 2 * v.shape[-1], dtype=v.dtype)[..., ::2]
            else:
                w = v[None]
            with pytest.raises((TypeError, ValueError)):
                fn(**dict(kw, **{name: w}))


def test_absent_operands(t):
    """What may not be absent is refused before the library is called."""
    required = {bd.expert_groups: ("ids",), bd.expert_combine: ("Y", "pos"), bd.expert_combine_bwd: ("dO", "pos", "Y"),
                bd.linear_f32_grouped: ("X", "W", "offsets"), bd.linear_f32_grouped_bwd: ("dY", "X", "W", "offsets", "Z"),
                bd.linear_q4_mx8_grouped: ("X8", "XE", "Q", "S", "offsets"), bd.block_norm_f32: ("U", "X"),
                bd.block_norm_mx8: ("U", "X"), bd.block_norm_f32_bwd: ("dY", "U", "S", "rstd_u", "rstd_s")}
    good = _good(t)
    for fn, names in required.items():
        for name in names:
            with pytest.raises((TypeError, ValueError, bd.GGError)) as e:
                fn(**dict(good[fn], **{name: None}))
            assert getattr(e.value, "status", None) != bd.GG_ERR_NO_DEVICE, (fn, name)


def test_gates_and_wanted_gradients(t):
    f = t.ones
    kw = _good(t)[bd.block_norm_f32_bwd]
    with pytest.raises(ValueError):                      # a row that is every row's has to be a vector
        bd.block_norm_f32(f(4, 8), f(4, 8), gate=f(8).expand(4, 8))
    with pytest.raises(ValueError):
        bd.block_norm_f32_bwd(**dict(kw, dgamma_u=None, accumulate=True))
    with pytest.raises(ValueError):
        bd.linear_f32_grouped_bwd(**dict(_good(t)[bd.linear_f32_grouped_bwd], dW=None, accumulate=True))
    with pytest.raises(ValueError):
        bd.linear_f32_grouped(f(4, 5), f(3, 5, 6), t.zeros(4, dtype=t.int32), act="tanh")
    with pytest.raises(ValueError):
        bd.expert_groups(t.zeros(4, 2, dtype=t.int32), 1025)
    with pytest.raises(bd.GGError) as e:                 # experts alone need no Y
        bd.expert_combine_bwd(f(4, 6), t.zeros(4, 2, dtype=t.int32), want=("dY",))
    assert e.value.status == bd.GG_ERR_NO_DEVICE
