"""Refusals of the dense layers and the norm through the C ABI, on the CPU:
arguments are checked before any HIP call, with made-up addresses that are
never dereferenced.  Calls that pass every check stop at the device check and
are made only without a GPU."""
import math

import pytest

from gemv_gemm_f32_amd import binding as bd
from test_abi import passes_checks

lib = bd.load()
BAD, ALIAS, OK = bd.GG_ERR_INVALID_ARG, bd.GG_ERR_ALIAS, bd.GG_OK

# addresses 256 MiB apart
A = [0x10000000 * i for i in range(1, 15)]
X, W, B, R, Z, Y, DX, DW, DB, WS, E, Q, S, P = A


def linear(tw=0, act=0, M=8, N=6, K=5, x=X, ldx=5, w=W, ldw=6, b=None, r=None, ldr=0, z=None,
           ldz=0, y=Y, ldy=6):
    return lib.linear_f32(tw, act, M, N, K, x, ldx, w, ldw, b, r, ldr, z, ldz, y, ldy, None)


@pytest.mark.parametrize("kw", [
    dict(tw=2), dict(tw=-1), dict(act=-1), dict(act=5), dict(M=-1), dict(N=-1), dict(K=-1),
    dict(M=1 << 31), dict(x=None), dict(w=None), dict(y=None), dict(x=X + 2), dict(b=B + 1),
    dict(ldx=4), dict(ldw=5), dict(tw=1, ldw=4), dict(ldy=5), dict(r=R, ldr=5), dict(z=Z, ldz=5),
    dict(ldy=1 << 31), dict(x=(1 << 64) - 16), dict(y=(1 << 64) - 64)])
def test_linear_refuses(kw):
    assert linear(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(y=X), dict(y=W + 4), dict(y=B, b=B), dict(z=Y, ldz=6), dict(z=X, ldz=6),
    dict(z=R, ldz=6, r=R, ldr=6),
    dict(r=Y, ldr=7),                                   # in place needs the same stride
    dict(r=Y + 4, ldr=6),                               # and the same address
    dict(K=6, ldx=6, x=Y, r=Y, ldr=6)])                 # the residual may, the input may not
def test_linear_alias(kw):
    assert linear(**kw) == ALIAS


def test_linear_passes():
    assert linear(M=0, x=None, w=None, y=None) == OK
    assert linear(N=0, x=None, w=None, y=None) == OK
    passes_checks(lambda: linear(r=Y, ldr=6))           # the residual updated in place
    passes_checks(lambda: linear(K=0, x=None, w=None, b=B))
    passes_checks(lambda: linear(b=B, r=R, ldr=6, z=Z, ldz=6, act=4))
    # the leading dimensions of absent operands do not matter
    passes_checks(lambda: linear(ldr=-5, ldz=-7))


def bwd(tw=0, act=2, acc=0, M=8, N=6, K=5, dy=Y, lddy=6, z=Z, ldz=6, x=X, ldx=5, w=W, ldw=6,
        dx=DX, lddx=5, dw=DW, lddw=6, db=DB, ws=WS, wsb=1 << 20):
    return lib.linear_f32_bwd(tw, act, acc, M, N, K, dy, lddy, z, ldz, x, ldx, w, ldw, dx, lddx,
                              dw, lddw, db, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(tw=2), dict(act=7), dict(acc=2), dict(acc=-1), dict(M=-1), dict(dy=None), dict(z=None),
    dict(x=None), dict(w=None), dict(lddy=5), dict(ldz=5), dict(ldx=4), dict(ldw=5), dict(lddx=4),
    dict(lddw=5), dict(tw=1, lddw=4), dict(db=DB + 2), dict(ws=None), dict(ws=WS + 4), dict(wsb=-1),
    dict(wsb=4 * (8 * 8 + 64 * 6) - 1), dict(act=0, z=None, wsb=4 * 64 * 6 - 1)])
def test_linear_bwd_refuses(kw):
    assert bwd(**kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(dx=Y, lddx=6), dict(dw=W), dict(dx=X), dict(dw=DX), dict(db=DX), dict(db=W),
    dict(ws=Z), dict(ws=DX), dict(dx=Z, lddx=6)])
def test_linear_bwd_alias(kw):
    assert bwd(**kw) == ALIAS


def test_linear_bwd_passes():
    assert bwd(dx=None, dw=None, db=None, dy=None) == OK
    assert bwd(M=0, dw=None, db=None, dy=None) == OK     # only an empty dX is asked for
    passes_checks(lambda: bwd(wsb=4 * (8 * 8 + 64 * 6)))
    passes_checks(lambda: bwd(dx=None, w=None))
    passes_checks(lambda: bwd(dw=None, x=None))
    passes_checks(lambda: bwd(act=0, z=None))
    passes_checks(lambda: bwd(M=0, dy=None, z=None, x=None, ws=None, wsb=0))   # zeros to dW, db


def test_linear_bwd_workspace_size():
    f = lib.linear_f32_bwd_ws_size
    assert f(0, 8, 6) == 4 * 64 * 6 and f(2, 8, 6) == 4 * (8 * 8 + 64 * 6)
    assert f(1, 0, 6) == 0 and f(1, 6, 0) == 0
    for bad in ((5, 8, 6), (-1, 8, 6), (0, -1, 6), (0, 8, 1 << 31)):
        assert f(*bad) == BAD
    big = (1 << 31) - 1
    assert f(2, big, big) == BAD                          # past 2^62 bytes
    assert f(2, big, 8) == 4 * (8 * big + 64 * 8)


def norm(M=8, K=96, x=X, ldx=96, r=None, ldr=0, g=B, eps=1e-5, s=None, lds=0, y=Y, ldy=96,
         rstd=None):
    return lib.rmsnorm_f32(M, K, x, ldx, r, ldr, g, eps, s, lds, y, ldy, rstd, None)


def norm8(M=8, K=96, x=X, ldx=96, r=None, ldr=0, g=B, eps=1e-5, s=None, lds=0, q=Q, ldq=96, e=E,
          lde=3):
    return lib.rmsnorm_mx8(M, K, x, ldx, r, ldr, g, eps, s, lds, q, ldq, e, lde, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(K=1 << 31), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf),
    dict(x=None), dict(x=X + 2), dict(ldx=95), dict(r=R, ldr=95), dict(g=B + 2), dict(s=S, lds=95)])
def test_norm_refuses(kw):
    assert norm(**kw) == BAD and norm8(**kw) == BAD


def test_norm_refuses_outputs():
    assert norm(y=None) == BAD and norm(ldy=95) == BAD and norm(rstd=P + 2) == BAD
    assert norm8(q=None) == BAD and norm8(e=None) == BAD
    assert norm8(ldq=95) == BAD and norm8(lde=2) == BAD


def test_norm_alias():
    assert norm(y=X) == ALIAS                                    # only S may be in place
    assert norm(s=X, lds=97) == ALIAS and norm(s=X + 4, lds=96) == ALIAS
    assert norm(s=Y, lds=96) == ALIAS and norm(rstd=Y) == ALIAS and norm(y=B) == ALIAS
    assert norm(s=B, lds=96, g=B) == ALIAS
    assert norm(x=B, g=B, s=B, lds=96) == ALIAS                  # S onto X that is gamma too
    assert norm8(q=X) == ALIAS and norm8(e=Q) == ALIAS


def test_norm_passes():
    assert norm(M=0, x=None, y=None) == OK and norm8(K=0, x=None, q=None, e=None) == OK
    passes_checks(lambda: norm(s=X, lds=96))
    passes_checks(lambda: norm(r=R, ldr=96, s=R, lds=96))
    passes_checks(lambda: norm(g=None, eps=0.0))
    passes_checks(lambda: norm8(r=R, ldr=96, s=X, lds=96))
    passes_checks(lambda: norm8(q=Q + 3, e=E + 1, ldq=99))       # bytes need no alignment


def nbwd(acc=0, M=8, K=96, dy=Y, lddy=96, s=S, lds=96, g=B, rstd=P, ds=None, ldds=0, dx=DX, lddx=96,
         dg=DB, ws=WS, wsb=8 * 96 * 4):
    return lib.rmsnorm_f32_bwd(acc, M, K, dy, lddy, s, lds, g, rstd, ds, ldds, dx, lddx, dg, ws,
                               wsb, None)


@pytest.mark.parametrize("kw", [
    dict(acc=2), dict(M=-1), dict(K=-1), dict(dy=None), dict(s=None), dict(rstd=None),
    dict(rstd=P + 1), dict(lddy=95), dict(lds=95), dict(lddx=95), dict(ds=R, ldds=95),
    dict(ws=None), dict(ws=WS + 8), dict(wsb=8 * 96 * 4 - 1), dict(g=B + 2), dict(dg=DB + 2)])
def test_norm_bwd_refuses(kw):
    assert nbwd(**kw) == BAD


def test_norm_bwd_alias():
    assert nbwd(dx=Y) == ALIAS and nbwd(dx=S) == ALIAS and nbwd(dg=B) == ALIAS
    assert nbwd(ws=DX) == ALIAS and nbwd(dg=DX) == ALIAS
    assert nbwd(ds=DX, ldds=97) == ALIAS
    assert nbwd(ds=Y, ldds=96, dx=Y) == ALIAS                    # dS may be dX, dY may not


def test_norm_bwd_passes():
    assert nbwd(dx=None, dg=None) == OK and nbwd(K=0) == OK
    passes_checks(lambda: nbwd(ds=DX, ldds=96))
    passes_checks(lambda: nbwd(dg=None, ws=None, wsb=0))
    passes_checks(lambda: nbwd(dx=None))
    passes_checks(lambda: nbwd(M=0, dy=None, s=None, rstd=None, ws=None, wsb=0))
    f = lib.rmsnorm_f32_bwd_ws_size
    assert f(8, 96) == 8 * 96 * 4 and f(0, 96) == 0 and f(1 << 20, 96) == 512 * 96 * 4
    assert f(-1, 96) == BAD and f(8, 1 << 31) == BAD


def packed(bits, act=0, M=8, N=64, K=100, x=X, ldx=100, xe=E, ldxe=4, q=Q, ldq=50, s=S, lds=2,
           b=None, r=None, ldr=0, y=Y, ldy=64, y8=None, ldy8=0, ye=None, ldye=0):
    f = lib.linear_q2_mx8 if bits == 2 else lib.linear_q4_mx8
    return f(act, M, N, K, x, ldx, xe, ldxe, q, ldq, s, lds, b, r, ldr, y, ldy, y8, ldy8, ye, ldye,
             None)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("kw", [
    dict(act=5), dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(x=None), dict(xe=None), dict(q=None),
    dict(s=None), dict(s=S + 1), dict(ldx=99), dict(ldxe=3), dict(lds=1), dict(b=B + 2), dict(ldy=63),
    dict(r=R, ldr=63), dict(y=None), dict(y=None, y8=P, ldy8=64), dict(y8=P, ldy8=64),
    dict(ye=P, ldye=2), dict(y8=P, ldy8=63, ye=WS, ldye=2), dict(y8=P, ldy8=64, ye=WS, ldye=1)])
def test_packed_refuses(bits, kw):
    assert packed(bits, **kw) == BAD


def test_packed_code_rows():
    assert packed(4, ldq=49) == BAD and packed(2, ldq=24) == BAD
    passes_checks(lambda: packed(2, ldq=25))


@pytest.mark.parametrize("bits", [2, 4])
def test_packed_alias(bits):
    assert packed(bits, y=X) == ALIAS and packed(bits, y=Q) == ALIAS and packed(bits, y=S) == ALIAS
    assert packed(bits, y=E) == ALIAS and packed(bits, y=B, b=B) == ALIAS
    assert packed(bits, r=Y, ldr=65) == ALIAS
    assert packed(bits, y8=Y, ldy8=64, ye=WS, ldye=2) == ALIAS
    assert packed(bits, y8=X, ldy8=64, ye=WS, ldye=2) == ALIAS
    assert packed(bits, y8=P, ldy8=64, ye=P, ldye=2) == ALIAS
    # 8 bits onto the residual's place
    assert packed(bits, y=None, r=P, ldr=64, y8=P, ldy8=64, ye=WS, ldye=2) == ALIAS


@pytest.mark.parametrize("bits", [2, 4])
def test_packed_passes(bits):
    assert packed(bits, M=0, x=None) == OK and packed(bits, N=0, q=None) == OK
    passes_checks(lambda: packed(bits, r=Y, ldr=64, b=B))
    passes_checks(lambda: packed(bits, y=None, y8=P, ldy8=64, ye=WS, ldye=2))
    passes_checks(lambda: packed(bits, K=0, x=None, xe=None, q=None, s=None))
    passes_checks(lambda: packed(bits, x=X + 1, q=Q + 3, xe=E + 1, ldr=-1))


@pytest.mark.parametrize("name", ["linear_f32", "linear_f32_bwd", "rmsnorm_f32", "rmsnorm_mx8",
                                  "rmsnorm_f32_bwd", "linear_q2_mx8", "linear_q4_mx8"])
def test_package_names(name):
    import gemv_gemm_f32_amd
    assert getattr(gemv_gemm_f32_amd, name) is getattr(bd, name)
