"""Sizes near 2^31 and grids near 2^32 threads.  On the CPU the launchers run
against a recorder in place of the HIP runtime, which prints each launch: grids
have to be ones that a launch takes, and the launches together have to cover
the output once.  On the GPU the largest of them that fit run in full."""
import os
import subprocess

import pytest

from gemv_gemm_f32_amd import binding as bd
from gemv_gemm_f32_amd.build import HIPCC
from gpu_util import host, torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemv_gemm_f32_amd", "csrc")
MOST = (1 << 31) - 1
UNITS = ("gemm_f32", "linear_f32", "linear_bwd", "linear_mx8")


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    """record(call, sizes ...): the launches that it makes, each as (kernel,
    grid x, grid y, threads, arguments)."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    d = tmp_path_factory.mktemp("recorder")
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-I", CSRC, "-w"]
    objs = []
    for src in [os.path.join(CSRC, u + ".hip") for u in UNITS] + [os.path.join(ROOT, "tests", "launch_recorder.cpp")]:
        objs.append(str(d / (os.path.basename(src) + ".o")))
        subprocess.run([HIPCC, "-x", "hip"] + flags + ["-c", src, "-o", objs[-1]], check=True,
                       capture_output=True, text=True, timeout=300)
    exe = str(d / "recorder")
    subprocess.run(["g++", "-o", exe] + objs + ["-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files"],
                   check=True, capture_output=True, text=True, timeout=120)

    def run(*args):
        r = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        lines = r.stdout.split("\n")[:-1]
        assert lines.pop() == "status 0", r.stdout
        out = []
        for ln in lines:
            w = ln.split()
            if not w[0].lstrip("-").isdigit():
                gx, gy, threads = (int(v) for v in w[1:4])
                assert 1 <= gx and gx * threads < 1 << 32 and 1 <= gy <= 65535, ln
                w = (w[0], gx, gy, threads, [int(v) for v in w[4:]])
            else:
                w = [int(v) for v in w]
            out.append(w)
        return out
    return run


@pytest.mark.parametrize("act", [0, 4])
@pytest.mark.parametrize("M", [1, 16, 1024, 1025, 2114445424, 2114445425, 2114445438, MOST - 1023, MOST - 1022,
                               MOST - 15, MOST])
def test_chunks_of_the_element_pass(record, M, act):
    """The gradients' element pass: its chunks of rows meet, end at M and are
    as many as the grid has."""
    if act == 0:
        dz, cs = record("bwd_bias", M, 1, 0)
        assert "dz_kernel" in dz[0] and "column_sum" in cs[0]
    else:
        dz, cs = record("bwd_bias", M, 3, act)
    chunks = dz[2]
    assert dz[4][0] == M and cs[4][0] == chunks <= 64
    ends = [record("rows_of_chunk", M, i)[0] for i in range(chunks)]
    assert ends[0][0] == 0 and ends[-1][1] == M
    assert all(a < b for a, b in ends) and all(p[1] == q[0] for p, q in zip(ends, ends[1:]))


def _rectangles(launches, M, N):
    """The rectangles (row, column, rows, columns) that launches write, which
    have to cover an M x N output with leading dimension N once."""
    rects = []
    for name, gx, gy, threads, a in launches:
        m, n, off, ld = a[0], a[1], a[3], a[4]
        assert ld == N and m > 0 and n > 0, (name, a)
        rects.append((off // N, off % N, m, n))
        assert rects[-1][0] + m <= M and rects[-1][1] + n <= N
    assert sum(m * n for _, _, m, n in rects) == M * N
    for i, (r, c, m, n) in enumerate(rects):
        for r2, c2, m2, n2 in rects[:i]:
            assert r >= r2 + m2 or r2 >= r + m or c >= c2 + n2 or c2 >= c + n
    return rects


LARGE = [(MOST, 1, 1), (MOST, 1, 200), (1, MOST, 1), (MOST - 127, 1, 1), (MOST - 126, 1, 4), (MOST, 30, 5),
         (9, MOST, 1), (9, MOST, 64), (1 << 30, 65, 8), (190000, 200000, 128), (262145, 262143, 100),
         (1 << 29, 64, 4), ((1 << 29) + 1, 64, 4), (64, 1 << 30, 7)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_products_of_large_outputs(record, M, N, K, ta, tb):
    launches = record("gemm", M, N, K, ta, tb)
    for (r, c, m, n), (name, gx, _, _, a) in zip(_rectangles(launches, M, N), launches):
        assert "gemm_f32_" in name and a[2] == K
        assert m <= MOST - 127 and n <= MOST - 127              # rows of the last tile stay below 2^31
        assert a[5] == (r if ta else r * K) and a[6] == (c * K if tb else c)
        assert r % 128 == 0 and c % 128 == 0 and a[7] * a[8] == gx
        assert a[7] >= -(-m // 128) and a[8] >= -(-n // 64)


@pytest.mark.parametrize("M,tw", [(1, 0), (3, 0), (4, 0), (1, 1), (2, 1), (8, 1)])
@pytest.mark.parametrize("N", [1, 2047, 2048, 1 << 25, (1 << 25) + 1, (1 << 26) + 1, (1 << 27) + 1, MOST])
def test_few_rows_over_many_columns(record, M, N, tw):
    launches = record("linear", M, N, 3, tw)
    assert len(launches) == -(-N // (1 << 25))
    for (r, c, m, n), (name, _, _, _, a) in zip(_rectangles(launches, M, N), launches):
        assert "linear_few" in name and m == M and a[5] == 0 and a[6] == (c * 3 if tw else c)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("both", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, MOST, 5), (16, MOST, 200), (17, MOST, 100), (1, 1 << 28, 1), (1, (1 << 28) + 1, 1),
                                   (MOST, 1, 1), (MOST, 130, 300), ((1 << 30) + 1, 40, 64), (1 << 20, 1 << 17, 1536),
                                   (500, 12288, 1536), (64, 4096, 4096), (1, 1536, 12288)])
def test_packed_layers_of_large_outputs(record, M, N, K, both, bits):
    launches = record("packed", bits, M, N, K, both)
    if M * N < 1 << 28:
        assert len(launches) == 1
    for (r, c, m, n), (name, _, _, _, a) in zip(_rectangles(launches, M, N), launches):
        assert "packed_" in name and a[2] == K and c % 32 == 0
        assert a[5:9] == [r * K, r * -(-K // 32), c * -(-K * bits // 8), c * -(-K // 64)]
        assert a[9:13] == ([r * N + c, r * -(-N // 32) + c // 32, c, r * N + c] if both else [-1] * 4)


@pytest.mark.parametrize("K", [1, 31, 32, 33, (1 << 30) + 5, MOST - 32, MOST - 31, MOST - 30, MOST - 1, MOST])
def test_walk_along_k(record, K):
    """The staged kernels' slabs of 32 columns: as many as K has, the last one's
    places clamped to the last column.  (On the GPU one tile walks the longest
    of them for over a minute, so that it is not run there.)"""
    (slabs,), places = record("k_walk", K)
    assert slabs == -(-K // 32)
    assert places == [min((slabs - 1) * 32 + k, K - 1) for k in range(32)]


@pytest.mark.parametrize("M,N,K", [(346, 768, 768), (2048, 2048, 2048), (1 << 24, 64, 16)])
def test_ordinary_products_take_one_launch(record, M, N, K):
    assert len(record("gemm", M, N, K, 0, 0)) == 1
    assert len(record("linear", M, N, K, 1)) == 1


@pytest.mark.parametrize("M,N,K,tw", [(MOST, 1, 1, 0), (MOST, 2, 9, 1), (9, MOST, 3, 1), (9, MOST, 3, 0),
                                      (200000, 190000, 128, 0)])
def test_layers_of_large_outputs(record, M, N, K, tw):
    launches = record("linear", M, N, K, tw)
    for (r, c, m, n), (name, _, _, _, a) in zip(_rectangles(launches, M, N), launches):
        assert m <= MOST - 127 and n <= MOST - 127 and a[5] == r * K and a[6] == (c * K if tw else c)


@pytest.mark.gpu
def test_bias_gradient_of_most_rows():
    """2^31 - 1 rows of one column, zeros but for ones at the border of the last
    chunks and in the last rows: small integers, so the sum is exact."""
    t = torch()
    dY = t.zeros((MOST, 1), device="cuda")
    for r in (0, 63 * (1 << 25) - 1, 63 * (1 << 25), MOST - 17, MOST - 16, MOST - 1):
        dY[r] = 1
    _, _, db = bd.linear_f32_bwd(dY, None, t.ones((1, 1), device="cuda"), want=("db",))
    got = host(db)[0]
    del dY
    t.cuda.empty_cache()
    assert got == 6


def _equal(Y, f, step=1 << 28):
    """Whether the long vector Y is f(first, end) piece by piece."""
    return all(bool((Y[i:i + step] == f(i, min(i + step, Y.numel()))).all()) for i in range(0, Y.numel(), step))


def _pattern(i, j):
    t = torch()
    return (t.arange(i, j, device="cuda") % 251).float()


@pytest.mark.gpu
def test_layer_of_most_rows():
    """2^31 - 1 rows through a 1 x 1 layer with bias and a residual updated in
    place: small integers, exact."""
    t = torch()
    X = t.empty((MOST, 1), device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        X[i:j, 0] = _pattern(i, j)
    Y = t.full((MOST, 1), 3.0, device="cuda")
    bd.linear_f32(X, t.full((1, 1), 2.0, device="cuda"), bias=t.ones(1, device="cuda"), residual=Y, Y=Y)
    ok = _equal(Y[:, 0], lambda i, j: 2 * _pattern(i, j) + 4)
    del X, Y
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
@pytest.mark.parametrize("tw", [0, 1])
def test_layer_of_most_columns(tw):
    """9 rows over 2^31 - 1 columns: the tile kernels."""
    t = torch()
    W = t.empty(MOST, device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        W[i:j] = _pattern(i, j)
    X = t.arange(1, 10, device="cuda").float()[:, None].contiguous()
    Y = bd.linear_f32(X, W[:, None] if tw else W[None], trans_w=bool(tw))
    ok = [_equal(Y[m], lambda i, j: _pattern(i, j) * (m + 1)) for m in range(9)]
    del W, Y
    t.cuda.empty_cache()
    assert all(ok)


@pytest.mark.gpu
@pytest.mark.parametrize("tw", [0, 1])
def test_two_rows_over_most_columns(tw):
    """Bias, pre-activations and a residual updated in place past the columns
    of one launch."""
    t = torch()
    W = t.empty(MOST, device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        W[i:j] = _pattern(i, j)
    X = t.tensor([[1.0], [2.0]], device="cuda")
    Y = t.full((2, MOST), -5.0, device="cuda")
    Z = t.empty((2, MOST), device="cuda")
    bd.linear_f32(X, W[:, None] if tw else W[None], bias=W, residual=Y, Z=Z, Y=Y, act="relu", trans_w=bool(tw))
    ok = [_equal(Z[m], lambda i, j: _pattern(i, j) * (m + 2)) and
          _equal(Y[m], lambda i, j: _pattern(i, j) * (m + 2) - 5) for m in range(2)]
    del W, Y, Z
    t.cuda.empty_cache()
    assert all(ok)


def _e4m3(q):
    return q.view(torch().float8_e4m3fn).float()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [2, 4])
def test_packed_token_of_most_columns(bits):
    """One row of one column over 2^31 - 1 outputs, in fp32 and 8 bits: odd
    halves, exact in both."""
    t = torch()
    Q = t.empty(MOST, dtype=t.uint8, device="cuda")
    half = (1 << bits) - 1
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        Q[i:j] = (_pattern(i, j).to(t.uint8) & half)
    S = t.ones(MOST, dtype=t.float16, device="cuda")
    X8 = t.full((1, 1), 0x38, dtype=t.uint8, device="cuda")                    # 1
    XE = t.full((1, 1), 127, dtype=t.uint8, device="cuda")
    f = bd.linear_q2_mx8 if bits == 2 else bd.linear_q4_mx8
    Y, Y8, YE = f(X8, XE, Q[:, None], S[:, None], out="both")

    def want(i, j):
        return (_pattern(i, j).to(t.uint8) & half).float() - half / 2

    def of_8_bits(i, j):
        e = YE[0, i // 32:-(-j // 32)].float() - 127
        return _e4m3(Y8[0, i:j]) * t.exp2(e).repeat_interleave(32)[:j - i]
    ok = _equal(Y[0], want) and all(
        bool((of_8_bits(i, min(i + (1 << 28), MOST)) == Y[0, i:i + (1 << 28)]).all()) for i in range(0, MOST, 1 << 28))
    del Q, S, Y, Y8, YE
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
def test_packed_layer_of_most_rows():
    """2^31 - 1 rows of one column, the residual updated in place."""
    t = torch()
    X8 = t.empty((MOST, 1), dtype=t.uint8, device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        X8[i:j, 0] = (_pattern(i, j).to(t.uint8) & 7) + 0x38                  # 1, 1.125, ...
    XE = t.full((MOST, 1), 127, dtype=t.uint8, device="cuda")
    Y = t.full((MOST, 1), 2.0, device="cuda")
    bd.linear_q4_mx8(X8, XE, t.full((1, 1), 15, dtype=t.uint8, device="cuda"),
                     t.ones((1, 1), dtype=t.float16, device="cuda"), residual=Y, Y=Y)
    ok = _equal(Y[:, 0], lambda i, j: 7.5 * _e4m3(X8[i:j, 0]) + 2)
    del X8, XE, Y
    t.cuda.empty_cache()
    assert ok
