"""The layers on grouped rows at sizes near 2^31: on the CPU the counts that
their kernels and launchers go by, on the GPU outputs of the most columns, in
values that are exact."""
import subprocess

import pytest

from gemv_gemm_f32_amd import binding as bd
from gpu_util import torch
from test_groups_host import _hipcc, record  # noqa: F401 (a fixture)
from test_largest_sizes import MOST, _e4m3, _equal, _pattern

HOST = r"""
#include <stdio.h>
#include <stdlib.h>
#include "gemm_f32_tile.hpp"
#include "groups.hpp"
using namespace gg;
#define CHECK(c) do { if (!(c)) { printf("FAIL line %d: %s\n", __LINE__, #c); exit(1); } } while (0)
template <int J> void runs(int64_t k) {
    int64_t n = 0;
    for (int j0 = 0; j0 < k; j0 = next_run<J>(j0, (int)k)) CHECK(j0 == n++ * J && (int64_t)j0 + J - 1 <= INT32_MAX);
    CHECK(n == k / J + (k % J != 0));
}
int main() {
    for (int64_t n : {int64_t(0), int64_t(1), int64_t(31), int64_t(32), int64_t(33), int64_t(1) << 30, int64_t(INT32_MAX) - 128,
                      int64_t(INT32_MAX) - 127, int64_t(INT32_MAX) - 63, int64_t(INT32_MAX) - 1, int64_t(INT32_MAX)})
        for (int size : {1, 2, 4, 8, 16, 32, 64, 128, 256}) {
            const int64_t tiles = tiles_of((int)n, size);
            CHECK(tiles == n / size + (n % size != 0));
        }
    /* the walk along k: slabs, and which places of the last one lie behind K */
    for (int64_t K : {int64_t(1), int64_t(31), int64_t(32), int64_t(33), int64_t(1) << 30, int64_t(INT32_MAX) - 32,
                      int64_t(INT32_MAX) - 31, int64_t(INT32_MAX) - 30, int64_t(INT32_MAX) - 1, int64_t(INT32_MAX)}) {
        const int64_t slabs = slabs_to<32, unsigned>((int)K);
        CHECK(slabs == K / 32 + (K % 32 != 0));
        const int64_t k0 = (slabs - 1) * 32;
        for (int k = 0; k < 32; ++k)
            for (int n : {1, 4, 32}) CHECK(past_k<unsigned>((unsigned)k0 + k, n, (int)K) == (k0 + k + n > K));
    }
    /* a token's entries, J at a time */
    for (int64_t k : {0, 1, 7, 8, 9, 1 << 20, INT32_MAX - 8, INT32_MAX - 7, INT32_MAX - 3, INT32_MAX - 1, INT32_MAX}) {
        runs<4>(k);
        runs<8>(k);
    }
    printf("ALL OK\n");
}
"""


def test_counts_of_any_size(tmp_path):
    src, obj, exe = tmp_path / "host.cpp", tmp_path / "host.o", tmp_path / "host"
    src.write_text(HOST)
    _hipcc(src, obj)
    subprocess.run(["g++", "-o", str(exe), str(obj), "-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files"],
                   check=True, capture_output=True, text=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ALL OK" in r.stdout, r.stdout + r.stderr


# (W stored N x K, or K x N where it has rows of up to 2^22 columns or none)
@pytest.mark.parametrize("M,N,K,E,v", [(16, 1 << 29, 1, 16, 1), (8, 1 << 30, 1, 8, 1), (8, (1 << 30) - 4, 1, 8, 1),
                                       (4, MOST, 1, 4, 1), (1, MOST, 1, 1, 1), (16, 1 << 29, 1, 1024, 1),
                                       (16, MOST, 0, 16, 0), (1, MOST, 0, 1, 0), (16, 1 << 22, 3, 16, 0)])
def test_few_rows_over_many_columns(record, M, N, K, E, v):  # noqa: F811
    """Fewer than 2^31 tiles of 32 x 32 are one launch, whatever its kernel."""
    (name, groups), = record("forward", M, N, K, E, v)
    assert "grouped_" in name and groups >= -(-N // 64) * (1 if E == 1 else min(M, 16))


def _columns():
    """A vector of MOST columns."""
    t = torch()
    v = t.empty(MOST, device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        v[i:j] = _pattern(i, j)
    return v


def _ints(*values):
    return torch().tensor(values, dtype=torch().int32, device="cuda")


def _every_row(Y, f):
    return all(_equal(Y[m], lambda i, j: f(m, i, j)) for m in range(Y.shape[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3])
def test_layer_of_most_columns(M):
    """W stored N x K: the kernel for few rows and the tiles."""
    t = torch()
    W = _columns()
    X = t.arange(1, M + 1, device="cuda").float()[:, None].contiguous()
    Y = t.full((M, MOST), -1.0, device="cuda")
    bd.linear_f32_grouped(X, W[None, :, None], _ints(0, M), Y=Y, trans_w=True)
    ok = _every_row(Y, lambda m, i, j: _pattern(i, j) * (m + 1))
    del W, Y
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
def test_rows_of_sixteen_experts_over_many_columns():
    """More columns than a grid of the kernel for few rows holds; one matrix for
    all experts."""
    t = torch()
    N = 1 << 29
    W = _columns()[:N].clone()
    Y = t.full((16, N), -1.0, device="cuda")
    bd.linear_f32_grouped(t.arange(1, 17, device="cuda").float()[:, None].contiguous(), W[None, :, None].expand(16, N, 1),
                          _ints(*range(17)), Y=Y, trans_w=True)
    ok = _every_row(Y, lambda m, i, j: _pattern(i, j) * (m + 1))
    del W, Y
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3])
def test_bias_of_most_columns(M):
    """W stored K x N, which has rows this long for K = 0 alone."""
    t = torch()
    b = _columns()
    Y = t.full((M, MOST), -1.0, device="cuda")
    bd.linear_f32_grouped(t.empty((M, 0), device="cuda"), t.empty((1, 0, MOST), device="cuda"), _ints(0, M), bias=b[None],
                          Y=Y)
    ok = _every_row(Y, lambda m, i, j: _pattern(i, j))
    del b, Y
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
@pytest.mark.parametrize("tw", [0, 1])
def test_weight_gradient_of_no_rows_over_most_columns(tw):
    t = torch()
    dW = t.full((1, MOST, 1) if tw else (1, 1, MOST), 7.0, device="cuda")
    bd.linear_f32_grouped_bwd(t.empty((0, MOST), device="cuda"), t.empty((0, 1), device="cuda"), dW, _ints(0, 0), dW=dW,
                              want=("dW",), trans_w=bool(tw))
    ok = _equal(dW.view(-1), lambda i, j: t.zeros(j - i, device="cuda"))
    del dW
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
def test_bias_gradient_of_most_columns():
    t = torch()
    dY = _columns()
    Z = t.ones((1, MOST), device="cuda")
    Z[0, ::3] = -1
    db = t.full((1, MOST), 7.0, device="cuda")
    bd.linear_f32_grouped_bwd(dY[None], None, t.empty((1, 0, MOST), device="cuda"), _ints(0, 1), Z=Z, act="relu", db=db,
                              want=("db",))
    ok = _equal(db[0], lambda i, j: _pattern(i, j) * (t.arange(i, j, device="cuda") % 3 != 0))
    del dY, Z, db
    t.cuda.empty_cache()
    assert ok


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [2, 4])
def test_packed_layer_of_most_columns(bits):
    """One row of one column in fp32 and 8 bits: odd halves, exact in both."""
    t = torch()
    half = (1 << bits) - 1
    Q = t.empty(MOST, dtype=t.uint8, device="cuda")
    for i in range(0, MOST, 1 << 28):
        j = min(i + (1 << 28), MOST)
        Q[i:j] = _pattern(i, j).to(t.uint8) & half
    S = t.ones(MOST, dtype=t.float16, device="cuda")
    X8 = t.full((1, 1), 0x38, dtype=t.uint8, device="cuda")                    # 1
    XE = t.full((1, 1), 127, dtype=t.uint8, device="cuda")
    f = bd.linear_q2_mx8_grouped if bits == 2 else bd.linear_q4_mx8_grouped
    Y = t.full((1, MOST), -9.0, device="cuda")
    Y8 = t.zeros((1, MOST), dtype=t.uint8, device="cuda")
    YE = t.zeros((1, -(-MOST // 32)), dtype=t.uint8, device="cuda")
    f(X8, XE, Q[None, :, None], S[None, :, None], _ints(0, 1), Y=Y, Y8=Y8, YE=YE, out="both")

    def of_8_bits(i, j):
        e = YE[0, i // 32:-(-j // 32)].float() - 127
        return _e4m3(Y8[0, i:j]) * t.exp2(e).repeat_interleave(32)[:j - i]
    ok = _equal(Y[0], lambda i, j: (_pattern(i, j).to(t.uint8) & half).float() - half / 2) and _equal(Y[0], of_8_bits)
    del Q, S, Y, Y8, YE
    t.cuda.empty_cache()
    assert ok
