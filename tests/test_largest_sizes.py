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
