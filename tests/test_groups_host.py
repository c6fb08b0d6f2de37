"""What the grouped kernels' safety and coverage rest on, on the CPU: the rows
of a group stay inside whatever its offsets hold, a launch has a workgroup for
every tile that any sizes need, tiles are handed out once each, and grids are
ones that a launch takes.  groups.hpp compiled for the host, and the launchers
of the grouped layers with a recorder in place of the HIP runtime."""
import os
import subprocess

import pytest

from gemv_gemm_f32_amd.build import HIPCC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemv_gemm_f32_amd", "csrc")
FLAGS = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-I", CSRC, "-w"]

HOST = r"""
#include <stdio.h>
#include <stdlib.h>
#include <random>
#include <vector>
#include "groups.hpp"
using namespace gg;
#define CHECK(c) do { if (!(c)) { printf("FAIL line %d: %s\n", __LINE__, #c); exit(1); } } while (0)
int main() {
    std::mt19937 rng(1);
    const int wild[] = {0, 1, -1, 7, 100, 101, 99, INT32_MAX, INT32_MIN, INT32_MIN + 1, INT32_MAX - 1, 50};
    for (int M : {0, 1, 64, 100, INT32_MAX})
        for (int a : wild)
            for (int b : wild) {
                const int32_t o[2] = {a, b};
                int first, count;
                group_rows({o, 1, M}, 0, first, count);
                CHECK(first >= 0 && count >= 0 && first <= M && count <= M - first);
                if (0 <= a && a <= b && b <= M) CHECK(first == a && count == b - a);
                group_rows({o, 1, M}, 1, first, count);      /* no such group */
                CHECK(first == 0 && count == 0);
            }
    for (int BM : {1, 4, 8, 16, 32, 64, 128})
        for (int round = 0; round < 2000; ++round) {
            const int E = 1 + rng() % 40, M = rng() % 500;
            std::vector<int> size(E);
            for (int i = 0; i < M; ++i) ++size[rng() % (1 + rng() % E)];
            int64_t tiles = 0;
            for (int s : size) tiles += (s + BM - 1) / BM;
            CHECK(tiles <= tiles_most(M, E, BM));
        }
    /* reached: every group with one row more than whole tiles */
    CHECK(tiles_most(65 * 5, 5, 64) == 10 && tiles_most(3, 5, 64) == 3 && tiles_most(0, 5, 64) == 0);
    CHECK(tiles_most(INT32_MAX, 1024, 32) == ((int64_t)INT32_MAX + 1024 * 31) / 32);
    for (int n = 1; n < 700; ++n) {
        std::vector<char> seen(n);
        for (int b = 0; b < n; ++b) {
            const int t = xcd_run(b, n);
            CHECK(t >= 0 && t < n && !seen[t]);
            seen[t] = 1;
        }
    }
    CHECK(xcd_run(INT32_MAX - 1, INT32_MAX) >= 0);
    for (int64_t n : {int64_t(1), int64_t(1) << 20, (int64_t(1) << 20) + 1, int64_t(INT32_MAX)}) {
        const dim3 g = grid_of(n);
        CHECK((int64_t)g.x * g.y >= n && (int64_t)g.x * g.y < n + g.x && g.y <= 65535);
        CHECK((uint64_t)g.x * 1024 < (uint64_t)1 << 32 && (g.y == 1 || g.x % 8 == 0));
    }
    printf("ALL OK\n");
}
"""


def _hipcc(src, out, *more):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    subprocess.run([HIPCC, "-x", "hip"] + FLAGS + ["-c", str(src), "-o", str(out)], check=True, capture_output=True,
                   text=True, timeout=300)


def test_groups_on_the_host(tmp_path):
    src, obj, exe = tmp_path / "host.cpp", tmp_path / "host.o", tmp_path / "host"
    src.write_text(HOST)
    _hipcc(src, obj)
    subprocess.run(["g++", "-o", str(exe), str(obj), "-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files"],
                   check=True, capture_output=True, text=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ALL OK" in r.stdout, r.stdout + r.stderr


RECORDER = r"""
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <map>
#include <string>
#include "kernels.hpp"
using namespace gg;
static std::map<const void *, std::string> &names() { static std::map<const void *, std::string> n; return n; }
extern "C" {
void **__hipRegisterFatBinary(const void *) { static void *m; return &m; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterVar(void **, void *, char *, const char *, int, size_t, int, int) {}
void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *, void *, void *, void *,
                           int *) { names()[host] = name; }
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { abort(); }
hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **, size_t, hipStream_t) {
    printf("%s %u %u %u\n", names().at(f).c_str(), g.x, g.y, b.x * b.y * b.z);
    return hipSuccess;
}
}
template <class T> static T *at(int64_t n) { return reinterpret_cast<T *>((uintptr_t)n << 44); }
int main(int argc, char **argv) {
    const std::string call = argv[1];
    const auto n = [&](int i) { return argc > i ? (int)atoll(argv[i]) : 0; };
    const int M = n(2), N = n(3), K = n(4), E = n(5), v = n(6);
    hipError_t e = hipErrorUnknown;
    if (call == "forward")
        e = launch_linear_grouped({v == 1, 0, M, N, K, E, 0, at<float>(1), at<float>(2), nullptr, nullptr, at<int32_t>(3),
                                   nullptr, at<float>(4), K, v ? K : N, (int64_t)N * K, 0, 0, N}, 256, nullptr);
    if (call == "backward")
        e = launch_linear_grouped_bwd({v == 1, false, 1, M, N, K, E, 0, at<float>(1), at<float>(2), at<float>(3),
                                       at<float>(4), nullptr, at<int32_t>(5), at<float>(6), at<float>(7), at<float>(8),
                                       at<float>(9), N, N, K, v ? K : N, (int64_t)N * K, K, v ? K : N, (int64_t)N * K, N},
                                      256, nullptr);
    if (call == "packed") {
        const PackedGrouped a{{0, M, N, K, at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), at<uint16_t>(4), nullptr, nullptr,
                               at<float>(5), nullptr, nullptr, K, (K + 31) / 32, K, (K + 63) / 64, 0, N, 0, 0},
                              nullptr, at<int32_t>(6), E, 0, (int64_t)N * K, N, 0};
        e = launch_packed_grouped(v, a, 256, nullptr);
    }
    printf("status %d\n", (int)e);
}
"""


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    d = tmp_path_factory.mktemp("grouped_recorder")
    rec = d / "recorder.cpp"
    rec.write_text(RECORDER)
    objs = []
    for src in [os.path.join(CSRC, u + ".hip") for u in ("linear_grouped", "linear_mx8_grouped")] + [str(rec)]:
        objs.append(str(d / (os.path.basename(src) + ".o")))
        _hipcc(src, objs[-1])
    exe = str(d / "recorder")
    subprocess.run(["g++", "-o", exe] + objs + ["-no-pie", "-Wl,--unresolved-symbols=ignore-in-object-files"], check=True,
                   capture_output=True, text=True, timeout=120)

    def run(*args):
        r = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=60)
        lines = r.stdout.split("\n")[:-1]
        assert r.returncode == 0 and lines.pop() == "status 0", r.stdout + r.stderr
        out = []
        for ln in lines:
            name, gx, gy, threads = ln.split()
            gx, gy, threads = int(gx), int(gy), int(threads)
            assert gx * threads < 1 << 32 and gy <= 65535 and threads <= 1024, ln
            out.append((name, gx * gy))
        return out
    return run


MOST = (1 << 31) - 1
SIZES = [(1, 1, 1, 1), (8, 2304, 768, 8), (8192, 2048, 1024, 8), (MOST, 1, 1, 1), (MOST, 1000, 4, 1024),
         (1 << 20, 1 << 16, 64, 3), (5, 1 << 22, 16, 1024), (700, 1 << 22, 32, 2)]


@pytest.mark.parametrize("v", [0, 1])
@pytest.mark.parametrize("M,N,K,E", SIZES)
def test_grids_of_the_layer(record, M, N, K, E, v):
    (name, groups), = record("forward", M, N, K, E, v)
    assert "grouped_" in name and groups >= -(-M // 64) * -(-N // 64)
    launches = record("backward", M, N, K, E, v)
    # the biases' sums are a wave each of 64 columns in the last launch's first workgroups
    assert len(launches) == 3 and "dz" in launches[0][0]
    assert launches[1][1] >= -(-M // 64) * -(-K // 64)
    assert launches[2][1] >= E * -(-N // 64) * -(-K // 64) + -(-E * -(-N // 64) // 16)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("M,N,K,E", SIZES)
def test_grids_of_the_packed_layer(record, M, N, K, E, bits):
    (name, groups), = record("packed", M, N, K, E, bits)
    assert "packed_" in name and groups >= -(-M // 128) * -(-N // 256)
