"""AddressSanitizer and UndefinedBehaviorSanitizer build (gcc, any finding
aborts), on the CPU, of the argument checks of the layers: api_layers.hip
compiled as host C++ with launchers that launch nothing, called with the
largest and smallest sizes, wrapping ranges, absent operands and valid calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemv_gemm_f32_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]

STUBS = r"""
#include <hip/hip_runtime.h>
#include "kernels.hpp"
namespace gg {
hipError_t launch_linear(bool, int, int, int, int, const float *, int64_t, const float *, int64_t,
                         const float *, const float *, int64_t, float *, int64_t, float *, int64_t,
                         int, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_linear_bwd(bool, int, bool, int, int, int, const float *, int64_t, const float *,
                             int64_t, const float *, int64_t, const float *, int64_t, float *,
                             int64_t, float *, int64_t, float *, float *, int, hipStream_t) {
    return hipErrorNotSupported;
}
hipError_t launch_rmsnorm(const RmsNorm &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_rmsnorm_bwd(const RmsNormBwd &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_packed_linear(int, const PackedLinear &, int, hipStream_t) {
    return hipErrorNotSupported;
}
}
"""

MAIN = r"""
#include <stdio.h>
#include <math.h>
#include "gemvgemm.h"
static int failures = 0;
static void expect(long long got, long long want, const char *what) {
    if (got != want) { printf("FAIL %s: %lld, want %lld\n", what, got, want); ++failures; }
}
/* a call that passes the checks: no device here, or a stub launcher */
static void valid(int got, const char *what) {
    if (got != GG_ERR_NO_DEVICE && got != GG_ERR_LAUNCH) { printf("FAIL %s: %d\n", what, got); ++failures; }
}
#define P(n) ((float *)((uintptr_t)(n) << 32))
#define U(n) ((uint8_t *)((uintptr_t)(n) << 32))
#define H(n) ((uint16_t *)((uintptr_t)(n) << 32))
int main(void) {
    const int64_t big = 2147483647;
    float *top = (float *)(UINTPTR_MAX - 63);
    gg_stream_t s = NULL;
    valid(linear_f32(0, 4, 8, 6, 5, P(1), 5, P(2), 6, P(3), P(4), 6, P(5), 6, P(6), 6, s), "linear");
    valid(linear_f32(1, 0, 8, 6, 5, P(1), 5, P(2), 5, NULL, P(6), 6, NULL, -9, P(6), 6, s), "in place");
    expect(linear_f32(0, 0, big, big, big, top, big, P(2), big, NULL, NULL, 0, NULL, 0, P(6), big, s),
           GG_ERR_INVALID_ARG, "wrapping X");
    expect(linear_f32(0, 0, big, big, big, P(1), big, P(1), big, NULL, NULL, 0, NULL, 0, P(1), big, s),
           GG_ERR_ALIAS, "everything at one place");
    expect(linear_f32_bwd_ws_size(2, big, big), GG_ERR_INVALID_ARG, "workspace past 2^62");
    expect(linear_f32_bwd_ws_size(2, big, 8), 4 * (8 * big + 64 * 8), "tall workspace");
    expect(linear_f32_bwd_ws_size(0, 5, 7), 4 * 64 * 7, "workspace of column sums");
    expect(linear_f32_bwd(0, 2, 0, big, big, 1, P(1), big, P(2), big, P(3), 1, P(4), big, P(5), 1,
                          P(6), big, P(7), top, big, s), GG_ERR_INVALID_ARG, "wrapping workspace");
    valid(linear_f32_bwd(0, 2, 1, 8, 6, 5, P(1), 6, P(2), 6, P(3), 5, P(4), 6, P(5), 5, P(6), 6, P(7),
                         P(8), 1 << 20, s), "bwd");
    expect(linear_f32_bwd(0, 2, 1, 0, 0, 0, NULL, 0, NULL, 0, NULL, 0, NULL, 0, P(5), 5, P(6), 6, P(7),
                          NULL, 0, s), GG_OK, "nothing to do");
    valid(rmsnorm_f32(8, 96, P(1), 96, P(2), 96, P(3), 1e-5f, P(2), 96, P(4), 96, P(5), s), "norm");
    expect(rmsnorm_f32(8, 96, P(1), 96, NULL, 0, NULL, NAN, NULL, 0, P(4), 96, NULL, s),
           GG_ERR_INVALID_ARG, "eps NaN");
    expect(rmsnorm_f32(big, big, top, big, NULL, 0, NULL, 0.f, NULL, 0, P(4), big, NULL, s),
           GG_ERR_INVALID_ARG, "wrapping rows");
    valid(rmsnorm_mx8(8, 96, P(1), 96, NULL, 0, NULL, 0.f, NULL, 0, U(4), 96, U(5), 3, s), "norm8");
    expect(rmsnorm_f32_bwd_ws_size(big, big), 4LL * 512 * big, "norm workspace");
    valid(rmsnorm_f32_bwd(1, 8, 96, P(1), 96, P(2), 96, P(3), P(4), P(5), 96, P(5), 96, P(6), P(7),
                          8 * 96 * 4, s), "norm bwd");
    expect(rmsnorm_f32_bwd(1, 8, 96, P(1), 96, P(2), 96, P(3), P(4), P(5), 96, P(5), 96, P(6), P(7),
                           8 * 96 * 4 - 1, s), GG_ERR_INVALID_ARG, "short norm workspace");
    valid(linear_q4_mx8(1, 8, 64, 100, U(1), 100, U(2), 4, U(3), 50, H(4), 2, P(5), P(6), 64, P(6), 64,
                        U(7), 64, U(8), 2, s), "packed");
    expect(linear_q2_mx8(0, big, big, big, (uint8_t *)top, big, U(2), big, U(3), big, H(4), big, NULL,
                         NULL, 0, P(6), big, NULL, 0, NULL, 0, s), GG_ERR_INVALID_ARG, "wrapping X8");
    expect(linear_q2_mx8(0, big, big, big, U(1), big, U(1), big, U(1), big, H(1), big, NULL, NULL, 0,
                         P(1), big, U(1), big, U(1), big, s), GG_ERR_ALIAS, "packed at one place");
    printf("%s\n", failures ? "FAILED" : "ALL OK");
    return failures != 0;
}
"""


def test_layer_checks_under_sanitizers(tmp_path):
    if not (shutil.which("gcc") and shutil.which("g++")):
        pytest.skip("gcc/g++ are not installed")
    for name in ("libasan.so", "libubsan.so"):
        p = subprocess.run(["gcc", "-print-file-name=" + name], capture_output=True, text=True).stdout.strip()
        if not (os.path.isabs(p) and os.path.exists(p)):
            pytest.skip("the gcc sanitizer runtimes are not installed")
    api, stubs, main = tmp_path / "api.cpp", tmp_path / "stubs.cpp", tmp_path / "main.c"
    text = open(os.path.join(CSRC, "api_layers.hip")).read()
    api.write_text(text.replace('"../../include/gemvgemm.h"',
                                '"%s"' % os.path.join(ROOT, "include", "gemvgemm.h")))
    stubs.write_text(STUBS)
    main.write_text(MAIN)
    lib, exe = tmp_path / "libchecks.so", tmp_path / "main"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", "-I", CSRC] + SAN + [str(api), str(stubs), "-o", str(lib),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"],
                   check=True, capture_output=True, text=True, timeout=300)
    subprocess.run(["gcc", "-std=c99", "-g", "-I", os.path.join(ROOT, "include")] + SAN +
                   [str(main), "-o", str(exe), str(lib), "-Wl,-rpath," + str(tmp_path)],
                   check=True, capture_output=True, text=True, timeout=120)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and "ALL OK" in r.stdout, r.stdout + r.stderr
