"""AddressSanitizer and UndefinedBehaviorSanitizer build (gcc, any finding
aborts), on the CPU, of the argument checks of the layers with experts and of
the norms around a block: api_experts.hip compiled as host C++ with launchers
that launch nothing, called with the largest and smallest sizes, wrapping
ranges, absent operands and valid calls."""
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
hipError_t launch_expert_groups(const ExpertGroups &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_expert_combine(const ExpertCombine &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_expert_combine_bwd(const ExpertCombineBwd &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_linear_grouped(const LinearGrouped &, int, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_linear_grouped_bwd(const LinearGroupedBwd &, int, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_packed_grouped(int, const PackedGrouped &, int, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_block_norm(const BlockNorm &, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_block_norm_bwd(const BlockNormBwd &, hipStream_t) { return hipErrorNotSupported; }
int64_t grouped_dz_tiles(int64_t M, int64_t E) {
    const int64_t n = (M + E * 127) / 128;
    return n < M ? n : M;
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
#define P(n) ((float *)((uintptr_t)(n) << 40))
#define I(n) ((int32_t *)((uintptr_t)(n) << 40))
#define U(n) ((uint8_t *)((uintptr_t)(n) << 40))
#define H(n) ((uint16_t *)((uintptr_t)(n) << 40))
int main(void) {
    const int64_t big = 2147483647, wide = (int64_t)1 << 62;
    float *top = (float *)(UINTPTR_MAX - 63);
    float *low = (float *)4096;          /* from where 2^64 bytes less 2^34 fit */
    int32_t *lowi = (int32_t *)low;
    gg_stream_t s = NULL;
    valid(expert_groups(8, 2, 5, I(1), 2, I(2), I(3), I(4), 2, s), "groups");
    valid(expert_groups(big, 1, 1024, I(1), 1, I(2), I(3), I(4), 1, s), "most pairs");
    expect(expert_groups(big, big, 5, I(1), big, I(2), I(3), I(4), big, s), GG_ERR_INVALID_ARG, "too many pairs");
    expect(expert_groups(8, 2, 5, (int32_t *)top, 2, I(2), I(3), I(4), 2, s), GG_ERR_INVALID_ARG, "wrapping ids");
    valid(expert_combine(8, 2, 16, 96, P(1), 96, I(2), 2, P(3), 2, P(4), 96, P(4), 96, s), "combine");
    expect(expert_combine(big, big, big, big, top, big, I(2), big, NULL, 0, NULL, 0, P(4), big, s), GG_ERR_INVALID_ARG,
           "wrapping Y");
    expect(expert_combine(big, big, big, big, low, big, lowi, big, NULL, 0, NULL, 0, low, big, s), GG_ERR_ALIAS,
           "combine at one place");
    valid(expert_combine_bwd(8, 2, 16, 96, P(1), 96, P(2), 96, I(3), 2, P(4), 2, P(5), 96, P(6), 2, s), "combine_bwd");
    expect(expert_combine_bwd(big, big, big, big, P(1), big, top, big, I(3), big, NULL, 0, P(5), big, P(6), big, s),
           GG_ERR_INVALID_ARG, "wrapping expert results");
    valid(linear_f32_grouped(0, 4, 8, 6, 5, 3, 9, P(1), 5, I(2), I(3), P(4), 6, 30, P(5), 6, P(6), 6, P(7), 6, s), "grouped");
    expect(linear_f32_grouped(0, 4, 8, 6, 5, 1024, 9, P(1), 5, I(2), I(3), P(4), 6, wide, P(5), 6, P(6), 6, P(7), 6, s),
           GG_ERR_INVALID_ARG, "experts past the address space");
    expect(linear_f32_grouped(0, 0, big, big, big, 1024, big, top, big, I(2), I(3), P(4), big, 0, NULL, 0, NULL, 0, P(7),
                              big, s), GG_ERR_INVALID_ARG, "largest everything");
    expect(linear_f32_grouped_bwd_ws_size(2, big, big, 1024), GG_ERR_INVALID_ARG, "workspace past 2^62");
    expect(linear_f32_grouped_bwd_ws_size(2, big, 8, 1024), 4 * (8 * big + (big + 1024LL * 127) / 128 * 8), "tall workspace");
    valid(linear_f32_grouped_bwd(1, 2, 1, 8, 6, 5, 3, 9, P(1), 6, P(2), 6, P(3), 5, I(4), I(5), P(6), 5, 30, P(7), 5, P(8),
                                 5, 30, P(9), 6, P(10), 1 << 20, s), "grouped_bwd");
    expect(linear_f32_grouped_bwd(1, 2, 1, 8, 6, 5, 3, 9, P(1), 6, P(2), 6, P(3), 5, I(4), I(5), P(6), 5, 30, P(7), 5, P(8),
                                  5, wide, P(9), 6, P(10), 1 << 20, s), GG_ERR_INVALID_ARG, "gradients past the space");
    expect(linear_f32_grouped_bwd(0, 2, 0, big, big, big, 1024, big, P(1), big, P(2), big, P(3), big, NULL, I(5), P(6), big,
                                  0, P(7), big, P(8), big, 0, P(9), big, top, big, s), GG_ERR_INVALID_ARG, "largest bwd");
    valid(linear_q4_mx8_grouped(1, 8, 64, 100, 3, 9, U(1), 100, U(2), 4, I(3), I(4), U(5), 50, 3200, H(6), 2, 128, P(7), 64,
                                P(8), 64, U(9), 64, U(10), 2, s), "packed");
    expect(linear_q2_mx8_grouped(0, 8, 64, 100, 1024, 9, U(1), 100, U(2), 4, I(3), I(4), U(5), 50, wide, H(6), 2, wide, NULL,
                                 0, P(8), 64, NULL, 0, NULL, 0, s), GG_ERR_INVALID_ARG, "codes past the space");
    expect(linear_q2_mx8_grouped(0, big, big, big, 1024, big, U(1), big, U(2), big, I(3), I(4), U(5), big, 0, H(6), big, 0,
                                 NULL, 0, P(8), big, NULL, 0, NULL, 0, s), GG_ERR_INVALID_ARG, "too many tiles");
    valid(block_norm_f32(8, 96, P(1), 96, P(2), 96, P(3), P(4), 0, .5f, P(5), 1e-5f, P(2), 96, P(6), 96, P(7), P(8), s),
          "block norm in place");
    expect(block_norm_f32(big, big, top, big, P(2), big, NULL, NULL, 0, 1.f, NULL, 0.f, P(5), big, P(6), big, NULL, NULL, s),
           GG_ERR_INVALID_ARG, "wrapping rows");
    expect(block_norm_f32(8, 96, P(1), 96, P(2), 96, NULL, NULL, 0, NAN, NULL, 0.f, P(5), 96, P(6), 96, NULL, NULL, s),
           GG_ERR_INVALID_ARG, "alpha NaN");
    valid(block_norm_mx8(8, 96, P(1), 96, P(2), 96, NULL, P(4), 96, 1.f, NULL, 0.f, P(5), 96, U(6), 96, U(7), 3, s), "mx8");
    expect(block_norm_f32_bwd_ws_size(big, big), 8LL * 512 * big, "norm workspace");
    valid(block_norm_f32_bwd(1, 8, 96, P(1), 96, P(2), 96, P(3), 96, P(4), P(5), 0, 1.f, P(6), P(7), P(8), P(9), 96, P(10), 96,
                             P(9), 96, P(11), P(12), P(13), 0, P(14), 8 * 96 * 8, s), "block norm bwd");
    expect(block_norm_f32_bwd(1, 8, 96, P(1), 96, P(2), 96, P(3), 96, P(4), P(5), 0, 1.f, P(6), P(7), P(8), P(9), 96, P(10), 96,
                              P(9), 96, P(11), P(12), P(13), 0, P(14), 8 * 96 * 8 - 1, s), GG_ERR_INVALID_ARG, "short");
    expect(block_norm_f32_bwd(0, big, big, low, big, low, big, low, big, NULL, NULL, 0, 1.f, NULL, low, low, NULL, 0,
                              low, big, low, big, NULL, NULL, NULL, 0, NULL, 0, s), GG_ERR_ALIAS, "norms at one place");
    printf("%s\n", failures ? "FAILED" : "ALL OK");
    return failures != 0;
}
"""


def test_expert_checks_under_sanitizers(tmp_path):
    if not (shutil.which("gcc") and shutil.which("g++")):
        pytest.skip("gcc/g++ are not installed")
    for name in ("libasan.so", "libubsan.so"):
        p = subprocess.run(["gcc", "-print-file-name=" + name], capture_output=True, text=True).stdout.strip()
        if not (os.path.isabs(p) and os.path.exists(p)):
            pytest.skip("the gcc sanitizer runtimes are not installed")
    api, stubs, main = tmp_path / "api.cpp", tmp_path / "stubs.cpp", tmp_path / "main.c"
    text = open(os.path.join(CSRC, "api_experts.hip")).read()
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
