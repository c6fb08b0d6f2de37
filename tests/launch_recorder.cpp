// Stands in for the HIP runtime under the library's launchers, on the CPU:
// hipLaunchKernel prints the launch instead of making it.  One line per launch,
//   <kernel> <grid x> <grid y> <threads> <the kernel's arguments that matter>
// and the launcher's status at the end of a call.  Pointers are made up and
// never dereferenced; an output's place is printed as its distance from OUT.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>

#include "gemm_f32_tile.hpp"
#include "kernels.hpp"

using namespace gg;

namespace {
std::map<const void *, std::string> &names() {
    static std::map<const void *, std::string> n;
    return n;
}
template <class T>
T arg(void **a, int i) { return *static_cast<T *>(a[i]); }

const uintptr_t OUT = (uintptr_t)1 << 50;      // the output that a call writes
template <class T>
T *at(int64_t n) { return reinterpret_cast<T *>((uintptr_t)n << 44); }
long long from_out(const void *p) {
    return p ? (long long)(reinterpret_cast<uintptr_t>(p) - OUT) : 0;
}
}  // namespace

extern "C" {
void **__hipRegisterFatBinary(const void *) { static void *m; return &m; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterVar(void **, void *, char *, const char *, int, size_t, int, int) {}
void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *,
                           void *, void *, void *, int *) {
    names()[host] = name;
}
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { abort(); }

hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t, hipStream_t) {
    const std::string &n = names().at(f);
    const auto has = [&](const char *s) { return n.find(s) != std::string::npos; };
    printf("%s %u %u %u ", n.c_str(), g.x, g.y, b.x * b.y * b.z);
    if (has("dz_kernel")) {
        // M N chunk
        printf("%d %d %d\n", arg<int>(a, 1), arg<int>(a, 2), arg<int>(a, 3));
    } else if (has("column_sum")) {
        printf("%d %d\n", arg<int>(a, 0), arg<int>(a, 1));
    } else if (has("gemm_f32_") || has("linear_few")) {
        // M N K, the distance of C, its leading dimension, the distances of
        // both operands; tiles
        printf("%d %d %d %lld %lld %lld %lld", arg<int>(a, 0), arg<int>(a, 1), arg<int>(a, 2),
               from_out(arg<float *>(a, 7)) / 4, (long long)arg<int64_t>(a, 8),
               (long long)(arg<const float *>(a, 3) - at<float>(1)),
               (long long)(arg<const float *>(a, 5) - at<float>(2)));
        if (has("gemm_f32_")) printf(" %d %d", arg<int>(a, 10), arg<int>(a, 11));
        printf("\n");
    } else if (has("packed_")) {
        const PackedLinear p = arg<PackedLinear>(a, 0);
        printf("%d %d %d %lld %lld", p.M, p.N, p.K, from_out(p.Y) / 4, (long long)p.ldy);
        printf(" %lld %lld %lld %lld", (long long)(p.X - at<uint8_t>(1)), (long long)(p.XE - at<uint8_t>(2)),
               (long long)(p.Q - at<uint8_t>(3)), (long long)(p.S - at<uint16_t>(4)));
        printf(" %lld %lld", p.Y8 ? (long long)(p.Y8 - at<uint8_t>(5)) : -1,
               p.YE ? (long long)(p.YE - at<uint8_t>(6)) : -1);
        printf(" %lld %lld\n", p.bias ? (long long)(p.bias - at<float>(7)) : -1,
               p.R ? (long long)(p.R - at<float>(8)) : -1);
    } else {
        printf("\n");
    }
    return hipSuccess;
}
}

// <call> <sizes ...>
int main(int argc, char **argv) {
    const std::string call = argv[1];
    const auto n = [&](int i) { return argc > i ? (int)atoll(argv[i]) : 0; };
    float *out = reinterpret_cast<float *>(OUT);
    hipError_t e = hipErrorUnknown;
    if (call == "bwd_bias") {                   // M N act: column sums alone
        e = launch_linear_bwd(false, n(4), false, n(2), n(3), 1, at<float>(1), n(3), at<float>(2),
                              n(3), nullptr, 0, nullptr, 0, nullptr, 0, nullptr, 0, out, at<float>(3),
                              256, nullptr);
    } else if (call == "gemm") {                // M N K, A as K x M, B as N x K
        e = launch_gemm(!n(5), n(6), n(2), n(3), n(4), 1.f, at<float>(1), n(5) ? n(2) : n(4),
                        at<float>(2), n(6) ? n(4) : n(3), 0.f, out, n(3), 256, nullptr);
    } else if (call == "linear") {              // M N K, W as N x K
        e = launch_linear(n(5), 0, n(2), n(3), n(4), at<float>(1), n(4), at<float>(2),
                          n(5) ? n(4) : n(3), nullptr, nullptr, 0, nullptr, 0, out, n(3), 256, nullptr);
    } else if (call == "packed") {              // bits M N K, to 8 bits as well
        const int64_t N = n(4), K = n(5);
        const int64_t ldq = (K * n(2) + 7) / 8;
        const PackedLinear a{0, n(3), n(4), n(5), at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), at<uint16_t>(4),
                             n(6) ? at<float>(7) : nullptr, n(6) ? at<float>(8) : nullptr, out,
                             n(6) ? at<uint8_t>(5) : nullptr, n(6) ? at<uint8_t>(6) : nullptr,
                             K, (K + 31) / 32, ldq, (K + 63) / 64, n(6) ? N : 0, N, n(6) ? N : 0,
                             n(6) ? (N + 31) / 32 : 0};
        e = launch_packed_linear(n(2), a, 256, nullptr);
    } else if (call == "k_walk") {              // K -> slabs; places in the last one
        const int K = n(2), slabs = slabs_of<32>(K), k0 = (slabs - 1) * 32;
        printf("%d\n", slabs);
        for (int k = 0; k < 32; ++k) printf("%d ", clamp_k(k0, k, K - 1));
        printf("\n");
        e = hipSuccess;
    } else if (call == "rows_of_chunk") {       // M chunk index -> first row, end
        const RowRange r = dz_rows(n(2), dz_chunk(n(2)), n(3));
        printf("%lld %lld\n", (long long)r.first, (long long)r.end);
        e = hipSuccess;
    }
    printf("status %d\n", (int)e);
    return 0;
}
