// experts.hip -- the way of tokens to their experts and back: the order of
// (token, expert) pairs by expert, and the weighted sum of a token's expert
// results with its gradients.
#include <hip/hip_runtime.h>

#include "kernels.hpp"
#include "wave.hpp"

namespace gg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));   // rows may start at any float

// ---------------------------------------------------------------------------
// Grouping is a counting sort that keeps the order of equal keys.  One
// workgroup does it all: entries are few (a training batch has some 10^5), so
// what counts is the launch, the barriers and each wave's walk, and no second
// launch or exchange between workgroups.  Each of W waves takes a run of entries,
// counts its experts in an LDS row of its own (integers: their order does not
// matter), the rows are scanned over waves and experts, and the wave walks its
// run again, 64 entries at a time in order: entries of one expert find each
// other by a ballot per bit of the key, and their rank is the number of
// earlier lanes among them.  Entries without an expert have the key E and come
// last.
template <int W>
__global__ __launch_bounds__(64 * W) void expert_groups_kernel(ExpertGroups a, int bits) {
    constexpr int THREADS = 64 * W;
    __shared__ int count[W * (MAX_EXPERTS + 1)];      // W rows of E + 1
    __shared__ int wave_total[W];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bins = a.E + 1;
    for (int i = tid; i < W * bins; i += THREADS) count[i] = 0;
    __syncthreads();

    // fewer than 2^31 entries, so that sums of places fit 32 bits
    const unsigned k = a.k, n = (unsigned)a.T * k;
    const unsigned per = ((n + W - 1) / W + 63) / 64 * 64;
    const unsigned first = min(per * wave, n), end = min(first + per, n);
    int *mine = count + wave * bins;
    const auto key_of = [&](unsigned i) {
        const int e = a.ids[a.ldi == a.k ? (int64_t)i : i / k * a.ldi + i % k];
        return e >= 0 && e < a.E ? e : a.E;
    };
    constexpr int U = 8;                              // loads in flight
    for (unsigned base = first; base < end; base += 64 * U) {
        int key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) key[u] = key_of(min(base + 64 * u + lane, end - 1));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (base + 64 * u + lane < end) atomicAdd(mine + key[u], 1);
    }
    __syncthreads();

    // counts to places: over the waves of one expert, then over experts, a
    // round of THREADS bins at a time
    int before = 0;
    for (int b0 = 0; b0 < bins; b0 += THREADS) {
        const int b = b0 + tid;
        int total = 0;
        if (b < bins)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int c = count[w * bins + b];
                count[w * bins + b] = total;
                total += c;
            }
        int incl = total;                             // inclusive over the wave
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 63) wave_total[wave] = incl;
        __syncthreads();
        int start = before + incl - total;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < wave) start += wave_total[w];
            before += wave_total[w];
        }
        if (b < bins) {
#pragma unroll
            for (int w = 0; w < W; ++w) count[w * bins + b] += start;
            a.offsets[b] = start;                     // bin E starts where the last group ends
        }
        __syncthreads();
    }

    for (unsigned base = first; base < end; base += 64 * U) {
        int key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) key[u] = key_of(min(base + 64 * u + lane, end - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned i = base + 64 * u + lane;
            const bool there = i < end;
            uint64_t same = __ballot(there);
            for (int bit = 0; bit < bits; ++bit) {
                const uint64_t set = __ballot(key[u] >> bit & 1);
                same &= key[u] >> bit & 1 ? set : ~set;
            }
            if (there) {
                const int rank = __popcll(same & ((1ull << lane) - 1));
                const int at = mine[key[u]] + rank;
                a.rows[at] = (int)(i / k);
                a.pos[i / k * a.ldp + i % k] = key[u] < a.E ? at : -1;
            }
            // the last of the equal lanes moves the expert's place on, after
            // all have read it: LDS takes a wave's accesses in order
#if defined(__HIP_DEVICE_COMPILE__)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#endif
            if (there && (same >> lane) == 1) mine[key[u]] += __popcll(same);
#if defined(__HIP_DEVICE_COMPILE__)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#endif
        }
    }
}

// ---------------------------------------------------------------------------
// Joining: bound by memory.  A wave takes a token and U spans of 256 columns,
// 4 columns per lane and span, adds the token's rows of Y in the order of its
// choice, and writes each value of out once.
__device__ __forceinline__ v4f get(const float *row, int64_t col, int K) {
    v4f x = {0.f, 0.f, 0.f, 0.f};
    if (col + 4 <= K) {
        x = *reinterpret_cast<const v4f_any *>(row + col);
    } else if (col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) x[c] = row[col + c];
    }
    return x;
}

__device__ __forceinline__ void put(float *row, int64_t col, int K, const v4f &x) {
    if (col + 4 <= K) {
        *reinterpret_cast<v4f_any *>(row + col) = x;
    } else if (col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) row[col + c] = x[c];
    }
}

template <int U>
__global__ __launch_bounds__(256) void expert_combine_kernel(ExpertCombine a, int spans) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t units = (int64_t)a.T * spans;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + wave; unit < units; unit += (int64_t)gridDim.x * 4) {
        const int64_t t = unit / spans;
        const int64_t col = (unit % spans) * (256 * U) + 4 * lane;
        v4f sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] = v4f{0.f, 0.f, 0.f, 0.f};
            if (a.R) sum[u] = get(a.R + t * a.ldr, col + 256 * u, a.K);
        }
        const int32_t *pos = a.pos + t * a.ldp;
        const float *w = a.w ? a.w + t * a.ldw : nullptr;
#pragma unroll 2
        for (int j = 0; j < a.k; ++j) {
            const int p = pos[j];
            if (p < 0 || p >= a.M) continue;          // uniform
            const float f = w ? w[j] : 1.f;
            const float *row = a.Y + (int64_t)p * a.ldy;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const v4f y = get(row, col + 256 * u, a.K);
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[u][c] = __builtin_fmaf(f, y[c], sum[u][c]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) put(a.out + t * a.ldo, col + 256 * u, a.K, sum[u]);
    }
}

// Gradients: W waves take a token, a wave every W-th span of 256 columns, and
// up to J of its entries at a time, whose products with dO stay in registers
// until the row's end.
template <int W, int J>
__global__ __launch_bounds__(256) void expert_combine_bwd_kernel(ExpertCombineBwd a) {
    constexpr int TOKENS = 4 / W;
    __shared__ float red[4][J];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave / W, part = wave % W;
    for (int64_t base = (int64_t)blockIdx.x * TOKENS; base < a.T; base += (int64_t)gridDim.x * TOKENS) {
        const bool live = base + sub < a.T;
        const int64_t t = live ? base + sub : a.T - 1;
        const float *dO = a.dO + t * a.ldo;
        for (int j0 = 0; j0 < a.k; j0 += J) {
            int p[J];
            float f[J], dot[J];
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const int j = min(j0 + i, a.k - 1);
                p[i] = a.pos[t * a.ldp + j];
                if (j0 + i >= a.k || p[i] >= a.M || !live) p[i] = -1;
                f[i] = a.w ? a.w[t * a.ldw + j] : 1.f;
                dot[i] = 0.f;
            }
            for (int64_t col = part * 256 + 4 * lane; col < a.K; col += W * 256) {
                const v4f d = get(dO, col, a.K);
                v4f y[J];
                if (a.dw)
#pragma unroll
                    for (int i = 0; i < J; ++i)
                        if (p[i] >= 0) y[i] = get(a.Y + (int64_t)p[i] * a.ldy, col, a.K);
#pragma unroll
                for (int i = 0; i < J; ++i) {
                    if (p[i] < 0) continue;           // uniform
                    v4f o;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        o[c] = f[i] * d[c];
                        if (a.dw) dot[i] = __builtin_fmaf(d[c], y[i][c], dot[i]);
                    }
                    if (a.dY) put(a.dY + (int64_t)p[i] * a.lddy, col, a.K, o);
                }
            }
            if (a.dw == nullptr) continue;            // uniform
#pragma unroll
            for (int i = 0; i < J; ++i) dot[i] = wave64_sum(dot[i]);
            if constexpr (W > 1) {
                if (lane == 0)
#pragma unroll
                    for (int i = 0; i < J; ++i) red[wave][i] = dot[i];
                __syncthreads();
                if (part == 0)
#pragma unroll
                    for (int i = 0; i < J; ++i) {
#pragma unroll
                        for (int w = 1; w < W; ++w) dot[i] += red[wave + w][i];
                    }
                __syncthreads();
            }
            if (live && part == 0 && lane == 0)
#pragma unroll
                for (int i = 0; i < J; ++i)
                    if (j0 + i < a.k) a.dw[t * a.lddw + j0 + i] = dot[i];
        }
    }
}

constexpr int64_t MAX_GROUPS = 1 << 20;
inline unsigned groups(int64_t n) { return (unsigned)(n < MAX_GROUPS ? n : MAX_GROUPS); }

}  // namespace

hipError_t launch_expert_groups(const ExpertGroups &a, hipStream_t s) {
    int bits = 0;
    while (a.E >> bits) ++bits;                       // keys up to E
    // one wave needs no barriers: the better choice for the few entries of
    // generated tokens
    if ((int64_t)a.T * a.k <= 512) return launch(expert_groups_kernel<1>, dim3(1), dim3(64), s, a, bits);
    return launch(expert_groups_kernel<16>, dim3(1), dim3(1024), s, a, bits);
}

hipError_t launch_expert_combine(const ExpertCombine &a, hipStream_t s) {
    // four spans per wave where that still gives every SIMD a wave, else one
    const int64_t wide = ((int64_t)a.K + 1023) / 1024, narrow = ((int64_t)a.K + 255) / 256;
    if (wide * a.T >= 4096)
        return launch(expert_combine_kernel<4>, dim3(groups((wide * a.T + 3) / 4)), dim3(256), s, a, (int)wide);
    return launch(expert_combine_kernel<1>, dim3(groups((narrow * a.T + 3) / 4)), dim3(256), s, a, (int)narrow);
}

hipError_t launch_expert_combine_bwd(const ExpertCombineBwd &a, hipStream_t s) {
    if (a.K > 256) return launch(expert_combine_bwd_kernel<4, 4>, dim3(groups(a.T)), dim3(256), s, a);
    return launch(expert_combine_bwd_kernel<1, 4>, dim3(groups(((int64_t)a.T + 3) / 4)), dim3(256), s, a);
}

}  // namespace gg
