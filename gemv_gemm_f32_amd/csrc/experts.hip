// experts.hip -- the way of tokens to their experts and back: the order of
// (token, expert) pairs by expert, and the weighted sum of a token's expert
// results with its gradients.
#include <hip/hip_runtime.h>

#include "groups.hpp"
#include "kernels.hpp"
#include "wave.hpp"

namespace gg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));   // rows may start at any float

// ---------------------------------------------------------------------------
// Grouping is a counting sort that keeps the order of equal keys.  A wave takes
// a run of entries, counts its experts in an LDS row of its own (integers:
// their order does not matter), the rows are scanned over waves and experts, and
// the wave walks its run again, 64 entries at a time in order: entries of one
// expert find each other by a ballot per bit of the key, and their rank is the
// number of earlier lanes among them.  Entries without an expert have the key E
// and come last.
//
// Few entries are one workgroup's work, in one launch (512 tokens, 8 of 64 experts).
// More are bound by the scattered stores of rows, a cache line per lane, and are
// spread over workgroups: one launch counts each workgroup's experts into rows (all
// of which the last launch writes), a second finds the places, and a third writes
// rows: the call has no workspace, so that rows holds the counts until every
// workgroup has read them (8,192 tokens, 8 of 128 experts: 12.8 us in 64 workgroups).
// launch_expert_groups has the border, with both sides' times.
struct Entries {
    const ExpertGroups &a;
    unsigned k;
    // fewer than 2^31 entries, so that sums of places fit 32 bits
    __device__ __forceinline__ explicit Entries(const ExpertGroups &g) : a(g), k(g.k) {}
    __device__ __forceinline__ unsigned number() const { return (unsigned)a.T * k; }
    __device__ __forceinline__ int key(unsigned i) const {
        const int e = a.ids[a.ldi == a.k ? (int64_t)i : i / k * a.ldi + i % k];
        return e >= 0 && e < a.E ? e : a.E;
    }
    __device__ __forceinline__ int32_t &pos(unsigned i) const {
        return a.pos[a.ldp == a.k ? (int64_t)i : i / k * a.ldp + i % k];
    }
    static constexpr int U = 8;                       // loads in flight
    // adds a run's counts to bin[0 .. E] in LDS
    __device__ __forceinline__ void count(int *bin, unsigned first, unsigned end) const {
        const unsigned lane = threadIdx.x & 63;
        for (unsigned base = first; base < end; base += 64 * U) {
            int e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) e[u] = key(min(base + 64 * u + lane, end - 1));
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (base + 64 * u + lane < end) atomicAdd(bin + e[u], 1);
        }
    }
    // store(i, key, place) for a run whose experts' next places are in `next`, an
    // LDS row of the wave's own
    template <class Store>
    __device__ __forceinline__ void place(int *next, unsigned first, unsigned end, int bits, Store store) const {
        const unsigned lane = threadIdx.x & 63;
        for (unsigned base = first; base < end; base += 64 * U) {
            int e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) e[u] = key(min(base + 64 * u + lane, end - 1));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (base + 64 * u >= end) break;      // uniform
                const unsigned i = base + 64 * u + lane;
                const bool there = i < end;
                uint64_t same = __ballot(there);
                for (int bit = 0; bit < bits; ++bit) {
                    const uint64_t set = __ballot(e[u] >> bit & 1);
                    same &= e[u] >> bit & 1 ? set : ~set;
                }
                if (there) store(i, e[u], next[e[u]] + __popcll(same & ((1ull << lane) - 1)));
                // the last of the equal lanes moves the expert's place on, after
                // all have read it: LDS takes a wave's accesses in order
                in_order();
                if (there && (same >> lane) == 1) next[e[u]] += __popcll(same);
                in_order();
            }
        }
    }
    static __device__ __forceinline__ void in_order() {
#if defined(__HIP_DEVICE_COMPILE__)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#endif
    }
};

// Sums of value(b) over the bins before b, for all bins: out(b, sum), by the
// W waves of a workgroup, a round of their threads at a time.
template <int W, class Value, class Out>
__device__ __forceinline__ void scan_bins(int bins, Value value, Out out) {
    __shared__ int wave_total[W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before = 0;
    for (int b0 = 0; b0 < bins; b0 += 64 * W) {
        const int b = b0 + (int)threadIdx.x, v = b < bins ? value(b) : 0, incl = wave64_scan(v);
        if (lane == 63) wave_total[wave] = incl;
        __syncthreads();
        int start = before + incl - v;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < wave) start += wave_total[w];
            before += wave_total[w];
        }
        if (b < bins) out(b, start);
        __syncthreads();
    }
}

template <int W>
__global__ __launch_bounds__(64 * W) void expert_groups_kernel(ExpertGroups a, int bits) {
    __shared__ int count[W * (MAX_EXPERTS + 1)];      // W rows of E + 1
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int bins = a.E + 1;
    for (int i = threadIdx.x; i < W * bins; i += 64 * W) count[i] = 0;
    __syncthreads();
    const Entries all(a);
    const unsigned n = all.number(), per = ((n + W - 1) / W + 63) / 64 * 64;
    const unsigned first = min(per * wave, n), end = min(first + per, n);
    int *mine = count + wave * bins;
    all.count(mine, first, end);
    __syncthreads();
    // counts to places: over the waves of one expert, then over experts
    const auto over_waves = [&](int b) {
        int total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int c = count[w * bins + b];
            count[w * bins + b] = total;
            total += c;
        }
        return total;
    };
    scan_bins<W>(bins, over_waves, [&](int b, int start) {
#pragma unroll
        for (int w = 0; w < W; ++w) count[w * bins + b] += start;
        a.offsets[b] = start;                         // bin E starts where the last group ends
    });
    all.place(mine, first, end, bits, [&](unsigned i, int e, int at) {
        a.rows[at] = (int)(i / all.k);
        all.pos(i) = e < a.E ? at : -1;
    });
}

// The same over workgroups of PW waves, each with `per` entries, a multiple of
// 64 PW.  Every workgroup adds up the counts of all: a thread per expert, or with 16
// waves as many as there are, so that few loads follow each other.
template <int PW>
__global__ __launch_bounds__(64 * PW) void expert_count_kernel(ExpertGroups a, unsigned per) {
    __shared__ int count[MAX_EXPERTS + 1];
    for (int b = threadIdx.x; b <= a.E; b += 64 * PW) count[b] = 0;
    __syncthreads();
    const Entries all(a);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned first = min(per * blockIdx.x + per / PW * wave, all.number());
    all.count(count, first, min(first + per / PW, all.number()));
    __syncthreads();
    for (int b = threadIdx.x; b <= a.E; b += 64 * PW) a.rows[(int64_t)blockIdx.x * (a.E + 1) + b] = count[b];
}

template <int PW>
__global__ __launch_bounds__(64 * PW) void expert_place_kernel(ExpertGroups a, unsigned per, int bits) {
    constexpr int THREADS = 64 * PW, SUMS = (PW > 4 ? THREADS : 0) + MAX_EXPERTS + 1;
    __shared__ int count[PW * (MAX_EXPERTS + 1)], total[PW > 4 ? SUMS : 1], earlier[SUMS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int bins = a.E + 1, parts = PW > 4 ? max(THREADS / bins, 1) : 1;
    for (int i = threadIdx.x; i < PW * bins; i += THREADS) count[i] = 0;
    // entry i of a table of parts x bins: all entries of expert i % bins in each
    // parts-th workgroup, and those of them in earlier ones
    const auto add_up = [&](int i) {
        const int b = parts > 1 ? i % bins : i;
        int sum = 0, before = 0;
#pragma unroll 8
        for (int g = parts > 1 ? i / bins : 0; g < (int)gridDim.x; g += parts) {
            const int c = a.rows[(int64_t)g * bins + b];
            sum += c;
            before += g < (int)blockIdx.x ? c : 0;
        }
        earlier[i] = before;
        return sum;
    };
    if constexpr (PW > 4)
        for (int i = threadIdx.x; i < parts * bins; i += THREADS) total[i] = add_up(i);
    __syncthreads();
    const Entries all(a);
    const unsigned first = min(per * blockIdx.x + per / PW * wave, all.number());
    const unsigned end = min(first + per / PW, all.number());
    int *mine = count + wave * bins;
    all.count(mine, first, end);
    const auto all_of = [&](int b) {
        if constexpr (PW > 4) {
            int sum = total[b];
            for (int p = 1; p < parts; ++p) sum += total[p * bins + b];
            return sum;
        } else {
            return add_up(b);
        }
    };
    scan_bins<PW>(bins, all_of, [&](int b, int start) {
        if (blockIdx.x == 0) a.offsets[b] = start;
        int at = start;
        for (int p = 0; p < parts; ++p) at += earlier[p * bins + b];
#pragma unroll
        for (int w = 0; w < PW; ++w) {
            const int c = count[w * bins + b];
            count[w * bins + b] = at;
            at += c;
        }
    });
    // no place is -1, so that its complement marks an entry without an expert
    all.place(mine, first, end, bits, [&](unsigned i, int e, int at) { all.pos(i) = e < a.E ? at : ~at; });
}

__global__ __launch_bounds__(256) void expert_rows_kernel(ExpertGroups a) {
    const Entries all(a);
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all.number(); i += (uint64_t)gridDim.x * 256) {
        const int at = all.pos((unsigned)i);
        a.rows[at < 0 ? ~at : at] = (int)((unsigned)i / all.k);
        if (at < 0) all.pos((unsigned)i) = -1;
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
// until the row's end.  Rows are loaded whether an entry has one or not (then
// row 0), so that no load waits for a branch.
template <int W, int J>
__global__ __launch_bounds__(256) void expert_combine_bwd_kernel(ExpertCombineBwd a) {
    constexpr int TOKENS = 4 / W;
    __shared__ float red[4][J];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave / W, part = wave % W;
    const bool read = a.dw && a.M > 0;
    for (int64_t base = (int64_t)blockIdx.x * TOKENS; base < a.T; base += (int64_t)gridDim.x * TOKENS) {
        const bool live = base + sub < a.T;
        const int64_t t = live ? base + sub : a.T - 1;
        const float *dO = a.dO + t * a.ldo;
        for (int j0 = 0; j0 < a.k; j0 = next_run<J>(j0, a.k)) {
            int p[J];
            float f[J], dot[J];
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const int j = min(j0 + i, a.k - 1);
                p[i] = a.pos[t * a.ldp + j];
                f[i] = a.w ? a.w[t * a.ldw + j] : 1.f;
            }
#pragma unroll
            for (int i = 0; i < J; ++i) {
                if (j0 + i >= a.k || p[i] >= a.M || !live) p[i] = -1;
                dot[i] = 0.f;
            }
#pragma unroll 2
            for (int64_t col = part * 256 + 4 * lane; col < a.K; col += W * 256) {
                const v4f d = get(dO, col, a.K);
                v4f y[J];
                if (read)
#pragma unroll
                    for (int i = 0; i < J; ++i) y[i] = get(a.Y + (int64_t)max(p[i], 0) * a.ldy, col, a.K);
#pragma unroll
                for (int i = 0; i < J; ++i) {
                    v4f o;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        o[c] = f[i] * d[c];
                        if (read) dot[i] = __builtin_fmaf(d[c], y[i][c], dot[i]);
                    }
                    if (a.dY && p[i] >= 0) put(a.dY + (int64_t)p[i] * a.lddy, col, a.K, o);
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
                    if (j0 + i < a.k) a.dw[t * a.lddw + j0 + i] = p[i] < 0 ? 0.f : dot[i];
        }
    }
}

// Short rows, of up to 4 TEAM columns: TEAM lanes per token, so that a wave's loads
// serve 64 / TEAM of them.  Entries without a row load row 0 (of one at least) and
// leave it out.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v) {
    return TEAM == 16 ? row16_sum(v) : half32_sum(v);
}

template <int TEAM>
__global__ __launch_bounds__(256) void expert_combine_short_kernel(ExpertCombine a) {
    constexpr int TOKENS = 256 / TEAM;
    const int col = threadIdx.x % TEAM * 4;
    for (int64_t base = (int64_t)blockIdx.x * TOKENS; base < a.T; base += (int64_t)gridDim.x * TOKENS) {
        const int64_t want = base + threadIdx.x / TEAM, t = min(want, (int64_t)a.T - 1);
        v4f sum = {0.f, 0.f, 0.f, 0.f};
        if (a.R) sum = get(a.R + t * a.ldr, col, a.K);
        if (a.M > 0)
#pragma unroll 4
            for (int j = 0; j < a.k; ++j) {
                const int p = a.pos[t * a.ldp + j];
                const float f = a.w ? a.w[t * a.ldw + j] : 1.f;
                const bool there = p >= 0 && p < a.M;
                const v4f y = get(a.Y + (there ? (int64_t)p : 0) * a.ldy, col, a.K);
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = there ? __builtin_fmaf(f, y[c], sum[c]) : sum[c];
            }
        if (want < a.T) put(a.out + t * a.ldo, col, a.K, sum);
    }
}

template <int TEAM>
__global__ __launch_bounds__(256) void expert_combine_bwd_short_kernel(ExpertCombineBwd a) {
    constexpr int TOKENS = 256 / TEAM, J = 4;
    const int col = threadIdx.x % TEAM * 4;
    const bool read = a.dw && a.M > 0;
    for (int64_t base = (int64_t)blockIdx.x * TOKENS; base < a.T; base += (int64_t)gridDim.x * TOKENS) {
        const int64_t want = base + threadIdx.x / TEAM, t = min(want, (int64_t)a.T - 1);
        const v4f d = get(a.dO + t * a.ldo, col, a.K);
        for (int j0 = 0; j0 < a.k; j0 = next_run<J>(j0, a.k)) {
            int p[J];
            v4f y[J];
            float f[J];
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const int j = min(j0 + i, a.k - 1);
                p[i] = a.pos[t * a.ldp + j];
                f[i] = a.w ? a.w[t * a.ldw + j] : 1.f;
                if (want >= a.T || j0 + i >= a.k || p[i] >= a.M) p[i] = -1;
            }
#pragma unroll
            for (int i = 0; i < J; ++i) {
                y[i] = v4f{0.f, 0.f, 0.f, 0.f};
                if (read) y[i] = get(a.Y + (int64_t)max(p[i], 0) * a.ldy, col, a.K);
            }
#pragma unroll
            for (int i = 0; i < J; ++i) {
                v4f o;
                float dot = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[c] = f[i] * d[c];
                    dot = __builtin_fmaf(d[c], y[i][c], dot);
                }
                if (a.dY && p[i] >= 0) put(a.dY + (int64_t)p[i] * a.lddy, col, a.K, o);
                if (a.dw == nullptr) continue;        // uniform
                dot = team_sum<TEAM>(dot);
                if (want < a.T && j0 + i < a.k && col == 0) a.dw[t * a.lddw + j0 + i] = p[i] < 0 ? 0.f : dot;
            }
        }
    }
}

constexpr int64_t MAX_GROUPS = 1 << 20;
inline unsigned groups(int64_t n) { return (unsigned)(n < MAX_GROUPS ? n : MAX_GROUPS); }

template <int PW>
hipError_t count_and_place(const ExpertGroups &a, int64_t n, int64_t groups, int bits, hipStream_t s) {
    const unsigned per = (unsigned)(((n + groups - 1) / groups + 64 * PW - 1) / (64 * PW) * (64 * PW));
    const unsigned grid = (unsigned)((n + per - 1) / per);
    const hipError_t e = launch(expert_count_kernel<PW>, dim3(grid), dim3(64 * PW), s, a, per);
    return e == hipSuccess ? launch(expert_place_kernel<PW>, dim3(grid), dim3(64 * PW), s, a, per, bits) : e;
}

}  // namespace

hipError_t launch_expert_groups(const ExpertGroups &a, hipStream_t s) {
    int bits = 0;
    while (a.E >> bits) ++bits;                       // keys up to E
    const int64_t n = (int64_t)a.T * a.k;
    // one workgroup: of four waves for the few entries of generated tokens (8
    // entries of 64 experts 3.1 us, on 16 waves 3.8; 512 3.8 / 4.2; 768 4.2 / 4.3)
    if (n <= 768) return launch(expert_groups_kernel<4>, dim3(1), dim3(256), s, a, bits);
    // or several, of 1,024 entries and more, as many as their counts fit into rows,
    // where there are 8 at least (8192 entries of 64 experts 9.5 us, 10.2 in one; 4096
    // 10.2 / 7.2); each reads the counts of all, so up to 128, or one per 4,096
    // entries (on 4 waves each, 262,144 of 256 experts 22.4, in 64 23.4, in 256 28.3;
    // 1,048,576 of 128 in 256 35.3, in 128 40.4)
    const int64_t room = n / (a.E + 1), cap = n >= 4096 * 256 ? 256 : n >= 4096 * 128 ? n / 4096 : 128;
    const int64_t most = n / 1024 < cap ? n / 1024 : cap, groups = room < most ? room : most;
    if (groups < 8) return launch(expert_groups_kernel<16>, dim3(1), dim3(1024), s, a, bits);
    // 16 waves each where entries or experts are many (262,144 entries of 256 experts
    // 17.0 us, 22.5 on 4; 100,000 of 64 12.4 / 14.9; 65,536 of 1,000 16.4 / 23.7, of 128
    // 13.2 / 12.5; 8192 of 8 11.2 / 8.9; 96,000 of 64 12.1 / 13.9)
    hipError_t e = n >= 81920 || a.E >= 512 ? count_and_place<16>(a, n, groups, bits, s)
                                            : count_and_place<4>(a, n, groups, bits, s);
    if (e == hipSuccess)
        e = launch(expert_rows_kernel, dim3((unsigned)(n < (1 << 20) ? (n + 255) / 256 : 4096)), dim3(256), s, a);
    return e;
}

// Threads per token where rows are short (us, 8192 tokens of 8 entries, on 16 or 32
// threads and on a wave: K = 64 5.6 / 13.0, gradients 7.6 / 21.9; K = 128 7.9 / 17.9,
// gradients 13.6 / 25.5; one token of 8, K = 64: 3.5 / 3.9, gradients 4.2 / 6.1).
int team_of(int K) { return K <= 64 ? 16 : K <= 128 ? 32 : 0; }

hipError_t launch_expert_combine(const ExpertCombine &a, hipStream_t s) {
    if (const int team = team_of(a.K)) {
        const dim3 grid(groups(((int64_t)a.T * team + 255) / 256));
        return launch(team == 16 ? expert_combine_short_kernel<16> : expert_combine_short_kernel<32>, grid, dim3(256), s, a);
    }
    // four spans per wave where that still gives every SIMD a wave, else one
    const int64_t wide = ((int64_t)a.K + 1023) / 1024, narrow = ((int64_t)a.K + 255) / 256;
    if (wide * a.T >= 4096)
        return launch(expert_combine_kernel<4>, dim3(groups((wide * a.T + 3) / 4)), dim3(256), s, a, (int)wide);
    return launch(expert_combine_kernel<1>, dim3(groups((narrow * a.T + 3) / 4)), dim3(256), s, a, (int)narrow);
}

template <int W>
hipError_t combine_bwd(const ExpertCombineBwd &a, hipStream_t s) {
    const dim3 grid(groups(((int64_t)a.T + 4 / W - 1) / (4 / W)));
    if (a.k == 1) return launch(expert_combine_bwd_kernel<W, 1>, grid, dim3(256), s, a);
    if (a.k == 2) return launch(expert_combine_bwd_kernel<W, 2>, grid, dim3(256), s, a);
    if (a.k <= 4) return launch(expert_combine_bwd_kernel<W, 4>, grid, dim3(256), s, a);
    return launch(expert_combine_bwd_kernel<W, 8>, grid, dim3(256), s, a);
}

hipError_t launch_expert_combine_bwd(const ExpertCombineBwd &a, hipStream_t s) {
    if (const int team = team_of(a.K)) {
        const dim3 grid(groups(((int64_t)a.T * team + 255) / 256));
        return launch(team == 16 ? expert_combine_bwd_short_kernel<16> : expert_combine_bwd_short_kernel<32>, grid,
                      dim3(256), s, a);
    }
    // four waves per token where each has a span, or where tokens are few (us, in
    // one wave / in four: 8192 tokens, 2 entries, 2048 columns 70 / 62; 8192, 8, 512
    // 58 / 88; 2048, 2, 768 6.5 / 7.8; 346, 2, 768 4.5 / 4.0; 1, 8, 1536 12.6 / 7.3)
    if (a.K >= 1024 || (a.K > 256 && a.T < 1024)) return combine_bwd<4>(a, s);
    return combine_bwd<1>(a, s);
}

}  // namespace gg
