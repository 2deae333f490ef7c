// Tokens to their experts and back.  A slot is one of the top_k choices of a
// token, slot s = t * top_k + j; the rows of an expert are its slots in slot
// order, the experts one after the other.
//
// Sort: a stable counting sort over at most 1024 experts.  A CTA takes runs of
// 1024 or 4096 slots, each of its 16 warps consecutive ones of a run in two or
// eight steps of 32.  In a step the lanes with one expert find one another by a
// ballot for each bit of the expert's number; a lane's rank is the warp's
// count of that expert so far plus its equals in lower lanes, and the lowest of
// them moves the count on.  Exclusive sums of the counts over warps, CTAs and
// experts turn ranks into rows.  The slots of the rows are put in order in
// shared memory first, so that an expert's leave the CTA together.  Only
// integers are added, so the result is the same every time.  More than one
// CTA: a first kernel leaves every CTA's counts in the workspace and every CTA
// of the second adds up the ones before its own (at most 512 rows of
// num_experts integers from L2).
//
// Bound: latency, a chain of loads, shared memory and barriers.  What depends
// on nothing is therefore done for all steps at once.
#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMany = 8;  // steps of a warp in a run, with many slots
constexpr int kSortFew = 2;   // and with few

// The experts of this lane's slots s, s + apart, ... (-1: dropped, or behind the last slot).
template <int N>
__device__ __forceinline__ void slot_experts(const ExpertSortArgs& a, int64_t s, int apart, int (&e)[N]) {
    int64_t id[N];
    if (a.ids64) {
#pragma unroll
        for (int b = 0; b < N; ++b) id[b] = __ldg(static_cast<const long long*>(a.ids) + min(s + b * apart, a.slots - 1));
    } else {
#pragma unroll
        for (int b = 0; b < N; ++b) id[b] = __ldg(static_cast<const int*>(a.ids) + min(s + b * apart, a.slots - 1));
    }
#pragma unroll
    for (int b = 0; b < N; ++b) e[b] = s + b * apart < a.slots && id[b] >= 0 && id[b] < a.num_experts ? (int)id[b] : -1;
}

// Exclusive sum over the warp; total gets the sum.
__device__ __forceinline__ int warp_scan(int v, int lane, int& total) {
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return s - v;
}

template <int STEPS>
__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const __grid_constant__ ExpertSortArgs a) {
    pdl_wait();
    pdl_next();  // the second kernel ranks its slots meanwhile
    extern __shared__ int counts[];
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads) counts[e] = 0;
    __syncthreads();
    for (int run = 0; run < a.runs; ++run) {
        int e[STEPS];
        slot_experts<STEPS>(a, ((int64_t)blockIdx.x * a.runs + run) * (STEPS * kSortThreads) + threadIdx.x, kSortThreads, e);
#pragma unroll
        for (int b = 0; b < STEPS; ++b)
            if (e[b] >= 0) atomicAdd(&counts[e[b]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.num_experts + e] = counts[e];
}

// Exclusive sums of n[0 .. E) by one warp, given to out(e, sum); returns the
// sum of all.  A lane takes E / 32 neighbours.
template <typename F> __device__ __forceinline__ int expert_scan(const int* n, int E, int lane, F&& out) {
    const int per = (E + 31) >> 5, e0 = lane * per;
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += e0 + i < E ? n[e0 + i] : 0;
    int all;
    int s = warp_scan(mine, lane, all);
    for (int i = 0; i < per; ++i) {
        if (e0 + i >= E) break;
        const int v = n[e0 + i];
        out(e0 + i, s);
        s += v;
    }
    return all;
}

template <int STEPS>
__global__ void __launch_bounds__(kSortThreads, 2) expert_place_kernel(const __grid_constant__ ExpertSortArgs a) {
    // at[w][e]: warp w's slots of expert e in this run, then the number of
    // them in lower warps; mine[e]: this CTA's slots of e in this run;
    // place[e]: the first of their places among the run's; first[e]: the row of
    // the CTA's next slot of e; total[e]: slots of e in all; order: the run's
    // (slot, row) in row order
    constexpr int kRun = kSortThreads * STEPS;
    extern __shared__ __align__(8) int smem[];
    const int E = a.num_experts;
    int2* order = reinterpret_cast<int2*>(smem);
    int* place = reinterpret_cast<int*>(order + kRun);
    int* first = place + E;
    int* total = first + E;
    int* mine = total + E;
    int* at = mine + E;
    __shared__ int kept, here;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = gridDim.x == 1;
    int* counts = at + warp * E;
    const unsigned below = (1u << lane) - 1u;
    pdl_next();
    // with a first kernel, which has waited, only its counts are to be waited for
    if (alone) pdl_wait();
    int64_t s0 = (int64_t)blockIdx.x * a.runs * kRun + warp * (32 * STEPS) + lane;
    int e[STEPS];
    slot_experts<STEPS>(a, s0, 32, e);
    for (int i = threadIdx.x; i < (kSortWarps + 3) * E; i += kSortThreads) first[i] = 0;
    __syncthreads();
    for (int run = 0; run < a.runs; ++run, s0 += kRun) {
        if (run > 0) slot_experts<STEPS>(a, s0, 32, e);
        unsigned same[STEPS];
#pragma unroll
        for (int b = 0; b < STEPS; ++b) same[b] = __ballot_sync(0xffffffffu, e[b] >= 0);
        for (int bit = 0; bit < a.expert_bits; ++bit) {
#pragma unroll
            for (int b = 0; b < STEPS; ++b) {
                const bool set = (e[b] >> bit) & 1;
                const unsigned m = __ballot_sync(0xffffffffu, set);
                same[b] &= set ? m : ~m;
            }
        }
        int rank[STEPS];
#pragma unroll
        for (int b = 0; b < STEPS; ++b) {
            const int low = __popc(same[b] & below);
            rank[b] = e[b] >= 0 ? counts[e[b]] + low : 0;
            __syncwarp();
            if (e[b] >= 0 && low == 0) counts[e[b]] = rank[b] + __popc(same[b]);
            __syncwarp();
        }
        __syncthreads();
        // exclusive sums over the warps, an expert a thread
        for (int x = threadIdx.x; x < E; x += kSortThreads) {
            int n[kSortWarps], s = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) n[w] = at[w * E + x];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                at[w * E + x] = s;
                s += n[w];
            }
            mine[x] = s;
            if (alone) total[x] = s;
        }
        if (run == 0 && !alone) {
            pdl_wait();
            // the CTAs' counts: a thread takes a column of every so manieth CTA
            constexpr int U = 16;
            const int cols = (min(E, kSortThreads) + 31) & ~31, rows = kSortThreads / cols;
            const int r0 = (int)threadIdx.x / cols;
            for (int x = (int)threadIdx.x % cols; x < E && r0 < rows; x += cols) {
                int all = 0, before = 0;
                for (int c0 = r0; c0 < (int)gridDim.x; c0 += rows * U) {
                    int n[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int c = c0 + u * rows;
                        n[u] = c < (int)gridDim.x ? __ldcg(a.counts + c * E + x) : 0;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        all += n[u];
                        before += c0 + u * rows < (int)blockIdx.x ? n[u] : 0;
                    }
                }
                atomicAdd(&total[x], all);
                atomicAdd(&first[x], before);
            }
        }
        __syncthreads();
        // and over the experts: of this run, and (once) of all
        if (warp == 0) {
            const int n = expert_scan(mine, E, lane, [&](int x, int s) { place[x] = s; });
            if (lane == 0) here = n;
        } else if (warp == 1 && run == 0) {
            const int n = expert_scan(total, E, lane, [&](int x, int s) {
                first[x] += s;
                if (blockIdx.x == 0) a.group_offsets[x] = s;
            });
            if (lane == 0) {
                kept = n;
                if (blockIdx.x == 0) a.group_offsets[E] = n;
            }
        }
        __syncthreads();
        int row[STEPS], to[STEPS];
#pragma unroll
        for (int b = 0; b < STEPS; ++b) {
            const int x = e[b] < 0 ? 0 : e[b];
            const int in = counts[x] + rank[b];
            row[b] = e[b] < 0 ? -1 : first[x] + in;
            to[b] = place[x] + in;
        }
        const int behind = kept;
#pragma unroll
        for (int b = 0; b < STEPS; ++b) {
            const int64_t s = s0 + b * 32;
            if (row[b] >= 0) order[to[b]] = make_int2((int)s, row[b]);
            if (s < a.slots) {
                a.row_of_slot[s] = row[b];
                if (s >= behind) a.slot_of_row[s] = -1;  // the rows behind the last group
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < here; i += kSortThreads) a.slot_of_row[order[i].y] = order[i].x;
        if (run + 1 < a.runs) {
            // the next run's slots come behind this one's
            for (int x = threadIdx.x; x < E; x += kSortThreads) first[x] += mine[x];
            for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) at[i] = 0;
            __syncthreads();
        }
    }
}

// ---- rows

// A row index inside [0, num_rows), or -1.
__device__ __forceinline__ int64_t row_at(const ExpertRowsArgs& a, int64_t slot) {
    const int r = __ldg(a.row_of_slot + slot);
    return r >= 0 && r < a.num_rows ? r : -1;
}

constexpr int kRowThreads = 256;

// rows[r(t, j)] = x[t]: a thread reads one 16-byte vector of a token and writes it to each of its rows.
__global__ void __launch_bounds__(kRowThreads) expert_dispatch_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    const int64_t n = a.tokens * a.nvec;
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kRowThreads) {
        const int64_t t = i / a.nvec;
        const int v = (int)(i - t * a.nvec);
        const uint4 x = ld_stream(a.token_in + t * a.token_bytes + (int64_t)v * 16);
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t r = row_at(a, t * a.top_k + j);
            if (r >= 0) st_vec(a.rows_out + r * a.rows_out_bytes + (int64_t)v * 16, x);
        }
    }
}

// y[t] = cast(sum_j w[t, j] rows[r(t, j)]), FP32, in the order of j.
template <typename T, bool W>
__global__ void __launch_bounds__(kRowThreads) expert_combine_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    constexpr int B = 4;
    const int64_t n = a.tokens * a.nvec;
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kRowThreads) {
        const int64_t t = i / a.nvec;
        const int v = (int)(i - t * a.nvec);
        float acc[V];
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
        for (int j0 = 0; j0 < a.top_k; j0 += B) {
            uint4 x[B];
            float w[B];
#pragma unroll
            for (int u = 0; u < B; ++u) {
                const int64_t s = t * a.top_k + j0 + u;
                const int64_t r = j0 + u < a.top_k ? row_at(a, s) : -1;
                x[u] = make_uint4(0, 0, 0, 0);
                w[u] = 0.0f;
                if (r >= 0) {
                    x[u] = ld_stream(a.rows_in + r * a.rows_in_bytes + (int64_t)v * 16);
                    w[u] = W ? __ldg(a.weights + s) : 1.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < B; ++u) {
                float f[V];
                unpack<T>(x[u], f);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = W ? fmaf(w[u], f[e], acc[e]) : acc[e] + f[e];
            }
        }
        st_vec(a.token_out + t * a.token_bytes + (int64_t)v * 16, pack<T>(acc));
    }
}

// drows[r(t, j)] = cast(w[t, j] dy[t]); dw[t, j] = <dy[t], rows[r(t, j)]>, one CTA a token.
template <typename T, bool W, bool DW>
__global__ void __launch_bounds__(kRowThreads) expert_combine_bwd_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    __shared__ float red[2][32];
    int bank = 0;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t s = t * a.top_k + j;
            const int64_t r = row_at(a, s);
            // plain loads of what the outputs may overwrite (dweights over
            // weights, drows over rows): the compiler keeps them ahead of the
            // stores to the same place, as it need not with read-only loads
            const float w = W ? a.weights[s] : 1.0f;
            float dot = 0.0f;
            if (r >= 0) {
                for (int v = threadIdx.x; v < a.nvec; v += blockDim.x) {
                    const uint4 g4 = ld_stream(a.token_in + t * a.token_bytes + (int64_t)v * 16);
                    float g[V], o[V];
                    unpack<T>(g4, g);
                    if constexpr (DW) {
                        float x[V];
                        unpack<T>(*reinterpret_cast<const uint4*>(a.rows_in + r * a.rows_in_bytes + (int64_t)v * 16), x);
#pragma unroll
                        for (int e = 0; e < V; ++e) dot = fmaf(g[e], x[e], dot);
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = w * g[e];
                    st_vec(a.rows_out + r * a.rows_out_bytes + (int64_t)v * 16, W ? pack<T>(o) : g4);
                }
            }
            if constexpr (DW) {
                dot = block_sum(dot, red, bank);
                if (threadIdx.x == 0) a.dweights[s] = dot;
            }
        }
    }
}

unsigned row_grid(const ExpertRowsArgs& a) {
    const int64_t n = (a.tokens * a.nvec + kRowThreads - 1) / kRowThreads;
    return (unsigned)(n < 0x7fffffff ? n : 0x7fffffff);
}

template <typename T>
cudaError_t launch_combine_bwd(const ExpertRowsArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.tokens < 0x7fffffff ? a.tokens : 0x7fffffff);
    const unsigned threads = a.nvec >= kRowThreads ? kRowThreads : (a.nvec + 31) / 32 * 32;
    if (a.weights)
        return a.dweights ? launch_pdl(expert_combine_bwd_kernel<T, true, true>, grid, threads, 0, s, a)
                          : launch_pdl(expert_combine_bwd_kernel<T, true, false>, grid, threads, 0, s, a);
    return a.dweights ? launch_pdl(expert_combine_bwd_kernel<T, false, true>, grid, threads, 0, s, a)
                      : launch_pdl(expert_combine_bwd_kernel<T, false, false>, grid, threads, 0, s, a);
}

// Shape of the sort.  One CTA up to a run of eight steps (a second launch would
// cost more than the steps); then as many CTAs of two steps as there are slots
// for, up to 148, or of eight steps, up to 512, and more runs at last.  (The
// number of SMs is not asked for: the workspace's size must not depend on the
// current device.)
struct SortShape {
    int64_t steps, runs, ctas;
};
SortShape sort_shape(int64_t slots) {
    SortShape s{kSortFew, 1, 1};
    if (slots > kSortThreads * kSortFew && (slots <= kSortThreads * kSortMany || slots > kSortThreads * kSortFew * 148))
        s.steps = kSortMany;
    const int64_t run = s.steps * kSortThreads;
    s.runs = (slots + run * 512 - 1) / (run * 512);
    s.ctas = (slots + run * s.runs - 1) / (run * s.runs);
    return s;
}

template <int STEPS> cudaError_t launch_sort(const ExpertSortArgs& a, unsigned ctas, cudaStream_t s) {
    if (ctas > 1) {
        const cudaError_t e = launch_pdl(expert_count_kernel<STEPS>, ctas, kSortThreads, (size_t)a.num_experts * 4, s, a);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = ((size_t)2 * STEPS * kSortThreads + (size_t)(kSortWarps + 4) * (size_t)a.num_experts) * 4;
    const cudaError_t e = allow_smem((const void*)expert_place_kernel<STEPS>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(expert_place_kernel<STEPS>, ctas, kSortThreads, smem, s, a);
}

}  // namespace

size_t expert_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
    const int64_t n = sort_shape(slots).ctas;
    return n > 1 ? (size_t)n * (size_t)num_experts * sizeof(int32_t) : 0;
}

cudaError_t launch_expert_sort(ExpertSortArgs a, cudaStream_t s) {
    const SortShape sh = sort_shape(a.slots);
    a.runs = (int32_t)sh.runs;
    a.expert_bits = 0;
    while ((1 << a.expert_bits) < a.num_experts) ++a.expert_bits;
    return sh.steps == kSortFew ? launch_sort<kSortFew>(a, (unsigned)sh.ctas, s)
                                : launch_sort<kSortMany>(a, (unsigned)sh.ctas, s);
}

cudaError_t launch_expert_dispatch(const ExpertRowsArgs& a, cudaStream_t s) {
    return launch_pdl(expert_dispatch_kernel, row_grid(a), kRowThreads, 0, s, a);
}

cudaError_t launch_expert_combine(int dtype, const ExpertRowsArgs& a, cudaStream_t s) {
    if (dtype == 0)
        return a.weights ? launch_pdl(expert_combine_kernel<__nv_bfloat16, true>, row_grid(a), kRowThreads, 0, s, a)
                         : launch_pdl(expert_combine_kernel<__nv_bfloat16, false>, row_grid(a), kRowThreads, 0, s, a);
    return a.weights ? launch_pdl(expert_combine_kernel<float, true>, row_grid(a), kRowThreads, 0, s, a)
                     : launch_pdl(expert_combine_kernel<float, false>, row_grid(a), kRowThreads, 0, s, a);
}

cudaError_t launch_expert_combine_bwd(int dtype, const ExpertRowsArgs& a, cudaStream_t s) {
    return dtype == 0 ? launch_combine_bwd<__nv_bfloat16>(a, s) : launch_combine_bwd<float>(a, s);
}

}  // namespace muse
