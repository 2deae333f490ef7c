// Tokens to their experts and back.  A slot is one of the top_k choices of a
// token, slot s = t * top_k + j; the rows of an expert are its slots in slot
// order, the experts one after the other.
//
// Sort: a stable counting sort over at most 1024 experts.  A CTA takes runs of
// 4096 slots, each of its 32 warps 128 consecutive ones of a run in four
// steps.  In a step the lanes with one expert find one another by a ballot
// for each bit of the expert's number; a lane's rank is the warp's count of
// that expert so far plus its equals in lower lanes, and the lowest of them
// moves the count on.  Exclusive sums of the counts over warps, CTAs and
// experts turn ranks into rows.  Only integers are added, so the result is the
// same every time.  More than one CTA: a first kernel leaves every CTA's
// counts in the workspace and every CTA of the second adds up the ones before
// its own (at most 512 rows of num_experts integers from L2).
#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

// The expert of slot s, or -1 when the slot is dropped.
__device__ __forceinline__ int slot_expert(const ExpertSortArgs& a, int64_t s) {
    if (s >= a.slots) return -1;
    const int64_t e = a.ids64 ? __ldg(static_cast<const long long*>(a.ids) + s) : (int64_t)__ldg(static_cast<const int*>(a.ids) + s);
    return e >= 0 && e < a.num_experts ? (int)e : -1;
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

constexpr int kSortSteps = 4;
constexpr int kSortRun = kSortThreads * kSortSteps;

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const __grid_constant__ ExpertSortArgs a) {
    pdl_begin();
    extern __shared__ int counts[];
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads) counts[e] = 0;
    __syncthreads();
    for (int run = 0; run < a.runs; ++run) {
        const int64_t s0 = ((int64_t)blockIdx.x * a.runs + run) * kSortRun + threadIdx.x;
        int e[kSortSteps];
#pragma unroll
        for (int b = 0; b < kSortSteps; ++b) e[b] = slot_expert(a, s0 + b * kSortThreads);
#pragma unroll
        for (int b = 0; b < kSortSteps; ++b)
            if (e[b] >= 0) atomicAdd(&counts[e[b]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.num_experts + e] = counts[e];
}

// Lanes of the warp whose expert is e too (for lanes with an expert); `bits`
// of an expert's number count.
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, e >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool set = (e >> b) & 1;
        const unsigned m = __ballot_sync(0xffffffffu, set);
        same &= set ? m : ~m;
    }
    return same;
}

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const __grid_constant__ ExpertSortArgs a) {
    pdl_begin();
    // at[w][e]: warp w's slots of expert e in this run, then the number of
    // them in lower warps (odd stride: a column is read by the lanes of one
    // warp); first[e]: the row of this CTA's next slot of e; total[e]: slots
    // of e in all, then in this run
    extern __shared__ int smem[];
    const int E = a.num_experts, stride = E | 1;
    int* at = smem;
    int* first = smem + kSortWarps * stride;
    int* total = first + E;
    __shared__ int kept;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = gridDim.x == 1;
    int* mine = at + warp * stride;
    const unsigned below = (1u << lane) - 1u;
    for (int i = threadIdx.x; i < kSortWarps * stride + 2 * E; i += kSortThreads) smem[i] = 0;
    __syncthreads();
    if (!alone) {
        // a warp takes every 32nd CTA's counts, a lane an expert
        constexpr int U = 8;
        for (int e = lane; e < E; e += 32) {
            int all = 0, before = 0;
            for (int c0 = warp; c0 < (int)gridDim.x; c0 += kSortWarps * U) {
                int n[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * kSortWarps;
                    n[u] = c < (int)gridDim.x ? __ldcg(a.counts + (int64_t)c * E + e) : 0;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    all += n[u];
                    before += c0 + u * kSortWarps < (int)blockIdx.x ? n[u] : 0;
                }
            }
            if (all) atomicAdd(&total[e], all);
            if (before) atomicAdd(&first[e], before);
        }
    }
    for (int run = 0; run < a.runs; ++run) {
        const int64_t s0 = ((int64_t)blockIdx.x * a.runs + run) * kSortRun + warp * (32 * kSortSteps) + lane;
        int e[kSortSteps], rank[kSortSteps];
#pragma unroll
        for (int b = 0; b < kSortSteps; ++b) e[b] = slot_expert(a, s0 + b * 32);
#pragma unroll
        for (int b = 0; b < kSortSteps; ++b) {
            const unsigned same = same_expert(e[b], a.expert_bits);
            const bool has = e[b] >= 0;
            rank[b] = has ? mine[e[b]] + __popc(same & below) : 0;
            __syncwarp();
            if (has && (same & below) == 0) mine[e[b]] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // exclusive sums over the warps, an expert a warp
        for (int x = warp; x < E; x += kSortWarps) {
            int n;
            at[lane * stride + x] = warp_scan(at[lane * stride + x], lane, n);
            if (lane == 0 && alone) total[x] = n;
        }
        __syncthreads();
        if (run == 0) {
            // and over the experts
            if (warp == 0) {
                int base = 0;
                for (int x0 = 0; x0 < E; x0 += 32) {
                    const int x = x0 + lane;
                    int n;
                    const int s = warp_scan(x < E ? total[x] : 0, lane, n);
                    if (x < E) {
                        first[x] += base + s;
                        if (blockIdx.x == 0) a.group_offsets[x] = base + s;
                    }
                    base += n;
                }
                if (lane == 0) {
                    kept = base;
                    if (blockIdx.x == 0) a.group_offsets[E] = base;
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int b = 0; b < kSortSteps; ++b) {
            const int64_t s = s0 + b * 32;
            if (s >= a.slots) continue;
            const int row = e[b] >= 0 ? first[e[b]] + mine[e[b]] + rank[b] : -1;
            a.row_of_slot[s] = row;
            if (row >= 0) a.slot_of_row[row] = (int)s;
            if (s >= kept) a.slot_of_row[s] = -1;  // the rows behind the last group
        }
        if (run + 1 < a.runs) {
            // the next run's slots come behind this one's
            __syncthreads();
            for (int x = threadIdx.x; x < E; x += kSortThreads) total[x] = 0;
            __syncthreads();
#pragma unroll
            for (int b = 0; b < kSortSteps; ++b)
                if (e[b] >= 0) atomicAdd(&total[e[b]], 1);
            __syncthreads();
            for (int x = threadIdx.x; x < E; x += kSortThreads) first[x] += total[x];
            for (int i = threadIdx.x; i < kSortWarps * stride; i += kSortThreads) at[i] = 0;
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

// CTAs of the sort, and runs a CTA takes: one run each up to 512 CTAs.
constexpr int64_t kSortMaxCtas = 512;
int64_t sort_runs(int64_t slots) { return (slots + kSortRun * kSortMaxCtas - 1) / (kSortRun * kSortMaxCtas); }
int64_t sort_ctas(int64_t slots) {
    const int64_t per = sort_runs(slots) * kSortRun;
    return (slots + per - 1) / per;
}

}  // namespace

size_t expert_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
    const int64_t n = sort_ctas(slots);
    return n > 1 ? (size_t)n * (size_t)num_experts * sizeof(int32_t) : 0;
}

cudaError_t launch_expert_sort(ExpertSortArgs a, cudaStream_t s) {
    const unsigned ctas = (unsigned)sort_ctas(a.slots);
    a.runs = (int32_t)sort_runs(a.slots);
    a.expert_bits = 0;
    while ((1 << a.expert_bits) < a.num_experts) ++a.expert_bits;
    if (ctas > 1) {
        const cudaError_t e = launch_pdl(expert_count_kernel, ctas, kSortThreads, (size_t)a.num_experts * 4, s, a);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = ((size_t)kSortWarps * (size_t)(a.num_experts | 1) + 2 * (size_t)a.num_experts) * 4;
    if (smem > 40 * 1024) {  // above the default 48 KB once the static part is added
        const cudaError_t e = cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(expert_place_kernel, ctas, kSortThreads, smem, s, a);
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
