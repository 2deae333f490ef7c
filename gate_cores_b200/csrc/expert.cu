// Tokens to their experts and back.  A slot is one of the top_k choices of a
// token, slot s = t * top_k + j; the rows of an expert are its slots in slot
// order, the experts one after the other.
//
// Sort: a stable counting sort over at most 1024 experts.  Each CTA takes a
// contiguous run of slots and each of its warps a contiguous part of the run.
// A warp counts its part per expert, 32 slots at a time (lanes with the same
// expert find one another with a warp match; the lowest of them adds for all).
// The counts become start positions by an exclusive sum over warps, CTAs and
// experts, and a second walk of the same slots hands out positions from them
// in slot order.  Only integers are added and each in a fixed order of its
// own counter, so the result is the same every time.  More than one CTA: a
// first kernel leaves every CTA's counts in the workspace and every CTA of the
// second adds up the ones before its own (at most 512 rows of num_experts
// integers from L2: a third launch for the sums would cost more).
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

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const __grid_constant__ ExpertSortArgs a) {
    pdl_begin();
    extern __shared__ int counts[];
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads) counts[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * a.run, s1 = min(s0 + a.run, a.slots);
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kSortThreads) {
        const int e = slot_expert(a, s);
        if (e >= 0) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.num_experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.num_experts + e] = counts[e];
}

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const __grid_constant__ ExpertSortArgs a) {
    pdl_begin();
    // at[w][e]: first the count, then the next position of warp w's slots of expert e (odd stride: a column of it is
    // read by the lanes of one warp); before[e], total[e]: slots of e in earlier CTAs, in all
    extern __shared__ int smem[];
    const int E = a.num_experts, stride = E | 1;
    int* at = smem;
    int* before = smem + kSortWarps * stride;
    int* total = before + E;
    __shared__ int kept;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kSortWarps * stride + 2 * E; i += kSortThreads) smem[i] = 0;
    __syncthreads();
    const int part = a.run / kSortWarps;  // a multiple of 32
    const int64_t s0 = (int64_t)blockIdx.x * a.run + (int64_t)warp * part;
    const int64_t s1 = min(s0 + part, a.slots);
    int* mine = at + warp * stride;
    const unsigned below = (1u << lane) - 1u;
    for (int64_t b = s0; b < s1; b += 32) {
        const int e = slot_expert(a, b + lane);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
    }
    if (gridDim.x > 1) {
        for (int c = warp; c < (int)gridDim.x; c += kSortWarps)
            for (int e = lane; e < E; e += 32) {
                const int n = __ldcg(a.counts + (int64_t)c * E + e);
                if (n) {
                    atomicAdd(&total[e], n);
                    if (c < (int)blockIdx.x) atomicAdd(&before[e], n);
                }
            }
    }
    __syncthreads();
    // exclusive sums over the warps, an expert a warp
    for (int e = warp; e < E; e += kSortWarps) {
        int n;
        const int s = warp_scan(at[lane * stride + e], lane, n);
        at[lane * stride + e] = s;
        if (lane == 0 && gridDim.x == 1) total[e] = n;
    }
    __syncthreads();
    // and over the experts: before[e] becomes this CTA's first position of expert e
    if (warp == 0) {
        int base = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int n;
            const int s = warp_scan(e < E ? total[e] : 0, lane, n);
            if (e < E) {
                before[e] += base + s;
                if (blockIdx.x == 0) a.group_offsets[e] = base + s;
            }
            base += n;
        }
        if (lane == 0) {
            kept = base;
            if (blockIdx.x == 0) a.group_offsets[E] = base;
        }
    }
    __syncthreads();
    for (int64_t b = s0; b < s1; b += 32) {
        const int64_t s = b + lane;
        const int e = slot_expert(a, s);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = before[e] + mine[e] + __popc(same & below);
        __syncwarp();
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
        if (s < s1) {
            a.row_of_slot[s] = row;
            if (row >= 0) a.slot_of_row[row] = (int)s;
            if (s >= kept) a.slot_of_row[s] = -1;  // the rows behind the last group
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

// Slots a CTA takes, a multiple of 1024 (32 a warp's step), and how many CTAs that makes.
struct SortShape {
    int64_t run, ctas;
};
constexpr int64_t kSortRun = 4096;
constexpr int64_t kSortMaxCtas = 512;
SortShape sort_shape(int64_t slots) {
    int64_t run = kSortRun;
    if (slots > kSortRun * kSortMaxCtas) run = ((slots + kSortMaxCtas - 1) / kSortMaxCtas + 1023) / 1024 * 1024;
    return SortShape{run, (slots + run - 1) / run};
}

}  // namespace

size_t expert_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
    const SortShape sh = sort_shape(slots);
    return sh.ctas > 1 ? (size_t)sh.ctas * (size_t)num_experts * sizeof(int32_t) : 0;
}

cudaError_t launch_expert_sort(ExpertSortArgs a, cudaStream_t s) {
    const SortShape sh = sort_shape(a.slots);
    a.run = (int32_t)sh.run;
    if (sh.ctas > 1) {
        const cudaError_t e = launch_pdl(expert_count_kernel, (unsigned)sh.ctas, kSortThreads, (size_t)a.num_experts * 4, s, a);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = ((size_t)kSortWarps * (size_t)(a.num_experts | 1) + 2 * (size_t)a.num_experts) * 4;
    if (smem > 40 * 1024) {  // above the default 48 KB once the static part is added
        const cudaError_t e = cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(expert_place_kernel, (unsigned)sh.ctas, kSortThreads, smem, s, a);
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
