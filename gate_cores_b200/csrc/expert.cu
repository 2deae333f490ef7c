// Tokens to their experts and back.  A slot is one of the top_k choices of a
// token, slot s = t * top_k + j; the rows of an expert are its slots in slot
// order, the experts one after the other.
//
// Sort: a stable counting sort over at most 1024 experts.  A CTA takes runs of
// 1024, 2560 or 4096 slots, each of its 16 warps consecutive ones of a run in
// two, five or eight steps of 32.  In a step the lanes with one expert find one another by a
// ballot for each bit of the expert's number; a lane's rank is the warp's
// count of that expert so far plus its equals in lower lanes, and the lowest of
// them moves the count on.  Exclusive sums of the counts over warps, CTAs and
// experts turn ranks into rows.  The slots of the rows are put in order in
// shared memory first, so that an expert's leave the CTA together.  Only
// integers are added, so the result is the same every time.  More than one
// CTA: a first kernel leaves every CTA's counts in the workspace, and every CTA
// of the last adds up the ones before its own from L2, or finds them added up
// by a kernel between the two.
//
// Bound: latency, a chain of loads, shared memory and barriers.  What depends
// on nothing is therefore done for all steps at once.
#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMany = 8;  // steps of a warp in a run, with many slots,
constexpr int kSortSome = 5;  // fewer
constexpr int kSortFew = 2;   // and few

// The experts of this lane's slots s, s + apart, ... (-1: dropped, or behind the
// last slot).  From L2: the last kernel reads them before its own wait, on the
// word of the first that whatever wrote them has completed, and so does not
// depend on what an L1 may still hold.
template <int N>
__device__ __forceinline__ void slot_experts(const ExpertSortArgs& a, int64_t s, int apart, int (&e)[N]) {
    int64_t id[N];
    if (a.ids64) {
#pragma unroll
        for (int b = 0; b < N; ++b) id[b] = __ldcg(static_cast<const long long*>(a.ids) + min(s + b * apart, a.slots - 1));
    } else {
#pragma unroll
        for (int b = 0; b < N; ++b) id[b] = __ldcg(static_cast<const int*>(a.ids) + min(s + b * apart, a.slots - 1));
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
    pdl_next();  // the last kernel ranks its slots meanwhile
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

// Exclusive sums of the CTAs' counts over the CTAs, in their place, and the sums
// of all behind them.  A CTA takes 32 experts, each of its warps as many
// neighbouring CTAs' counts as 32 warps need for all.
constexpr int kMaxSortCtas = 512;
__global__ void __launch_bounds__(1024) expert_scan_kernel(const __grid_constant__ ExpertSortArgs a, int ctas) {
    constexpr int kRows = kMaxSortCtas / 32;
    __shared__ int part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int x = blockIdx.x * 32 + lane, rows = (ctas + 31) / 32, c0 = warp * rows;
    const int mine = x < a.num_experts ? min(rows, ctas - c0) : 0;  // (none: zero or less)
    int* counts = a.counts + (int64_t)c0 * a.num_experts + x;
    pdl_next();  // this CTA began on the first kernel's word, which so holds for the last as well
    pdl_wait();
    int n[kRows], sum = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) n[i] = i < mine ? __ldcg(counts + i * a.num_experts) : 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) sum += n[i];
    part[warp][lane] = sum;
    __syncthreads();
    int all;  // of expert blockIdx.x * 32 + warp
    part[lane][warp] = warp_scan(part[lane][warp], lane, all);
    const int e = blockIdx.x * 32 + warp;
    if (lane == 0 && e < a.num_experts) a.counts[ctas * a.num_experts + e] = all;
    __syncthreads();
    sum = part[warp][lane];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (i < mine) counts[i * a.num_experts] = sum;
        sum += n[i];
    }
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
    // with a first kernel, which has waited, only counts are to be waited for
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
        if (run == 0 && a.scanned) {
            pdl_wait();
            for (int x = threadIdx.x; x < E; x += kSortThreads) {
                first[x] = __ldcg(a.counts + blockIdx.x * E + x);
                total[x] = __ldcg(a.counts + gridDim.x * E + x);
            }
        } else if (run == 0 && !alone) {
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
// Bound: HBM, each token's row and each expert's row once.  A token takes
// 2^lanes neighbouring threads (up to 256; with few tokens as many as its row
// has places for), each of them U vectors of its row and B of its rows at a
// time, so that a thread has about four 16-byte loads on their way whatever
// top_k is.  (Rows one after the other, a vector at a time: one bf16 row of
// 7168 for each of 4096 tokens 37 us against 24.  More at once costs resident
// warps: eight loads for eight rows of 4096 105 us against 92 at 8192 tokens.)

constexpr int kRowThreads = 256;

// A row index inside [0, num_rows), or -1.
__device__ __forceinline__ int64_t row_at(const ExpertRowsArgs& a, int64_t slot) {
    const int r = __ldg(a.row_of_slot + slot);
    return r >= 0 && r < a.num_rows ? r : -1;
}

// rows[r(t, j)] = x[t].
template <int U>
__global__ void __launch_bounds__(kRowThreads) expert_dispatch_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    const int64_t thread = (int64_t)blockIdx.x * kRowThreads + threadIdx.x, t = thread >> a.lanes;
    if (t >= a.tokens) return;
    const int G = 1 << a.lanes;
    const char* in = a.token_in + t * a.token_bytes;
    for (int v0 = (int)(thread & (G - 1)); v0 < a.nvec; v0 += G * U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * G < a.nvec) x[u] = ld_stream(in + (v0 + u * G) * 16);
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t r = row_at(a, t * a.top_k + j);
            if (r < 0) continue;
            char* out = a.rows_out + r * a.rows_out_bytes;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + u * G < a.nvec) st_vec(out + (v0 + u * G) * 16, x[u]);
        }
    }
}

// y[t] = cast(sum_j w[t, j] rows[r(t, j)]), FP32, in the order of j; B rows at a time.
template <typename T, bool W, int B, int U>
__global__ void __launch_bounds__(kRowThreads) expert_combine_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    const int64_t thread = (int64_t)blockIdx.x * kRowThreads + threadIdx.x, t = thread >> a.lanes;
    if (t >= a.tokens) return;
    const int G = 1 << a.lanes;
    char* out = a.token_out + t * a.token_bytes;
    for (int v0 = (int)(thread & (G - 1)); v0 < a.nvec; v0 += G * U) {
        float acc[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[u][e] = 0.0f;
        for (int j0 = 0; j0 < a.top_k; j0 += B) {
            uint4 x[B][U];
            float w[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int64_t s = t * a.top_k + j0 + b;
                const int64_t r = j0 + b < a.top_k ? row_at(a, s) : -1;
                w[b] = W && r >= 0 ? __ldg(a.weights + s) : W ? 0.0f : 1.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[b][u] = make_uint4(0, 0, 0, 0);
                    if (r >= 0 && v0 + u * G < a.nvec)
                        x[b][u] = ld_stream(a.rows_in + r * a.rows_in_bytes + (v0 + u * G) * 16);
                }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[V];
                    unpack<T>(x[b][u], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[u][e] = W ? fmaf(w[b], f[e], acc[u][e]) : acc[u][e] + f[e];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * G < a.nvec) st_vec(out + (v0 + u * G) * 16, pack<T>(acc[u]));
    }
}

// Sums of B values (a power of two up to 8) over a warp.  Each exchange halves
// the values a lane is still in charge of: B - 1 + log2(32 / B) shuffles in
// place of 5 B.  The lanes whose upper log2 B bits are i end with sum i.
template <int B> __device__ __forceinline__ float warp_sums(float (&v)[B], int lane) {
    int o = 16;
#pragma unroll
    for (int n = B / 2; n > 0; n /= 2) {
        const bool high = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = high ? v[i + n] : v[i], send = high ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
        o /= 2;
    }
    float s = v[0];
    for (; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// drows[r(t, j)] = cast(w[t, j] dy[t]); dw[t, j] = <dy[t], rows[r(t, j)]>, B rows at a time.
template <typename T, bool W, bool DW, int B>
__global__ void __launch_bounds__(kRowThreads) expert_combine_bwd_kernel(const __grid_constant__ ExpertRowsArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    __shared__ float red[kRowThreads / 32][B];
    const int64_t t = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> a.lanes;
    const int G = 1 << a.lanes, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool live = t < a.tokens;  // the others go along for the barriers
    const char* in = a.token_in + t * a.token_bytes;
    for (int j0 = 0; j0 < a.top_k; j0 += B) {
        int64_t r[B];
        float w[B], dot[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int64_t s = t * a.top_k + j0 + b;
            r[b] = live && j0 + b < a.top_k ? row_at(a, s) : -1;
            // plain loads of what the outputs may overwrite (dweights over
            // weights, drows over rows): the compiler keeps them ahead of the
            // stores to the same place, as it need not with read-only loads
            w[b] = W && r[b] >= 0 ? a.weights[s] : 1.0f;
            dot[b] = 0.0f;
        }
        for (int v = threadIdx.x & (G - 1); v < a.nvec && live; v += G) {
            const uint4 g4 = ld_stream(in + v * 16);
            uint4 x[B];
            if constexpr (DW) {
#pragma unroll
                for (int b = 0; b < B; ++b)
                    x[b] = r[b] >= 0 ? *reinterpret_cast<const uint4*>(a.rows_in + r[b] * a.rows_in_bytes + v * 16)
                                     : make_uint4(0, 0, 0, 0);
            }
            float g[V];
            unpack<T>(g4, g);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (r[b] < 0) continue;
                if constexpr (DW) {
                    float f[V];
                    unpack<T>(x[b], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) dot[b] = fmaf(g[e], f[e], dot[b]);
                }
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = w[b] * g[e];
                st_vec(a.rows_out + r[b] * a.rows_out_bytes + v * 16, W ? pack<T>(o) : g4);
            }
        }
        if constexpr (DW) {
            if (G >= 32) {
                // sum b: in lanes 32 / B * b .. of every warp of the token, then over its warps
                const float s = warp_sums<B>(dot, lane);
                __syncthreads();
                if (lane % (32 / B) == 0) red[warp][lane / (32 / B)] = s;
                __syncthreads();
                const int b = threadIdx.x & (G - 1);  // the token's first threads take a sum each
                if (live && b < B && j0 + b < a.top_k) {
                    float all = 0.0f;
                    for (int i = 0; i < G / 32; ++i) all += red[warp + i][b];
                    a.dweights[t * a.top_k + j0 + b] = all;
                }
            } else {
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    for (int o = G / 2; o > 0; o /= 2) dot[b] += __shfl_xor_sync(0xffffffffu, dot[b], o);
                    if (live && (threadIdx.x & (G - 1)) == 0 && j0 + b < a.top_k) a.dweights[t * a.top_k + j0 + b] = dot[b];
                }
            }
        }
    }
}

// Threads of a token (their log2, at most `most`) at U vectors a thread, and
// the CTAs that makes.
unsigned row_grid(ExpertRowsArgs& a, int U, int most) {
    a.lanes = 0;
    while ((1 << a.lanes) < most && (U << a.lanes) < a.nvec) ++a.lanes;
    return (unsigned)(((a.tokens << a.lanes) + kRowThreads - 1) / kRowThreads);
}
// Where no sum over a token's threads is to be had: rows of few tokens over
// several CTAs (one token, eight rows of 4096: 2.4 us against 3.7).
int row_threads(const ExpertRowsArgs& a) { return a.tokens <= 2 * (int64_t)sm_count() ? 4096 : kRowThreads; }

template <typename T, bool W, int B>
cudaError_t launch_combine_bwd_b(ExpertRowsArgs a, cudaStream_t s) {
    const unsigned grid = row_grid(a, 1, kRowThreads);
    return a.dweights ? launch_pdl(expert_combine_bwd_kernel<T, W, true, B>, grid, kRowThreads, 0, s, a)
                      : launch_pdl(expert_combine_bwd_kernel<T, W, false, B>, grid, kRowThreads, 0, s, a);
}

template <typename T, bool W>
cudaError_t launch_combine_bwd(const ExpertRowsArgs& a, cudaStream_t s) {
    if (a.top_k == 1) return launch_combine_bwd_b<T, W, 1>(a, s);
    if (a.top_k == 2) return launch_combine_bwd_b<T, W, 2>(a, s);
    return launch_combine_bwd_b<T, W, 4>(a, s);  // (eight: 208 us against 176 for eight rows of 4096)
}

template <typename T, bool W, int B, int U>
cudaError_t launch_combine_bu(ExpertRowsArgs a, cudaStream_t s) {
    const unsigned grid = row_grid(a, U, row_threads(a));
    return launch_pdl(expert_combine_kernel<T, W, B, U>, grid, kRowThreads, 0, s, a);
}

template <typename T, bool W>
cudaError_t launch_combine(const ExpertRowsArgs& a, cudaStream_t s) {
    if (a.top_k == 1) return launch_combine_bu<T, W, 1, 2>(a, s);
    if (a.top_k == 2) return launch_combine_bu<T, W, 2, 2>(a, s);
    return launch_combine_bu<T, W, 4, 1>(a, s);
}

// Shape of the sort.  One CTA up to a run of eight steps (as two launches 4096
// slots take 4.2 us against 5.5, which the second launch costs the host).  Then
// two, five or eight steps: the fewest of these that keep the CTAs within a wave
// of two an SM, and eight with more runs at last.  On B200, us, 64 experts: 262144
// slots two steps 7.7, five 8.5, eight 8.2; 350000 two 10.5, five 10.3, eight
// 11.4; 500000 11.5, 9.5 and 11.4; 642008 five 9.9, eight 11.1; 2097152 eight
// 21.8, five 23.6.  Between 303105 and 500000 slots more kinds of CTA would be
// 4 to 18 % faster (350000: three steps 8.5, four 8.9; 500000: four 9.2), at
// 606208 four no longer (11.5 against 9.8).  (The number of SMs is not asked for:
// the workspace's size must not depend on the current device.)
//
// Every CTA adds up the counts of all itself while that is little work, CTAs^2
// times experts of it.  Beyond, a kernel between the two does it once.  Itself
// and by the kernel: 65536 slots of 256 experts (1.0 M) 6.0 and 6.9 us, 131072 of
// 64 (1.0 M) 6.4 and 6.6; 321004 of 128 (2.0 M) 10.8 and 8.7, 642008 of 64 (4.0 M)
// 10.9 and 9.7; of 512, with eight steps, 27.7 and 15.8.
constexpr int64_t kSortWave = 2 * 148;
constexpr int64_t kSortOwnSums = 1536 << 10;
struct SortShape {
    int64_t steps, runs, ctas;
};
SortShape sort_shape(int64_t slots, int64_t num_experts) {
    constexpr int64_t few = kSortThreads * kSortFew, many = kSortThreads * kSortMany;
    SortShape s{kSortFew, 1, 1};
    if (slots > few && slots <= many) s.steps = kSortMany;
    else if (slots > few * kSortWave) s.steps = slots <= (int64_t)kSortThreads * kSortSome * kSortWave ? kSortSome : kSortMany;
    const int64_t run = s.steps * kSortThreads;
    s.runs = (slots + run * kMaxSortCtas - 1) / (run * kMaxSortCtas);
    s.ctas = (slots + run * s.runs - 1) / (run * s.runs);
    return s;
}

template <int STEPS> cudaError_t launch_sort(const ExpertSortArgs& a, unsigned ctas, cudaStream_t s) {
    if (ctas > 1) {
        const cudaError_t e = launch_pdl(expert_count_kernel<STEPS>, ctas, kSortThreads, (size_t)a.num_experts * 4, s, a);
        if (e != cudaSuccess) return e;
        if (a.scanned) {
            const unsigned blocks = (unsigned)(a.num_experts + 31) / 32;
            const cudaError_t f = launch_pdl(expert_scan_kernel, blocks, 1024, 0, s, a, (int)ctas);
            if (f != cudaSuccess) return f;
        }
    }
    const size_t smem = ((size_t)2 * STEPS * kSortThreads + (size_t)(kSortWarps + 4) * (size_t)a.num_experts) * 4;
    const cudaError_t e = allow_smem((const void*)expert_place_kernel<STEPS>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(expert_place_kernel<STEPS>, ctas, kSortThreads, smem, s, a);
}

}  // namespace

size_t expert_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
    const int64_t n = sort_shape(slots, num_experts).ctas;
    return n > 1 ? (size_t)(n + 1) * (size_t)num_experts * sizeof(int32_t) : 0;
}

cudaError_t launch_expert_sort(ExpertSortArgs a, cudaStream_t s) {
    const SortShape sh = sort_shape(a.slots, a.num_experts);
    a.runs = (int32_t)sh.runs;
    a.scanned = sh.ctas > 1 && sh.ctas * sh.ctas * a.num_experts > kSortOwnSums;
    a.expert_bits = 0;
    while ((1 << a.expert_bits) < a.num_experts) ++a.expert_bits;
    switch (sh.steps) {
        case kSortFew: return launch_sort<kSortFew>(a, (unsigned)sh.ctas, s);
        case kSortSome: return launch_sort<kSortSome>(a, (unsigned)sh.ctas, s);
        default: return launch_sort<kSortMany>(a, (unsigned)sh.ctas, s);
    }
}

cudaError_t launch_expert_dispatch(ExpertRowsArgs a, cudaStream_t s) {
    const unsigned grid = row_grid(a, 2, row_threads(a));
    return launch_pdl(expert_dispatch_kernel<2>, grid, kRowThreads, 0, s, a);
}

cudaError_t launch_expert_combine(int dtype, const ExpertRowsArgs& a, cudaStream_t s) {
    if (dtype == 0)
        return a.weights ? launch_combine<__nv_bfloat16, true>(a, s) : launch_combine<__nv_bfloat16, false>(a, s);
    return a.weights ? launch_combine<float, true>(a, s) : launch_combine<float, false>(a, s);
}

cudaError_t launch_expert_combine_bwd(int dtype, const ExpertRowsArgs& a, cudaStream_t s) {
    if (dtype == 0)
        return a.weights ? launch_combine_bwd<__nv_bfloat16, true>(a, s) : launch_combine_bwd<__nv_bfloat16, false>(a, s);
    return a.weights ? launch_combine_bwd<float, true>(a, s) : launch_combine_bwd<float, false>(a, s);
}

}  // namespace muse
