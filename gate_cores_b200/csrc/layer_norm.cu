// Layer norm and its gradient.
//   forward:  c = x - mean(x), r = 1 / sqrt(mean(c^2) + eps), y = c r w + b
//   backward: g = dy w, n = c r; dx = r (g - mean(g) - n mean(g n)),
//             dgain += dy n, dbias += dy (sums over the rows)
//
// A row's 16-byte vectors are dealt to the lanes of a part of a warp, a warp,
// or several warps, at most NV to a lane, and stay in its registers from the
// load to the last use: HBM sees each input once.  The variance and sum g c
// are taken of centred elements, never as a difference of two large sums.  A
// row on several warps costs one barrier all the same: a warp centres its
// elements on its own mean m_w by shuffles, and the warps exchange
//   m_w, d_w = sum (x - m_w), Q_w = sum (x - m_w)^2, G_w = sum g,
//   C_w = sum g (x - m_w),
// from which, with n_w elements in warp w and D_w = m_w - mean,
//   mean = m_0 + sum (n_w (m_w - m_0) + d_w) / H,   sum c^2 = sum Q_w + 2 D_w d_w + n_w D_w^2,
//   sum g c = sum C_w + G_w D_w.
// d_w is what the rounding of m_w left; FP32 rows keep it, so that elements far
// from zero lose nothing to the mean's sum.  bf16 rows take it as 0 and round
// m_w correctly instead (mean_of): a row of one value, at most 2^15 times 8 bits,
// has an exact sum and so its value as mean, and centred elements of exactly 0.
// (A mean off by its last place left 2.4e-4 of 1000 elements of 2576, which
// 1 / sqrt(eps) made 0.24.)  A bf16 row of more than one value has a variance of
// at least (2^-8 |mean|)^2 / H or so, so that the mean's last place is at most
// 2^-17 sqrt(H) in y.
//
// Bound: HBM.  The next rows are on their way while a row is reduced: every
// lane copies its own vectors of a later row into its own places in shared
// memory (cp.async) and waits for its own copies only, so that neither
// registers nor barriers pay for the rows in flight.  (Measured against core
// 1's ring of whole-row bulk copies with a second row sum: 131072 x 256 bf16
// 44.2 us there, 22.4 here; 16384 x 1280 23.2 and 15.3; 8192 x 4096 26.3 and
// 24.0.)  The parameter gradients leave one partial row per CTA, added in a
// fixed order by a second kernel.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

constexpr int kLnMaxWarps = 16;  // of a CTA

template <typename T> __host__ __device__ constexpr bool keeps_rest() { return std::is_same<T, float>::value; }

// sum / n; of bf16 rows with what the product by the rounded 1 / n leaves of the sum added back.
template <typename T> __device__ __forceinline__ float mean_of(float sum, float n, float inv_n) {
    const float m = sum * inv_n;
    if constexpr (keeps_rest<T>()) return m;
    return fmaf(fmaf(-m, n, sum), inv_n, m);
}

// How a CTA's threads share rows: `lanes` threads a row (L < 32: a part of a
// warp), groups of them taking rows of their own.
struct Deal {
    int lanes, group, in_row, lane, warp_in_row;
};
template <int L> __device__ __forceinline__ Deal deal(int warps) {
    Deal d;
    d.lanes = L < 32 ? L : 32 * warps;
    d.group = (int)threadIdx.x / d.lanes;
    d.in_row = (int)threadIdx.x - d.group * d.lanes;
    d.lane = threadIdx.x & 31;
    d.warp_in_row = d.in_row >> 5;
    return d;
}
// Barrier of one group's warps (a row on several warps).
__device__ __forceinline__ void group_sync(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// A lane's vectors of a row: slot i holds vector in_row + i * lanes.  The
// launcher takes as few slots as hold the row, so that every slot but the last
// is full in every lane; `last` says whether the last one is.
template <int NV, int P>
__device__ __forceinline__ void center(f32x2 (&x)[NV][P], bool last, float m) {
    const f32x2 m2 = f2_make(-m, -m);
    const float e = last ? -m : 0.0f;  // idle: stays zero
    const f32x2 e2 = f2_make(e, e);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < P; ++q) x[i][q] = f2_add(x[i][q], i < NV - 1 ? m2 : e2);
    }
}
template <int NV, int P, typename F>
__device__ __forceinline__ float lane_sum(F&& term) {
    f32x2 acc[2] = {f2_make(0.0f, 0.0f), f2_make(0.0f, 0.0f)};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < P; ++q) acc[q & 1] = term(i, q, acc[q & 1]);
    }
    return f2_sum(acc[0]) + f2_sum(acc[1]);
}
// A lane's copy of 16 bytes into its own place in shared memory; zeros without
// a read where `on` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
// A row's vectors into the lane's places (`place` bytes from one to the next).
template <int NV>
__device__ __forceinline__ void copy_row(uint32_t to, uint32_t place, const char* from, int slot, bool live, bool last) {
    if (live) {
#pragma unroll
        for (int i = 0; i < NV - 1; ++i) copy16(to + i * place, from + i * slot);
        copy16(to + (NV - 1) * place, last ? from + (NV - 1) * slot : from, last);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) copy16(to + i * place, from, false);  // nothing is read
    }
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of this thread's copies but those of its latest N rows have landed.
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// D rows on their way.  PARAMS: gain + offset and bias wait in shared memory
// (ones and zeros where there are none); otherwise they are read from global
// memory for every row.
template <typename T, int NV, int L, int D, bool PARAMS>
__global__ void __launch_bounds__(32 * kLnMaxWarps) layer_norm_kernel(const __grid_constant__ LayerNormArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N, P = V / 2, SV = V / 4;
    constexpr bool REST = keeps_rest<T>();
    constexpr int W = PARAMS && NV < 8 ? 8 : kLnMaxWarps;  // warps of a row at most, a power of two
    // {m_w, Q_w, d_w, n_w} of the warps of a row, two banks
    __shared__ float4 part[2][kLnMaxWarps];
    extern __shared__ __align__(16) unsigned char smem[];  // [D][NV][threads] vectors; PARAMS: then [gain | bias]
    float* params = reinterpret_cast<float*>(smem + (size_t)D * NV * blockDim.x * 16);
    const Deal d = deal<L>(a.warps);
    const int nvec = a.width / V;
    const bool many = L == 32 && a.warps > 1;
    const bool last = d.in_row + (NV - 1) * d.lanes < nvec;
    const float width = (float)a.width, inv_width = 1.0f / width;
    // elements of this warp's part of a row
    const float here = L == 32 ? (float)((32 * (NV - 1) + __popc(__ballot_sync(0xffffffffu, last))) * V) : width;
    const float inv_here = 1.0f / here;
    const int groups = (int)blockDim.x / d.lanes;
    const int64_t step = (int64_t)gridDim.x * groups;
    // rows of the warp's first group, so that its lanes leave the loop together
    const int first = L < 32 ? ((int)threadIdx.x >> 5) * (32 / L) : d.group;
    const int ahead = d.group - first;
    int64_t base = (int64_t)blockIdx.x * groups + first;
    const char* in = static_cast<const char*>(a.x) + (base + ahead) * a.x_stride * (int64_t)sizeof(T) + d.in_row * 16;
    char* out = static_cast<char*>(a.out) + (base + ahead) * a.out_stride * (int64_t)sizeof(T) + d.in_row * 16;
    const int64_t in_step = step * a.x_stride * (int64_t)sizeof(T), out_step = step * a.out_stride * (int64_t)sizeof(T);
    const int slot = d.lanes * 16;  // bytes between a lane's vectors

    const bool first_slot = NV > 1 || last;
    // this lane's places; `get` is the next to be read, and filled again then
    // (rows on warps have no register to spare for a `put` of the same value;
    // rows on parts of a warp spill without one: 131072 x 120 bf16 17.6 us, 14.4 with)
    unsigned char* const home = smem + threadIdx.x * 16;
    const uint32_t home_addr = (uint32_t)__cvta_generic_to_shared(home);
    const uint32_t place = blockDim.x * 16, row_bytes = NV * place;
    uint32_t put = 0, get = 0;
    int64_t next = base + ahead;
    auto fetch = [&](uint32_t put) {
        // (behind the last row nothing is copied: no copy is left when the
        // kernel ends; a part of a warp without a row sums what was there
        // before, for nobody)  Where an idle lane has no vector of its own,
        // the row's start is given (and not read).
        if (next < a.rows) copy_row<NV>(home_addr + put, place, first_slot ? in : in - d.in_row * 16, slot, true, last);
        copies_end();
        next += step;
        in += in_step;
    };
#pragma unroll
    for (int k = 0; k < D; ++k) fetch(k * row_bytes);
    if constexpr (PARAMS) {
        // the k-th four columns of all vectors lie together: a warp's 16-byte
        // reads of neighbouring vectors then meet no bank twice
#pragma unroll 4
        for (int c = threadIdx.x; c < a.width / 4; c += blockDim.x) {
            float4 g = make_float4(1.0f, 1.0f, 1.0f, 1.0f), b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (a.gain) {
                g = __ldg(reinterpret_cast<const float4*>(a.gain) + c);
                g.x += a.gain_offset; g.y += a.gain_offset; g.z += a.gain_offset; g.w += a.gain_offset;
            }
            if (a.bias) b = __ldg(reinterpret_cast<const float4*>(a.bias) + c);
            const int at = c % SV * nvec + c / SV;
            reinterpret_cast<float4*>(params)[at] = g;
            reinterpret_cast<float4*>(params + a.width)[at] = b;
        }
        __syncthreads();
    }
    const float4* wp = PARAMS ? reinterpret_cast<const float4*>(params) + d.in_row
                              : reinterpret_cast<const float4*>(a.gain) + d.in_row * SV;
    const float4* bp = PARAMS ? reinterpret_cast<const float4*>(params + a.width) + d.in_row
                              : reinterpret_cast<const float4*>(a.bias) + d.in_row * SV;
    const f32x2 off2 = f2_make(a.gain_offset, a.gain_offset);
    int bank = 0;
    for (; base < a.rows; base += step) {
        const bool live = base + ahead < a.rows;
        f32x2 x[NV][P];
        copies_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) to_pairs<T>(*reinterpret_cast<const uint4*>(home + get + i * place), x[i]);

        const float m = mean_of<T>(group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); })), here, inv_here);
        // the sum has used all of the row, so its places are free
        fetch(L < 32 ? put : get);
        if (L < 32) put = put + row_bytes == D * row_bytes ? 0 : put + row_bytes;
        get = get + row_bytes == D * row_bytes ? 0 : get + row_bytes;
        center<NV, P>(x, last, m);
        float rest = 0.0f;
        if constexpr (REST) rest = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); }));
        float sq = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(x[i][q], x[i][q], s); }));
        float shift = REST ? rest * inv_here : 0.0f;  // mean - m
        if (many) {
            float4* p = part[bank] + d.group * a.warps;
            if (d.lane == 0) p[d.warp_in_row] = make_float4(m, sq, rest, here);
            group_sync(d.group, d.lanes);
            // lane l takes the part of warp l modulo W; the mean as m_0 + off
            const bool on = (d.lane & (W - 1)) < a.warps;
            const float4 o = p[on ? d.lane & (W - 1) : 0];
            const float n = on ? o.w : 0.0f, rw = on ? o.z : 0.0f;
            const float m0 = p[0].x, dm = o.x - m0;
            const float off = group_sum<W>(fmaf(n, dm, rw)) * inv_width;
            const float dw = dm - off;
            sq = group_sum<W>(on ? o.y + dw * fmaf(2.0f, rw, n * dw) : 0.0f);
            shift = off - (m - m0);
            bank ^= 1;
        } else if constexpr (REST) {
            sq = fmaf(-shift, rest, sq);  // about m + shift
        }
        sq = sq < 0.0f ? 0.0f : sq;  // a rounding below a sum of zero (a NaN stays)
        const float r = inv_rms_fast(sq, inv_width, a.eps);
        const f32x2 r2 = f2_make(r, r), s2 = f2_make(-shift * r, -shift * r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x2 o[P];
#pragma unroll
            for (int q = 0; q < P; ++q) o[q] = f2_fma(x[i][q], r2, s2);
            if (i < NV - 1 || last) {
                const int at = PARAMS ? i * d.lanes : i * d.lanes * SV;
#pragma unroll
                for (int k = 0; k < SV; ++k) {
                    if constexpr (PARAMS) {
                        const float4 g = wp[at + k * nvec], b = bp[at + k * nvec];
                        o[2 * k] = f2_fma(o[2 * k], f2_make(g.x, g.y), f2_make(b.x, b.y));
                        o[2 * k + 1] = f2_fma(o[2 * k + 1], f2_make(g.z, g.w), f2_make(b.z, b.w));
                    } else {
                        if (a.gain) {
                            const float4 g = __ldg(wp + at + k);
                            o[2 * k] = f2_mul(o[2 * k], f2_add(f2_make(g.x, g.y), off2));
                            o[2 * k + 1] = f2_mul(o[2 * k + 1], f2_add(f2_make(g.z, g.w), off2));
                        }
                        if (a.bias) {
                            const float4 b = __ldg(bp + at + k);
                            o[2 * k] = f2_add(o[2 * k], f2_make(b.x, b.y));
                            o[2 * k + 1] = f2_add(o[2 * k + 1], f2_make(b.z, b.w));
                        }
                    }
                }
                if (live) st_vec(out + i * slot, from_pairs<T>(o));
            }
        }
        out += out_step;
    }
}

// Backward.  A CTA takes `groups` rows at a time (a tile), in two steps.  First
// as in the forward: the lanes of a row bring it to registers, sum, and write
// dx; mean and r go to shared memory.  Then, after a barrier, the threads turn
// from rows to columns: a thread owns NB vectors' columns in every row of its
// set (where a row has fewer vectors than the CTA has threads, sets of threads
// share the tile's rows), reads x and dy once more where the copies left them
// and keeps dgain and dbias in registers.  Rows in the first step are wide and
// columns in the second are few, so neither needs many registers; with both in
// one step the lanes of a row hold its columns' gradients too, rows go over
// four times the warps and twice the instructions (8192 x 4096 bf16: 57 us
// that way).  A second barrier frees the tile's places for the rows after the
// next tile.
//
// L and W (lanes of a row within a warp, warps of a row), and with them the
// CTA, are compile-time constants here: the kernel issues half as many
// instructions on addresses as on arithmetic otherwise.
constexpr int kLnBwdNv = 4;  // vectors a lane takes of a row at most: of bf16, x and dy w then take 32 registers each
template <typename T, int NV, int L, int W> struct LnBwd {
    static constexpr int lanes = L < 32 ? L : 32 * W;
    // columns take 16 registers a bf16 vector, 8 an FP32 one: at most 2 and 4 of them a thread
    static constexpr int cols = std::is_same<T, float>::value ? 4 : 2;
    // rows of a tile: 8 warps of them, or, where those are too few threads for
    // the columns, two rows
    static constexpr int eight = W >= 8 ? 1 : 8 / W;
    static constexpr int groups = L < 32 ? 256 / L : eight * cols >= NV ? eight : 2;
    static constexpr int threads = lanes * groups;
    static constexpr int NB = (lanes * NV + threads - 1) / threads;
};

template <typename T, int NV, int L, int W>
__global__ void __launch_bounds__(LnBwd<T, NV, L, W>::threads, LnBwd<T, NV, L, W>::threads <= 256 ? 2 : 1)
    layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
    pdl_begin();
    using S = LnBwd<T, NV, L, W>;
    constexpr int V = Vec<T>::N, P = V / 2, SV = V / 4;
    constexpr int D = 2;  // tiles on their way or in use
    constexpr int NB = S::NB;
    constexpr int groups = S::groups, threads = S::threads;
    constexpr bool REST = keeps_rest<T>();
    constexpr bool many = W > 1;
    // {m_w, Q_w, G_w, C_w} and {d_w, n_w} of the warps of a row
    __shared__ float4 part[groups * W];
    __shared__ float2 more[groups * W];
    // of the tile's rows: bf16 (r, -mean r), FP32 (m, shift, r): n = x r - mean r, and ((x - m) - shift) r
    __shared__ float4 stat[groups];
    extern __shared__ __align__(16) unsigned char smem[];  // [D][x, dy][NV][threads] vectors, then gain + offset
    float* params = reinterpret_cast<float*>(smem + D * 2 * NV * threads * 16);
    const Deal d = deal<L>(W);
    const int nvec = a.width / V;
    const bool last = d.in_row + (NV - 1) * d.lanes < nvec;
    const float width = (float)a.width, inv_width = 1.0f / width;
    const float here = L == 32 ? (float)((32 * (NV - 1) + __popc(__ballot_sync(0xffffffffu, last))) * V) : width;
    const float inv_here = 1.0f / here;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t base = (int64_t)blockIdx.x * groups;  // the tile's first row
    const char* xin = static_cast<const char*>(a.x) + (base + d.group) * a.x_stride * (int64_t)sizeof(T) + d.in_row * 16;
    const char* gin = static_cast<const char*>(a.dy) + (base + d.group) * a.dy_stride * (int64_t)sizeof(T) + d.in_row * 16;
    char* out = static_cast<char*>(a.out) + (base + d.group) * a.out_stride * (int64_t)sizeof(T) + d.in_row * 16;
    const int64_t x_step = step * a.x_stride * (int64_t)sizeof(T), g_step = step * a.dy_stride * (int64_t)sizeof(T);
    const int64_t out_step = step * a.out_stride * (int64_t)sizeof(T);
    constexpr int slot = S::lanes * 16;

    const bool first_slot = NV > 1 || last;
    unsigned char* const home = smem + threadIdx.x * 16;
    const uint32_t home_addr = (uint32_t)__cvta_generic_to_shared(home);
    constexpr uint32_t place = threads * 16, tile_bytes = 2 * NV * place;
    int64_t next = base + d.group;
    auto fetch = [&](uint32_t put) {
        const bool live = next < a.rows;
        copy_row<NV>(home_addr + put, place, first_slot ? xin : xin - d.in_row * 16, slot, live, last);
        copy_row<NV>(home_addr + put + NV * place, place, first_slot ? gin : gin - d.in_row * 16, slot, live, last);
        copies_end();
        next += step;
        xin += x_step;
        gin += g_step;
    };
#pragma unroll
    for (int k = 0; k < D; ++k) fetch(k * tile_bytes);
    // gain + offset, laid out as in the forward
#pragma unroll 4
    for (int c = threadIdx.x; c < a.width / 4; c += threads) {
        float4 g = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        if (a.gain) {
            g = __ldg(reinterpret_cast<const float4*>(a.gain) + c);
            g.x += a.gain_offset; g.y += a.gain_offset; g.z += a.gain_offset; g.w += a.gain_offset;
        }
        reinterpret_cast<float4*>(params)[c % SV * nvec + c / SV] = g;
    }
    // of an idle slot the first vector's, to no effect: its dy is 0
    const float4* wp = reinterpret_cast<const float4*>(params) + (first_slot ? d.in_row : 0);
    const int last_at = last ? (NV - 1) * S::lanes : 0;
    __syncthreads();

    // columns: vectors col + i * threads (NB > 1), or those of set `set`
    const int sets = nvec < threads ? threads / nvec : 1;
    const int set = sets > 1 ? (int)threadIdx.x / nvec : 0;
    const int col = (int)threadIdx.x - set * nvec;
    uint32_t at[NB];  // of the vector in the tile's first row (row g: + g * lanes * 16)
    bool own[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int v = col + i * threads;
        own[i] = set < sets && v < nvec;
        at[i] = own[i] ? (uint32_t)(v / S::lanes) * place + (uint32_t)(v % S::lanes) * 16 : 0u;
    }
    f32x2 acc_g[NB][P], acc_b[NB][P];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
#pragma unroll
        for (int q = 0; q < P; ++q) acc_g[i][q] = acc_b[i][q] = f2_make(0.0f, 0.0f);
    }

    uint32_t get = 0;
    for (; base < a.rows; base += step) {
        const bool live = base + d.group < a.rows;
        f32x2 x[NV][P], g[NV][P];  // g: dy w
        copies_wait<D - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            to_pairs<T>(*reinterpret_cast<const uint4*>(home + get + i * place), x[i]);
            to_pairs<T>(*reinterpret_cast<const uint4*>(home + get + (NV + i) * place), g[i]);
#pragma unroll
            for (int k = 0; k < SV; ++k) {
                const float4 w = wp[(i < NV - 1 ? i * S::lanes : last_at) + k * nvec];
                g[i][2 * k] = f2_mul(g[i][2 * k], f2_make(w.x, w.y));
                g[i][2 * k + 1] = f2_mul(g[i][2 * k + 1], f2_make(w.z, w.w));
            }
        }
        const float m = mean_of<T>(group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); })), here, inv_here);
        float sg = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(g[i][q], s); }));
        center<NV, P>(x, last, m);
        float rest = 0.0f;
        if constexpr (REST) rest = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); }));
        float sq = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(x[i][q], x[i][q], s); }));
        float gc = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(g[i][q], x[i][q], s); }));
        float shift = REST ? rest * inv_here : 0.0f;
        if constexpr (many) {
            const int p0 = d.group * W;
            if (d.lane == 0) {
                part[p0 + d.warp_in_row] = make_float4(m, sq, sg, gc);
                more[p0 + d.warp_in_row] = make_float2(rest, here);
            }
            group_sync(d.group, S::lanes);
            // lane l takes the part of warp l modulo W2; the mean as m_0 + off
            constexpr int W2 = W > 4 ? 8 : W > 2 ? 4 : 2;
            const bool on = (d.lane & (W2 - 1)) < W;
            const float4 o = part[p0 + (on ? d.lane & (W2 - 1) : 0)];
            const float2 e = more[p0 + (on ? d.lane & (W2 - 1) : 0)];
            const float m0 = part[p0].x, dm = o.x - m0;
            const float off = group_sum<W2>(on ? fmaf(e.y, dm, e.x) : 0.0f) * inv_width;
            const float dw = dm - off;
            sq = group_sum<W2>(on ? o.y + dw * fmaf(2.0f, e.x, e.y * dw) : 0.0f);
            sg = group_sum<W2>(on ? o.z : 0.0f);
            gc = group_sum<W2>(on ? fmaf(o.z, dw, o.w) : 0.0f);
            shift = off - (m - m0);
        } else if constexpr (REST) {
            sq = fmaf(-shift, rest, sq);
            gc = fmaf(-shift, sg, gc);
        }
        sq = sq < 0.0f ? 0.0f : sq;
        const float r = inv_rms_fast(sq, inv_width, a.eps);
        if (d.in_row == 0) {
            // a tile's place without a row: its zeros add nothing
            if constexpr (REST) stat[d.group] = live ? make_float4(m, shift, r, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            // nor does a row of one value, whose n is 0, as x r and the rounded mean r need not be equal (without eps it
            // is NaN).  Its squares sum to 0; another row's may, by underflow, where the mean is below 2^-60 at most.
            else stat[d.group] = live && !(sq == 0.0f && fabsf(m) >= 0x1p-60f && a.eps > 0.0f)
                                     ? make_float4(r, -(m + shift) * r, 0.0f, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        const float k = -r * r * gc * inv_width;  // dx = r g - r mean(g) + k n
        const f32x2 r2 = f2_make(r, r), s2 = f2_make(-shift * r, -shift * r), k2 = f2_make(k, k);
        const f32x2 nm2 = f2_make(-r * sg * inv_width, -r * sg * inv_width);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x2 o[P];
#pragma unroll
            for (int q = 0; q < P; ++q) o[q] = f2_fma(f2_fma(x[i][q], r2, s2), k2, f2_fma(r2, g[i][q], nm2));
            if (live && (i < NV - 1 || last)) st_vec(out + i * slot, from_pairs<T>(o));
        }
        out += out_step;
        __syncthreads();

        const unsigned char* tile = smem + get;
        auto add_row = [&](int row) {
            const float4 st = stat[row];
            const uint32_t to = (uint32_t)row * (uint32_t)slot;
#pragma unroll
            for (int i = 0; i < NB; ++i) {  // (what is not the thread's own goes nowhere in the end)
                f32x2 cx[P], cg[P];
                to_pairs<T>(*reinterpret_cast<const uint4*>(tile + to + at[i]), cx);
                to_pairs<T>(*reinterpret_cast<const uint4*>(tile + to + at[i] + NV * place), cg);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    f32x2 n;
                    if constexpr (REST)
                        n = f2_mul(f2_add(f2_add(cx[q], f2_make(-st.x, -st.x)), f2_make(-st.y, -st.y)), f2_make(st.z, st.z));
                    else
                        n = f2_fma(cx[q], f2_make(st.x, st.x), f2_make(st.y, st.y));
                    acc_g[i][q] = f2_fma(cg[q], n, acc_g[i][q]);
                    acc_b[i][q] = f2_add(cg[q], acc_b[i][q]);
                }
            }
        };
        if (sets == 1) {
#pragma unroll
            for (int row = 0; row < (groups <= 8 ? groups : 0); ++row) add_row(row);
#pragma unroll 2
            for (int row = groups <= 8 ? groups : 0; row < groups; ++row) add_row(row);
        } else {
#pragma unroll 2
            for (int row = set < sets ? set : groups; row < groups; row += sets) add_row(row);
        }
        __syncthreads();
        fetch(get);
        get = get == 0 ? tile_bytes : 0;
    }
    copies_wait<0>();  // the last ones were of no row

    // one partial row of each gradient per CTA: the sets' added in their order
    if (!a.part_gain && !a.part_bias) return;
    float* acc_s = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* to = which == 0 ? a.part_gain : a.part_bias;
        if (!to) continue;
        to += (int64_t)blockIdx.x * a.width;
        if (sets > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (!own[i]) continue;
            float* p = sets > 1 ? acc_s + (int64_t)set * a.width + col * V : to + (int64_t)(col + i * threads) * V;
#pragma unroll
            for (int q = 0; q < SV; ++q) st_vec(p + 4 * q, from_pairs<float>((which == 0 ? acc_g[i] : acc_b[i]) + 2 * q));
        }
        if (sets == 1) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += threads) {
            float s = acc_s[c];
            for (int u = 1; u < sets; ++u) s += acc_s[u * a.width + c];
            to[c] = s;
        }
    }
}

// Sums of the partial rows, of both gradients in one launch: a CTA takes 32
// columns, each of its 64 groups of 8 threads (4 columns a thread) every 64th
// partial row in order, with up to 8 loads on their way (all of the usual 296
// rows' at once); the groups' sums are added in a fixed order.
constexpr int kSumCols = 32;
constexpr int kSumThreads = 512;
constexpr int kSumGroups = kSumThreads / (kSumCols / 4);
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 xor4(const float4& a, int o) {
    return make_float4(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o),
                       __shfl_xor_sync(0xffffffffu, a.z, o), __shfl_xor_sync(0xffffffffu, a.w, o));
}
__global__ void __launch_bounds__(kSumThreads)
    layer_norm_sum_kernel(const float* __restrict__ part0, float* __restrict__ out0, const float* __restrict__ part1,
                          float* __restrict__ out1, int parts, int width) {
    pdl_begin();
    constexpr int Q = kSumCols / 4, kWarps = kSumThreads / 32, U = 8;
    __shared__ float4 sums[kWarps][Q];
    const int blocks = (width + kSumCols - 1) / kSumCols;
    const bool second = !part0 || (int)blockIdx.x >= blocks;
    const float* part = second ? part1 : part0;
    float* out = second ? out1 : out0;
    const int q = threadIdx.x % Q, group = threadIdx.x / Q, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = ((int)blockIdx.x % blocks) * kSumCols + 4 * q;
    const bool on = c < width;  // widths are multiples of 4
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = group; p0 < parts; p0 += U * kSumGroups) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * kSumGroups;
            v[u] = on && p < parts ? __ldcg(reinterpret_cast<const float4*>(part + (int64_t)p * width + c))
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) s = add4(s, v[u]);
    }
    s = add4(s, xor4(s, 8));
    s = add4(s, xor4(s, 16));
    if (lane < Q) sums[warp][q] = s;
    __syncthreads();
    if (warp != 0) return;
    s = sums[lane / Q][q];
#pragma unroll
    for (int w = 32 / Q; w < kWarps; w += 32 / Q) s = add4(s, sums[w + lane / Q][q]);
    s = add4(s, xor4(s, 8));
    s = add4(s, xor4(s, 16));
    if (lane < Q && on) *reinterpret_cast<float4*>(out + c) = s;
}

// How rows of nvec vectors are dealt with: lanes of a row within a warp (a
// power of two from 4 on) or warps of it, vectors a lane, rows a CTA takes at
// a time, its threads.
struct Shape {
    int lanes, warps, nv, groups, threads;
};
// At most max_nv vectors a lane and about `most` warps a CTA.
Shape shape_of(int nvec, int max_nv, int most, int64_t rows) {
    Shape s{4, 1, 1, 1, 32};
    while (s.lanes < 32 && s.lanes * max_nv < nvec) s.lanes *= 2;
    if (s.lanes == 32) s.warps = (nvec + 32 * max_nv - 1) / (32 * max_nv);
    s.nv = (nvec + s.lanes * s.warps - 1) / (s.lanes * s.warps);
    const int per_warp = 32 / s.lanes;  // rows of a warp
    s.groups = most / s.warps > 1 ? most / s.warps : 1;  // warps, or sets of warps, of a CTA
    // few rows: over as many CTAs as there are SMs first
    const int64_t want = (rows + (int64_t)sm_count() * per_warp - 1) / ((int64_t)sm_count() * per_warp);
    if (want < s.groups) s.groups = want < 1 ? 1 : (int)want;
    s.threads = 32 * s.warps * s.groups;
    s.groups *= per_warp;
    return s;
}

template <typename T, int NV, int L, int D, bool PARAMS>
cudaError_t launch_fwd(LayerNormArgs a, const Shape& sh, cudaStream_t s) {
    a.warps = sh.warps;
    const size_t smem = (size_t)D * NV * sh.threads * 16 + (PARAMS ? (size_t)a.width * 8 : 0);
    auto kern = layer_norm_kernel<T, NV, L, D, PARAMS>;
    const cudaError_t e = allow_smem((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (a.rows + sh.groups - 1) / sh.groups;
    const int64_t most = (int64_t)blocks_per_sm((const void*)kern, sh.threads, smem) * sm_count();
    if (grid > most) grid = most;
    return launch_pdl(kern, (unsigned)grid, (unsigned)sh.threads, smem, s, a);
}

// Vectors a lane takes of a row, rows on their way and warps of a CTA, measured
// on B200 (16384 x 1280 and 8192 x 4096 bf16): 8 vectors, depth 2, 8 warps 15.3
// and 25.2 us; depth 3 16.6 and 26.7; 16 warps 15.6 and 26.9.
constexpr int kLnFwdNv = 8;
constexpr int kLnFwdDepth = 2;
constexpr int kLnFwdWarps = 8;
constexpr int kLnWide = 8192;                // columns
constexpr int kLnWidest = 16384;
constexpr size_t kLnSmem = 220 * 1024;  // of an SM, for one CTA
// Few rows (at most this many an SM): latency counts, so a row goes over as
// many warps as take it two vectors a lane, and the parameters come straight
// from global memory (4096 bf16 columns: 128 rows 3.6 us against 4.9 the other
// way, 296 rows 3.2 against 3.7, 1184 rows 6.5 against 5.8).
constexpr int kLnFewRows = 2;
constexpr int kLnFewNv = 2;

template <typename T, int D, bool PARAMS, int NV>
cudaError_t launch_fwd_nv(const LayerNormArgs& a, const Shape& sh, cudaStream_t s) {
    // a row that four lanes do not hold has more than four vectors for each of its lanes
    if constexpr (NV <= 4) return launch_fwd<T, NV, 4, D, PARAMS>(a, sh, s);
    else switch (sh.lanes) {
        case 4: return launch_fwd<T, NV, 4, D, PARAMS>(a, sh, s);
        case 8: return launch_fwd<T, NV, 8, D, PARAMS>(a, sh, s);
        case 16: return launch_fwd<T, NV, 16, D, PARAMS>(a, sh, s);
        default: return launch_fwd<T, NV, 32, D, PARAMS>(a, sh, s);
    }
}

template <typename T>
cudaError_t launch_fwd_t(const LayerNormArgs& a, cudaStream_t s) {
    const int nvec = a.width / Vec<T>::N;
    if (a.rows <= (int64_t)kLnFewRows * sm_count() && nvec > 32 * kLnFewNv && nvec <= 32 * kLnFewNv * kLnMaxWarps)
        return launch_fwd<T, kLnFewNv, 32, 1, false>(a, shape_of(nvec, kLnFewNv, 1, a.rows), s);
    const Shape sh = shape_of(nvec, kLnFwdNv, kLnFwdWarps, a.rows);
    // rows whose parameters leave room for one CTA an SM: it takes 16 warps
    // and the rows on their way that fit (up to kLnWidest columns one each),
    // wider ones read the parameters for every row (16384 x 9000 bf16: 149 us
    // that way)
    if (a.width > kLnWide) {
        const Shape wide = shape_of(nvec, kLnFwdNv, kLnMaxWarps, a.rows);
        // (64 KB: FP32 rows do not get there; and from 1025 vectors on, seven or
        // eight a lane, of rows for which two do not fit eight)
        if constexpr (Vec<T>::N > 4)
            if (a.width > kLnWidest) return launch_fwd<T, 8, 32, kLnFwdDepth, false>(a, wide, s);
        const size_t two = (size_t)2 * wide.nv * wide.threads * 16 + (size_t)a.width * 8;
        if (two > kLnSmem) return launch_fwd<T, 8, 32, 1, true>(a, wide, s);
        return wide.nv == 8 ? launch_fwd<T, 8, 32, 2, true>(a, wide, s) : launch_fwd<T, 7, 32, 2, true>(a, wide, s);
    }
    switch (sh.nv) {
        case 1: return launch_fwd_nv<T, kLnFwdDepth, true, 1>(a, sh, s);
        case 2: return launch_fwd_nv<T, kLnFwdDepth, true, 2>(a, sh, s);
        case 3: return launch_fwd_nv<T, kLnFwdDepth, true, 3>(a, sh, s);
        case 4: return launch_fwd_nv<T, kLnFwdDepth, true, 4>(a, sh, s);
        case 5: return launch_fwd_nv<T, kLnFwdDepth, true, 5>(a, sh, s);
        case 6: return launch_fwd_nv<T, kLnFwdDepth, true, 6>(a, sh, s);
        case 7: return launch_fwd_nv<T, kLnFwdDepth, true, 7>(a, sh, s);
        case 8: return launch_fwd_nv<T, kLnFwdDepth, true, 8>(a, sh, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, int NV, int L, int W>
cudaError_t launch_bwd(LayerNormArgs a, float* dgain, float* dbias, cudaStream_t s) {
    using S = LnBwd<T, NV, L, W>;
    if (!dgain) a.part_gain = nullptr;
    if (!dbias) a.part_bias = nullptr;
    // the ring (which holds the sets' gradients at the end, at most 32 bytes a thread) and the gain
    const size_t smem = (size_t)2 * 2 * NV * S::threads * 16 + (size_t)a.width * 4;
    auto kern = layer_norm_bwd_kernel<T, NV, L, W>;
    cudaError_t e = allow_smem((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (a.rows + S::groups - 1) / S::groups;
    const int64_t most = (int64_t)blocks_per_sm((const void*)kern, S::threads, smem) * sm_count();
    if (grid > most) grid = most;
    // the caller's workspace holds at most this many partial rows
    const int64_t cap = (int64_t)(row_bwd_gain_scratch_bytes(a.rows, a.width) / sizeof(float)) / a.width;
    if (grid > cap) grid = cap;
    e = launch_pdl(kern, (unsigned)grid, (unsigned)S::threads, smem, s, a);
    if (e != cudaSuccess || !(dgain || dbias)) return e;
    const int blocks = (a.width + kSumCols - 1) / kSumCols;
    return launch_pdl(layer_norm_sum_kernel, (unsigned)(blocks * ((dgain ? 1 : 0) + (dbias ? 1 : 0))), kSumThreads, 0, s,
                      dgain ? (const float*)a.part_gain : nullptr, dgain, dbias ? (const float*)a.part_bias : nullptr,
                      dbias, (int)grid, a.width);
}

// Vectors a lane: those that the lanes need for the row (at most kLnBwdNv).
template <typename T, int L, int W>
cudaError_t launch_bwd_nv(const LayerNormArgs& a, float* dgain, float* dbias, cudaStream_t s) {
    const int lanes = L < 32 ? L : 32 * W;
    const int nv = (a.width / Vec<T>::N + lanes - 1) / lanes;
    // (rows of one or two: those that four lanes hold)
    if constexpr (L == 4) {
        if (nv == 1) return launch_bwd<T, 1, L, W>(a, dgain, dbias, s);
        if (nv == 2) return launch_bwd<T, 2, L, W>(a, dgain, dbias, s);
    }
    constexpr bool f32 = std::is_same<T, float>::value;
    if constexpr (W <= 3 || f32) {
        if (nv <= 3) return launch_bwd<T, 3, L, W>(a, dgain, dbias, s);
    }
    // (the FP32 rows that three or six warps take have three)
    if constexpr (f32 && W % 3 == 0) return cudaErrorInvalidValue;
    else return launch_bwd<T, 4, L, W>(a, dgain, dbias, s);
}

template <typename T>
cudaError_t launch_bwd_t(const LayerNormArgs& a, float* dgain, float* dbias, cudaStream_t s) {
    const int nvec = a.width / Vec<T>::N;
    if (nvec <= 4 * kLnBwdNv) return launch_bwd_nv<T, 4, 1>(a, dgain, dbias, s);
    if (nvec <= 8 * kLnBwdNv) return launch_bwd_nv<T, 8, 1>(a, dgain, dbias, s);
    if (nvec <= 16 * kLnBwdNv) return launch_bwd_nv<T, 16, 1>(a, dgain, dbias, s);
    // Warps of a row at four vectors a lane; of an FP32 row, whose vectors make
    // fewer registers, at three where that leaves no more lanes idle (16384 x
    // 2304 82 us against 91; bf16 8192 x 2600 39.5 against 37.5, so not there).
    // Seven warps of a bf16 row spill registers that eight do not (8192 x 7168
    // 97 us against 87).
    constexpr bool f32 = std::is_same<T, float>::value;
    const int four = (nvec + 127) / 128, three = (nvec + 95) / 96;
    const int warps = f32 && three <= 8 && 96 * three <= 128 * four ? three : four;
    switch (!f32 && warps == 7 ? 8 : warps) {
        case 1: return launch_bwd_nv<T, 32, 1>(a, dgain, dbias, s);
        case 2: return launch_bwd_nv<T, 32, 2>(a, dgain, dbias, s);
        case 3: return launch_bwd_nv<T, 32, 3>(a, dgain, dbias, s);
        case 4: return launch_bwd_nv<T, 32, 4>(a, dgain, dbias, s);
        case 5: return launch_bwd_nv<T, 32, 5>(a, dgain, dbias, s);
        case 6: return launch_bwd_nv<T, 32, 6>(a, dgain, dbias, s);
        case 7:
            if constexpr (f32) return launch_bwd_nv<T, 32, 7>(a, dgain, dbias, s);
            break;
        case 8: return launch_bwd_nv<T, 32, 8>(a, dgain, dbias, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s) {
    return dtype == 0 ? launch_fwd_t<__nv_bfloat16>(a, s) : launch_fwd_t<float>(a, s);
}

cudaError_t launch_layer_norm_bwd(int dtype, LayerNormArgs a, float* dgain, float* dbias, cudaStream_t s) {
    return dtype == 0 ? launch_bwd_t<__nv_bfloat16>(a, dgain, dbias, s) : launch_bwd_t<float>(a, dgain, dbias, s);
}

}  // namespace muse
