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
// from zero lose nothing to the mean's sum (a bf16 element is known to 2^-9 of
// itself, and d_w is taken as 0).
//
// Bound: HBM.  The next row's loads are in flight while a row is reduced.
// In the backward a lane owns the same columns in every row and keeps their
// gain and bias gradients in registers; a CTA leaves one partial row of each
// and a second kernel adds them in a fixed order.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

// Warps of a CTA (rows on fewer warps share one).
constexpr int kLnWarps = 8;
constexpr int kLnMaxWarps = 16;  // of the widest rows

template <typename T> __host__ __device__ constexpr bool keeps_rest() { return std::is_same<T, float>::value; }

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
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const f32x2 c = f2_add(x[i][q], m2);
            x[i][q] = i < NV - 1 || last ? c : x[i][q];  // idle: stays zero
        }
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
// Sum over the first `warps` lanes (the others hold 0), in every lane.
__device__ __forceinline__ float warps_sum(float v, int warps) {
    for (int o = 1; o < warps; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

// PARAMS: gain + offset and bias wait in shared memory (ones and zeros where
// there are none); otherwise (rows too wide for that) they are read from
// global memory for every row.
template <typename T, int NV, int L, bool PARAMS>
__global__ void __launch_bounds__(32 * (PARAMS ? kLnWarps : kLnMaxWarps), PARAMS ? 2 : 1)
    layer_norm_kernel(const __grid_constant__ LayerNormArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N, P = V / 2, SV = V / 4;
    constexpr bool REST = keeps_rest<T>();
    // {m_w, Q_w, d_w, n_w} of the warps of a row, two banks
    __shared__ float4 part[2][kLnMaxWarps];
    extern __shared__ __align__(16) float params[];  // PARAMS: [gain | bias]
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

    uint4 raw[NV];
    auto load = [&](bool live) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            raw[i] = live && (i < NV - 1 || last) ? ld_stream(in + i * slot) : make_uint4(0, 0, 0, 0);
    };
    load(base + ahead < a.rows);
    if constexpr (PARAMS) {
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            params[c] = a.gain ? __ldg(a.gain + c) + a.gain_offset : 1.0f;
            params[a.width + c] = a.bias ? __ldg(a.bias + c) : 0.0f;
        }
        __syncthreads();
    }
    const float4* wp = reinterpret_cast<const float4*>(PARAMS ? params : a.gain) + d.in_row * SV;
    const float4* bp = reinterpret_cast<const float4*>(PARAMS ? params + a.width : a.bias) + d.in_row * SV;
    const f32x2 off2 = f2_make(a.gain_offset, a.gain_offset);
    int bank = 0;
    for (; base < a.rows; base += step) {
        const bool live = base + ahead < a.rows;
        f32x2 x[NV][P];
#pragma unroll
        for (int i = 0; i < NV; ++i) to_pairs<T>(raw[i], x[i]);
        in += in_step;
        load(base + step + ahead < a.rows);

        const float m = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); })) * inv_here;
        center<NV, P>(x, last, m);
        float rest = 0.0f;
        if constexpr (REST) rest = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); }));
        float sq = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(x[i][q], x[i][q], s); }));
        float shift = REST ? rest * inv_here : 0.0f;  // mean - m
        if (many) {
            float4* p = part[bank] + d.group * a.warps;
            if (d.lane == 0) p[d.warp_in_row] = make_float4(m, sq, rest, here);
            group_sync(d.group, d.lanes);
            // lane w takes warp w's part; the mean as m_0 + off
            const float4 o = p[d.lane < a.warps ? d.lane : 0];
            const float n = d.lane < a.warps ? o.w : 0.0f, rw = d.lane < a.warps ? o.z : 0.0f;
            const float m0 = __shfl_sync(0xffffffffu, o.x, 0), dm = o.x - m0;
            const float off = warps_sum(fmaf(n, dm, rw), a.warps) * inv_width;
            const float D = dm - off;
            sq = warps_sum(d.lane < a.warps ? o.y + D * fmaf(2.0f, rw, n * D) : 0.0f, a.warps);
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
                const int at = i * d.lanes * SV;
#pragma unroll
                for (int k = 0; k < SV; ++k) {
                    if constexpr (PARAMS) {
                        const float4 g = wp[at + k], b = bp[at + k];
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

// Vectors a lane takes of a row in the backward: its columns' two gradients
// take 16 registers a bf16 vector.
constexpr int kLnBwdNv = 2;

template <typename T, int NV, int L, int MAXW>
__global__ void __launch_bounds__(32 * MAXW, MAXW == kLnWarps ? 2 : 1)
    layer_norm_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N, P = V / 2, SV = V / 4;
    constexpr bool REST = keeps_rest<T>();
    // {m_w, Q_w, G_w, C_w} and {d_w, n_w} of the warps of a row, two banks
    __shared__ float4 part[2][MAXW];
    __shared__ float2 more[2][MAXW];
    extern __shared__ __align__(16) float acc_s[];  // the groups' gradients, at the end
    const Deal d = deal<L>(a.warps);
    const int nvec = a.width / V;
    const bool many = L == 32 && a.warps > 1;
    const bool last = d.in_row + (NV - 1) * d.lanes < nvec;
    const float width = (float)a.width, inv_width = 1.0f / width;
    const float here = L == 32 ? (float)((32 * (NV - 1) + __popc(__ballot_sync(0xffffffffu, last))) * V) : width;
    const float inv_here = 1.0f / here;
    const int groups = (int)blockDim.x / d.lanes;
    const int64_t step = (int64_t)gridDim.x * groups;
    const int first = L < 32 ? ((int)threadIdx.x >> 5) * (32 / L) : d.group;
    const int ahead = d.group - first;
    int64_t base = (int64_t)blockIdx.x * groups + first;
    const char* xin = static_cast<const char*>(a.x) + (base + ahead) * a.x_stride * (int64_t)sizeof(T) + d.in_row * 16;
    const char* gin = static_cast<const char*>(a.dy) + (base + ahead) * a.dy_stride * (int64_t)sizeof(T) + d.in_row * 16;
    char* out = static_cast<char*>(a.out) + (base + ahead) * a.out_stride * (int64_t)sizeof(T) + d.in_row * 16;
    const int64_t x_step = step * a.x_stride * (int64_t)sizeof(T), g_step = step * a.dy_stride * (int64_t)sizeof(T);
    const int64_t out_step = step * a.out_stride * (int64_t)sizeof(T);
    const int slot = d.lanes * 16;

    uint4 rx[NV], rg[NV];
    auto load = [&](bool live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool on = live && (i < NV - 1 || last);
            rx[i] = on ? ld_stream(xin + i * slot) : make_uint4(0, 0, 0, 0);
            rg[i] = on ? ld_stream(gin + i * slot) : make_uint4(0, 0, 0, 0);
        }
    };
    load(base + ahead < a.rows);
    f32x2 w[NV][P], acc_g[NV][P], acc_b[NV][P];
    {
        const f32x2 zero = f2_make(0.0f, 0.0f), off2 = f2_make(a.gain_offset, a.gain_offset);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = i < NV - 1 || last ? (d.in_row + i * d.lanes) * V : 0;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                w[i][q] = f2_make(1.0f, 1.0f);
                if (a.gain) {
                    const float2 g2 = __ldg(reinterpret_cast<const float2*>(a.gain + col) + q);
                    w[i][q] = f2_add(f2_make(g2.x, g2.y), off2);
                }
                acc_g[i][q] = acc_b[i][q] = zero;
            }
        }
    }
    int bank = 0;
    for (; base < a.rows; base += step) {
        const bool live = base + ahead < a.rows;
        f32x2 x[NV][P], g[NV][P];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            to_pairs<T>(rx[i], x[i]);
            to_pairs<T>(rg[i], g[i]);
        }
        xin += x_step;
        gin += g_step;
        load(base + step + ahead < a.rows);

        const float m = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); })) * inv_here;
        float sg = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(g[i][q], w[i][q], s); }));
        center<NV, P>(x, last, m);
        float rest = 0.0f;
        if constexpr (REST) rest = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_add(x[i][q], s); }));
        float sq = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(x[i][q], x[i][q], s); }));
        float gc = group_sum<L>(lane_sum<NV, P>([&](int i, int q, f32x2 s) { return f2_fma(f2_mul(g[i][q], w[i][q]), x[i][q], s); }));
        float shift = REST ? rest * inv_here : 0.0f;
        if (many) {
            const int at = d.group * a.warps;
            if (d.lane == 0) {
                part[bank][at + d.warp_in_row] = make_float4(m, sq, sg, gc);
                more[bank][at + d.warp_in_row] = make_float2(rest, here);
            }
            group_sync(d.group, d.lanes);
            // lane w takes warp w's part; the mean as m_0 + off
            const bool on = d.lane < a.warps;
            const float4 o = part[bank][at + (on ? d.lane : 0)];
            const float2 e = more[bank][at + (on ? d.lane : 0)];
            const float m0 = __shfl_sync(0xffffffffu, o.x, 0), dm = o.x - m0;
            const float off = warps_sum(on ? fmaf(e.y, dm, e.x) : 0.0f, a.warps) * inv_width;
            const float D = dm - off;
            sq = warps_sum(on ? o.y + D * fmaf(2.0f, e.x, e.y * D) : 0.0f, a.warps);
            sg = warps_sum(on ? o.z : 0.0f, a.warps);
            gc = warps_sum(on ? fmaf(o.z, D, o.w) : 0.0f, a.warps);
            shift = off - (m - m0);
            bank ^= 1;
        } else if constexpr (REST) {
            sq = fmaf(-shift, rest, sq);
            gc = fmaf(-shift, sg, gc);
        }
        sq = sq < 0.0f ? 0.0f : sq;
        const float r = inv_rms_fast(sq, inv_width, a.eps);
        const float k = -r * r * gc * inv_width;  // dx = r g - r mean(g) + k n
        const f32x2 r2 = f2_make(r, r), s2 = f2_make(-shift * r, -shift * r), k2 = f2_make(k, k);
        const f32x2 nm2 = f2_make(-r * sg * inv_width, -r * sg * inv_width);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x2 o[P];
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const f32x2 n = f2_fma(x[i][q], r2, s2);
                o[q] = f2_fma(n, k2, f2_fma(f2_mul(r2, w[i][q]), g[i][q], nm2));
                if (L == 32 || live) acc_g[i][q] = f2_fma(g[i][q], n, acc_g[i][q]);  // idle slots: g is 0
                acc_b[i][q] = f2_add(g[i][q], acc_b[i][q]);
            }
            if (live && (i < NV - 1 || last)) st_vec(out + i * slot, from_pairs<T>(o));
        }
        out += out_step;
    }

    // one partial row of each gradient per CTA: the groups' added in their order
    if (!a.part_gain && !a.part_bias) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* to = which == 0 ? a.part_gain : a.part_bias;
        if (!to) continue;
        to += (int64_t)blockIdx.x * a.width;
        if (groups == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i == NV - 1 && !last) continue;
#pragma unroll
                for (int k = 0; k < SV; ++k)
                    st_vec(to + (d.in_row + i * d.lanes) * V + 4 * k,
                           from_pairs<float>((which == 0 ? acc_g[i] : acc_b[i]) + 2 * k));
            }
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i == NV - 1 && !last) continue;
#pragma unroll
            for (int k = 0; k < SV; ++k)
                st_vec(acc_s + (int64_t)d.group * a.width + (d.in_row + i * d.lanes) * V + 4 * k,
                       from_pairs<float>((which == 0 ? acc_g[i] : acc_b[i]) + 2 * k));
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            float s = acc_s[c];
            for (int u = 1; u < groups; ++u) s += acc_s[u * a.width + c];
            to[c] = s;
        }
    }
}

// How rows of nvec vectors are dealt with at most max_nv vectors a lane: lanes
// of a row within a warp (a power of two from 4 on) or warps of it, vectors a
// lane, threads of a CTA.
struct Shape {
    int lanes, warps, nv, threads;
};
Shape shape_of(int nvec, int max_nv) {
    Shape s{4, 1, 1, 32 * kLnWarps};
    while (s.lanes < 32 && s.lanes * max_nv < nvec) s.lanes *= 2;
    if (s.lanes == 32) {
        s.warps = (nvec + 32 * max_nv - 1) / (32 * max_nv);
        s.threads = 32 * (s.warps >= kLnWarps ? s.warps : kLnWarps / s.warps * s.warps);
    }
    s.nv = (nvec + s.lanes * s.warps - 1) / (s.lanes * s.warps);
    return s;
}
int64_t groups_of(const Shape& s) { return s.threads / (s.lanes * s.warps); }

template <typename T, int NV, int L, bool PARAMS>
cudaError_t launch_fwd(LayerNormArgs a, const Shape& sh, cudaStream_t s) {
    a.warps = sh.warps;
    const size_t smem = PARAMS ? (size_t)a.width * 8 : 0;
    auto kern = layer_norm_kernel<T, NV, L, PARAMS>;
    if (smem > 40 * 1024) {  // above the default 48 KB once the static part is added
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t groups = groups_of(sh);
    int64_t grid = (a.rows + groups - 1) / groups;
    const int64_t most = (int64_t)blocks_per_sm((const void*)kern, sh.threads, smem) * sm_count();
    if (grid > most) grid = most;
    return launch_pdl(kern, (unsigned)grid, (unsigned)sh.threads, smem, s, a);
}

constexpr int kLnFwdNv = 8;

template <typename T, bool PARAMS, int NV>
cudaError_t launch_fwd_nv(const LayerNormArgs& a, const Shape& sh, cudaStream_t s) {
    if (sh.lanes == 32) return launch_fwd<T, NV, 32, PARAMS>(a, sh, s);
    if constexpr (PARAMS) {  // a part of a warp
        if (sh.lanes == 16) return launch_fwd<T, NV, 16, true>(a, sh, s);
        if (sh.lanes == 8) return launch_fwd<T, NV, 8, true>(a, sh, s);
        return launch_fwd<T, NV, 4, true>(a, sh, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, bool PARAMS>
cudaError_t launch_fwd_p(const LayerNormArgs& a, const Shape& sh, cudaStream_t s) {
    switch (sh.nv) {
        case 1: return launch_fwd_nv<T, PARAMS, 1>(a, sh, s);
        case 2: return launch_fwd_nv<T, PARAMS, 2>(a, sh, s);
        case 3: return launch_fwd_nv<T, PARAMS, 3>(a, sh, s);
        case 4: return launch_fwd_nv<T, PARAMS, 4>(a, sh, s);
        case 5: return launch_fwd_nv<T, PARAMS, 5>(a, sh, s);
        case 6: return launch_fwd_nv<T, PARAMS, 6>(a, sh, s);
        case 7: return launch_fwd_nv<T, PARAMS, 7>(a, sh, s);
        case 8: return launch_fwd_nv<T, PARAMS, 8>(a, sh, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_fwd_t(const LayerNormArgs& a, cudaStream_t s) {
    const int nvec = a.width / Vec<T>::N;
    const Shape sh = shape_of(nvec, kLnFwdNv);
    // the parameters of wider rows would leave room for one CTA
    return sh.warps <= kLnWarps && a.width <= 8192 ? launch_fwd_p<T, true>(a, sh, s) : launch_fwd_p<T, false>(a, sh, s);
}

template <typename T, int NV, int L, int MAXW>
cudaError_t launch_bwd(LayerNormArgs a, const Shape& sh, float* dgain, float* dbias, cudaStream_t s) {
    a.warps = sh.warps;
    const int64_t groups = groups_of(sh);
    if (!dgain) a.part_gain = nullptr;
    if (!dbias) a.part_bias = nullptr;
    const size_t smem = groups > 1 && (dgain || dbias) ? (size_t)groups * (size_t)a.width * sizeof(float) : 0;
    auto kern = layer_norm_bwd_kernel<T, NV, L, MAXW>;
    int64_t grid = (a.rows + groups - 1) / groups;
    const int64_t most = (int64_t)blocks_per_sm((const void*)kern, sh.threads, smem) * sm_count();
    if (grid > most) grid = most;
    // the caller's workspace holds at most this many partial rows
    const int64_t cap = (int64_t)(row_bwd_gain_scratch_bytes(a.rows, a.width) / sizeof(float)) / a.width;
    if (grid > cap) grid = cap;
    cudaError_t e = launch_pdl(kern, (unsigned)grid, (unsigned)sh.threads, smem, s, a);
    if (e == cudaSuccess && dgain) e = launch_param_grad_reduce(a.part_gain, (int)grid, a.width, dgain, s);
    if (e == cudaSuccess && dbias) e = launch_param_grad_reduce(a.part_bias, (int)grid, a.width, dbias, s);
    return e;
}

template <typename T, int NV>
cudaError_t launch_bwd_nv(const LayerNormArgs& a, const Shape& sh, float* dgain, float* dbias, cudaStream_t s) {
    if (sh.warps > kLnWarps) return launch_bwd<T, NV, 32, kLnMaxWarps>(a, sh, dgain, dbias, s);
    if (sh.lanes == 32) return launch_bwd<T, NV, 32, kLnWarps>(a, sh, dgain, dbias, s);
    if (sh.lanes == 16) return launch_bwd<T, NV, 16, kLnWarps>(a, sh, dgain, dbias, s);
    if (sh.lanes == 8) return launch_bwd<T, NV, 8, kLnWarps>(a, sh, dgain, dbias, s);
    return launch_bwd<T, NV, 4, kLnWarps>(a, sh, dgain, dbias, s);
}

template <typename T>
cudaError_t launch_bwd_t(const LayerNormArgs& a, float* dgain, float* dbias, cudaStream_t s) {
    const Shape sh = shape_of(a.width / Vec<T>::N, kLnBwdNv);
    return sh.nv == 1 ? launch_bwd_nv<T, 1>(a, sh, dgain, dbias, s) : launch_bwd_nv<T, 2>(a, sh, dgain, dbias, s);
}

}  // namespace

cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s) {
    return dtype == 0 ? launch_fwd_t<__nv_bfloat16>(a, s) : launch_fwd_t<float>(a, s);
}

cudaError_t launch_layer_norm_bwd(int dtype, LayerNormArgs a, float* dgain, float* dbias, cudaStream_t s) {
    return dtype == 0 ? launch_bwd_t<__nv_bfloat16>(a, dgain, dbias, s) : launch_bwd_t<float>(a, dgain, dbias, s);
}

}  // namespace muse
