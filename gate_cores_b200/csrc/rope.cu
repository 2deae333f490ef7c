// Rotary positions without a norm: Q [tokens, hq, head_dim] and K [tokens,
// hk, head_dim], of each head the first 2 * half elements rotated,
//   y_a = a c - b s,   y_b = a s + b c,   (c, s) = scale (cos, sin)(pos f_i),
// the members (a, b) of pair i adjacent (2i, 2i + 1) or half the rotated part
// apart (i, i + half); the elements behind the rotated part are copied.  The
// gradient is the same rotation by -pos f_i.
//
// Angle.  Only the fraction of a turn matters, so f_i enters as
// F = frac(f_i / 2 pi) in units of 2^-64 turns, and pos * F modulo 2^64 is the
// fraction at any 32-bit position: one integer product, no range reduction,
// and at position 2^31 still good to 2^-33 turns.  The nearest quarter
// turn is taken off in integers as well, which leaves at most an eighth of a
// turn for sincospif.  In FP32 the product pos f_i alone would be off by 0.004
// radians at position 131072.
//
// Bound: HBM, one read and one write of Q and K (in place: of their rotated
// part).  `split` warps take one token's heads; a warp keeps the token's
// (cos, sin) table in shared memory (each lane computes at most four of its
// at most 128 pairs) and gives each lane one place within a head, so a lane
// loads its own few pairs from the table once and then walks the heads, each
// item's place refilled with a later head's as soon as it is stored: four to six
// 16-byte loads a lane stay on their way.  (Refilling all places together after
// the last store: 321 us against 256 for 69632 tokens of 48 bf16 heads of 128.)
#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"

namespace muse {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

// Position of token t (the rule of core 3).  Packed documents: a search for
// the last boundary <= t with 32 probes a round; every index read lies in
// [0, num_seqs - 1] whatever the array holds.  All lanes return it.
__device__ __forceinline__ int32_t rope_position(const RopeArgs& a, int64_t t, int lane) {
    if (a.pos_mode == 0) return __ldg(a.positions + t);
    if (a.pos_mode == 1) return (int32_t)(t % a.seqlen);
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
        const int chunk = (hi - lo + 31) >> 5;
        const int probe = lo + lane * chunk;
        const bool le = probe < hi && (int64_t)__ldg(a.cu_seqlens + probe) <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int nlo = lo + (m ? 31 - __clz(m) : 0) * chunk;
        hi = min(hi, nlo + chunk);
        lo = nlo;
    }
    return (int32_t)(t - __ldg(a.cu_seqlens + lo));
}

// scale * (cos, sin) of pos * f radians; sign -1 turns the other way.  NaN for a
// frequency that is not finite, at every position (the conversions to integers
// below would make it no turn at all).
__device__ __forceinline__ float2 rope_unit(double f, int32_t pos, float scale, float sign) {
    // f / 2 pi as a sum of two doubles (1 / 2 pi = 0.15915494309189535 + -9.839338337591243e-18)
    const double hi = f * 0.15915494309189535;
    const double lo = fma(f, -9.839338337591243e-18, fma(f, 0.15915494309189535, -hi));
    // whole turns off to the nearest: exact (hi - floor(hi) would round for small negative hi)
    const unsigned long long F = (unsigned long long)(__double2ll_rn((hi - rint(hi)) * 0x1p64)) +
                                 (unsigned long long)__double2ll_rn(lo * 0x1p64);
    const unsigned long long p = F * (unsigned long long)(long long)pos;
    const unsigned n = (unsigned)((p + (1ull << 61)) >> 62);  // nearest quarter turn, modulo 4
    const long long rest = (long long)(p - ((unsigned long long)n << 62));  // [-2^61, 2^61): an eighth of a turn
    float s, c;
    // in units of pi; rounded once, so that slow pairs keep 24 bits of their sine and -pos turns exactly back
    const bool number = (__double2hiint(f) & 0x7ff00000) != 0x7ff00000;
    sincospif(number ? (float)rest * 0x1p-63f : CUDART_NAN_F, &s, &c);
    float cs = (n & 1u) ? s : c, sn = (n & 1u) ? c : s;
    if (n == 1u || n == 2u) cs = -cs;
    if (n >= 2u) sn = -sn;
    return make_float2(cs * scale, sn * scale * sign);
}

// The warp's table of the token's half pairs.
__device__ __forceinline__ void rope_table(const RopeArgs& a, int64_t t, int lane, float2* table) {
    const int32_t pos = rope_position(a, t, lane);
    for (int i = lane; i < a.half; i += 32) table[i] = rope_unit(__ldg(a.inv_freq + i), pos, a.scale, a.sign);
    __syncwarp();
}

__device__ __forceinline__ void turn(float& x, float& y, float2 u) {
    const float x0 = x, y0 = y;
    x = fmaf(-y0, u.y, x0 * u.x);
    y = fmaf(x0, u.y, y0 * u.x);
}

// Whole 16-byte vectors.  An item is what a lane takes of a head at once:
// adjacent pairs: one vector; halves (half a multiple of the vector): the two
// vectors that hold both members of V pairs, or two neighbouring vectors
// behind the rotated part.  items <= 32 of them make a head; 32 / items heads
// a step.
template <typename T, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    constexpr int NV = HALVES ? 2 : 1;        // vectors of an item
    constexpr int NP = HALVES ? V : V / 2;    // pairs of an item
    // items in flight, as many as the registers of four CTAs an SM hold: one more
    // of the halves spills (8 bytes of bf16, 32 of FP32; 69632 tokens of 48 bf16
    // heads 253.9 us with two, 256.7 with three, 279.8 with four; 8192 tokens of 40
    // FP32 heads 54.5 with three, 56.3 with four)
    constexpr int B = !HALVES ? 6 : V > 4 ? 2 : 3;
    __shared__ __align__(16) float2 tables[kRopeWarps][kMaxHalfDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = unit / a.split;
    if (t >= a.tokens) return;
    const int part = (int)(unit % a.split);
    const int nvh = a.head_dim / V;
    const int hv = a.half / V;  // HALVES: vectors from a pair's first member to its second
    const int per_step = 32 / a.items;
    const int sub = lane / a.items, item = lane - sub * a.items;
    // byte offsets of the item's vectors within a head; nrot rotated pairs
    int off0 = item * 16, off1 = off0, nrot, first = 0;
    bool two = false;
    if constexpr (HALVES) {
        nrot = item < hv ? V : 0;
        first = item * V;
        off1 = (item + hv) * 16;
        two = true;
        if (item >= hv) {
            const int v = 2 * hv + 2 * (item - hv);
            off0 = v * 16;
            off1 = off0 + 16;
            two = v + 1 < nvh;
        }
    } else {
        first = item * NP;
        nrot = min(max(a.half - first, 0), NP);  // less than NP: the rotated part ends inside this vector, or before it
    }
    const bool on = sub < per_step;
    const int heads = a.hq + a.hk;
    const int head_bytes = a.head_dim * (int)sizeof(T);
    const char* q = static_cast<const char*>(a.q) + t * a.q_stride * (int64_t)sizeof(T);
    const char* k = static_cast<const char*>(a.k) + t * a.k_stride * (int64_t)sizeof(T);
    char* qo = static_cast<char*>(a.q_out) + t * a.q_out_stride * (int64_t)sizeof(T);
    char* ko = static_cast<char*>(a.k_out) + t * a.k_out_stride * (int64_t)sizeof(T);
    const int stride = per_step * a.split;  // heads between a lane's items
    int h0 = on ? part * per_step + sub : heads;

    uint4 x[B][NV];
    auto load = [&](uint4 (&to)[NV], int hu) {
        if (hu < heads) {
            const char* p = hu < a.hq ? q + (int64_t)hu * head_bytes : k + (int64_t)(hu - a.hq) * head_bytes;
            to[0] = ld_stream(p + off0);
            if constexpr (HALVES)
                if (two) to[1] = ld_stream(p + off1);
        }
    };
#pragma unroll
    for (int u = 0; u < B; ++u) load(x[u], h0 + u * stride);  // in flight while the table is made
    float2* table = tables[warp];
    rope_table(a, t, lane, table);
    float2 cs[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) cs[p] = p < nrot ? table[first + p] : make_float2(1.0f, 0.0f);

#pragma unroll 1
    while (h0 < heads) {
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const int hu = h0 + u * stride;
            if (hu >= heads) break;
            char* p = hu < a.hq ? qo + (int64_t)hu * head_bytes : ko + (int64_t)(hu - a.hq) * head_bytes;
            if (nrot > 0) {
                float f[NV * V];
                unpack<T>(x[u][0], f);
                if constexpr (HALVES) {
                    unpack<T>(x[u][1], f + V);
#pragma unroll
                    for (int i = 0; i < V; ++i) turn(f[i], f[V + i], cs[i]);
                    x[u][1] = pack<T>(f + V);
                } else {
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        // selected, not multiplied by (1, 0): an infinity beside an unrotated element stays where it is
                        if (i < nrot) turn(f[2 * i], f[2 * i + 1], cs[i]);
                    }
                }
                uint4 y = pack<T>(f);
                if constexpr (!HALVES && V > 4) {
                    // the rotated part ends inside this vector, a pair a word: the other words keep their very bits
                    // (a NaN of 16 bits changes when it is packed)
                    if (nrot <= 1) y.y = x[u][0].y;
                    if (nrot <= 2) y.z = x[u][0].z;
                    if (nrot <= 3) y.w = x[u][0].w;
                }
                x[u][0] = y;
            }
            st_vec(p + off0, x[u][0]);
            if constexpr (HALVES)
                if (two) st_vec(p + off1, x[u][1]);
            load(x[u], hu + B * stride);
        }
        h0 += B * stride;
    }
}

// Halves whose distance is no whole number of vectors.  A warp takes as many
// heads at a time as fit kPairVecs vectors, brings them to shared memory 16
// bytes a lane, turns their pairs there element by element and stores them 16
// bytes a lane; the next heads are loaded meanwhile.  (Pairs straight from
// global memory, 2 or 4 bytes a lane: 101 us against 29 for 16384 tokens of 32
// bf16 heads of 80, 20 rotated.)
constexpr int kPairVecs = 128;
constexpr int kPairSlots = kPairVecs / 32;

// i / n for i < 512 and 0 < n <= 128, by m = ceil(2^16 / n): m n - 2^16 < n,
// so that i m / 2^16 is above i / n by less than i / 2^16 < 1 / n.
__device__ __forceinline__ int div_small(int i, uint32_t m) { return (int)(((uint32_t)i * m) >> 16); }

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(const __grid_constant__ RopeArgs a) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    __shared__ float2 tables[kRopeWarps][kMaxHalfDim];
    __shared__ __align__(16) uint4 staged[kRopeWarps][kPairVecs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = unit / a.split;
    if (t >= a.tokens) return;
    const int part = (int)(unit % a.split);
    const char* q = static_cast<const char*>(a.q) + t * a.q_stride * (int64_t)sizeof(T);
    const char* k = static_cast<const char*>(a.k) + t * a.k_stride * (int64_t)sizeof(T);
    char* qo = static_cast<char*>(a.q_out) + t * a.q_out_stride * (int64_t)sizeof(T);
    char* ko = static_cast<char*>(a.k_out) + t * a.k_out_stride * (int64_t)sizeof(T);
    const int heads = a.hq + a.hk;
    const int head_bytes = a.head_dim * (int)sizeof(T);
    const int take = a.items;                // vectors of a head that are brought (in place: those with rotated elements)
    const int at_once = kPairVecs / take;    // heads
    const uint32_t m_take = (65536u + take - 1) / take, m_half = (65536u + a.half - 1) / a.half;

    // this lane's vectors of heads h0 .. h0 + at_once - 1
    auto offset = [&](int u, int h0, int& h) {
        const int v = lane + 32 * u, in = div_small(v, m_take);
        h = v < at_once * take ? h0 + in : heads;
        return (v - in * take) * 16;
    };
    uint4 x[kPairSlots];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kPairSlots; ++u) {
            int h;
            const int off = offset(u, h0, h);
            if (h < heads)
                x[u] = ld_stream((h < a.hq ? q + (int64_t)h * head_bytes : k + (int64_t)(h - a.hq) * head_bytes) + off);
        }
    };
    int h0 = part * at_once;
    load(h0);
    float2* table = tables[warp];
    rope_table(a, t, lane, table);
    uint4* box = staged[warp];
    T* elements = reinterpret_cast<T*>(box);
    for (; h0 < heads; h0 += at_once * a.split) {
#pragma unroll
        for (int u = 0; u < kPairSlots; ++u) box[lane + 32 * u] = x[u];  // (past the heads: not used)
        load(h0 + at_once * a.split);
        __syncwarp();
        const int pairs = min(at_once, heads - h0) * a.half;
        for (int e = lane; e < pairs; e += 32) {
            const int h = div_small(e, m_half), i = e - h * a.half;
            T* p = elements + h * take * V + i;
            float f = (float)p[0], g = (float)p[a.half];
            turn(f, g, table[i]);
            p[0] = (T)f;
            p[a.half] = (T)g;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kPairSlots; ++u) {
            int h;
            const int off = offset(u, h0, h);
            if (h < heads)
                st_vec((h < a.hq ? qo + (int64_t)h * head_bytes : ko + (int64_t)(h - a.hq) * head_bytes) + off, box[lane + 32 * u]);
        }
        __syncwarp();
    }
}

__global__ void rope_frequencies_kernel(const __grid_constant__ RopeFreqArgs a) {
    pdl_begin();
    const int i = threadIdx.x;
    if (i < a.n) a.out[i] = a.inv_freq[i];
}

template <typename T>
cudaError_t launch_rope_t(RopeArgs a, bool halves, cudaStream_t s) {
    constexpr int V = Vec<T>::N;
    const bool vectors = !halves || a.half % V == 0;
    const int nvh = a.head_dim / V;
    int steps;
    if (!vectors) {
        a.items = a.in_place ? (2 * a.half + V - 1) / V : nvh;
        const int per_step = kPairVecs / a.items;
        steps = (a.hq + a.hk + per_step - 1) / per_step;
    } else {
        // what is behind the rotated part is left alone in place
        if (halves) {
            const int hv = a.half / V, rest = nvh - 2 * hv;
            a.items = hv + (a.in_place ? 0 : (rest + 1) / 2);
        } else {
            a.items = a.in_place ? (2 * a.half + V - 1) / V : nvh;
        }
        const int per_step = 32 / a.items;
        steps = (a.hq + a.hk + per_step - 1) / per_step;
    }
    // one warp takes a token; where that leaves most of the GPU idle, up to
    // eight share one, down to a step each
    a.split = 1;
    while (a.split < kRopeWarps && a.split < steps && a.tokens * a.split < (int64_t)sm_count() * kRopeWarps * 2) a.split *= 2;
    const int64_t grid = (a.tokens * a.split + kRopeWarps - 1) / kRopeWarps;
    if (!vectors) return launch_pdl(rope_pairs_kernel<T>, (unsigned)grid, kRopeThreads, 0, s, a);
    return halves ? launch_pdl(rope_kernel<T, true>, (unsigned)grid, kRopeThreads, 0, s, a)
                  : launch_pdl(rope_kernel<T, false>, (unsigned)grid, kRopeThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_rope(int dtype, bool halves, const RopeArgs& a, cudaStream_t s) {
    return dtype == 0 ? launch_rope_t<__nv_bfloat16>(a, halves, s) : launch_rope_t<float>(a, halves, s);
}

cudaError_t launch_rope_frequencies(const RopeFreqArgs& a, cudaStream_t s) {
    return launch_pdl(rope_frequencies_kernel, 1u, (unsigned)kMaxHalfDim, 0, s, a);
}

}  // namespace muse
