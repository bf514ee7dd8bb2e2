// la.cuh -- what the kernels of linear attention with a fixed decay a head share: the norm and rotation
// of keys and queries.  How a warp holds rows of a state, and the sums along them, are gdn.cuh's.
//
// The operation, per head h of group g with the state S (head_dim x d_state, d_state contiguous):
//   S <- e^log_decay S + v k^T,   y = scale * S q
// A row of S needs nothing of the other rows.
//
// Angles: position * inv_freq can be 1e5 and more, where fp32 has two digits left behind the point.  So a
// frequency becomes a 64-bit fraction of a turn a position; its product with the position, modulo 2^64,
// is the angle modulo a whole turn to 2^-32 or better, whatever the position.  Integers do it, because fp64
// arithmetic runs at a hundredth of fp32's rate here.
#pragma once

#include "gdn.cuh"

namespace ms {
namespace la {

using namespace gdn;

// Norm and rotation of a call.
struct QkPrep {
    const float *kw, *qw, *inv_freq;
    const int32_t *pos;
    float eps;
    int norm, half, inter;  // half: pairs turned, rot_dim / 2
};

// e^l as the sum of two fp32 numbers: a head that remembers 1 / |l| tokens multiplies what rounding a single one to 24 bits
// takes by that many.  The logarithm's own error is relative to l, so that it is no larger than one such rounding over that time.
__device__ __forceinline__ float2 decay_of(float l) {
    const float hi = expf(l);
    return make_float2(hi, hi > 1e-30f && hi < 1.0f ? hi * (l - logf(hi)) : 0.0f);
}
// S <- d S + v k on two of a row's values at a time.
__device__ __forceinline__ uint64_t decayed_add(uint64_t hi, uint64_t lo, uint64_t S, uint64_t v, uint64_t k) {
    return fma2(hi, S, fma2(lo, S, mul2(v, k)));
}

// Turns a position, as a fraction of 2^64 (0 <= f; exact to 2^-62 of itself or 2^-64).
__device__ __forceinline__ uint64_t turns(float f) {
    const uint32_t bits = __float_as_uint(f), e = (bits >> 23) & 255u;
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - (int)(e ? e : 1u);                  // f = m 2^-s
    const uint64_t K = 2935890503282001226ull;              // 2^64 / (2 pi)
    const uint64_t hi = __umul64hi(m, K), lo = m * K;
    if (s <= 0) return s > -64 ? lo << -s : 0;
    if (s < 64) return (lo >> s) | (hi << (64 - s));
    return s < 128 ? hi >> (s - 64) : 0;
}
// Cosine and sine of `pos` steps of t.
__device__ __forceinline__ float2 turned(uint64_t t, int32_t pos) {
    const int32_t a = (int32_t)((uint64_t)((int64_t)pos * (int64_t)t) >> 32);  // in 2^-32 of a turn, from -1/2 to 1/2
    float2 r;
    sincospif((float)a * 4.656612873077393e-10f, &r.y, &r.x);                  // (2^-31: half turns)
    return r;
}

// One row's norm and rotation in registers: a lane holds 8 consecutive values of N, LPR = N / 8 lanes a row.
// w: the lane's 8 weights; table: cosine and sine of the row's `half` angles.  All 32 lanes take part.
template <int N>
__device__ __forceinline__ void norm_rotate(float (&x)[8], const float (&w)[8], const QkPrep &p, const float2 *table, int lane) {
    constexpr int LPR = N / 8;
    if (p.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<LPR>(ss) * (1.0f / N) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
    }
    if (p.half) {
        const int idx = lane & (LPR - 1);
        if (p.inter) {
            if (idx * 4 < p.half) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t = table[idx * 4 + e];
                    const float a = x[2 * e], b = x[2 * e + 1];
                    x[2 * e] = a * t.x - b * t.y;
                    x[2 * e + 1] = b * t.x + a * t.y;
                }
            }
        } else {
            const int far = p.half / 8;  // lanes between the halves of a pair
            const bool first = idx < far, in = idx < 2 * far;
            const int with = in ? (first ? lane + far : lane - far) : lane;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_sync(0xffffffffu, x[e], with);
                const float2 t = in ? table[(first ? idx : idx - far) * 8 + e] : make_float2(1.0f, 0.0f);
                x[e] = first ? x[e] * t.x - o * t.y : (in ? x[e] * t.x + o * t.y : x[e]);
            }
        }
    }
}

template <int N>
__device__ __forceinline__ void norm_weights(const float *w, int lane, float (&to)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) to[e] = w ? __ldg(w + (lane & (N / 8 - 1)) * 8 + e) : 1.0f;
}

// The checks of a call's norm and rotation.
inline int check_prep(int N, int32_t qk_norm, float eps, const int32_t *pos, const float *inv_freq, int32_t rot_dim) {
    if (rot_dim < 0 || (rot_dim && (!pos || !inv_freq)) || (qk_norm && !(eps >= 0.0f))) return MAMBA_EINVAL;
    if (rot_dim > N || rot_dim % 16) return MAMBA_EUNSUPPORTED;
    return MAMBA_OK;
}
inline QkPrep make_prep(int32_t qk_norm, const float *kw, const float *qw, float eps, const int32_t *pos,
                        const float *inv_freq, int32_t rot_dim, int32_t inter) {
    QkPrep p;
    p.kw = qk_norm ? kw : nullptr;
    p.qw = qk_norm ? qw : nullptr;
    p.inv_freq = inv_freq;
    p.pos = pos;
    p.eps = eps;
    p.norm = qk_norm != 0;
    p.half = rot_dim / 2;
    p.inter = inter != 0;
    return p;
}

}  // namespace la
}  // namespace ms
