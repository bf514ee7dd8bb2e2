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
// takes by that many.  The logarithm's own error is 2^-24 of l, no larger than one such rounding over that time, or 2^-45.
// The first is taken from below and the second is never zero, unless e^l is, so that an infinite state stays infinite: of
// numbers of opposite signs, or of a zero, it would make NaN.
__device__ __forceinline__ float2 decay_of(float l) {
    const float e = expf(l);
    if (!(e > 0.0f && e <= 1.0f)) return make_float2(e, 0.0f);
    const float hi = e - e * 0x1p-21f;                                // (expf is off by 2^-22 of itself at most)
    const float d = l - logf(hi);                                     // e^l = hi e^d
    return make_float2(hi, fmaxf(hi * fmaf(0.5f * d, d, d), 0x1p-149f));
}
// S <- d S + x, and d S + v k, on two of a row's values at a time.
__device__ __forceinline__ uint64_t decayed(uint64_t hi, uint64_t lo, uint64_t S, uint64_t x) { return fma2(hi, S, fma2(lo, S, x)); }
__device__ __forceinline__ uint64_t decayed_add(uint64_t hi, uint64_t lo, uint64_t S, uint64_t v, uint64_t k) {
    return decayed(hi, lo, S, mul2(v, k));
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
    // in 2^-32 of a turn, from -1/2 to 1/2; without signs, since the product passes 2^63 and is meant to wrap
    const int32_t a = (int32_t)(uint32_t)(((uint64_t)(int64_t)pos * t) >> 32);
    float2 r;
    sincospif((float)a * 4.656612873077393e-10f, &r.y, &r.x);                  // (2^-31: half turns)
    return r;
}

// One row's norm and rotation in registers, N / (2 V) lanes a row, 2 V values a lane: V from `a` and V from `b` of the row.
// Where halves are rotated against each other these are the two halves of V pairs, so that no lane needs another's
// values but for the sum of squares; elsewhere b is a + V.  Either way lane idx turns the angles V idx .. V idx + V - 1.
template <int V>
struct LaneRow {
    int a, b, angle;
    bool turns;  // whether this lane's values are among those rotated
    __device__ __forceinline__ LaneRow(const QkPrep &p, int idx) : angle(V * idx), turns(V * idx < p.half) {
        const bool halves = turns && !p.inter;
        a = halves ? V * idx : 2 * V * idx;
        b = halves ? p.half + V * idx : 2 * V * idx + V;
    }
};
// w: the lane's weights; t: cosines and sines of its angles.  All lanes of the row take part.
template <int N, int V>
__device__ __forceinline__ void norm_rotate(float (&x)[2 * V], const float (&w)[2 * V], const QkPrep &p, const float2 (&t)[V],
                                            const LaneRow<V> &l) {
    if (p.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(sum_lanes<N / (2 * V)>(ss) * (1.0f / N) + p.eps);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) x[e] *= r * w[e];
    }
    auto turn = [](float &u, float &v, float2 t) {
        const float a = u, b = v;
        u = a * t.x - b * t.y;
        v = b * t.x + a * t.y;
    };
    if (l.turns && p.inter) {
#pragma unroll
        for (int e = 0; e < V; ++e) turn(x[2 * e], x[2 * e + 1], t[e]);
    } else if (l.turns) {
#pragma unroll
        for (int e = 0; e < V; ++e) turn(x[e], x[V + e], t[e]);
    }
}
template <int V>
__device__ __forceinline__ void norm_weights(const float *w, const LaneRow<V> &l, float (&to)[2 * V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        to[e] = w ? __ldg(w + l.a + e) : 1.0f;
        to[V + e] = w ? __ldg(w + l.b + e) : 1.0f;
    }
}
// V values, as they are stored, and in fp32.
template <typename T, int V> struct Some;
template <int V> struct Some<bf16, V> {
    uint2 v[V / 4];
    __device__ __forceinline__ void load(const bf16 *p) {
        if constexpr (V == 8) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            v[0] = make_uint2(x.x, x.y), v[1] = make_uint2(x.z, x.w);
        } else {
            v[0] = *reinterpret_cast<const uint2 *>(p);
        }
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            f[4 * i] = __uint_as_float(v[i].x << 16), f[4 * i + 1] = __uint_as_float(v[i].x & 0xffff0000u);
            f[4 * i + 2] = __uint_as_float(v[i].y << 16), f[4 * i + 3] = __uint_as_float(v[i].y & 0xffff0000u);
        }
    }
};
template <int V> struct Some<float, V> {
    float4 v[V / 4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) v[i] = reinterpret_cast<const float4 *>(p)[i];
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) f[4 * i] = v[i].x, f[4 * i + 1] = v[i].y, f[4 * i + 2] = v[i].z, f[4 * i + 3] = v[i].w;
    }
};

// The checks of a layer (check_desc's, and check_layer's for the compiled shapes) with what belongs to a convolution and to steps
// replaced: these layers have neither.
inline mamba_layer_desc without_conv(const mamba_layer_desc &d) {
    mamba_layer_desc u = d;
    u.conv_kernel = 2;
    u.num_spec = 0;
    u.conv_dtype = u.dt_dtype = d.act_dtype;
    return u;
}
inline int check_la_desc(const mamba_layer_desc *d) {
    if (!d) return MAMBA_EINVAL;
    const mamba_layer_desc u = without_conv(*d);
    return check_desc(&u);
}
inline int check_la_layer(const mamba_layer_desc *d) {
    if (!d) return MAMBA_EINVAL;
    const mamba_layer_desc u = without_conv(*d);
    return check_layer(&u);
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
