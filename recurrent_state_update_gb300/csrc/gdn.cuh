// gdn.cuh -- what the kernels of the gated delta rule share: the layout of a head's state over a
// warp, the reductions along its rows, the gates, and 8-element loads and stores.
//
// The operation, per head h of group g with the state S (head_dim x d_state, d_state contiguous):
//   a = exp(Delta * A),  Delta = softplus(dt + dt_bias),  b = sigmoid(beta)
//   u = b * (v - a * S k),   S <- a * S + u k^T,   y = scale * S q
// with k and q scaled to unit length.  A row of S needs nothing of the other rows, so rows are
// spread over warps and blocks at will; each row needs two sums over its d_state values, S k and
// S q of the OLD state, because S q of the new one is a * (S q) + u * (k . q).
#pragma once

#include "common.cuh"

namespace ms {
namespace gdn {

constexpr float kNormEps = 1e-6f;  // added to the squared length of k and q before the root
constexpr int kMaxTok = 8;         // tokens of one decode call

// The gates' and scalings' switches of a call.
struct Gates {
    const float *A, *dt_bias;
    int dt_bf16, dt_softplus, beta_sigmoid, l2norm;
    float scale;
};

// log of the decay a of one token and head (<= 0 for A <= 0), from the raw step.
__device__ __forceinline__ float log_decay(const Gates &g, float dt, int h) {
    const float s = dt + (g.dt_bias ? g.dt_bias[h] : 0.0f);
    return (g.dt_softplus ? softplus_f(s) : s) * g.A[h];
}
__device__ __forceinline__ float write_gate(const Gates &g, float beta) {
    return g.beta_sigmoid ? __fdividef(1.0f, 1.0f + expf(-beta)) : beta;
}
// The factor that scales a key or query of squared length ss.
__device__ __forceinline__ float unit_factor(const Gates &g, float ss) {
    return g.l2norm ? rsqrtf(ss + kNormEps) : 1.0f;
}

// Two fp32 values in a register pair, for the two-wide multiply-add.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Eight consecutive values <-> fp32, past L1 (each state byte is used once per call).
__device__ __forceinline__ void load8_stream(const bf16 *p, float (&f)[8]) {
    unpack16(__ldcs(reinterpret_cast<const uint4 *>(p)), f);
}
__device__ __forceinline__ void load8_stream(const float *p, float (&f)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p)), b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void store8_stream(bf16 *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p), pack16(f));
}
__device__ __forceinline__ void store8_stream(float *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                                    __float_as_uint(f[3])));
    __stcs(reinterpret_cast<uint4 *>(p) + 1, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                                        __float_as_uint(f[6]), __float_as_uint(f[7])));
}
// The same through the caches (keys and queries, which every block of a head reads).
__device__ __forceinline__ void load8(const bf16 *p, float (&f)[8]) {
    unpack16(*reinterpret_cast<const uint4 *>(p), f);
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <typename T>
__device__ __forceinline__ void load_row(const T *p, uint64_t (&v)[4]) {
    float f[8];
    load8_stream(p, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}
__device__ __forceinline__ void load_row_shared(const float *p, uint64_t (&v)[4]) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
// Eight state values on their way: loaded now, unpacked when they are needed.
struct RawBf16 {
    uint4 w;
    __device__ __forceinline__ void load(const bf16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void unpack(uint64_t (&v)[4]) const {
        float f[8];
        unpack16(w, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
    }
};
struct RawF32 {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const uint4 *>(p));
        b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void unpack(uint64_t (&v)[4]) const {
        v[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
        v[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        v[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
        v[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
    }
};
template <typename T> struct RawOf;
template <> struct RawOf<bf16> { using type = RawBf16; };
template <> struct RawOf<float> { using type = RawF32; };
template <typename T>
__device__ __forceinline__ void store_row(T *p, const uint64_t (&v)[4]) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) unpair(v[e], f[2 * e], f[2 * e + 1]);
    store8_stream(p, f);
}

// How a warp holds rows of S: LPR lanes a row with PIECES times 8 consecutive values each (a piece of all lanes
// after the other), RPW rows side by side, RT rows a lane (row r * RPW + lane / LPR of the warp's RPW * RT).
template <int N, int RT_, int PIECES = 1>
struct RowMap {
    static constexpr int LPR = N / (8 * PIECES), RPW = 32 / LPR, RT = RT_, ROWS = RPW * RT, PAIRS = 4 * PIECES;
    static constexpr int SHARE = LPR / RT;   // lanes of a row's that end up with the same row's sum
    static_assert(LPR >= RT, "more sums than lanes of a row");
};

// Sums val[0..NV) over the M*2 lanes that differ in the lane bits 2M-1 .. 0.  Halves the number of
// sums with each exchange while there is more than one (NV - 1 exchanges, where a butterfly of each
// sum would take NV * log2): lane l ends with the sum of index l / (2M / NV).
template <int NV, int M>
__device__ __forceinline__ float reduce_rows(float (&val)[NV], int lane) {
    if constexpr (M == 0) {
        static_assert(NV == 1, "as many lanes as sums");
        return val[0];
    } else if constexpr (NV == 1) {
        val[0] += __shfl_xor_sync(0xffffffffu, val[0], M);
        return reduce_rows<1, M / 2>(val, lane);
    } else {
        float half[NV / 2];
        const bool up = lane & M;
#pragma unroll
        for (int j = 0; j < NV / 2; ++j) {
            const float keep = up ? val[NV / 2 + j] : val[j], send = up ? val[j] : val[NV / 2 + j];
            half[j] = keep + __shfl_xor_sync(0xffffffffu, send, M);
        }
        return reduce_rows<NV / 2, M / 2>(half, lane);
    }
}

// Sum over the LPR lanes of a row, in every one of them.
template <int LPR>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int m = LPR / 2; m; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// S x of the rows a warp holds, that of row r in the lanes of index r, where a lane's index is (its place in
// the row) / SHARE.
template <typename Map>
__device__ __forceinline__ float row_sum(const uint64_t (&S)[Map::RT][Map::PAIRS], const uint64_t (&x)[Map::PAIRS], int lane) {
    float val[Map::RT];
#pragma unroll
    for (int r = 0; r < Map::RT; ++r) {
        uint64_t p = mul2(S[r][0], x[0]);
#pragma unroll
        for (int e = 1; e < Map::PAIRS; ++e) p = fma2(S[r][e], x[e], p);
        float lo, hi;
        unpair(p, lo, hi);
        val[r] = lo + hi;
    }
    return reduce_rows<Map::RT, Map::LPR / 2>(val, lane);
}
// S <- a S + u (rk k)^T, u of row r from the lanes of index r; a may differ by column (int8 codes carry their
// scale in it).
template <typename Map>
__device__ __forceinline__ void write_rows(uint64_t (&S)[Map::RT][Map::PAIRS], const uint64_t (&a)[Map::PAIRS],
                                           const uint64_t (&k)[Map::PAIRS], float u, float rk, int lane) {
    const float own = u * rk;
#pragma unroll
    for (int r = 0; r < Map::RT; ++r) {
        const float uk = __shfl_sync(0xffffffffu, own, (lane & ~(Map::LPR - 1)) + r * Map::SHARE);
        const uint64_t uk2 = pair(uk, uk);
#pragma unroll
        for (int e = 0; e < Map::PAIRS; ++e) S[r][e] = fma2(a[e], S[r][e], mul2(uk2, k[e]));
    }
}
// One token on the rows a warp holds: the new states, and scale * S q of the row of this lane's index.  k, q:
// this lane's 8 values, unscaled; rk, rq: their factors (rq with the output scale); ukq: their scaled
// product k . q with the output scale (S q of the new state is a * (S q) + u * (k . q)); v: the row's value.
template <typename Map>
__device__ __forceinline__ float token_rows(uint64_t (&S)[Map::RT][Map::PAIRS], const uint64_t (&k)[Map::PAIRS],
                                            const uint64_t (&q)[Map::PAIRS], float rk, float rq, float ukq, float a,
                                            float b, float v, int lane) {
    const float sq = row_sum<Map>(S, q, lane);
    const float u = b * (v - a * rk * row_sum<Map>(S, k, lane));
    uint64_t as[Map::PAIRS];
#pragma unroll
    for (int e = 0; e < Map::PAIRS; ++e) as[e] = pair(a, a);
    write_rows<Map>(S, as, k, u, rk, lane);
    return fmaf(a * rq, sq, u * ukq);
}

// Checks that hold for every call on a layer; the state shapes are those of the decode kernels.
inline int check_layer(const mamba_layer_desc *d) {
    const int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    return mamba_decode_supported(d);
}
inline Gates make_gates(const mamba_layer_desc *d, const float *A, const float *dt_bias, int dt_softplus,
                        int beta_sigmoid, int qk_l2norm, float scale) {
    Gates g;
    g.A = A;
    g.dt_bias = dt_bias;
    g.dt_bf16 = d->dt_dtype == MAMBA_BF16;
    g.dt_softplus = dt_softplus != 0;
    g.beta_sigmoid = beta_sigmoid != 0;
    g.l2norm = qk_l2norm != 0;
    g.scale = scale;
    return g;
}

}  // namespace gdn
}  // namespace ms
