// gdn_step.cu -- the recurrent step of the gated delta rule over a slot pool, for one token or a
// few drafted ones a request, and for one token on int8 cache entries.
//
// Mathematics and row layout: gdn.cuh.  Both are streaming passes: an element of the state is read
// once and written once (once a draft) for about 8 floating operations, so device memory bounds
// them, and a call of few rows is bound by the latency of one load, two short chains of shuffles
// and one store.  Rows of a head are independent but for the int8 scales' maxima, so a block takes a few
// of them, or there all of a head's.
#include "gdn.cuh"
#include "int8_entry.h"

namespace ms {

using namespace gdn;

namespace {

constexpr float kLeast = 1e-35f;  // a column no larger has codes of zero (127 over it could overflow)

struct StepArgs {
    void *pool;
    int64_t stride, num_slots;  // elements
    const int32_t *slot, *scratch;
    int ntok;
    const void *xbc, *dt, *beta;
    Gates gates;
    void *y;
    int32_t *err;
    int H, G, HG, Cd, splits;
};

// A token's scalars and this lane's keys and queries.
template <typename Map, typename ActT>
struct TokenIn {
    uint64_t k[4], q[4];
    float rk, rq, ukq, a, b;
    float kk, qq, kq;  // this lane's parts of the lengths and of k . q
    __device__ __forceinline__ void load_vectors(const ActT *row, int HP, int GN, int grp, int N, int lane) {
        const int c = (lane & (Map::LPR - 1)) * 8;
        unpack(row + HP + grp * N + c, row + HP + GN + grp * N + c);
    }
    __device__ __forceinline__ void unpack(const ActT *ksrc, const ActT *qsrc) {
        float kf[8], qf[8];
        load8(ksrc, kf);
        load8(qsrc, qf);
        kk = qq = kq = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            kk = fmaf(kf[e], kf[e], kk);
            qq = fmaf(qf[e], qf[e], qq);
            kq = fmaf(kf[e], qf[e], kq);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[e] = pair(kf[2 * e], kf[2 * e + 1]);
            q[e] = pair(qf[2 * e], qf[2 * e + 1]);
        }
    }
    __device__ __forceinline__ void load_scalars(const Gates &g, int h, const void *dt, const void *beta, int64_t th) {
        const float dtv = load_scalar(dt, th, g.dt_bf16), bv = load_scalar(beta, th, g.dt_bf16);
        rk = unit_factor(g, sum_lanes<Map::LPR>(kk));
        rq = unit_factor(g, sum_lanes<Map::LPR>(qq)) * g.scale;
        ukq = sum_lanes<Map::LPR>(kq) * rk * rq;
        a = expf(log_decay(g, dtv, h));
        b = write_gate(g, bv);
    }
};

// The row checks of a step: its slot, or -1 for a row that is skipped (padding, or flagged).
__device__ __forceinline__ int32_t step_slot(const StepArgs &p, int i) {
    const int32_t s = p.slot[i];
    if (s == -1) return -1;
    bool bad = s < -1 || s >= p.num_slots;
    if (p.scratch)
        for (int j = 0; j < p.ntok; ++j) {
            const int32_t d = p.scratch[(int64_t)i * p.ntok + j];
            bad |= d < -1 || d >= p.num_slots;
        }
    if (bad && threadIdx.x == 0) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
    return bad ? -1 : s;
}

// One token.  Block (head and share of its rows, batch row).
template <typename StateT, typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(64) k_gdn_step(const StepArgs p) {
    using Map = RowMap<N, RT>;
    using Raw = typename RawOf<StateT>::type;
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t s = step_slot(p, i);
    if (s < 0) return;
    const int row0 = (split * (blockDim.x >> 5) + warp) * Map::ROWS;
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE;
    StateT *state = static_cast<StateT *>(p.pool) + s * p.stride + ((int64_t)h * P + row0 + sub) * N +
                    (lane & (Map::LPR - 1)) * 8;
    Raw raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].load(state + r * Map::RPW * N);
    const int vrow = row0 + idx * Map::RPW + sub;
    const int64_t th = (int64_t)i * p.H + h;
    const ActT *xbc = static_cast<const ActT *>(p.xbc) + (int64_t)i * p.Cd;
    const float v = to_f32(xbc[h * P + vrow]);
    TokenIn<Map, ActT> in;
    in.load_vectors(xbc, p.H * P, p.G * N, h / p.HG, N, lane);
    in.load_scalars(p.gates, h, p.dt, p.beta, th);
    uint64_t S[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].unpack(S[r]);
    const float out = token_rows<Map>(S, in.k, in.q, in.rk, in.rq, in.ukq, in.a, in.b, v, lane);
    if ((lane & (Map::SHARE - 1)) == 0) static_cast<ActT *>(p.y)[th * P + vrow] = from_f32<ActT>(out);
#pragma unroll
    for (int r = 0; r < RT; ++r) store_row(state + r * Map::RPW * N, S[r]);
}

// Several tokens in order, the state after each into its scratch slot when there are some, else the last
// one's into the row's own.  Block (head and share of its rows, batch row).  While the state is on its way the
// tokens' keys, queries, values and scalars are brought to shared memory, a token to each LPR lanes, so that
// the tokens follow one another without a wait on memory: 4 tokens into scratch slots for 48 rows of 32 heads of
// 128 x 128 take 43.0 us, 0.88 of what a copy of those bytes takes (48.5 with each token's loads where it is used),
// for 61 rows of 128 heads of 64 x 128 99.6 us, 0.96 (111.8).
template <typename StateT, typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(64) k_gdn_tokens_step(const StepArgs p) {
    using Map = RowMap<N, RT>;
    using Raw = typename RawOf<StateT>::type;
    __shared__ __align__(16) float ks[kMaxTok][N], qs[kMaxTok][N];
    __shared__ float vs[kMaxTok][2 * Map::ROWS], scalars[kMaxTok][5];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int32_t s = step_slot(p, i);
    if (s < 0) return;
    const int row0 = split * warps * Map::ROWS;  // the block's
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE, col = (lane & (Map::LPR - 1)) * 8;
    const int lrow = warp * Map::ROWS + idx * Map::RPW + sub;
    StateT *pool = static_cast<StateT *>(p.pool);
    const int64_t off = ((int64_t)h * P + row0 + warp * Map::ROWS + sub) * N + col;
    Raw raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].load(pool + s * p.stride + off + (int64_t)r * Map::RPW * N);
    const ActT *xbc = static_cast<const ActT *>(p.xbc) + (int64_t)i * p.ntok * p.Cd;
    for (int base = 0; base < p.ntok; base += warps * Map::RPW) {
        const int own = base + warp * Map::RPW + sub, j = min(own, p.ntok - 1);
        TokenIn<Map, ActT> in;
        in.load_vectors(xbc + (int64_t)j * p.Cd, p.H * P, p.G * N, h / p.HG, N, lane);
        in.load_scalars(p.gates, h, p.dt, p.beta, ((int64_t)i * p.ntok + j) * p.H + h);
        if (own == j) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                *reinterpret_cast<ulonglong2 *>(&ks[j][col + 2 * e]) = make_ulonglong2(in.k[e], in.k[e + 1]);
                *reinterpret_cast<ulonglong2 *>(&qs[j][col + 2 * e]) = make_ulonglong2(in.q[e], in.q[e + 1]);
            }
            if (col == 0) {
                float *to = scalars[j];
                to[0] = in.rk, to[1] = in.rq, to[2] = in.ukq, to[3] = in.a, to[4] = in.b;
            }
        }
    }
    for (int e = threadIdx.x; e < p.ntok * warps * Map::ROWS; e += blockDim.x) {
        const int j = e / (warps * Map::ROWS), r = e % (warps * Map::ROWS);
        vs[j][r] = to_f32(xbc[(int64_t)j * p.Cd + h * P + row0 + r]);
    }
    uint64_t S[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].unpack(S[r]);
    __syncthreads();
    ActT *y = static_cast<ActT *>(p.y) + ((int64_t)i * p.ntok * p.H + h) * P + row0 + lrow;
    for (int j = 0; j < p.ntok; ++j, y += (int64_t)p.H * P) {
        uint64_t k[4], q[4];
        load_row_shared(&ks[j][col], k);
        load_row_shared(&qs[j][col], q);
        const float *in = scalars[j];
        const float out = token_rows<Map>(S, k, q, in[0], in[1], in[2], in[3], in[4], vs[j][lrow], lane);
        if ((lane & (Map::SHARE - 1)) == 0) *y = from_f32<ActT>(out);
        const int32_t d = p.scratch ? p.scratch[(int64_t)i * p.ntok + j] : (j == p.ntok - 1 ? s : -1);
        if (d >= 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r) store_row(pool + d * p.stride + off + (int64_t)r * Map::RPW * N, S[r]);
        }
    }
}

struct Int8Args {
    unsigned char *store;
    int64_t num_entries, entry_bytes, scale_off;
    const int32_t *entry;
    const void *xbc, *dt, *beta;
    Gates gates;
    void *y;
    int32_t *err;
    int H, G, HG, Cd;
};

// Codes to fp32 and back without conversion instructions, which run at a quarter of the rate: a byte
// with its sign bit flipped, as the low mantissa bits of 2^23, is 2^23 + 128 + code; and a sum with 1.5 * 2^23
// rounds to the nearest integer, ties to even, and holds it in its low bits.
__device__ __forceinline__ void codes_to_f32(uint2 w, uint64_t (&v)[4]) {
    const uint32_t x[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
    const uint64_t bias = pair(-8388736.0f, -8388736.0f);  // -(2^23 + 128)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = __byte_perm(x[e >> 1], 0x4b000000u, 0x7440u | (e & 1) * 2);
        const uint32_t hi = __byte_perm(x[e >> 1], 0x4b000000u, 0x7441u + (e & 1) * 2);
        v[e] = pair(__uint_as_float(lo), __uint_as_float(hi));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v[e]) : "l"(bias));
    }
}
__device__ __forceinline__ uint2 f32_to_codes(const uint64_t (&v)[4], const uint64_t (&inv)[4]) {
    const uint64_t round = pair(12582912.0f, 12582912.0f);
    uint32_t half[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t f = fma2(v[e], inv[e], round);  // (at most 127 and a rounding error: the nearest integer needs no bound)
        float lo, hi;
        unpair(f, lo, hi);
        half[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
    }
    return make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
}

// The larger of two magnitudes, or NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Block (head, batch row): all rows of the head, because a scale covers a column of it.  Codes become fp32
// on load; what belongs to a column (its scale, key and query) is made once for the block; the new state is
// scaled by the new column maxima (over the warps through shared memory) and rounded to the grid of
// step max/127, as the int8 store does; a column that holds a NaN or an infinity has no such grid and gets a NaN as
// its scale, so that it reads as NaN from then on.  At 192 rows of 32 heads of 128 x 128 a step moves 213 MB in
// 54.4 us, 0.57 of what a copy moves.  That is latency: 30 million warp instructions (9 a value: two products, the
// update, the maximum, and bytes to fp32 and back) fill 45 % of the issue slots and 33 % of the memory's time, because
// 168 registers a thread leave 11 warps an SM, whose blocks each load once, meet at three barriers and store, with
// nothing of another head on its way meanwhile.
template <typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(P / RowMap<N, RT>::ROWS * 32) k_gdn_step_int8(const Int8Args p) {
    using Map = RowMap<N, RT>;
    constexpr int WARPS = P / Map::ROWS;
    // by column: largest magnitudes by warp; keys and queries times the scales; scales; keys; what codes are
    // formed with
    __shared__ __align__(16) float top[WARPS][N], ks[N], qs[N], sa[N], kf[N], inv[N];
    __shared__ float scalars[5];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t e = p.entry[i];
    if (e == -1) return;  // padding row
    if (e < -1 || e >= p.num_entries) {
        if (threadIdx.x == 0) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        return;
    }
    unsigned char *ent = p.store + e * p.entry_bytes;
    const int col = (lane & (Map::LPR - 1)) * 8, sub = lane / Map::LPR, row0 = warp * Map::ROWS;
    const int idx = (lane & (Map::LPR - 1)) / Map::SHARE, vrow = row0 + idx * Map::RPW + sub;
    unsigned char *codes = ent + ((int64_t)h * P + row0 + sub) * N + col;
    float *scales = reinterpret_cast<float *>(ent + p.scale_off) + (int64_t)h * N;
    uint2 raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r] = __ldcs(reinterpret_cast<const uint2 *>(codes + r * Map::RPW * N));
    const int64_t th = (int64_t)i * p.H + h;
    const ActT *xbc = static_cast<const ActT *>(p.xbc) + (int64_t)i * p.Cd;
    const ActT *ksrc = xbc + p.H * P + (h / p.HG) * N, *qsrc = ksrc + p.G * N;
    const float v = to_f32(xbc[h * P + vrow]);
    for (int c = threadIdx.x; c < N; c += 32 * WARPS) {
        const float sc = scales[c], k = to_f32(ksrc[c]);
        ks[c] = k * sc;
        qs[c] = to_f32(qsrc[c]) * sc;
        sa[c] = sc;
        kf[c] = k;
    }
    if (warp == WARPS - 1) {  // the token's scalars, once for the block
        TokenIn<Map, ActT> in;
        in.unpack(ksrc + col, qsrc + col);
        in.load_scalars(p.gates, h, p.dt, p.beta, th);
        if (lane == 0) scalars[0] = in.rk, scalars[1] = in.rq, scalars[2] = in.ukq, scalars[3] = in.a, scalars[4] = in.b;
    }
    uint64_t S[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) codes_to_f32(raw[r], S[r]);
    __syncthreads();
    const float a = scalars[3], rk = scalars[0];
    uint64_t k[4], x[4];
    load_row_shared(qs + col, x);
    const float sq = row_sum<Map>(S, x, lane);
    load_row_shared(ks + col, x);
    const float u = scalars[4] * (v - a * rk * row_sum<Map>(S, x, lane));
    const float out = fmaf(a * scalars[1], sq, u * scalars[2]);
    if ((lane & (Map::SHARE - 1)) == 0) static_cast<ActT *>(p.y)[th * P + vrow] = from_f32<ActT>(out);
    load_row_shared(kf + col, k);
    load_row_shared(sa + col, x);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = mul2(x[c], pair(a, a));
    write_rows<Map>(S, x, k, u, rk, lane);
    {
        float m[8] = {};
#pragma unroll
        for (int r = 0; r < RT; r += 2)
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // (of two rows at a time: the maximum takes three numbers)
                float lo, hi, lo2 = 0.0f, hi2 = 0.0f;
                unpair(S[r][c], lo, hi);
                if (r + 1 < RT) unpair(S[r + 1][c], lo2, hi2);
                asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m[2 * c]) : "f"(lo), "f"(lo2));
                asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m[2 * c + 1]) : "f"(hi), "f"(hi2));
            }
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int o = Map::LPR; o < 32; o *= 2) m[c] = max_nan(m[c], __shfl_xor_sync(0xffffffffu, m[c], o));
        if (sub == 0) {
            reinterpret_cast<float4 *>(&top[warp][col])[0] = make_float4(m[0], m[1], m[2], m[3]);
            reinterpret_cast<float4 *>(&top[warp][col])[1] = make_float4(m[4], m[5], m[6], m[7]);
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < N; c += 32 * WARPS) {
        float t = top[0][c];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) t = max_nan(t, top[w][c]);
        inv[c] = t > kLeast ? 127.0f / t : 0.0f;
        scales[c] = t < INFINITY ? t / 127.0f : NAN;  // what a column no longer holds stays visible in its scale
    }
    __syncthreads();
    uint64_t to[4];
    load_row_shared(inv + col, to);
#pragma unroll
    for (int r = 0; r < RT; ++r) __stcs(reinterpret_cast<uint2 *>(codes + r * Map::RPW * N), f32_to_codes(S[r], to));
}

// Blocks of two warps (one, where a head has no more rows) with 8 rows a lane: 256 rows of 32 heads of 128 x 128
// in bf16 take 83.8 us, 0.95 of what a copy of those bytes takes; 89.8 with 16 rows a lane.  Measured with an
// earlier form of the arithmetic, eight warps a block took 104 us, four 98, two 97, and 4 or 2 rows a lane 103
// and 150 (the token's own scalars cost a warp as much as a few rows).  Of narrower heads 8 rows a lane are as
// many as there are sums for its lanes: 6.8 us for 300 rows of 8 heads of 64 x 64, and 7.6 with 4.
template <typename StateT, typename ActT, int P, int N, int RT>
int launch_step(StepArgs &a, int batch, cudaStream_t st) {
    constexpr int rows = RowMap<N, RT>::ROWS, warps = P / rows < 2 ? P / rows : 2;
    a.splits = P / (rows * warps);
    const dim3 grid((unsigned)(a.H * a.splits), (unsigned)batch);
    auto kern = a.ntok == 1 && !a.scratch ? k_gdn_step<StateT, ActT, P, N, RT> : k_gdn_tokens_step<StateT, ActT, P, N, RT>;
    if (launch_pdl(kern, grid, dim3(32 * warps), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <typename StateT, typename ActT>
int dispatch_step(StepArgs &a, int batch, int P, int N, cudaStream_t st) {
    if (P == 128 && N == 128) return launch_step<StateT, ActT, 128, 128, 8>(a, batch, st);
    if (P == 64 && N == 128) return launch_step<StateT, ActT, 64, 128, 8>(a, batch, st);
    if (P == 64 && N == 64) return launch_step<StateT, ActT, 64, 64, 8>(a, batch, st);
    if (P == 32 && N == 64) return launch_step<StateT, ActT, 32, 64, 8>(a, batch, st);
    if (P == 16 && N == 16) return launch_step<StateT, ActT, 16, 16, 1>(a, batch, st);
    return MAMBA_EUNSUPPORTED;
}

// Many rows a lane, whose products and maxima then cost a warp less for each: at 192 rows of 32 heads of
// 128 x 128, 16 rows a lane (4 warps a block, three blocks an SM) took 54.3 us, 8 rows 69.8, 4 rows 74.7;
// at 600 rows of 8 heads of 64 x 64, 8 rows 13.5 us, 4 rows 14.5; at 800 rows of 12 heads of 32 x 64, 15.4 and
// 16.2.  Heads of 64 x 128 fill a block of 4 warps with 8 rows a lane: 56.0 us at 100 rows of 128 heads,
// against 59.9 with 16.  Keeping only the codes and forming the new state twice, for twice the warps an SM,
// took 70.8 us at the first of these sizes: half as many instructions again.
template <typename ActT, int P, int N, int RT>
int launch_int8(const Int8Args &a, int batch, cudaStream_t st) {
    const dim3 grid((unsigned)a.H, (unsigned)batch), block(P / RowMap<N, RT>::ROWS * 32);
    if (launch_pdl(k_gdn_step_int8<ActT, P, N, RT>, grid, block, 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <typename ActT>
int dispatch_int8(const Int8Args &a, int batch, int P, int N, cudaStream_t st) {
    if (P == 128 && N == 128) return launch_int8<ActT, 128, 128, 16>(a, batch, st);
    if (P == 64 && N == 128) return launch_int8<ActT, 64, 128, 8>(a, batch, st);
    if (P == 64 && N == 64) return launch_int8<ActT, 64, 64, 8>(a, batch, st);
    if (P == 32 && N == 64) return launch_int8<ActT, 32, 64, 8>(a, batch, st);
    if (P == 16 && N == 16) return launch_int8<ActT, 16, 16, 1>(a, batch, st);
    return MAMBA_EUNSUPPORTED;
}

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" int gdn_state_update(const mamba_layer_desc *d, void *ssm_pool, int64_t ssm_slot_stride, int64_t num_slots,
                                const int32_t *slot_ids, const int32_t *scratch_slots, int32_t batch, int32_t ntok,
                                const void *xbc, const void *dt, const void *beta, const float *A, const float *dt_bias,
                                int32_t dt_softplus, int32_t beta_sigmoid, int32_t qk_l2norm, float scale, void *y,
                                int32_t *err_word, void *stream) {
    MS_TRACE("gdn_state_update");
    int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (batch < 0 || batch > 65535 || ntok < 1 || ntok > kMaxTok) return MAMBA_EINVAL;
    if (batch == 0) return MAMBA_OK;
    if (!ssm_pool || !slot_ids || !xbc || !dt || !beta || !A || !y) return MAMBA_EINVAL;
    const int H = d->nheads, P = d->head_dim, N = d->d_state, G = d->n_groups;
    if (num_slots <= 0 || ssm_slot_stride < (int64_t)H * P * N) return MAMBA_EINVAL;
    if ((rc = check_layer(d)) != MAMBA_OK) return rc;
    const size_t sb = dtype_bytes(d->state_dtype), ab = dtype_bytes(d->act_dtype);
    if (!aligned16(ssm_pool) || ((size_t)ssm_slot_stride * sb) % 16 != 0 || !aligned16(xbc) || (uintptr_t)y % ab != 0)
        return MAMBA_EALIGN;
    StepArgs a;
    a.pool = ssm_pool; a.stride = ssm_slot_stride; a.num_slots = num_slots;
    a.slot = slot_ids; a.scratch = scratch_slots; a.ntok = ntok;
    a.xbc = xbc; a.dt = dt; a.beta = beta;
    a.gates = make_gates(d, A, dt_bias, dt_softplus, beta_sigmoid, qk_l2norm, scale);
    a.y = y; a.err = err_word; a.H = H; a.G = G; a.HG = H / G; a.Cd = mamba_conv_dim(d);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool sbf = d->state_dtype == MAMBA_BF16, abf = d->act_dtype == MAMBA_BF16;
    if (sbf && abf) return dispatch_step<bf16, bf16>(a, batch, P, N, st);
    if (sbf) return dispatch_step<bf16, float>(a, batch, P, N, st);
    if (abf) return dispatch_step<float, bf16>(a, batch, P, N, st);
    return dispatch_step<float, float>(a, batch, P, N, st);
}

extern "C" int gdn_state_update_int8(const mamba_layer_desc *d, void *store, int64_t num_entries, const int32_t *entries,
                                     int32_t batch, const void *xbc, const void *dt, const void *beta, const float *A,
                                     const float *dt_bias, int32_t dt_softplus, int32_t beta_sigmoid, int32_t qk_l2norm,
                                     float scale, void *y, int32_t *err_word, void *stream) {
    MS_TRACE("gdn_state_update_int8");
    int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (batch < 0 || batch > 65535) return MAMBA_EINVAL;
    if (batch == 0) return MAMBA_OK;
    if (!store || !entries || !xbc || !dt || !beta || !A || !y || num_entries <= 0) return MAMBA_EINVAL;
    if ((rc = check_layer(d)) != MAMBA_OK) return rc;
    if (!aligned16(store) || !aligned16(xbc) || (uintptr_t)y % dtype_bytes(d->act_dtype) != 0) return MAMBA_EALIGN;
    const EntryLayout lay = entry_layout(d);
    Int8Args a;
    a.store = static_cast<unsigned char *>(store);
    a.num_entries = num_entries; a.entry_bytes = (int64_t)lay.total; a.scale_off = (int64_t)lay.scales;
    a.entry = entries; a.xbc = xbc; a.dt = dt; a.beta = beta;
    a.gates = make_gates(d, A, dt_bias, dt_softplus, beta_sigmoid, qk_l2norm, scale);
    a.y = y; a.err = err_word; a.H = d->nheads; a.G = d->n_groups; a.HG = a.H / a.G; a.Cd = mamba_conv_dim(d);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->act_dtype == MAMBA_BF16 ? dispatch_int8<bf16>(a, batch, d->head_dim, d->d_state, st)
                                      : dispatch_int8<float>(a, batch, d->head_dim, d->d_state, st);
}
