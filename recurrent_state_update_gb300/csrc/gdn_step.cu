// gdn_step.cu -- the recurrent step of the gated delta rule over a slot pool, for one token or a
// few drafted ones a request, and for one token on int8 cache entries.
//
// Mathematics and row layout: gdn.cuh.  Both are streaming passes: an element of the state is read
// once and written once (once a draft) for about 8 floating operations, so device memory bounds
// them, and a call of few rows is bound by the latency of one load, two short chains of shuffles
// and one store.  Rows of a head are independent, so a block takes as many of them as keep the
// GPU busy: 16 a warp in long launches, 4 a warp over more blocks in short ones.
#include "gdn.cuh"
#include "int8_entry.h"

namespace ms {

using namespace gdn;

namespace {

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
    float k[8], q[8], rk, rq, ukq, a, b, v;
    __device__ __forceinline__ void load(const Gates &g, const ActT *row, int HP, int GN, int h, int grp, int P, int N,
                                         int vrow, const void *dt, const void *beta, int64_t th, int lane) {
        const int c = (lane & (Map::LPR - 1)) * 8;
        load8(row + HP + grp * N + c, k);
        load8(row + HP + GN + grp * N + c, q);
        v = to_f32(row[h * P + vrow]);
        const float dtv = load_scalar(dt, th, g.dt_bf16), bv = load_scalar(beta, th, g.dt_bf16);
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            kk = fmaf(k[e], k[e], kk);
            qq = fmaf(q[e], q[e], qq);
            kq = fmaf(k[e], q[e], kq);
        }
        kk = sum_lanes<Map::LPR>(kk);
        qq = sum_lanes<Map::LPR>(qq);
        kq = sum_lanes<Map::LPR>(kq);
        rk = unit_factor(g, kk);
        rq = unit_factor(g, qq) * g.scale;
        ukq = kq * rk * rq;
        a = expf(log_decay(g, dtv, h));
        b = write_gate(g, bv);
    }
};

// Block (head and share of its rows, batch row).
template <typename StateT, typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(256) k_gdn_step(const StepArgs p) {
    using Map = RowMap<N, RT>;
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t s = p.slot[i];
    if (s == -1) return;  // padding row
    bool bad = s < -1 || s >= p.num_slots;
    if (p.scratch)
        for (int j = 0; j < p.ntok; ++j) {
            const int32_t d = p.scratch[(int64_t)i * p.ntok + j];
            bad |= d < -1 || d >= p.num_slots;
        }
    if (bad) {
        if (threadIdx.x == 0) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        return;
    }
    const int row0 = (split * (blockDim.x >> 5) + warp) * Map::ROWS;
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE;
    StateT *pool = static_cast<StateT *>(p.pool);
    const int64_t off = ((int64_t)h * P + row0 + sub) * N + (lane & (Map::LPR - 1)) * 8;
    float S[RT][8];
#pragma unroll
    for (int r = 0; r < RT; ++r) load8_stream(pool + s * p.stride + off + (int64_t)r * Map::RPW * N, S[r]);
    const int vrow = row0 + (idx % RT) * Map::RPW + sub;
    const ActT *xbc = static_cast<const ActT *>(p.xbc);
    ActT *y = static_cast<ActT *>(p.y);
    for (int j = 0; j < p.ntok; ++j) {
        const int64_t t = (int64_t)i * p.ntok + j;
        TokenIn<Map, ActT> in;
        in.load(p.gates, xbc + t * p.Cd, p.H * P, p.G * N, h, h / p.HG, P, N, vrow, p.dt, p.beta, t * p.H + h, lane);
        const float out = token_rows<Map>(S, in.k, in.q, in.rk, in.rq, in.ukq, in.a, in.b, in.v, lane);
        if (idx >= RT && (lane & (Map::SHARE - 1)) == 0) y[(t * p.H + h) * P + vrow] = from_f32<ActT>(out);
        const int32_t d = p.scratch ? p.scratch[t] : (j == p.ntok - 1 ? s : -1);
        if (d >= 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r) store8_stream(pool + d * p.stride + off + (int64_t)r * Map::RPW * N, S[r]);
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

// Block (head, batch row): all rows of the head, because a scale covers a column of it.  Codes
// become fp32 on load; the new state is scaled by the new column maxima (a maximum over the warps
// through shared memory: the order of its updates does not matter) and rounded to the grid of
// step max/127, as the int8 store does.
template <typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(P / RowMap<N, RT>::ROWS * 32) k_gdn_step_int8(const Int8Args p) {
    using Map = RowMap<N, RT>;
    __shared__ int top[N];  // column maxima of |S|, as the bits of non-negative floats
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t e = p.entry[i];
    if (e == -1) return;  // padding row
    if (e < -1 || e >= p.num_entries) {
        if (threadIdx.x == 0) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        return;
    }
    for (int c = threadIdx.x; c < N; c += blockDim.x) top[c] = 0;
    unsigned char *ent = p.store + e * p.entry_bytes;
    const int col = (lane & (Map::LPR - 1)) * 8, sub = lane / Map::LPR, row0 = warp * Map::ROWS;
    const int idx = (lane & (Map::LPR - 1)) / Map::SHARE, vrow = row0 + (idx % RT) * Map::RPW + sub;
    unsigned char *codes = ent + ((int64_t)h * P + row0 + sub) * N + col;
    float *scales = reinterpret_cast<float *>(ent + p.scale_off) + (int64_t)h * N + col;
    uint2 raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r] = __ldcs(reinterpret_cast<const uint2 *>(codes + r * Map::RPW * N));
    float sc[8];
    load8(scales, sc);
    TokenIn<Map, ActT> in;
    in.load(p.gates, static_cast<const ActT *>(p.xbc) + (int64_t)i * p.Cd, p.H * P, p.G * N, h, h / p.HG, P, N, vrow, p.dt,
            p.beta, (int64_t)i * p.H + h, lane);
    float S[RT][8];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t w = c < 4 ? raw[r].x : raw[r].y;
            S[r][c] = (float)(int8_t)(w >> (8 * (c & 3))) * sc[c];
        }
    const float out = token_rows<Map>(S, in.k, in.q, in.rk, in.rq, in.ukq, in.a, in.b, in.v, lane);
    if (idx >= RT && (lane & (Map::SHARE - 1)) == 0)
        static_cast<ActT *>(p.y)[((int64_t)i * p.H + h) * P + vrow] = from_f32<ActT>(out);
    __syncthreads();  // top is zero, and every thread has its scales
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float m = 0.0f;
#pragma unroll
        for (int r = 0; r < RT; ++r) m = fmaxf(m, fabsf(S[r][c]));
#pragma unroll
        for (int o = Map::LPR; o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (sub == 0) atomicMax(&top[col + c], __float_as_int(m));
    }
    __syncthreads();
    float inv[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float m = __int_as_float(top[col + c]);
        inv[c] = m > 0.0f ? 127.0f / m : 0.0f;
        if (warp == 0 && sub == 0) scales[c] = m / 127.0f;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int code = max(-127, min(127, __float2int_rn(S[r][c] * inv[c])));
            w[c >> 2] |= (uint32_t)(code & 0xff) << (8 * (c & 3));
        }
        __stcs(reinterpret_cast<uint2 *>(codes + r * Map::RPW * N), make_uint2(w[0], w[1]));
    }
}

// Launches with RT rows a lane and as many warps a block as `rows` of the head need.
template <typename StateT, typename ActT, int P, int N, int RT>
int launch_step(StepArgs &a, int batch, int warps, cudaStream_t st) {
    a.splits = P / (RowMap<N, RT>::ROWS * warps);
    const dim3 grid((unsigned)(a.H * a.splits), (unsigned)batch);
    if (launch_pdl(k_gdn_step<StateT, ActT, P, N, RT>, grid, dim3(32 * warps), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <typename StateT, typename ActT>
int dispatch_step(StepArgs &a, int batch, int P, int N, cudaStream_t st) {
    if (P == 128 && N == 128) return launch_step<StateT, ActT, 128, 128, 8>(a, batch, 8, st);
    if (P == 64 && N == 128) return launch_step<StateT, ActT, 64, 128, 8>(a, batch, 4, st);
    if (P == 64 && N == 64) return launch_step<StateT, ActT, 64, 64, 4>(a, batch, 4, st);
    if (P == 32 && N == 64) return launch_step<StateT, ActT, 32, 64, 4>(a, batch, 2, st);
    if (P == 16 && N == 16) return launch_step<StateT, ActT, 16, 16, 1>(a, batch, 1, st);
    return MAMBA_EUNSUPPORTED;
}

template <typename ActT, int P, int N, int RT>
int launch_int8(const Int8Args &a, int batch, cudaStream_t st) {
    const dim3 grid((unsigned)a.H, (unsigned)batch), block(P / RowMap<N, RT>::ROWS * 32);
    if (launch_pdl(k_gdn_step_int8<ActT, P, N, RT>, grid, block, 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <typename ActT>
int dispatch_int8(const Int8Args &a, int batch, int P, int N, cudaStream_t st) {
    if (P == 128 && N == 128) return launch_int8<ActT, 128, 128, 8>(a, batch, st);
    if (P == 64 && N == 128) return launch_int8<ActT, 64, 128, 8>(a, batch, st);
    if (P == 64 && N == 64) return launch_int8<ActT, 64, 64, 4>(a, batch, st);
    if (P == 32 && N == 64) return launch_int8<ActT, 32, 64, 4>(a, batch, st);
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
