// la_step.cu -- the recurrent step of linear attention over a slot pool, with the norm and rotation of its
// keys and queries, and these two on their own for a prefill.
//
// The step is a streaming pass: an element of the state is read once and written once (once a draft) for
// five floating operations, so device memory bounds it, and a call of few rows is bound by the latency of one
// load, the norm, and one store.
#include "la.cuh"

namespace ms {

using namespace la;

namespace {

struct StepArgs {
    void *pool;
    int64_t stride, num_slots;  // elements
    const int32_t *slot, *scratch;
    int ntok;
    const void *xbc;
    const float *log_decay;
    QkPrep prep;
    float scale;
    void *y;
    int32_t *err;
    int H, G, HG, Cd, splits;
};

// Block (head and share of its rows, batch row).  While the state is on its way the block forms its tokens' angles,
// an angle a thread, and then their keys and queries, a row of either to each LPR lanes, in shared memory in
// fp32, so that the tokens follow one another without a wait on memory.
template <typename StateT, typename ActT, int P, int N, int RT>
__global__ void __launch_bounds__(64) k_la_step(const StepArgs p) {
    using Map = RowMap<N, RT>;
    using Raw = typename RawOf<StateT>::type;
    __shared__ __align__(16) float kq[2 * kMaxTok][N];  // a token's key and query
    __shared__ float2 table[kMaxTok][N / 2];
    __shared__ float vs[kMaxTok][2 * Map::ROWS];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int32_t s = p.slot[i];
    if (s == -1) return;  // padding row
    bool bad = s < -1 || s >= p.num_slots;
    if (p.scratch)
        for (int j = 0; j < p.ntok; ++j) {
            const int32_t d = p.scratch[(int64_t)i * p.ntok + j];
            bad |= d < -1 || d >= p.num_slots;
        }
    if (bad) {
        if (tid == 0) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        return;
    }
    const int row0 = split * warps * Map::ROWS;  // the block's
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE, col = (lane & (Map::LPR - 1)) * 8;
    StateT *pool = static_cast<StateT *>(p.pool);
    const int64_t off = ((int64_t)h * P + row0 + warp * Map::ROWS + sub) * N + col;
    Raw raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].load(pool + s * p.stride + off + (int64_t)r * Map::RPW * N);
    const ActT *xbc = static_cast<const ActT *>(p.xbc) + (int64_t)i * p.ntok * p.Cd;
    const ActT *keys = xbc + p.H * P + (h / p.HG) * N, *queries = keys + p.G * N;
    const float2 decay = decay_of(p.log_decay[h]);
    for (int e = tid; e < p.ntok * p.prep.half; e += blockDim.x) {
        const int j = e / p.prep.half, a = e % p.prep.half;
        table[j][a] = turned(turns(p.prep.inv_freq[a]), p.prep.pos[(int64_t)i * p.ntok + j]);
    }
    for (int e = tid; e < p.ntok * warps * Map::ROWS; e += blockDim.x) {
        const int j = e / (warps * Map::ROWS), r = e % (warps * Map::ROWS);
        vs[j][r] = to_f32(xbc[(int64_t)j * p.Cd + h * P + row0 + r]);
    }
    __syncthreads();
    for (int base = warp * Map::RPW; base < 2 * p.ntok; base += warps * Map::RPW) {  // (the same of all lanes of a warp)
        const int own = base + sub, t = min(own, 2 * p.ntok - 1);
        float x[8], w[8];
        load8(((t & 1) ? queries : keys) + (int64_t)(t >> 1) * p.Cd + col, x);
        norm_weights<N>((t & 1) ? p.prep.qw : p.prep.kw, lane, w);
        norm_rotate<N>(x, w, p.prep, table[t >> 1], lane);
        if (own == t) {
            const float f = (t & 1) ? p.scale : 1.0f;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4 *>(&kq[t][col + e]) = make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f);
        }
    }
    uint64_t S[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].unpack(S[r]);
    const uint64_t dh = pair(decay.x, decay.x), dl = pair(decay.y, decay.y);
    __syncthreads();
    ActT *y = static_cast<ActT *>(p.y) + ((int64_t)i * p.ntok * p.H + h) * P + row0 + warp * Map::ROWS + idx * Map::RPW + sub;
    for (int j = 0; j < p.ntok; ++j, y += (int64_t)p.H * P) {
        uint64_t k[4], q[4];
        load_row_shared(&kq[2 * j][col], k);
        load_row_shared(&kq[2 * j + 1][col], q);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float v = vs[j][warp * Map::ROWS + r * Map::RPW + sub];
            const uint64_t v2 = pair(v, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) S[r][e] = decayed_add(dh, dl, S[r][e], v2, k[e]);
        }
        const float out = row_sum<Map>(S, q, lane);
        if ((lane & (Map::SHARE - 1)) == 0) *y = from_f32<ActT>(out);
        const int32_t d = p.scratch ? p.scratch[(int64_t)i * p.ntok + j] : (j == p.ntok - 1 ? s : -1);
        if (d >= 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r) store_row(pool + d * p.stride + off + (int64_t)r * Map::RPW * N, S[r]);
        }
    }
}

template <typename StateT, typename ActT, int P, int N, int RT>
int launch_step(StepArgs &a, int batch, cudaStream_t st) {
    constexpr int rows = RowMap<N, RT>::ROWS, warps = P / rows < 2 ? P / rows : 2;
    a.splits = P / (rows * warps);
    const dim3 grid((unsigned)(a.H * a.splits), (unsigned)batch);
    if (launch_pdl(k_la_step<StateT, ActT, P, N, RT>, grid, dim3(32 * warps), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
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

// ---- norm and rotation on their own ----

constexpr int kPrepThreads = 256, kPrepItems = 4;  // threads a block; pieces of 8 values a thread has on its way

struct PrepArgs {
    const void *k, *q;
    void *k_out, *q_out;
    int64_t ks, qs, kos, qos;  // token strides, elements
    int T, G, per;             // per: tokens of a pass of a block
    QkPrep prep;
};

// Streaming: 2 G N values a token in and out.  A block takes `per` tokens at a time, as many as fill its
// threads' pieces: their angles go to shared memory, an angle a thread and step (each shared by all heads of
// the token), while the pieces are on their way.
template <typename ActT, int N>
__global__ void __launch_bounds__(kPrepThreads) k_la_qk_prep(const PrepArgs p) {
    constexpr int LPR = N / 8;
    extern __shared__ __align__(16) float2 angles[];  // [per][half]
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, col = (tid & (LPR - 1)) * 8, half = p.prep.half;
    float kw[8], qw[8];
    norm_weights<N>(p.prep.kw, lane, kw);
    norm_weights<N>(p.prep.qw, lane, qw);
    const ActT *k = static_cast<const ActT *>(p.k), *q = static_cast<const ActT *>(p.q);
    ActT *ko = static_cast<ActT *>(p.k_out), *qo = static_cast<ActT *>(p.q_out);
    const int rows = p.per * 2 * p.G;  // rows (a head's key or query) of a pass
    for (int64_t t0 = (int64_t)blockIdx.x * p.per; t0 < p.T; t0 += (int64_t)gridDim.x * p.per) {
        const int n = (int)min((int64_t)p.per, p.T - t0);
        for (int base = 0; base < rows; base += kPrepItems * kPrepThreads / LPR) {
            float x[kPrepItems][8];
            int at[kPrepItems];  // row of the pass, or -1
#pragma unroll
            for (int i = 0; i < kPrepItems; ++i) {
                const int r = base + (i * kPrepThreads + tid) / LPR, j = r / (2 * p.G), g = r % (2 * p.G);
                at[i] = j < n && (!p.prep.pos || p.prep.pos[t0 + j] >= 0) ? r : -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
                if (at[i] >= 0)
                    load8(g < p.G ? k + (t0 + j) * p.ks + g * N + col : q + (t0 + j) * p.qs + (g - p.G) * N + col, x[i]);
            }
            if (base == 0 && half) {
                __syncthreads();  // the last pass has read its angles
                for (int e = tid; e < n * half; e += kPrepThreads)
                    angles[e] = turned(turns(p.prep.inv_freq[e % half]), p.prep.pos[t0 + e / half]);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kPrepItems; ++i) {
                const int r = max(at[i], 0), j = r / (2 * p.G), g = r % (2 * p.G);
                norm_rotate<N>(x[i], g < p.G ? kw : qw, p.prep, angles + j * half, lane);
                if (at[i] < 0) continue;
                ActT *to = g < p.G ? ko + (t0 + j) * p.kos + g * N + col : qo + (t0 + j) * p.qos + (g - p.G) * N + col;
                store8_stream(to, x[i]);
            }
        }
    }
}

template <typename ActT, int N>
int launch_prep(PrepArgs &a, cudaStream_t st) {
    constexpr int rows = kPrepItems * kPrepThreads * 8 / N;
    a.per = rows / (2 * a.G) < 1 ? 1 : rows / (2 * a.G);
    const int64_t passes = ((int64_t)a.T + a.per - 1) / a.per;
    const unsigned grid = (unsigned)(passes < 152 * 8 ? passes : 152 * 8);
    if (launch_pdl(k_la_qk_prep<ActT, N>, dim3(grid), dim3(kPrepThreads), (size_t)a.per * a.prep.half * sizeof(float2), st, a) !=
        cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}

template <typename ActT>
int dispatch_prep(PrepArgs &a, int N, cudaStream_t st) {
    if (N == 16) return launch_prep<ActT, 16>(a, st);
    if (N == 32) return launch_prep<ActT, 32>(a, st);
    if (N == 64) return launch_prep<ActT, 64>(a, st);
    if (N == 128) return launch_prep<ActT, 128>(a, st);
    if (N == 256) return launch_prep<ActT, 256>(a, st);
    return MAMBA_EUNSUPPORTED;
}

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" int la_state_update(const mamba_layer_desc *d, void *ssm_pool, int64_t ssm_slot_stride, int64_t num_slots,
                               const int32_t *slot_ids, const int32_t *scratch_slots, int32_t batch, int32_t ntok,
                               const void *xbc, const float *log_decay, int32_t qk_norm, const float *k_weight,
                               const float *q_weight, float eps, const int32_t *positions, const float *inv_freq,
                               int32_t rot_dim, int32_t interleaved, float scale, void *y, int32_t *err_word, void *stream) {
    MS_TRACE("la_state_update");
    int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (batch < 0 || batch > 65535 || ntok < 1 || ntok > kMaxTok) return MAMBA_EINVAL;
    if (batch == 0) return MAMBA_OK;
    if (!ssm_pool || !slot_ids || !xbc || !log_decay || !y) return MAMBA_EINVAL;
    const int H = d->nheads, P = d->head_dim, N = d->d_state, G = d->n_groups;
    if (num_slots <= 0 || ssm_slot_stride < (int64_t)H * P * N) return MAMBA_EINVAL;
    if ((rc = check_layer(d)) != MAMBA_OK) return rc;
    if ((rc = check_prep(N, qk_norm, eps, positions, inv_freq, rot_dim)) != MAMBA_OK) return rc;
    if (!aligned16(ssm_pool) || ((size_t)ssm_slot_stride * dtype_bytes(d->state_dtype)) % 16 != 0 || !aligned16(xbc) ||
        (uintptr_t)y % dtype_bytes(d->act_dtype) != 0)
        return MAMBA_EALIGN;
    StepArgs a;
    a.pool = ssm_pool; a.stride = ssm_slot_stride; a.num_slots = num_slots;
    a.slot = slot_ids; a.scratch = scratch_slots; a.ntok = ntok;
    a.xbc = xbc; a.log_decay = log_decay; a.scale = scale;
    a.prep = make_prep(qk_norm, k_weight, q_weight, eps, positions, inv_freq, rot_dim, interleaved);
    a.y = y; a.err = err_word; a.H = H; a.G = G; a.HG = H / G; a.Cd = mamba_conv_dim(d);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool sbf = d->state_dtype == MAMBA_BF16, abf = d->act_dtype == MAMBA_BF16;
    if (sbf && abf) return dispatch_step<bf16, bf16>(a, batch, P, N, st);
    if (sbf) return dispatch_step<bf16, float>(a, batch, P, N, st);
    if (abf) return dispatch_step<float, bf16>(a, batch, P, N, st);
    return dispatch_step<float, float>(a, batch, P, N, st);
}

extern "C" int la_qk_norm_rope(const mamba_layer_desc *d, const void *k, int64_t k_stride, const void *q, int64_t q_stride,
                               int32_t tokens, int32_t qk_norm, const float *k_weight, const float *q_weight, float eps,
                               const int32_t *positions, const float *inv_freq, int32_t rot_dim, int32_t interleaved,
                               void *k_out, int64_t k_out_stride, void *q_out, int64_t q_out_stride, void *stream) {
    MS_TRACE("la_qk_norm_rope");
    int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (tokens < 0) return MAMBA_EINVAL;
    if (tokens == 0) return MAMBA_OK;
    const int N = d->d_state, G = d->n_groups;
    if (!k || !q || !k_out || !q_out) return MAMBA_EINVAL;
    const int64_t strides[4] = {k_stride, q_stride, k_out_stride, q_out_stride};
    for (int64_t s : strides)
        if (s < (int64_t)G * N) return MAMBA_EINVAL;
    if (N != 16 && N != 32 && N != 64 && N != 128 && N != 256) return MAMBA_EUNSUPPORTED;
    if ((rc = check_prep(N, qk_norm, eps, positions, inv_freq, rot_dim)) != MAMBA_OK) return rc;
    const size_t ab = dtype_bytes(d->act_dtype);
    for (int64_t s : strides)
        if ((size_t)s * ab % 16 != 0) return MAMBA_EALIGN;
    if (!aligned16(k) || !aligned16(q) || !aligned16(k_out) || !aligned16(q_out)) return MAMBA_EALIGN;
    PrepArgs a;
    a.k = k; a.q = q; a.k_out = k_out; a.q_out = q_out;
    a.ks = k_stride; a.qs = q_stride; a.kos = k_out_stride; a.qos = q_out_stride;
    a.T = tokens; a.G = G;
    a.prep = make_prep(qk_norm, k_weight, q_weight, eps, positions, inv_freq, rot_dim, interleaved);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->act_dtype == MAMBA_BF16 ? dispatch_prep<bf16>(a, N, st) : dispatch_prep<float>(a, N, st);
}
