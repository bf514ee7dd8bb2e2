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
template <typename StateT, typename ActT, int P, int N, int RT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) k_la_step(const StepArgs p) {
    using Map = RowMap<N, RT>;
    using Raw = typename RawOf<StateT>::type;
    __shared__ __align__(16) float kq[2 * kMaxTok][N];  // a token's key and query
    __shared__ __align__(16) float2 table[kMaxTok][N / 2];
    __shared__ float vs[kMaxTok][WARPS * Map::ROWS];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int i = blockIdx.y, h = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    const int row0 = split * WARPS * Map::ROWS;  // the block's
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE, col = (lane & (Map::LPR - 1)) * 8;
    StateT *pool = static_cast<StateT *>(p.pool);
    const int64_t off = ((int64_t)h * P + row0 + warp * Map::ROWS + sub) * N + col;
    Raw raw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) raw[r].load(pool + s * p.stride + off + (int64_t)r * Map::RPW * N);
    const ActT *xbc = static_cast<const ActT *>(p.xbc) + (int64_t)i * p.ntok * p.Cd;
    const ActT *keys = xbc + p.H * P + (h / p.HG) * N, *queries = keys + p.G * N;
    const float2 decay = decay_of(p.log_decay[h]);
    for (int e = tid; e < p.ntok * p.prep.half; e += 32 * WARPS) {
        const int j = e / p.prep.half, a = e % p.prep.half;
        table[j][a] = turned(turns(p.prep.inv_freq[a]), p.prep.pos[(int64_t)i * p.ntok + j]);
    }
    for (int e = tid; e < p.ntok * WARPS * Map::ROWS; e += 32 * WARPS) {
        const int j = e / (WARPS * Map::ROWS), r = e % (WARPS * Map::ROWS);
        vs[j][r] = to_f32(xbc[(int64_t)j * p.Cd + h * P + row0 + r]);
    }
    __syncthreads();
    const LaneRow<4> own(p.prep, lane & (Map::LPR - 1));
    for (int base = warp * Map::RPW; base < 2 * p.ntok; base += WARPS * Map::RPW) {  // (the same of all lanes of a warp)
        const int mine = base + sub, t = min(mine, 2 * p.ntok - 1);
        const ActT *from = ((t & 1) ? queries : keys) + (int64_t)(t >> 1) * p.Cd;
        Some<ActT, 4> lo, hi;
        lo.load(from + own.a);
        hi.load(from + own.b);
        float x[8], w[8];
        lo.get(x);
        hi.get(x + 4);
        norm_weights((t & 1) ? p.prep.qw : p.prep.kw, own, w);
        float2 turn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) turn[e] = own.turns ? table[t >> 1][own.angle + e] : make_float2(1.0f, 0.0f);
        norm_rotate<N, 4>(x, w, p.prep, turn, own);
        if (mine == t) {
            const float f = (t & 1) ? p.scale : 1.0f;
            *reinterpret_cast<float4 *>(&kq[t][own.a]) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
            *reinterpret_cast<float4 *>(&kq[t][own.b]) = make_float4(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
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
    constexpr int rows = RowMap<N, RT>::ROWS, most = sizeof(StateT) == 2 ? 4 : 2, warps = P / rows < most ? P / rows : most;
    a.splits = P / (rows * warps);
    const dim3 grid((unsigned)(a.H * a.splits), (unsigned)batch);
    if (launch_pdl(k_la_step<StateT, ActT, P, N, RT, warps>, grid, dim3(32 * warps), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

// Rows a lane and warps a block, in us at 256 rows of 32 heads of 128 x 128, 61 of 128 heads of 64 x 128, and 48 of the
// former with four drafts: fp32 states 160, 79 and 88 with 8 rows and two warps, 167, 82 and 101 with 4 rows, 170, 83 and 89
// with four warps; bf16 states, whose rows are half as many bytes for the same preparation, 90, 45 and 46 with 4 rows and four
// warps, 92, 46 and 50 with 8 rows and two warps, 97, 48 and 47 with 8 rows and four.  One warp a block took 100 to 160.
template <typename StateT, typename ActT>
int dispatch_step(StepArgs &a, int batch, int P, int N, cudaStream_t st) {
    constexpr int R = sizeof(StateT) == 2 ? 4 : 8;
    if (P == 128 && N == 128) return launch_step<StateT, ActT, 128, 128, R>(a, batch, st);
    if (P == 64 && N == 128) return launch_step<StateT, ActT, 64, 128, R>(a, batch, st);
    if (P == 64 && N == 64) return launch_step<StateT, ActT, 64, 64, 8>(a, batch, st);
    if (P == 32 && N == 64) return launch_step<StateT, ActT, 32, 64, 8>(a, batch, st);
    if (P == 16 && N == 16) return launch_step<StateT, ActT, 16, 16, 1>(a, batch, st);
    return MAMBA_EUNSUPPORTED;
}

// ---- norm and rotation on their own ----

constexpr int kPrepThreads = 128, kPrepAhead = 3;  // threads a block; rows of a lane on their way at a time

struct PrepArgs {
    const void *k, *q;
    void *k_out, *q_out;
    int64_t ks, qs, kos, qos;  // token strides, elements
    int T, G, rows, parts;     // rows: of a token's 2 G heads' keys and queries that a warp takes; parts: warps a token
    QkPrep prep;
};

// Streaming: 2 G N values a token in and out.  A warp takes a token's rows, or a part of them: its lanes' angles are then
// the same for all of them and stay in registers, each times the weights it meets, and warps need nothing of one another.
// Arithmetic goes two values an instruction: a lane's pairs (u, v) are held as eight u and eight v (see LaneRow).
// 16384 tokens of 32 + 32 heads of 128, 537 MB, take 93 us, 0.87 of what a copy takes; with one value an instruction 108 us, half
// of the issue slots, and with 4 values from each half, which are twice as many loads, 116.
template <typename ActT, int N, bool INTER>
__global__ void __launch_bounds__(kPrepThreads) k_la_qk_prep(const PrepArgs p) {
    constexpr int V = 8, LPR = N / (2 * V), RPW = 32 / LPR;
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int64_t id = (int64_t)blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5), t = id / p.parts;
    if (t >= p.T) return;
    const int32_t pos = p.prep.pos ? p.prep.pos[t] : 0;
    if (pos < 0) return;  // padding row
    const int lane = threadIdx.x & 31, sub = lane / LPR;
    const int begin = (int)(id % p.parts) * p.rows + sub, end = min(2 * p.G, (int)(id % p.parts + 1) * p.rows);
    const LaneRow<V> own(p.prep, lane & (LPR - 1));
    const ActT *k = static_cast<const ActT *>(p.k) + t * p.ks, *q = static_cast<const ActT *>(p.q) + t * p.qs;
    ActT *ko = static_cast<ActT *>(p.k_out) + t * p.kos, *qo = static_cast<ActT *>(p.q_out) + t * p.qos;
    Some<ActT, V> lo[kPrepAhead], hi[kPrepAhead];
    auto fetch = [&](int i, int r) {
        const ActT *from = r < p.G ? k + r * N : q + (r - p.G) * N;
        if (r < end) lo[i].load(from + own.a), hi[i].load(from + own.b);
    };
#pragma unroll
    for (int i = 0; i < kPrepAhead; ++i) fetch(i, begin + i * RPW);
    float2 turn[V];
#pragma unroll
    for (int e = 0; e < V; ++e)
        turn[e] = own.turns ? turned(turns(p.prep.inv_freq[own.angle + e]), pos) : make_float2(1.0f, 0.0f);
    // u' = uc u - us v, v' = vc v + vs u: cosines and sines times the weights
    uint64_t uc[V / 2], us[V / 2], vc[V / 2], vs[V / 2];
    int kind = -1;
    for (int base = begin; base - sub < end; base += kPrepAhead * RPW) {  // (the same for all lanes of a warp)
#pragma unroll
        for (int i = 0; i < kPrepAhead; ++i) {
            const int r = base + i * RPW;
            float x[2 * V] = {};
            if (r < end) lo[i].get(x), hi[i].get(x + V);
            fetch(i, r + kPrepAhead * RPW);
            if (kind != (r >= p.G)) {
                kind = r >= p.G;
                float w[2 * V], c[4][V];
                norm_weights(kind ? p.prep.qw : p.prep.kw, own, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float wu = INTER ? w[2 * e] : w[e], wv = INTER ? w[2 * e + 1] : w[V + e];
                    c[0][e] = wu * turn[e].x, c[1][e] = -wv * turn[e].y, c[2][e] = wv * turn[e].x, c[3][e] = wu * turn[e].y;
                }
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    uc[e] = pair(c[0][2 * e], c[0][2 * e + 1]), us[e] = pair(c[1][2 * e], c[1][2 * e + 1]);
                    vc[e] = pair(c[2][2 * e], c[2][2 * e + 1]), vs[e] = pair(c[3][2 * e], c[3][2 * e + 1]);
                }
            }
            uint64_t u[V / 2], v[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                u[e] = INTER ? pair(x[4 * e], x[4 * e + 2]) : pair(x[2 * e], x[2 * e + 1]);
                v[e] = INTER ? pair(x[4 * e + 1], x[4 * e + 3]) : pair(x[V + 2 * e], x[V + 2 * e + 1]);
            }
            if (p.prep.norm) {
                uint64_t ss = mul2(u[0], u[0]);
#pragma unroll
                for (int e = 1; e < V / 2; ++e) ss = fma2(u[e], u[e], ss);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) ss = fma2(v[e], v[e], ss);
                float s0, s1;
                unpair(ss, s0, s1);
                const float f = rsqrtf(sum_lanes<LPR>(s0 + s1) * (1.0f / N) + p.prep.eps);
                const uint64_t f2 = pair(f, f);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) u[e] = mul2(u[e], f2), v[e] = mul2(v[e], f2);
            }
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const uint64_t a = mul2(u[e], uc[e]), b = mul2(v[e], vc[e]);
                const uint64_t at = own.turns ? fma2(v[e], us[e], a) : a, bt = own.turns ? fma2(u[e], vs[e], b) : b;
                float y[4];
                unpair(at, y[0], y[1]);
                unpair(bt, y[2], y[3]);
                x[INTER ? 4 * e : 2 * e] = y[0], x[INTER ? 4 * e + 2 : 2 * e + 1] = y[1];
                x[INTER ? 4 * e + 1 : V + 2 * e] = y[2], x[INTER ? 4 * e + 3 : V + 2 * e + 1] = y[3];
            }
            if (r < end) {
                ActT *to = r < p.G ? ko + r * N : qo + (r - p.G) * N;
                const float first[V] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]},
                            second[V] = {x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]};
                store8_stream(to + own.a, first);
                store8_stream(to + own.b, second);
            }
        }
    }
}

// A warp's rows: all of a token's where tokens alone fill the SMs several times, else fewer.
template <typename ActT, int N>
int launch_prep(PrepArgs &a, cudaStream_t st) {
    constexpr int RPW = 32 * 16 / N;
    const int64_t passes = ((int64_t)2 * a.G + RPW - 1) / RPW, want = 152 * 64;  // passes of a warp over a token's rows; warps
    int64_t parts = (want + a.T - 1) / a.T;
    if (parts > passes) parts = passes;
    const int64_t per = (passes + parts - 1) / parts;
    a.rows = (int)per * RPW;
    a.parts = (int)((passes + per - 1) / per);
    const int64_t blocks = ((int64_t)a.T * a.parts + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    if (blocks > INT32_MAX) return MAMBA_EINVAL;
    auto kern = a.prep.inter ? k_la_qk_prep<ActT, N, true> : k_la_qk_prep<ActT, N, false>;
    if (launch_pdl(kern, dim3((unsigned)blocks), dim3(kPrepThreads), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
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
    int rc = check_la_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (batch < 0 || batch > 65535 || ntok < 1 || ntok > kMaxTok) return MAMBA_EINVAL;
    if (batch == 0) return MAMBA_OK;
    if (!ssm_pool || !slot_ids || !xbc || !log_decay || !y) return MAMBA_EINVAL;
    const int H = d->nheads, P = d->head_dim, N = d->d_state, G = d->n_groups;
    if (num_slots <= 0 || ssm_slot_stride < (int64_t)H * P * N) return MAMBA_EINVAL;
    if ((rc = check_la_layer(d)) != MAMBA_OK) return rc;
    if ((rc = check_prep(N, qk_norm, eps, positions, inv_freq, rot_dim)) != MAMBA_OK) return rc;
    if (!aligned16(ssm_pool) || ((size_t)ssm_slot_stride * dtype_bytes(d->state_dtype)) % 16 != 0 || !aligned16(xbc) ||
        (uintptr_t)y % dtype_bytes(d->act_dtype) != 0)
        return MAMBA_EALIGN;
    StepArgs a;
    a.pool = ssm_pool; a.stride = ssm_slot_stride; a.num_slots = num_slots;
    a.slot = slot_ids; a.scratch = scratch_slots; a.ntok = ntok;
    a.xbc = xbc; a.log_decay = log_decay; a.scale = scale;
    a.prep = make_prep(qk_norm, k_weight, q_weight, eps, positions, inv_freq, rot_dim, interleaved);
    a.y = y; a.err = err_word; a.H = H; a.G = G; a.HG = H / G; a.Cd = H * P + 2 * G * N;
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
    int rc = check_la_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (tokens < 0) return MAMBA_EINVAL;
    if (tokens == 0) return MAMBA_OK;
    const int N = d->d_state, G = d->n_groups;
    if (!k || !q || !k_out || !q_out) return MAMBA_EINVAL;
    const int64_t strides[4] = {k_stride, q_stride, k_out_stride, q_out_stride};
    for (int64_t s : strides)
        if (s < (int64_t)G * N) return MAMBA_EINVAL;
    if ((k_out == k && k_out_stride != k_stride) || (q_out == q && q_out_stride != q_stride)) return MAMBA_EINVAL;
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
