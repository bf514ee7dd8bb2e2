// gdn_scan.cu -- the gated delta rule over a varlen prefill batch: the call's checks and plan, and
// the token-by-token form in fp32 for fp32 states or activations and for the small state shapes.
//
// The token-by-token form keeps its rows of the state in registers and walks the sequence; the
// rows of a head are independent (gdn.cuh), so a block takes a few rows of one head: a token is
// then a chain (two dot products, five shuffles, one update; 0.28 us measured for heads of 128 x 128)
// that bounds the call while there are fewer warps than the SMs hold.  Keys and queries of 16 tokens are
// scaled once and staged in shared memory in fp32 for all warps of the block, the next 16 tokens'
// loads being in flight meanwhile.
#include "gdn_scan_tc.h"

namespace ms {

using namespace gdn;

namespace {

constexpr int kStage = 16;  // tokens staged in shared memory at a time
constexpr int64_t kManyRows = 32768;  // rows of all states together from which a lane takes most of them

constexpr int kPlanThreads = 1024;
constexpr int kMaxOrdered = 4096;  // sequences up to which the longest go first (the order is found by counting)

// Checks cu_seqlens and the slot ids, orders the sequences longest first (the longest chains start
// first), numbers the chunks and notes where each begins.
__global__ void __launch_bounds__(kPlanThreads) k_gdn_plan(const ScanParams p) {
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    __shared__ int ok, sums[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) ok = p.cu[0] == 0 && p.cu[p.nseq] == p.T;
    __syncthreads();
    // each thread numbers a run of sequences, from the sum of the runs before it
    const int run = (p.nseq + kPlanThreads - 1) / kPlanThreads, lo = min(p.nseq, tid * run), hi = min(p.nseq, lo + run);
    int n = 0;
    for (int s = lo; s < hi; ++s) {
        const int a = p.cu[s], b = p.cu[s + 1], len = b - a;
        if (b < a) ok = 0;  // (compared, not subtracted: a difference past 2^31 wraps; in order from 0 to T none does)
        const int32_t sl = p.slot[s];
        if (sl < -1 || sl >= p.num_slots) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        n += (len + kChunk - 1) / kChunk;
    }
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
    }
    if (lane == 31) sums[warp] = at;
    __syncthreads();
    if (!ok) {
        if (tid == 0) {
            flag_error(p.err, MAMBA_ERR_SEQLENS);
            p.meta[0] = 0;
            p.meta[1] = 0;
        }
        return;
    }
    int32_t *order = meta_order(p), *first = meta_chunks(p);
    int total = 0;
    at -= n;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) at += sums[w];
        total += sums[w];
    }
    for (int s = lo; s < hi; ++s) {
        first[s] = at;
        at += (p.cu[s + 1] - p.cu[s] + kChunk - 1) / kChunk;
    }
    if (tid == 0) {
        first[p.nseq] = total;
        p.meta[0] = 1;
        p.meta[1] = total;
    }
    __syncthreads();
    for (int c = tid; c < total; c += kPlanThreads) {  // a chunk's sequence: the last whose first chunk is not past it
        int a = 0, b = p.nseq - 1;
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (first[mid] <= c) a = mid;
            else b = mid - 1;
        }
        const int t0 = p.cu[a] + (c - first[a]) * kChunk;
        meta_table(p)[c] = make_int2(t0, min(kChunk, p.cu[a + 1] - t0));
    }
    for (int s = tid; s < p.nseq; s += kPlanThreads) {
        int r = s;
        if (p.nseq <= kMaxOrdered) {
            const int len = p.cu[s + 1] - p.cu[s];
            r = 0;
            for (int s2 = 0; s2 < p.nseq; ++s2) {
                const int l2 = p.cu[s2 + 1] - p.cu[s2];
                r += (l2 > len) || (l2 == len && s2 < s);
            }
        }
        order[r] = s;
    }
}

// Block (head and share of its rows, sequence in the plan's order).
template <typename StateT, typename ActT, int P, int N, int RT, int PIECES, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) k_gdn_tokens(const ScanParams p) {
    using Map = RowMap<N, RT, PIECES>;
    constexpr int ROWS = Map::ROWS * WARPS, SPLITS = P / ROWS;
    constexpr int SL = N / 8, GROUPS = 32 * WARPS / SL;  // staging: a token SL lanes
    constexpr int PASS = (kStage + GROUPS - 1) / GROUPS, VPASS = (kStage * ROWS + 32 * WARPS - 1) / (32 * WARPS);
    __shared__ __align__(16) float ks[kStage][N], qs[kStage][N];
    __shared__ float vs[kStage][ROWS];
    __shared__ float as[kStage], bs[kStage], kqs[kStage];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    if (p.meta[0] == 0) return;  // bad cu_seqlens (flagged): nothing is done
    const int s = meta_order(p)[blockIdx.y];
    const int h = blockIdx.x / SPLITS, split = blockIdx.x % SPLITS, grp = h / p.HG;
    const int t0 = p.cu[s], len = p.cu[s + 1] - t0;
    const int32_t slot = p.slot[s];
    if (len <= 0 || slot < -1 || slot >= p.num_slots) return;  // empty, or bad slot (flagged)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE;
    const int col = (lane & (SL - 1)) * 8, own = (lane & (Map::LPR - 1)) * 8;  // of staging, of the state
    const int brow = warp * Map::ROWS, row0 = split * ROWS + brow;
    const int lrow = brow + idx * Map::RPW + sub;  // the block's row whose sum this lane gets
    StateT *pool = static_cast<StateT *>(p.pool);
    const int64_t off = ((int64_t)h * P + row0 + sub) * N + own;
    uint64_t S[RT][Map::PAIRS] = {};  // (pairs of zeros)
    auto piece = [](uint64_t *v, int i) -> uint64_t(&)[4] { return *reinterpret_cast<uint64_t(*)[4]>(v + 4 * i); };
    auto columns = [&](const float *row, uint64_t (&x)[Map::PAIRS]) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) load_row_shared(row + own + i * Map::LPR * 8, piece(x, i));
    };
    auto write_state = [&](int32_t to) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                store_row(pool + to * p.stride + off + r * Map::RPW * N + i * Map::LPR * 8, piece(S[r], i));
    };
    if (slot >= 0 && p.has_init && p.has_init[s]) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                load_row(pool + slot * p.stride + off + r * Map::RPW * N + i * Map::LPR * 8, piece(S[r], i));
    }
    const ActT *v = static_cast<const ActT *>(p.v), *k = static_cast<const ActT *>(p.k), *q = static_cast<const ActT *>(p.q);
    ActT *y = static_cast<ActT *>(p.y);
    const int64_t rowk = (int64_t)p.G * N, rowv = (int64_t)p.H * P;
    const int group = tid / SL;
    float kr[PASS][8], qr[PASS][8], dtr[PASS], br[PASS];
    ActT vr[VPASS];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int j = base + i * GROUPS + group;
            if (i * GROUPS + group < kStage && j < len) {
                load8(k + (t0 + j) * rowk + (int64_t)grp * N + col, kr[i]);
                load8(q + (t0 + j) * rowk + (int64_t)grp * N + col, qr[i]);
                dtr[i] = load_scalar(p.dt, (int64_t)(t0 + j) * p.H + h, p.gates.dt_bf16);
                br[i] = load_scalar(p.beta, (int64_t)(t0 + j) * p.H + h, p.gates.dt_bf16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) kr[i][e] = qr[i][e] = 0.0f;
                dtr[i] = br[i] = 0.0f;
            }
        }
#pragma unroll
        for (int x = 0; x < VPASS; ++x) {
            const int c = tid + x * 32 * WARPS, j = base + c / ROWS;
            vr[x] = c < kStage * ROWS && j < len ? v[(t0 + j) * rowv + (int64_t)h * P + split * ROWS + c % ROWS]
                                                 : from_f32<ActT>(0.0f);
        }
    };
    fetch(0);
    for (int base = 0; base < len; base += kStage) {
        const int L = min(kStage, len - base);
        __syncthreads();  // the stage before is consumed
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kk = fmaf(kr[i][e], kr[i][e], kk);
                qq = fmaf(qr[i][e], qr[i][e], qq);
                kq = fmaf(kr[i][e], qr[i][e], kq);
            }
            kk = sum_lanes<SL>(kk);
            qq = sum_lanes<SL>(qq);
            kq = sum_lanes<SL>(kq);
            const float rk = unit_factor(p.gates, kk), rq = unit_factor(p.gates, qq) * p.gates.scale;
            const int j = i * GROUPS + group;
            if (j < kStage) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ks[j][col + e] = kr[i][e] * rk;
                    qs[j][col + e] = qr[i][e] * rq;
                }
                if (col == 0) {
                    as[j] = expf(log_decay(p.gates, dtr[i], h));
                    bs[j] = write_gate(p.gates, br[i]);
                    kqs[j] = kq * rk * rq;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < VPASS; ++x) {
            const int c = tid + x * 32 * WARPS;
            if (c < kStage * ROWS) vs[c / ROWS][c % ROWS] = to_f32(vr[x]);
        }
        __syncthreads();
        fetch(base + kStage);
        ActT *yt = y + (int64_t)(t0 + base) * rowv + (int64_t)h * P + split * ROWS + lrow;
        // with few values a lane the next token's operands wait in registers; with many, other warps hide them
        constexpr bool AHEAD = RT * PIECES <= 4;
        uint64_t kc[Map::PAIRS], qc[Map::PAIRS];
        float ac = as[0], bc = bs[0], kqc = kqs[0], vc = vs[0][lrow];
        columns(ks[0], kc);
        columns(qs[0], qc);
#pragma unroll 1
        for (int j = 0; j < L; ++j, yt += rowv) {
            uint64_t kn[Map::PAIRS], qn[Map::PAIRS];
            const int jn = min(j + 1, kStage - 1);
            float an, bn, kqn, vn;
            auto next = [&] {
                an = as[jn], bn = bs[jn], kqn = kqs[jn], vn = vs[jn][lrow];
                columns(ks[jn], kn);
                columns(qs[jn], qn);
            };
            if (AHEAD) next();
            const float out = token_rows<Map>(S, kc, qc, 1.0f, 1.0f, kqc, ac, bc, vc, lane);
            if (!AHEAD) next();
            if ((lane & (Map::SHARE - 1)) == 0) *yt = from_f32<ActT>(out);
#pragma unroll
            for (int e = 0; e < Map::PAIRS; ++e) kc[e] = kn[e], qc[e] = qn[e];
            ac = an, bc = bn, kqc = kqn, vc = vn;
            if (p.ckpt_slots) {
                const int32_t cs = ckpt_slot(p, s, base + j + 1, tid == 0 && blockIdx.x == 0);
                if (cs >= 0) write_state(cs);
            }
        }
    }
    if (slot >= 0) write_state(slot);
}

template <typename StateT, typename ActT, int P, int N, int RT, int PIECES, int WARPS>
int launch_tokens(const ScanParams &p, cudaStream_t st) {
    const dim3 grid((unsigned)(p.H * (P / (RowMap<N, RT, PIECES>::ROWS * WARPS))), (unsigned)p.nseq);
    if (launch_pdl(k_gdn_tokens<StateT, ActT, P, N, RT, PIECES, WARPS>, grid, dim3(32 * WARPS), 0, st, p) != cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}

// Rows a lane, and pieces of 8 columns: a token costs a warp of one piece about 90 instructions and 25 a row, so
// many rows keep the SMs' issue slots for the rows and few make many warps.  Measured on 32 heads of 128 x 128
// with fp32 states: 16 sequences of 500 tokens 0.95 ms with 8 rows, 1.18 with 4, 1.50 with 2; one of 1000
// tokens 0.45, 0.31, 0.29.  Two pieces spare an exchange but read twice the columns: 1.09 ms (4 rows) and 0.30 (2)
// there, yet for d_state 64, bf16 states: 64 sequences of 500 tokens of 8 heads of 64 x 64 0.39 ms with two
// pieces of 2 rows, 0.45 with one of 4; four of 500 tokens 0.19 (two pieces, a row) and 0.23 (one, 2 rows).
template <typename StateT, typename ActT>
int dispatch_tokens(const ScanParams &p, int P, int N, cudaStream_t st) {
    const int64_t rows = (int64_t)p.nseq * p.H * P;
    if (P == 128 && N == 128) {
        if (rows >= kManyRows) return launch_tokens<StateT, ActT, 128, 128, 8, 1, 4>(p, st);
        if (rows >= kManyRows / 4) return launch_tokens<StateT, ActT, 128, 128, 4, 1, 4>(p, st);
        return launch_tokens<StateT, ActT, 128, 128, 2, 1, 8>(p, st);
    }
    if (P == 64 && N == 128) {
        if (rows >= kManyRows) return launch_tokens<StateT, ActT, 64, 128, 8, 1, 4>(p, st);
        if (rows >= kManyRows / 4) return launch_tokens<StateT, ActT, 64, 128, 4, 1, 4>(p, st);
        return launch_tokens<StateT, ActT, 64, 128, 2, 1, 8>(p, st);
    }
    if (P == 64 && N == 64) {
        if (rows >= kManyRows) return launch_tokens<StateT, ActT, 64, 64, 2, 2, 4>(p, st);
        return launch_tokens<StateT, ActT, 64, 64, 1, 2, 4>(p, st);
    }
    if (P == 32 && N == 64) {
        if (rows >= kManyRows) return launch_tokens<StateT, ActT, 32, 64, 2, 2, 2>(p, st);
        return launch_tokens<StateT, ActT, 32, 64, 1, 2, 4>(p, st);
    }
    if (P == 16 && N == 16) return launch_tokens<StateT, ActT, 16, 16, 1, 1, 1>(p, st);
    return MAMBA_EUNSUPPORTED;
}

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" size_t gdn_chunk_scan_workspace_bytes(const mamba_layer_desc *d, int32_t total_tokens, int32_t nseq) {
    if (check_layer(d) != MAMBA_OK || total_tokens < 0 || nseq < 0) return 0;
    return scan_meta_bytes(total_tokens, nseq) + (chunked_eligible(d) ? chunked_workspace_bytes(d, total_tokens, nseq) : 0);
}

extern "C" int gdn_chunk_scan(const mamba_layer_desc *d, void *ssm_pool, int64_t ssm_slot_stride, int64_t num_slots,
                              const int32_t *cu_seqlens, int32_t nseq, int32_t total_tokens, const int32_t *slot_ids,
                              const uint8_t *has_initial_state, const int32_t *ckpt_slots, int32_t max_ckpt,
                              int32_t ckpt_interval, const void *v, const void *k, const void *q, const void *dt,
                              const void *beta, const float *A, const float *dt_bias, int32_t dt_softplus,
                              int32_t beta_sigmoid, int32_t qk_l2norm, float scale, void *y, void *workspace,
                              size_t workspace_bytes, int32_t *err_word, void *stream) {
    MS_TRACE("gdn_chunk_scan");
    int rc = check_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (nseq < 0 || nseq > 65535 || total_tokens < 0) return MAMBA_EINVAL;
    if (nseq == 0) return MAMBA_OK;
    if (!ssm_pool || !cu_seqlens || !slot_ids || !A || !workspace) return MAMBA_EINVAL;
    if (total_tokens > 0 && (!v || !k || !q || !dt || !beta || !y)) return MAMBA_EINVAL;
    const int H = d->nheads, P = d->head_dim, N = d->d_state, G = d->n_groups;
    if (num_slots <= 0 || ssm_slot_stride < (int64_t)H * P * N) return MAMBA_EINVAL;
    if (ckpt_slots && (max_ckpt <= 0 || ckpt_interval <= 0 || ckpt_interval % kChunk)) return MAMBA_EINVAL;
    if ((rc = check_layer(d)) != MAMBA_OK) return rc;
    if (workspace_bytes < gdn_chunk_scan_workspace_bytes(d, total_tokens, nseq)) return MAMBA_ENOSPACE;
    if (!aligned16(ssm_pool) || ((size_t)ssm_slot_stride * dtype_bytes(d->state_dtype)) % 16 != 0 || !aligned16(workspace) ||
        !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(y))
        return MAMBA_EALIGN;
    ScanParams p;
    p.pool = ssm_pool; p.stride = ssm_slot_stride; p.num_slots = num_slots;
    p.cu = cu_seqlens; p.slot = slot_ids; p.has_init = has_initial_state;
    p.ckpt_slots = ckpt_slots; p.max_ckpt = ckpt_slots ? max_ckpt : 0; p.ckpt_interval = ckpt_interval;
    p.nseq = nseq; p.T = total_tokens; p.H = H; p.G = G; p.HG = H / G;
    p.v = v; p.k = k; p.q = q; p.dt = dt; p.beta = beta;
    p.gates = make_gates(d, A, dt_bias, dt_softplus, beta_sigmoid, qk_l2norm, scale);
    p.y = y; p.err = err_word;
    p.meta = static_cast<int32_t *>(workspace);
    p.ws = static_cast<unsigned char *>(workspace) + scan_meta_bytes(total_tokens, nseq);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_pdl(k_gdn_plan, dim3(1), dim3(kPlanThreads), 0, st, p) != cudaSuccess) return MAMBA_ECUDA;
    if (total_tokens == 0) return launch_status();  // only empty sequences
    if (chunked_eligible(d)) return chunked_launch(p, P, st);
    const bool sbf = d->state_dtype == MAMBA_BF16, abf = d->act_dtype == MAMBA_BF16;
    if (sbf && abf) return dispatch_tokens<bf16, bf16>(p, P, N, st);
    if (sbf) return dispatch_tokens<bf16, float>(p, P, N, st);
    if (abf) return dispatch_tokens<float, bf16>(p, P, N, st);
    return dispatch_tokens<float, float>(p, P, N, st);
}
