// la_scan.cu -- linear attention over a varlen prefill batch: the call's checks and plan, and the
// token-by-token form in fp32 for fp32 activations and for the small state shapes.
//
// The token-by-token form keeps its rows of the state in registers and walks the sequence; the rows of a
// head are independent, so a block takes a few rows of one head.  A token is one update and one dot product a
// row, and only the update's multiply-add follows the token before.  Keys and queries of 16 tokens are staged
// in shared memory in fp32 for all warps of the block, the next 16 tokens' loads being in flight meanwhile.
// What bounds it is the issue of its instructions where there are many rows (16 sequences of 500 tokens of 32 heads of
// 128 x 128, 21 G operations, 767 us), and their latency, 0.23 us a token, where there are few.
#include "la_scan.h"

namespace ms {

using namespace la;

namespace {

constexpr int kStage = 16;            // tokens staged in shared memory at a time
constexpr int64_t kManyRows = 32768;  // rows of all states together from which a lane takes more of them

constexpr int kPlanThreads = 1024;

// Checks cu_seqlens and the slot ids, cuts the sequences into segments and puts the longest first (blocks start in
// that order, so that none that takes long starts last).
__global__ void __launch_bounds__(kPlanThreads) k_la_plan(const ScanParams p) {
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    __shared__ int bad, sums[kPlanThreads / 32], place[kPlanThreads];  // place: where the segments of each length go
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = p.cu[0] != 0 || p.cu[p.nseq] > p.T;
    place[tid] = 0;
    __syncthreads();
    const int run = (p.nseq + kPlanThreads - 1) / kPlanThreads, lo = min(p.nseq, tid * run), hi = min(p.nseq, lo + run);
    for (int s = lo; s < hi; ++s) {
        const int32_t sl = p.slot[s];
        if (p.cu[s + 1] < p.cu[s]) bad = 1;  // (compared, not subtracted: a difference past 2^31 wraps; in order from 0 none does)
        if (sl < -1 || sl >= p.num_slots) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            flag_error(p.err, MAMBA_ERR_SEQLENS);
            p.meta[0] = 0;
        }
        return;
    }
    auto segments = [&](int s) {  // none of a sequence whose slot is bad: it is left untouched
        const int32_t sl = p.slot[s];
        return sl < -1 || sl >= p.num_slots ? 0 : (int)(((int64_t)p.cu[s + 1] - p.cu[s] + p.seg_tokens - 1) / p.seg_tokens);
    };
    // longest first: place 0 is for the longest
    auto rank = [&](int tokens) { return kPlanThreads - 1 - min(kPlanThreads - 1, tokens / kChunk); };
    auto tokens_of = [&](int s, int i) { return min(p.seg_tokens, p.cu[s + 1] - p.cu[s] - i * p.seg_tokens); };
    int n = 0;
    for (int s = lo; s < hi; ++s) {
        const int m = segments(s);
        n += m;
        for (int i = 0; i < m; ++i) atomicAdd(&place[rank(tokens_of(s, i))], 1);
    }
    auto scan = [&](int v, int *total) {  // exclusive running sum over the threads
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        if (total) *total = all;
        return before + x - v;
    };
    int total, at = scan(n, &total);
    const int mine = place[tid];  // (scan has met all threads since the counts were taken)
    const int begin = scan(mine, nullptr);
    place[tid] = begin;
    __syncthreads();
    Segment *out = meta_segments(p);
    for (int s = lo; s < hi; ++s) {
        const int m = segments(s);
        for (int i = 0; i < m; ++i) {  // (the order among equals is not fixed, and no result depends on it)
            const int to = atomicAdd(&place[rank(tokens_of(s, i))], 1);
            const int32_t sl = p.slot[s];
            out[to] = {s, i, m - 1, at + s, p.cu[s] + i * p.seg_tokens, tokens_of(s, i), sl, sl >= 0 && p.has_init && p.has_init[s]};
        }
        at += m;
    }
    if (tid == 0) p.meta[0] = total, p.meta[1] = 0;
}

// Block (head and share of its rows, sequence in the plan's order).
template <typename StateT, typename ActT, int P, int N, int RT, int PIECES, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) k_la_tokens(const ScanParams p) {
    using Map = RowMap<N, RT, PIECES>;
    constexpr int ROWS = Map::ROWS * WARPS, SPLITS = P / ROWS;
    constexpr int SL = N / 8, GROUPS = 32 * WARPS / SL;  // staging: a token SL lanes
    constexpr int PASS = (kStage + GROUPS - 1) / GROUPS, VPASS = (kStage * ROWS + 32 * WARPS - 1) / (32 * WARPS);
    __shared__ __align__(16) float ks[kStage][N], qs[kStage][N];
    __shared__ float vs[kStage][ROWS];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    if ((int)blockIdx.y >= p.meta[0]) return;  // no such sequence: empty ones, bad slots, cu_seqlens refused (flagged)
    const Segment job = meta_segments(p)[blockIdx.y];  // (the whole sequence)
    const int h = blockIdx.x / SPLITS, split = blockIdx.x % SPLITS, grp = h / p.HG;
    const int s = job.seq, t0 = job.t0, len = job.len;
    const int32_t slot = job.slot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane / Map::LPR, idx = (lane & (Map::LPR - 1)) / Map::SHARE;
    const int col = (lane & (SL - 1)) * 8, own = (lane & (Map::LPR - 1)) * 8;  // of staging, of the state
    const int brow = warp * Map::ROWS, row0 = split * ROWS + brow;
    const int lrow = brow + idx * Map::RPW + sub;  // the block's row whose sum this lane gets
    const float2 decay = decay_of(p.log_decay[h]);
    const uint64_t dh = pair(decay.x, decay.x), dl = pair(decay.y, decay.y);
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
    if (job.seeded) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                load_row(pool + slot * p.stride + off + r * Map::RPW * N + i * Map::LPR * 8, piece(S[r], i));
    }
    const ActT *v = static_cast<const ActT *>(p.v), *k = static_cast<const ActT *>(p.k), *q = static_cast<const ActT *>(p.q);
    ActT *y = static_cast<ActT *>(p.y);
    const int64_t rowy = (int64_t)p.H * P;
    const int group = tid / SL;
    float kr[PASS][8], qr[PASS][8];
    ActT vr[VPASS];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int j = base + i * GROUPS + group;
            if (i * GROUPS + group < kStage && j < len) {
                load8(k + (int64_t)(t0 + j) * p.ks + (int64_t)grp * N + col, kr[i]);
                load8(q + (int64_t)(t0 + j) * p.qs + (int64_t)grp * N + col, qr[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) kr[i][e] = qr[i][e] = 0.0f;
            }
        }
#pragma unroll
        for (int x = 0; x < VPASS; ++x) {
            const int c = tid + x * 32 * WARPS, j = base + c / ROWS;
            vr[x] = c < kStage * ROWS && j < len ? v[(int64_t)(t0 + j) * p.vs + (int64_t)h * P + split * ROWS + c % ROWS]
                                                 : from_f32<ActT>(0.0f);
        }
    };
    fetch(0);
    for (int base = 0; base < len; base += kStage) {
        const int L = min(kStage, len - base);
        __syncthreads();  // the stage before is consumed
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int j = i * GROUPS + group;
            if (j < kStage) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    *reinterpret_cast<float4 *>(&ks[j][col + e]) = make_float4(kr[i][e], kr[i][e + 1], kr[i][e + 2], kr[i][e + 3]);
                    *reinterpret_cast<float4 *>(&qs[j][col + e]) =
                        make_float4(qr[i][e] * p.scale, qr[i][e + 1] * p.scale, qr[i][e + 2] * p.scale, qr[i][e + 3] * p.scale);
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
        ActT *yt = y + (int64_t)(t0 + base) * rowy + (int64_t)h * P + split * ROWS + lrow;
#pragma unroll 1
        for (int j = 0; j < L; ++j, yt += rowy) {
            uint64_t kc[Map::PAIRS], qc[Map::PAIRS];
            columns(ks[j], kc);
            columns(qs[j], qc);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float x = vs[j][brow + r * Map::RPW + sub];
                const uint64_t v2 = pair(x, x);
#pragma unroll
                for (int e = 0; e < Map::PAIRS; ++e) S[r][e] = decayed_add(dh, dl, S[r][e], v2, kc[e]);
            }
            const float out = row_sum<Map>(S, qc, lane);
            if ((lane & (Map::SHARE - 1)) == 0) *yt = from_f32<ActT>(out);
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
    if (launch_pdl(k_la_tokens<StateT, ActT, P, N, RT, PIECES, WARPS>, grid, dim3(32 * WARPS), 0, st, p) != cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}

// Rows a lane, pieces of 8 columns and warps a block.  A token costs a warp its keys and queries whatever its rows, so many
// rows keep the SMs' issue slots for the rows and few make many warps.  Measured with fp32 states and activations: 16 sequences
// of 500 tokens of 32 heads of 128 x 128 767 us with 8 rows, 818 with 4, 1230 with 2; one of 1000 tokens 329, 232 and 264; 8 of
// 500 of 128 heads of 64 x 128 760, 815, 1217; two of 1000 of 24 such heads 488, 340, 392.  Of 64 x 64 two pieces of 2 rows
// served 4 sequences of 500 tokens of 8 heads in 190 us and 24 of 40 heads in 371; one row 189 and 557, 4 rows of one piece
// 218 and 386.  Of 32 x 64, 12 heads, two pieces of 2 rows took 150 us for 100 sequences of 200 tokens and 198 for 4 of 500,
// of one row 185 and 188.
template <typename StateT, typename ActT>
int dispatch_tokens(const ScanParams &p, int P, int N, cudaStream_t st) {
    const bool many = (int64_t)p.nseq * p.H * P >= kManyRows;
    if (P == 128 && N == 128)
        return many ? launch_tokens<StateT, ActT, 128, 128, 8, 1, 4>(p, st) : launch_tokens<StateT, ActT, 128, 128, 4, 1, 4>(p, st);
    if (P == 64 && N == 128)
        return many ? launch_tokens<StateT, ActT, 64, 128, 8, 1, 4>(p, st) : launch_tokens<StateT, ActT, 64, 128, 4, 1, 4>(p, st);
    if (P == 64 && N == 64) return launch_tokens<StateT, ActT, 64, 64, 2, 2, 4>(p, st);
    if (P == 32 && N == 64)
        return many ? launch_tokens<StateT, ActT, 32, 64, 2, 2, 2>(p, st) : launch_tokens<StateT, ActT, 32, 64, 1, 2, 4>(p, st);
    if (P == 16 && N == 16) return launch_tokens<StateT, ActT, 16, 16, 1, 1, 1>(p, st);
    return MAMBA_EUNSUPPORTED;
}

int segment_tokens(const mamba_layer_desc *d, int T, int nseq) {
    return chunked_eligible(d) ? chunked_segment_tokens(d->nheads, T, nseq) : kWhole;
}

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" size_t la_chunk_scan_workspace_bytes(const mamba_layer_desc *d, int32_t total_tokens, int32_t nseq) {
    if (check_la_layer(d) != MAMBA_OK || total_tokens < 0 || total_tokens > kWhole || nseq < 0) return 0;
    // of the most segments that a batch of this many tokens or fewer is cut into: more tokens can be fewer, longer segments
    const int64_t segs = chunked_eligible(d) ? chunked_most_segments(d->nheads, total_tokens, nseq) : nseq;
    return scan_meta_bytes(segs) + (chunked_eligible(d) ? chunked_workspace_bytes(d, segs, nseq) : 0);
}

extern "C" int la_chunk_scan(const mamba_layer_desc *d, void *ssm_pool, int64_t ssm_slot_stride, int64_t num_slots,
                             const int32_t *cu_seqlens, int32_t nseq, int32_t total_tokens, const int32_t *slot_ids,
                             const uint8_t *has_initial_state, const int32_t *ckpt_slots, int32_t max_ckpt,
                             int32_t ckpt_interval, const void *v, int64_t v_stride, const void *k, int64_t k_stride,
                             const void *q, int64_t q_stride, const float *log_decay, float scale, void *y, void *workspace,
                             size_t workspace_bytes, int32_t *err_word, void *stream) {
    MS_TRACE("la_chunk_scan");
    int rc = check_la_desc(d);
    if (rc != MAMBA_OK) return rc;
    if (nseq < 0 || nseq > 65535 || total_tokens < 0 || total_tokens > kWhole) return MAMBA_EINVAL;
    if (nseq == 0) return MAMBA_OK;
    if (!ssm_pool || !cu_seqlens || !slot_ids || !log_decay || !workspace) return MAMBA_EINVAL;
    if (total_tokens > 0 && (!v || !k || !q || !y)) return MAMBA_EINVAL;
    const int H = d->nheads, P = d->head_dim, N = d->d_state, G = d->n_groups;
    if (num_slots <= 0 || ssm_slot_stride < (int64_t)H * P * N) return MAMBA_EINVAL;
    if (total_tokens > 0 && (v_stride < (int64_t)H * P || k_stride < (int64_t)G * N || q_stride < (int64_t)G * N))
        return MAMBA_EINVAL;
    if (ckpt_slots && (max_ckpt <= 0 || ckpt_interval <= 0 || ckpt_interval % kChunk)) return MAMBA_EINVAL;
    if ((rc = check_la_layer(d)) != MAMBA_OK) return rc;
    if (workspace_bytes < la_chunk_scan_workspace_bytes(d, total_tokens, nseq)) return MAMBA_ENOSPACE;
    const size_t ab = dtype_bytes(d->act_dtype);
    if (!aligned16(ssm_pool) || ((size_t)ssm_slot_stride * dtype_bytes(d->state_dtype)) % 16 != 0 || !aligned16(workspace) ||
        !aligned16(v) || !aligned16(k) || !aligned16(q) || !aligned16(y))
        return MAMBA_EALIGN;
    if (total_tokens > 0 && (v_stride * ab % 16 || k_stride * ab % 16 || q_stride * ab % 16)) return MAMBA_EALIGN;
    ScanParams p;
    p.pool = ssm_pool; p.stride = ssm_slot_stride; p.num_slots = num_slots;
    p.cu = cu_seqlens; p.slot = slot_ids; p.has_init = has_initial_state;
    p.ckpt_slots = ckpt_slots; p.max_ckpt = ckpt_slots ? max_ckpt : 0; p.ckpt_interval = ckpt_interval;
    p.nseq = nseq; p.T = total_tokens; p.H = H; p.G = G; p.HG = H / G;
    p.v = v; p.k = k; p.q = q; p.vs = v_stride; p.ks = k_stride; p.qs = q_stride;
    p.log_decay = log_decay; p.scale = scale;
    p.y = y; p.err = err_word;
    p.seg_tokens = segment_tokens(d, total_tokens, nseq);
    p.max_segs = (int)scan_max_segments(total_tokens, nseq, p.seg_tokens);
    if ((int64_t)p.max_segs * H > INT32_MAX) return MAMBA_EINVAL;
    p.meta = static_cast<int32_t *>(workspace);
    p.ws = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + scan_meta_bytes(p.max_segs));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_pdl(k_la_plan, dim3(1), dim3(kPlanThreads), 0, st, p) != cudaSuccess) return MAMBA_ECUDA;
    if (total_tokens == 0) return launch_status();  // only empty sequences
    if (chunked_eligible(d)) return chunked_launch(p, d, st);
    const bool sbf = d->state_dtype == MAMBA_BF16, abf = d->act_dtype == MAMBA_BF16;
    if (sbf && abf) return dispatch_tokens<bf16, bf16>(p, P, N, st);
    if (sbf) return dispatch_tokens<bf16, float>(p, P, N, st);
    if (abf) return dispatch_tokens<float, bf16>(p, P, N, st);
    return dispatch_tokens<float, float>(p, P, N, st);
}
