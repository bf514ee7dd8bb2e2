// batch_plan.cu -- the arguments of the varlen and step calls from the requests' lengths and block table.
//
// A few kilobytes in and out, so the call's latency is what counts: one launch while a block can sum all
// lengths by itself in passing (each block then does so, rather than wait for one that would), two launches
// beyond that.  Blocks share the tokens and the requests out by index.
#include "common.cuh"

namespace ms {

namespace {

constexpr int kThreads = 512, kOwn = 8, kOneLaunch = kThreads * kOwn;  // rows up to which every block sums for itself
constexpr int kTokensBlock = 4 * kThreads;                            // tokens a block takes, at least

struct PlanArgs {
    const int32_t *fresh, *past, *table;
    int64_t table_stride, num_slots;
    int rows, cols, block, max_tokens, max_ckpt;
    int32_t *cu, *slot, *src, *dst, *ckpt, *pos, *row, *err;
    uint8_t *init;
};

// Whether a row's own lengths are ones a request can have.
__device__ __forceinline__ bool row_ok(int32_t n, int32_t c) { return n >= 0 && c >= 0 && (int64_t)n + c <= INT32_MAX; }

// Exclusive running sum over the block's threads and the total.  64 bits: a sum of lengths may pass 2^31.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *shared) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) shared[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += shared[w];
        total += shared[w];
    }
    __syncthreads();
    return before + x - v;
}

// A request's outputs; n = 0 for all of them when the batch is refused.
__device__ void plan_row(const PlanArgs &p, int i, bool ok) {
    const int32_t n = ok ? p.fresh[i] : 0, c = ok ? p.past[i] : 0;
    const int32_t *pages = p.table + (int64_t)i * p.table_stride;
    bool bad = false;
    auto page = [&](int32_t tokens) {  // of the state after `tokens` >= 1 tokens
        const int32_t j = p.block ? (tokens - 1) / p.block : 0;
        const int32_t s = j < p.cols ? pages[j] : -1;
        bad |= s < 0 || s >= p.num_slots;
        return s;
    };
    int32_t to = -1, from = -1;
    if (n > 0) {
        to = page(c + n);
        from = c > 0 ? page(c) : to;
    }
    const bool aligned = n > 0 && p.block && c % p.block == 0;
    auto kept = [&](int k) -> int32_t {  // of checkpoint k: -1 where there is none to keep
        if (!aligned || (int64_t)k * p.block >= n) return -1;
        const int j = c / p.block + k - 1;
        return j < p.cols ? pages[j] : -2;
    };
    if (p.ckpt)
        for (int k = 1; k <= p.max_ckpt && aligned && (int64_t)k * p.block < n; ++k) {
            const int32_t s = kept(k);
            bad |= s < -1 || s >= p.num_slots;
        }
    if (bad) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
    p.slot[i] = bad ? -2 : to;
    if (p.init) p.init[i] = n > 0 && c > 0;
    if (p.src) {
        const bool moves = !bad && from != to;
        p.src[i] = moves ? from : -1;
        p.dst[i] = moves ? to : -1;
    }
    if (p.ckpt)
        for (int k = 1; k <= p.max_ckpt; ++k) p.ckpt[(int64_t)i * p.max_ckpt + k - 1] = bad ? -1 : kept(k);
}

__device__ __forceinline__ void plan_token(const PlanArgs &p, const int32_t *cu, int t, int total) {
    int32_t row = -1, pos = -1;
    if (t < total) {
        int a = 0, b = p.rows - 1;  // the last row that begins at or before t: rows of no tokens begin where the next does
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (cu[mid] <= t) a = mid;
            else b = mid - 1;
        }
        row = a;
        pos = p.past[a] + (t - cu[a]);
    }
    if (p.row) p.row[t] = row;
    if (p.pos) p.pos[t] = pos;
}

// ONE: every block sums the lengths into its shared memory; else cu is there already (k_batch_sums).
template <bool ONE>
__global__ void __launch_bounds__(kThreads) k_batch_plan(const PlanArgs p) {
    __shared__ int64_t sums[kThreads / 32];
    __shared__ int32_t mine[ONE ? kOneLaunch + 1 : 1];
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int32_t *cu = ONE ? mine : p.cu;
    int total;
    bool ok;
    if (ONE) {
        const int per = (p.rows + kThreads - 1) / kThreads;
        int32_t n[kOwn];
        int64_t sum = 0;
        bool good = true;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            const int i = tid * per + e;
            n[e] = 0;
            if (e < per && i < p.rows) {
                n[e] = p.fresh[i];
                good &= row_ok(n[e], p.past[i]);
            }
            sum += n[e];
        }
        int64_t all, at = block_scan(sum, all, sums);
        ok = __syncthreads_and(good) && all <= p.max_tokens;
        total = ok ? (int)all : 0;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            const int i = tid * per + e;
            if (e < per && i < p.rows) mine[i] = ok ? (int32_t)at : 0;
            at += n[e];
        }
        if (tid == 0) mine[p.rows] = total;
        if (!ok && tid == 0 && blockIdx.x == 0) flag_error(p.err, MAMBA_ERR_SEQLENS);
        __syncthreads();
        for (int i = blockIdx.x * kThreads + tid; i <= p.rows; i += gridDim.x * kThreads) p.cu[i] = mine[i];
    } else {
        total = p.cu[p.rows];
        ok = total > 0;  // (of a batch of no tokens every row is one of padding, refused or not)
    }
    for (int i = blockIdx.x * kThreads + tid; i < p.rows; i += gridDim.x * kThreads) plan_row(p, i, ok);
    if (p.pos || p.row)
        for (int64_t t = (int64_t)blockIdx.x * kThreads + tid; t < p.max_tokens; t += (int64_t)gridDim.x * kThreads)
            plan_token(p, cu, (int)t, total);
}

__global__ void __launch_bounds__(kThreads) k_batch_sums(const PlanArgs p) {
    __shared__ int64_t sums[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int per = (p.rows + kThreads - 1) / kThreads, lo = min(p.rows, (int)threadIdx.x * per), hi = min(p.rows, lo + per);
    int64_t sum = 0;
    bool good = true;
    for (int i = lo; i < hi; ++i) {
        sum += p.fresh[i];
        good &= row_ok(p.fresh[i], p.past[i]);
    }
    int64_t all, at = block_scan(sum, all, sums);
    const bool ok = __syncthreads_and(good) && all <= p.max_tokens;
    for (int i = lo; i < hi; ++i) {
        p.cu[i] = ok ? (int32_t)at : 0;
        at += p.fresh[i];
    }
    if (threadIdx.x == 0) {
        p.cu[p.rows] = ok ? (int32_t)all : 0;
        if (!ok) flag_error(p.err, MAMBA_ERR_SEQLENS);
    }
}

}  // namespace
}  // namespace ms

using namespace ms;

extern "C" int mamba_batch_plan(const int32_t *new_tokens, const int32_t *computed, int32_t rows, const int32_t *block_table,
                                int64_t table_stride, int32_t table_cols, int32_t block, int64_t num_slots, int32_t max_tokens,
                                int32_t max_ckpt, int32_t *cu_seqlens, int32_t *slot_ids, uint8_t *has_initial_state,
                                int32_t *copy_src, int32_t *copy_dst, int32_t *ckpt_slots, int32_t *positions,
                                int32_t *token_rows, int32_t *err_word, void *stream) {
    MS_TRACE("mamba_batch_plan");
    if (rows < 0 || rows > 65535 || max_tokens < 0 || block < 0 || num_slots <= 0 || !cu_seqlens) return MAMBA_EINVAL;
    if (rows > 0 && (!new_tokens || !computed || !block_table || !slot_ids || table_cols <= 0 || table_stride < table_cols))
        return MAMBA_EINVAL;
    if ((copy_src == nullptr) != (copy_dst == nullptr) || (ckpt_slots && max_ckpt <= 0)) return MAMBA_EINVAL;
    PlanArgs a;
    a.fresh = new_tokens; a.past = computed; a.table = block_table;
    a.table_stride = table_stride; a.num_slots = num_slots;
    a.rows = rows; a.cols = table_cols; a.block = block; a.max_tokens = max_tokens; a.max_ckpt = max_ckpt;
    a.cu = cu_seqlens; a.slot = slot_ids; a.src = copy_src; a.dst = copy_dst; a.ckpt = ckpt_slots;
    a.pos = positions; a.row = token_rows; a.err = err_word; a.init = has_initial_state;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t shares = (((positions || token_rows) ? max_tokens : 0) + (int64_t)kTokensBlock - 1) / kTokensBlock;
    const unsigned grid = (unsigned)(shares < 1 ? 1 : shares > 152 ? 152 : shares);
    const bool one = rows <= kOneLaunch;
    if (!one && launch_pdl(k_batch_sums, dim3(1), dim3(kThreads), 0, st, a) != cudaSuccess) return MAMBA_ECUDA;
    if (launch_pdl(one ? k_batch_plan<true> : k_batch_plan<false>, dim3(grid), dim3(kThreads), 0, st, a) != cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}
