// gdn_scan_tc.cu -- the chunked gated delta rule on the tcgen05 tensor cores.
//
// For a chunk of 64 tokens and a head with the state S (P x N) before it, with c_i the running sum
// of the log decays, unit keys and queries k_i, q_i of lengths |k_i|, |q_i| (after any scaling), and
// w_i = b_i |k_i|^2, what a token's write takes of what the state holds along its key:
//   (I + L) U = R,   L_ij = w_i (k_i . k_j) e^(c_i - c_j), j < i
//   R = diag(b |k|) V - diag(w e^c) K S^T  the values, less what the decayed state already returns
//   U = T R,  T = (I + L)^-1               what is written, along unit keys
//   Y = |q| (diag(e^c) Q S^T + A U),       A_ij = (q_i . k_j) e^(c_i - c_j), j <= i
//   S <- e^(c_64) S + (diag(e^(c_64 - c)) U)^T K
// So the gates and the keys' lengths, which may have any size, meet the values and the state in fp32; L, T and A
// hold nothing past 2, the most that w may be.
// T and A need no state, so k_gdn_prep forms them for all chunks of the batch at once; the chain
// from chunk to chunk, k_gdn_chain, has four products left, all of them transposed so that the
// value index is the row: its left operands S, R^T, U^T are the accumulators of the product
// before, rounded to 16 bits, and never leave tensor memory; T, A, K, Q are tiles in shared
// memory in the form the products read them.
//
// Number formats: the products run on fp16 operands (11 bits; bf16's 8 would put four times the
// output's own rounding into y), sums in fp32, and the state itself stays in fp32 in registers.
// Keys and queries are of unit length before they are rounded.  Values have bf16's range, so every
// row of the state (one value index) has a power of two, chosen anew for every chunk, that brings the largest
// of its state and of what is written to it (b |k| v) to [2^7, 2^8).  The chunk takes that no further than 151 times:
// a write moves a row's length (sqrt(128) times its largest value, at most) by |b k v| and nothing else makes it
// grow, so it stays below sqrt(128) + 64 = 75.3 times the largest, and |U| below twice that and one; 151 * 2^8 is
// inside fp16's 65504.  The row's power stands that high because fp16 rounds below 2^-14 to multiples of 2^-24: a
// row's small numbers (values that fall silent, what a decay over a chunk leaves) are held to 2^-12 of themselves or
// 2^-24 of the largest in the chunk.
#include <mutex>

#include <cuda_fp16.h>

#include "gdn_scan_tc.h"
#include "umma.cuh"

namespace ms {
namespace gdn {

using namespace umma;

namespace {

constexpr int C = kChunk, TN = 128;
constexpr uint32_t kPolls = umma::kWaitPolls;
constexpr float LOG2E = 1.4426950408889634f;

// Workspace of one chunk.  Per group the tiles of unit keys and queries, 64 rows x 128 fp16 in two
// 128-byte-swizzled blocks each, interleaved [K 0..63 | Q 0..63 | K 64..127 | Q 64..127] so that keys
// and queries stacked are one operand of 128 rows; per head T, A (64 x 64, swizzled) and the gates.
constexpr uint32_t kBlk = 64 * 128;          // one swizzled block of 64 rows
constexpr uint32_t kKqBytes = 4 * kBlk;
// |k| is the length that gives the rounded unit key the token's w exactly: its factor 1 - w on what the state holds
// along its key multiplies up over the tokens, and nothing dampens that where w comes near 2.
struct HeadGates {
    float f[C];    // b |k|
    float rk[C];   // w e^c
    float oq[C];   // |q| * scale
    __half ek[C];  // e^(c_64 - c), for operands of 11 bits
    __half g[C];   // e^c, as well
    bf16 near_f[C];  // b |k| to 8 bits, for the choice of a row's power of two
    float last, pad[3];  // e^(c_64)
};
constexpr uint32_t kGateBytes = sizeof(HeadGates);
constexpr uint32_t kHeadBytes = 2 * kBlk + kGateBytes;
static_assert(kGateBytes % 16 == 0, "bulk copy size");

struct WsLayout {
    unsigned char *base;
    int64_t heads, stride;  // of a chunk: offset of the heads' part, bytes
    WsLayout(unsigned char *b, int H, int G)
        : base(b), heads((int64_t)G * kKqBytes), stride((int64_t)G * kKqBytes + (int64_t)H * kHeadBytes) {}
    __host__ __device__ int64_t chunk_bytes() const { return stride; }
    __device__ unsigned char *kq(int chunk, int g) const { return base + chunk * stride + (int64_t)g * kKqBytes; }
    __device__ unsigned char *head(int chunk, int h) const { return base + chunk * stride + heads + (int64_t)h * kHeadBytes; }
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return idesc_bf16(M, N, false, b_mn_major) & ~((7u << 7) | (7u << 10));  // A and B format: fp16
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// mbar_wait as a short loop: unrolled, the waits alone were a third of k_gdn_chain's instructions, and a
// loop that does not stay in the instruction cache runs at the rate it is fetched.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < kPolls; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

// The same with one outcome for the whole warp, which has to arrive together: a wait gives up lane by lane, and
// lanes that disagree whether to go on would leave an election (elect_one) waiting for the others.
__device__ __forceinline__ bool warp_wait_for(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_for(bar, parity));
}

// The swizzled tiles want 1024-byte boundaries; the launches ask for that much more.
template <typename T>
__device__ __forceinline__ T *align1024(unsigned char *p) {
    return reinterpret_cast<T *>(p + (-smem_u32(p) & 1023u));  // (an offset, so that accesses stay shared-memory ones)
}

// ---------------------------------------------------------------------------------------
// what needs no state: unit keys and queries, T, A and the gates of every chunk
// ---------------------------------------------------------------------------------------

constexpr int kPrepThreads = 256;
// A decay below 2^-150 is zero in fp32; with no logs lower than that the running sum of 64 of them is rounded to 2^-11
// at most, so that what decays little after a token that forgets all is still told apart.
constexpr float kNothing = -150.0f;
constexpr float kSpan = 96.0f;  // largest base-2 exponent span of a block whose decays are factored

// T of one head on the way: L's diagonal 16 x 16 blocks in fp32 (two blocks start 16 banks apart), the
// rest of L in fp16, rows 144 bytes apart so that eight rows' 16 bytes miss one another's banks.  The blocks
// of (I + L)^-1 take the places of L's that are used.
struct Inverse {
    float diag[4][16 * 20 + 16];
    __half L[C][72];
};
// Decays within a 32-token half of the chunk and from the first half to the second, as a factor of the
// row times one of the column; w: see above.
struct Decays {
    float cum[C], w[C], near[C], far[32];
};

template <int HEADS>
struct PrepSmem {
    union {
        unsigned char kq[kKqBytes];  // until its product and its copy to the workspace are done
        Inverse inv[HEADS];
    };
    unsigned char out[HEADS][2 * kBlk];  // T | A
    HeadGates gates[HEADS];
    Decays dec[HEADS];
    float ss[2 * C];  // squared lengths of keys and queries
    float inv_unit[C];  // 1 over the lengths of the keys rounded
    uint64_t bar;
    uint32_t tmem;
    float half_sum[HEADS];
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 8 x 8 matrices of 16-bit elements from shared memory, as fragments (thread T: row T / 4, elements
// 2 (T % 4) and the next), or transposed; lane l points at row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// A 16 x 16 (row-major fragments) times B 16 x 8, added to D 16 x 8: for the blocks of 16 and 32 rows
// of (I + L)^-1, below the 64 rows of a tcgen05 tile.
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Address of this lane's row for a 16 x 16 block of a matrix with 72-element rows: fragments in the
// order of an A operand, and (transposed) of two B operands side by side.
__device__ __forceinline__ uint32_t block16(const __half (*m)[72], int row, int col, int lane) {
    return smem_u32(&m[row + (lane & 15)][col + (lane >> 4) * 8]);
}

// -T22 (L21 T11) as (T22 L21) T11 for 16 rows and 16 K columns: rows row.. of T22 at columns mid.., L21 in
// rows mid.., columns left.., T11 at (left, left).  The first product's sums are the second's left
// operand as they lie in the registers.
template <int K>
__device__ __forceinline__ void lower_left(const Inverse &v, int row, int mid, int left, float (&out)[2 * K][4], int lane) {
    uint32_t a[K][4], b[4];
#pragma unroll
    for (int k = 0; k < K; ++k) ldmatrix4(a[k], block16(v.L, row, mid + 16 * k, lane));
    float x[2 * K][4] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int n = 0; n < K; ++n) {
            ldmatrix4_trans(b, block16(v.L, mid + 16 * k, left + 16 * n, lane));
            mma16(x[2 * n], a[k], b[0], b[1]);
            mma16(x[2 * n + 1], a[k], b[2], b[3]);
        }
#pragma unroll
    for (int n = 0; n < 2 * K; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[n][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t xa[4] = {pack_f16x2(-x[2 * k][0], -x[2 * k][1]), pack_f16x2(-x[2 * k][2], -x[2 * k][3]),
                                pack_f16x2(-x[2 * k + 1][0], -x[2 * k + 1][1]),
                                pack_f16x2(-x[2 * k + 1][2], -x[2 * k + 1][3])};
#pragma unroll
        for (int n = 0; n < K; ++n) {
            ldmatrix4_trans(b, block16(v.L, left + 16 * k, left + 16 * n, lane));
            mma16(out[2 * n], xa, b[0], b[1]);
            mma16(out[2 * n + 1], xa, b[2], b[3]);
        }
    }
}

// T = (I + L)^-1 of one head by a pair of warps (w = 0, 1 of the pair).  The diagonal blocks of
// 16 by forward substitution in fp32, a column a thread; the blocks below them by products.
__device__ __forceinline__ void invert(Inverse &v, unsigned char *T, int w, int lane, int pair) {
    const int d = 2 * w + (lane >> 4), c = lane & 15;  // diagonal block and its column
    {
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float acc[2] = {r == c ? 1.0f : 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < r; m += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(&v.diag[d][r * 20 + m]);
                const float *lp = &l.x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < r) acc[e & 1] = fmaf(-lp[e], x[m + e], acc[e & 1]);
            }
            x[r] = acc[0] + acc[1];
            const int row = 16 * d + r, col = 16 * d + c;
            v.L[row][col] = __float2half_rn(x[r]);
            *reinterpret_cast<__half *>(T + swz128_offset(row, col)) = v.L[row][col];
        }
        // the block right of the first of the pair's two diagonal blocks
        *reinterpret_cast<uint4 *>(&v.L[32 * w + c][32 * w + 16 + (lane >> 4) * 8]) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    const int fr = lane >> 2, fc = (lane & 3) * 2;
    auto put = [&](int row, int col, float v0, float v1) {
        *reinterpret_cast<uint32_t *>(T + swz128_offset(row, col)) = pack_f16x2(v0, v1);
    };
    {
        float o[2][4];
        const int left = 32 * w, mid = left + 16;
        lower_left<1>(v, mid, mid, left, o, lane);
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = mid + fr + 8 * e, col = left + 8 * n + fc;
                *reinterpret_cast<uint32_t *>(&v.L[row][col]) = pack_f16x2(o[n][2 * e], o[n][2 * e + 1]);
                put(row, col, o[n][2 * e], o[n][2 * e + 1]);
            }
    }
    asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
    {
        float o[4][4];
        lower_left<2>(v, 32 + 16 * w, 32, 0, o, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) put(32 + 16 * w + fr + 8 * e, 8 * n + fc, o[n][2 * e], o[n][2 * e + 1]);
    }
}

// Block (chunk, group and share of its heads): two heads of a group share its keys' and queries' one product,
// K K^T over Q K^T.  0.5 MB of a 64-token chunk of 32 heads and 16 groups are read and 1.1 MB written; 8192 tokens
// take 57 us (3.6 TB/s).  Neither memory nor the issue slots (a third used) bound it but a block's own row of steps
// (loads, product, decays, the inverse); three blocks an SM run side by side, 70 KB of shared memory each.
template <int HEADS>
__global__ void __launch_bounds__(kPrepThreads, 3) k_gdn_prep(const ScanParams p, const WsLayout ws) {
    extern __shared__ __align__(1024) unsigned char prep_smem[];
    PrepSmem<HEADS> &sm = *align1024<PrepSmem<HEADS>>(prep_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int chunk = blockIdx.x;
    if (p.meta[0] == 0 || chunk >= p.meta[1]) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int2 where = meta_table(p)[chunk];
    const int64_t t0 = where.x;
    const int L = where.y;
    const int shares = p.HG / HEADS;
    const int g = blockIdx.y / shares, h0 = g * p.HG + (blockIdx.y % shares) * HEADS;
    // a token of a head a thread: its raw step and gate; no step and no write past the sequence's end
    float run = 0.0f, b = 0.0f;
    const int hh = tid / C, tok = tid & (C - 1);
    if (hh < HEADS && tok < L) {
        const int64_t th = (t0 + tok) * p.H + h0 + hh;
        run = load_scalar(p.dt, th, p.gates.dt_bf16);
        b = load_scalar(p.beta, th, p.gates.dt_bf16);
    }
    // unit keys (rows 0..63) and queries (64..127): 16 lanes a row, 16 rows a pass
    {
        const int r0 = tid >> 4, col = (tid & 15) * 8;
        uint4 raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (i * 16 + r0) & (C - 1);
            const bf16 *src = static_cast<const bf16 *>(i < 4 ? p.k : p.q) + ((t0 + row) * p.G + g) * TN + col;
            raw[i] = row < L ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
        }
        if (warp == 0) {
            tmem_alloc(&sm.tmem, 64);
            tmem_relinquish();
        }
        if (tid == 0) {
            mbar_init(&sm.bar, 1);
            fence_mbar_init();
        }
#pragma unroll
        for (int e = tid * 16; e < (int)kBlk; e += kPrepThreads * 16)  // T above its diagonal blocks
#pragma unroll
            for (int x = 0; x < HEADS; ++x) *reinterpret_cast<uint4 *>(sm.out[x] + e) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            unpack16(raw[i], f);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
            ss = sum_lanes<16>(ss);
            const float inv = ss > 0.0f ? rsqrtf(ss) : 0.0f;
            const int row = i * 16 + r0;  // of the stacked tile
            uint4 u;
            u.x = pack_f16x2(f[0] * inv, f[1] * inv);
            u.y = pack_f16x2(f[2] * inv, f[3] * inv);
            u.z = pack_f16x2(f[4] * inv, f[5] * inv);
            u.w = pack_f16x2(f[6] * inv, f[7] * inv);
            *reinterpret_cast<uint4 *>(sm.kq + (col >> 6) * 2 * kBlk + swz128_chunk(row, (col & 63) >> 3)) = u;
            if (i < 4) {  // what rounding made of the key's unit length goes into its length (see HeadGates)
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                float rr = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                    rr = fmaf(r.x, r.x, fmaf(r.y, r.y, rr));
                }
                rr = sum_lanes<16>(rr);
                if (col == 0) sm.inv_unit[row] = rr > 0.0f ? rsqrtf(rr) : 0.0f;
            }
            if (col == 0) sm.ss[row] = ss;
        }
    }
    // running sums of the log decays (base 2) over each head's two warps of tokens
    if (hh < HEADS) {
        if (tok < L) {
            run = log_decay(p.gates, run, h0 + hh) * LOG2E;
            if (run < kNothing) run = kNothing;  // (a NaN stays)
            b = write_gate(p.gates, b);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (tok == 31) sm.half_sum[hh] = run;
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    if (warp == 7 && elect_one()) {
        const uint32_t kq = smem_u32(sm.kq);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // rows 0..63: k_i . k_j, rows 64..127: q_i . k_j
            mma_bf16(tm, desc_kmajor(kq, 2 * kBlk, kk), desc_kmajor(kq, 2 * kBlk, kk), idesc_f16(128, C, false), kk > 0);
        mma_commit(&sm.bar);
        if (blockIdx.y % shares == 0) {
            bulk_s2g(ws.kq(chunk, g), sm.kq, kKqBytes);
            bulk_commit();
            bulk_wait_read<0>();  // the tile's memory is reused below
        }
    }
    // The decay e^(c_i - c_j), j <= i, is a row factor times a column factor.  From the first half of the
    // chunk to the second both are taken to the first half's last token, so both are at most 1; within a
    // half to its first token, where the column's is at least 1 and is used only while the half spans at
    // most 2^96 (wider ones form each decay from its own difference, below).
    if (hh < HEADS) {
        Decays &dec = sm.dec[hh];
        if (tok >= 32) run += sm.half_sum[hh];
        dec.cum[tok] = run;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + hh) : "memory");
        const float kk = sm.ss[tok], qq = sm.ss[C + tok], last = dec.cum[C - 1], e = exp2f(run);
        const float nk = sqrtf(kk) * unit_factor(p.gates, kk) * sm.inv_unit[tok], f = b * nk, w = f * nk;
        HeadGates &gt = sm.gates[hh];
        gt.f[tok] = f;
        gt.near_f[tok] = __float2bfloat16(f);
        gt.rk[tok] = w * e;
        dec.w[tok] = w;
        gt.ek[tok] = __float2half_rn(exp2f(last - run));
        gt.g[tok] = __float2half_rn(e);
        gt.oq[tok] = sqrtf(qq) * unit_factor(p.gates, qq) * p.gates.scale;
        if (tok == 0) gt.last = exp2f(last);
        dec.near[tok] = exp2f(fminf(dec.cum[tok & 32] - run, kSpan));
        if (tok < 32) dec.far[tok] = exp2f(dec.cum[31] - run);
    }
    const int bad = wait_for(&sm.bar, 0) ? 0 : 1;
    tc_fence_after();
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            flag_error(p.err, MAMBA_ERR_TIMEOUT);
            wait_for(&sm.bar, 0);
        }
    } else {
        const int q = warp & 3, hf = warp >> 2, i = (q & 1) * 32 + lane;  // row i of K K^T (q < 2) or Q K^T
        float dots[32];
        tmem_ld32(tm + ((uint32_t)(q * 32) << 16) + hf * 32, dots);
        // L (what T needs of it) and A of this thread's 32 columns
#pragma unroll 1
        for (int x = 0; x < HEADS; ++x) {
            const Decays &dec = sm.dec[x];
            const float ci = dec.cum[i], wi = q < 2 ? dec.w[i] : 1.0f;
            float w[32];
            if (hf < (q & 1)) {  // from the first half to the second
                const float f = exp2f(ci - dec.cum[31]) * wi;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(dec.far + j);
                    w[j] = dots[j] * (f * u.x);
                    w[j + 1] = dots[j + 1] * (f * u.y);
                    w[j + 2] = dots[j + 2] * (f * u.z);
                    w[j + 3] = dots[j + 3] * (f * u.w);
                }
            } else if (hf == (q & 1)) {  // within a half
                const int lim = q < 2 ? lane : lane + 1;  // columns below it count
                if (dec.cum[hf * 32] - dec.cum[hf * 32 + 31] <= kSpan) {
                    const float f = exp2f(ci - dec.cum[hf * 32]) * wi;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(dec.near + hf * 32 + j);
                        w[j] = j < lim ? dots[j] * (f * u.x) : 0.0f;
                        w[j + 1] = j + 1 < lim ? dots[j + 1] * (f * u.y) : 0.0f;
                        w[j + 2] = j + 2 < lim ? dots[j + 2] * (f * u.z) : 0.0f;
                        w[j + 3] = j + 3 < lim ? dots[j + 3] * (f * u.w) : 0.0f;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float v = dots[j] * wi * exp2_approx(ci - dec.cum[hf * 32 + j]);
                        w[j] = j < lim ? v : 0.0f;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) w[j] = 0.0f;
            }
            if (q < 2) {
                if (hf <= (q & 1)) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        *reinterpret_cast<uint4 *>(&sm.inv[x].L[i][hf * 32 + j]) =
                            make_uint4(pack_f16x2(w[j], w[j + 1]), pack_f16x2(w[j + 2], w[j + 3]),
                                       pack_f16x2(w[j + 4], w[j + 5]), pack_f16x2(w[j + 6], w[j + 7]));
                }
                if (hf == (q & 1)) {  // this row's part of its diagonal block of 16
                    float *dst = &sm.inv[x].diag[i >> 4][(i & 15) * 20];
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(dst + j) =
                            make_float4(lane & 16 ? w[j + 16] : w[j], lane & 16 ? w[j + 17] : w[j + 1],
                                        lane & 16 ? w[j + 18] : w[j + 2], lane & 16 ? w[j + 19] : w[j + 3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    *reinterpret_cast<uint4 *>(sm.out[x] + kBlk + swz128_chunk(i, hf * 4 + j / 8)) =
                        make_uint4(pack_f16x2(w[j], w[j + 1]), pack_f16x2(w[j + 2], w[j + 3]), pack_f16x2(w[j + 4], w[j + 5]),
                                   pack_f16x2(w[j + 6], w[j + 7]));
            }
        }
        __syncthreads();
        if (warp < 2 * HEADS) {
            const int x = warp >> 1;
            invert(sm.inv[x], sm.out[x], warp & 1, lane, x);
        }
        fence_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one()) {
#pragma unroll
            for (int x = 0; x < HEADS; ++x) {
                unsigned char *dst = ws.head(chunk, h0 + x);
                bulk_s2g(dst, sm.out[x], 2 * kBlk);
                bulk_s2g(dst + 2 * kBlk, &sm.gates[x], kGateBytes);
            }
            bulk_commit();
            bulk_wait_all();
        }
        if (warp == 7 && elect_one()) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tm, 64);
}

// ---------------------------------------------------------------------------------------
// the chain over a sequence's chunks
// ---------------------------------------------------------------------------------------

constexpr int kChainThreads = 256;       // four warps on the chain, four beside it
constexpr int kChainRegs = 208, kSideRegs = 48;  // (208 + 48) * 128 registers: what the block is launched with
constexpr int kRows = 128;               // rows of tensor memory; with head_dim 64 the upper half holds zeros
constexpr int kTop = 7;                  // a row's power of two brings its largest value to [2^kTop, 2^(kTop + 1))

// What the block waits for: keys, gates and values (two stages), queries, T and A from memory; the products X, U,
// Q S^T, the increment and Y; the values in registers.
enum { B_IN = 0, B_Q = 2, B_T, B_A, B_X, B_U, B_OI, B_S, B_Y, B_TAKEN, kBars };

struct ChainSmem {
    // q: a chunk's queries, and once they are used its outputs on their way to memory; v: its values, by token
    unsigned char k[2][2 * kBlk], q[2][2 * kBlk], T[kBlk], A[kBlk], v[2 * kBlk];
    HeadGates gates[4];
    float unscale[2][kRows];   // a chunk's inverse powers of two, by row
    uint64_t bar[kBars];
    uint32_t tmem;
    // the block's sequence, head, first token, tokens and chunks, and the first chunk's part of the workspace:
    // here and not in registers, of which the chain has none to spare (what is spilled comes back from L2:
    // next to this much shared memory almost no L1 is left)
    int s, h, t0, len, nc;
    const unsigned char *head0, *kq0;
    uint32_t armed[8], parity[8];  // what each warp leaves behind (Armed)
};

// The barriers ever armed with a copy or a product, and the last phase of each: what is waited for
// before a block that gave up lets go of its memory.
struct Armed {
    uint32_t bars = 0, parity = 0;
    __device__ __forceinline__ void operator()(int i, uint32_t phase) {
        bars |= 1u << i;
        parity = (parity & ~(1u << i)) | phase << i;
    }
};

// Tensor-memory columns: the state's 16-bit copy and X (or R^T over X) make way for the new state's
// increment, which is as wide as both.
constexpr uint32_t T_S = 0, T_X = 64, T_D = 0, T_U = 128, T_Y = 192;

template <int REGS>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// Barrier of one half of the block (1: the chain, 2: the side); whether any thread passed a non-zero
// value.
__device__ __forceinline__ bool half_sync_or(int half, int v) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(any)
        : "r"(v), "r"(half)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void max_abs(float &m, float a, float b) {
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(a), "f"(b));
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 fp32 columns of a warp's 32 lanes as matrix fragments, 16 lanes a load: element
// [half][4 n + 2 r + e] is lane 16 half + 8 r + T / 4, column 8 n + 2 (T % 4) + e.
__device__ __forceinline__ void tmem_frag2(uint32_t a, float (&v)[2][8]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a), "r"(a + (16u << 16))
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i >> 3][i & 7] = __uint_as_float(r[i]);
}
// 16 fp32 columns of this warp's lanes, on their way after the first call and there after the second: what
// stands between them hides the latency, and the second's operands keep the uses after it.
__device__ __forceinline__ void tmem_get(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_got(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// N pieces of 16 columns from a, each given to f(piece, values) with the next one on its way.
template <int N, typename F>
__device__ __forceinline__ void tmem_pieces(uint32_t a, F f) {
    uint32_t r[2][16];
    tmem_get(a, r[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        tmem_got(r[i & 1]);
        if (i + 1 < N) tmem_get(a + 16 * (i + 1), r[(i + 1) & 1]);
        f(i, r[i & 1]);
    }
}
// 8 32-bit columns (two 16-bit values each) of this warp's lanes; tmem_put_wait waits for all before it.
__device__ __forceinline__ void tmem_put8(uint32_t a, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// A tile to memory, tracked in the issuing thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// One sequence and head, as both halves of the block see it.
template <int P>
struct ChainJob {
    const ScanParams &p;
    const WsLayout &ws;
    const CUtensorMap &vmap, &ymap;
    ChainSmem &sm;

    __device__ __forceinline__ const unsigned char *head(int c) const { return sm.head0 + c * ws.chunk_bytes(); }
    __device__ __forceinline__ const unsigned char *kq(int c) const { return sm.kq0 + c * ws.chunk_bytes(); }
    __device__ __forceinline__ void load_keys(int c) const {
        uint64_t *bar = &sm.bar[B_IN + (c & 1)];
        mbar_arrive_expect_tx(bar, 2 * kBlk + kGateBytes);
        bulk_g2s(sm.k[c & 1], kq(c), kBlk, bar);
        bulk_g2s(sm.k[c & 1] + kBlk, kq(c) + 2 * kBlk, kBlk, bar);
        bulk_g2s(&sm.gates[c & 3], head(c) + 2 * kBlk, kGateBytes, bar);
    }
    __device__ __forceinline__ void load_queries(int c) const {
        mbar_arrive_expect_tx(&sm.bar[B_Q], 2 * kBlk);
        bulk_g2s(sm.q[c & 1], kq(c) + kBlk, kBlk, &sm.bar[B_Q]);
        bulk_g2s(sm.q[c & 1] + kBlk, kq(c) + 3 * kBlk, kBlk, &sm.bar[B_Q]);
    }
    __device__ __forceinline__ void load_values(int c) const {
        uint64_t *bar = &sm.bar[B_IN + (c & 1)];
        mbar_arrive_expect_tx(bar, C * P * 2);
        tma_load_2d(sm.v, &vmap, sm.h * P, sm.t0 + c * C, bar);
    }
    __device__ __forceinline__ void load_tile(int c, int i, unsigned char *dst, uint32_t off) const {
        mbar_arrive_expect_tx(&sm.bar[i], kBlk);
        bulk_g2s(dst, head(c) + off, kBlk, &sm.bar[i]);
    }
    // into L2, for loads that are needed within a thousand cycles of their issue
    __device__ __forceinline__ void prefetch(int c) const {
        bulk_prefetch(head(c), kHeadBytes);
        bulk_prefetch(kq(c), kKqBytes);
        asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&vmap)),
                     "r"(sm.h * P), "r"(sm.t0 + c * C)
                     : "memory");
    }
};

// The chain's four warps: warp w holds rows 32 w .. + 31 of the state, a row a thread.  Returns whether
// a wait gave up.
template <int P>
__device__ __forceinline__ bool chain_warps(const ChainJob<P> &J, Armed &arm) {
    const ScanParams &p = J.p;
    ChainSmem &sm = J.sm;
    const int row = threadIdx.x, warp = threadIdx.x >> 5;
    const uint32_t lanes = sm.tmem + ((uint32_t)(warp * 32) << 16);  // (of warp 0: tensor memory's first lane)
    const int32_t slot = p.slot[sm.s];
    auto pool_row = [&](int32_t to) {
        return static_cast<bf16 *>(p.pool) + to * p.stride + ((int64_t)sm.h * P + row) * TN;
    };
    float S[TN];  // times the row's power of two
    float top = 0.0f;  // the row's largest magnitude, as S holds it
    {
        const bool seeded = row < P && slot >= 0 && p.has_init && p.has_init[sm.s];
        const bf16 *src = pool_row(seeded ? slot : 0);
#pragma unroll
        for (int e = 0; e < TN; e += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (seeded)  // (volatile: one after the other, not all in registers at once)
                asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(src + e));
            float f[8];
            unpack16(w, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) S[e + i] = f[i], top = fmaxf(top, fabsf(f[i]));
        }
    }
    float scale = 1.0f, unscale = 1.0f;  // the power of two and its inverse
    int bad = 0;  // a wait gave up: all four warps leave at the next barrier

    auto store_state16 = [&](int e) {  // 16 columns of the state's copy for the products
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pk[i] = pack_f16x2(S[e + 2 * i], S[e + 2 * i + 1]);
        tmem_put8(lanes + T_S + e / 2, pk);
    };
    auto issue_x = [&](int c) {  // X = S K^T
        const uint32_t k = smem_u32(sm.k[c & 1]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(lanes + T_X, lanes + T_S + 8 * kk, desc_kmajor(k, kBlk, kk), idesc_f16(128, C, false), kk > 0);
        mma_commit(&sm.bar[B_X]);
    };
    auto write_state = [&](int32_t to) {
        if (row >= P) return;
        uint4 *dst = reinterpret_cast<uint4 *>(pool_row(to));
#pragma unroll
        for (int e = 0; e < TN; e += 8) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = S[e + i] * unscale;
            dst[e / 8] = pack16(f);
        }
    };

    // The row's values of chunk c, two tokens' each (with head_dim 64 the upper rows hold zeros), and the row's
    // power of two for it, by the largest of state and writes b |k| v.  Rows are their threads' own, so no other thread needs to know.
    uint32_t vals[C / 2];
    auto take_values = [&](int c) {
        if (!wait_for(&sm.bar[B_IN + (c & 1)], c >> 1 & 1)) bad = 1;
        const uint16_t *v = reinterpret_cast<const uint16_t *>(sm.v) + (row & (P - 1));
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            vals[i] = v[2 * i * P] | (uint32_t)v[(2 * i + 1) * P] << 16;
            if (row >= P) vals[i] = 0;
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.bar[B_TAKEN]);
        const int L = sm.len - c * C;
        if (__builtin_expect(L < C, 0)) {  // past the sequence's end the tile holds another's values
#pragma unroll
            for (int i = 0; i < C / 2; ++i) vals[i] = 2 * i + 1 < L ? vals[i] : (2 * i < L ? vals[i] & 0xffffu : 0u);
        }
    };
    auto choose_power = [&](int c) {
        __nv_bfloat162 m[4];  // (four chains of maxima: one would be the latency of 32)
#pragma unroll
        for (int n = 0; n < C / 8; ++n) {
            const uint4 fw = *reinterpret_cast<const uint4 *>(sm.gates[c & 3].near_f + 8 * n);
            const uint32_t f[4] = {fw.x, fw.y, fw.z, fw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 w = __habs2(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&vals[4 * n + i]),
                                                         *reinterpret_cast<const __nv_bfloat162 *>(&f[i])));
                m[i] = n ? __hmax2(m[i], w) : w;
            }
        }
        m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
        const float vmax = fmaxf(__low2float(m[0]), __high2float(m[0]));
        // biased exponents: E of the largest, old of the one that the present power brings to 2^kTop
        const float most = fmaxf(top * unscale, vmax);
        const uint32_t old = (__float_as_uint(unscale) >> 23) + kTop;
        const uint32_t E = most < INFINITY ? max(1u + kTop, __float_as_uint(most) >> 23) : old;
        if (E != old) {
            scale = __uint_as_float((254u + kTop - E) << 23);
            unscale = __uint_as_float((E - kTop) << 23);
            int shift = (int)old - (int)E;
            while (shift != 0) {  // (in two steps where no float holds their ratio)
                const int by = max(-126, min(126, shift));
                const float ratio = __uint_as_float((uint32_t)(127 + by) << 23);
                shift -= by;
#pragma unroll
                for (int e = 0; e < TN; ++e) S[e] *= ratio;
            }
        }
        sm.unscale[c & 1][row] = unscale;
#pragma unroll
        for (int e = 0; e < TN; e += 16) store_state16(e);
        tmem_put_wait();
    };

    for (int c = -1; c < sm.nc; ++c) {  // (from -1: only what readies the first chunk)
        const uint32_t ph = c & 1;
        const HeadGates &gt = sm.gates[c & 3];
        if (c >= 0) {
            // 1. X = S K^T
            if (warp == 0) {
                arm(B_X, ph);
                if (elect_one()) issue_x(c);
                if (!wait_for(&sm.bar[B_T], ph)) bad = 1;
            }
            // 2. R = b |k| V - w e^c X, rounded, over X (past the sequence's end the values, the keys and so X are zero)
            if (!wait_for(&sm.bar[B_X], ph)) bad = 1;
            tc_fence_after();
            {
                const uint64_t sc = pair(scale, scale);
#pragma unroll
                for (int n = 0; n < C / 16; ++n) {  // 16 tokens
                    uint32_t x[16], pk[8];
                    tmem_get(lanes + T_X + 16 * n, x);
                    tmem_got(x);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {  // two tokens, twice
                        const float4 f = *reinterpret_cast<const float4 *>(gt.f + 16 * n + 2 * i);
                        const float4 r = *reinterpret_cast<const float4 *>(gt.rk + 16 * n + 2 * i);
                        auto two = [&](int j, float f0, float f1, float r0, float r1) {
                            const uint32_t w = vals[8 * n + j];
                            const uint64_t v2 = mul2(mul2(pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), pair(f0, f1)), sc);
                            float lo, hi;
                            unpair(fma2(pair(-r0, -r1), pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), v2), lo, hi);
                            pk[j] = pack_f16x2(lo, hi);
                        };
                        two(i, f.x, f.y, r.x, r.y), two(i + 1, f.z, f.w, r.z, r.w);
                    }
                    tmem_put8(lanes + T_X + 8 * n, pk);  // (packed to the left: over what has been read)
                }
                tmem_put_wait();
            }
            tc_fence_before();
            if (half_sync_or(1, bad)) return true;
            tc_fence_after();
            // 3. U^T = R^T T^T (the side, which has time for it, issues the state's part of Y and the loads: code that
            // one warp runs once a chunk comes from far in the instruction cache, some 400 cycles a visit)
            if (warp == 0) {
                arm(B_U, ph);
                if (elect_one()) {
                    const uint32_t T = smem_u32(sm.T);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ts(lanes + T_U, lanes + T_X + kk * 8, desc_kmajor(T, kBlk, kk), idesc_f16(128, C, false), kk > 0);
                    mma_commit(&sm.bar[B_U]);
                }
            } else if (warp == 2) {
                if (!wait_for(&sm.bar[B_A], ph)) bad = 1;
            } else if (warp == 3) {
                if (!wait_for(&sm.bar[B_OI], ph)) bad = 1;  // the state's copy is read: the increment may take its columns
            }
            // 4. U^T rounded, as it is and times e^(c_64 - c) (a product of rounded numbers: a conversion from fp32
            // takes four times as long)
            if (!wait_for(&sm.bar[B_U], ph)) bad = 1;
            tc_fence_after();
            tmem_pieces<4>(lanes + T_U, [&](int n, const uint32_t (&u)[16]) {  // 16 tokens: both forms over their own columns
                const uint4 w0 = *reinterpret_cast<const uint4 *>(gt.ek + 16 * n);
                const uint4 w1 = *reinterpret_cast<const uint4 *>(gt.ek + 16 * n + 8);
                const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                uint32_t pk[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) pk[i] = pack_f16x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                tmem_put8(lanes + T_U + 16 * n, pk);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const __half2 e = __hmul2(*reinterpret_cast<const __half2 *>(&pk[i]), *reinterpret_cast<const __half2 *>(&w[i]));
                    pk[i] = *reinterpret_cast<const uint32_t *>(&e);
                }
                tmem_put8(lanes + T_U + 16 * n + 8, pk);
            });
            tmem_put_wait();
            tc_fence_before();
            if (half_sync_or(1, bad)) return true;
            tc_fence_after();
            // 5. the state's increment, over the columns of its copy and of R (both are read), and A's part of Y; meanwhile
            // the next values
            if (warp == 0) {
                arm(B_S, ph), arm(B_Y, ph);
                if (elect_one()) {
                    const uint32_t A = smem_u32(sm.A), k = smem_u32(sm.k[ph]);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ts(lanes + T_D, lanes + T_U + kk * 16 + 8, desc_mnmajor(k, kBlk, kk), idesc_f16(128, TN, true), kk > 0);
                    mma_commit(&sm.bar[B_S]);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ts(lanes + T_Y, lanes + T_U + kk * 16, desc_kmajor(A, kBlk, kk), idesc_f16(128, C, false), 1);
                    mma_commit(&sm.bar[B_Y]);
                }
            }
        }
        if (c + 1 < sm.nc) take_values(c + 1);
        if (c >= 0) {
            // 6. the new state, and its copy over the increment (a row's columns are its thread's own)
            const float last = gt.last;
            float tops[4] = {};
            if (!wait_for(&sm.bar[B_S], ph)) bad = 1;
            tc_fence_after();
#pragma unroll
            for (int n = 0; n < TN / 16; ++n) {
                uint32_t d[16];
                tmem_get(lanes + T_D + 16 * n, d);
                tmem_got(d);
#pragma unroll
                for (int i = 0; i < 16; ++i) S[16 * n + i] = fmaf(last, S[16 * n + i], __uint_as_float(d[i]));
#pragma unroll
                for (int i = 0; i < 16; i += 2) max_abs(tops[i / 2 & 3], S[16 * n + i], S[16 * n + i + 1]);
            }
            top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            if (p.ckpt_slots) {
                const int32_t cs = ckpt_slot(p, sm.s, min(sm.len, (c + 1) * C), threadIdx.x == 0 && sm.h == 0);
                if (__builtin_expect(cs >= 0, 0)) write_state(cs);
            }
        }
        if (c + 1 < sm.nc) choose_power(c + 1);
        tc_fence_before();
        if (half_sync_or(1, bad)) return true;
        tc_fence_after();
    }
    if (slot >= 0) write_state(slot);
    return false;
}

// The four warps beside the chain: they scale the next chunk's queries, issue the state's part of Y, take the
// outputs to memory, and load.  Warp w works on tensor-memory lanes 32 w .. + 31, as fragments of 32 values
// by 8 tokens.  Returns whether a wait gave up.
template <int P>
__device__ __forceinline__ bool side_warps(const ChainJob<P> &J, Armed &arm) {
    const ScanParams &p = J.p;
    ChainSmem &sm = J.sm;
    const int tid = threadIdx.x - 128, warp = tid >> 5, lane = tid & 31;
    const bool live = 32 * warp < P;  // this warp's rows are values
    const uint32_t lanes = sm.tmem + ((uint32_t)(warp * 32) << 16);
    // this lane's 16 bytes (8 values of a token) of the outputs' tile, for 8 tokens from 8 n
    auto token_row = [&](const unsigned char *tile, int n) {
        return smem_u32(tile) + (warp >> 1) * kBlk + swz128_chunk(8 * n + (lane & 7), 4 * (warp & 1) + (lane >> 3));
    };
    int bad = 0;  // the same in all lanes of a warp
    for (int c = -1; c < sm.nc; ++c) {
        const int c1 = c + 1;
        if (c >= 0 && warp == 0) {
            // the state's part of Y, once the state's copy is there (X is formed of it)
            if (!warp_wait_for(&sm.bar[B_X], c & 1)) bad = 1;
            tc_fence_after();
            if (!bad) {
                arm(B_OI, c & 1);
                if (elect_one()) {
                    const uint32_t q = smem_u32(sm.q[c & 1]), tm = sm.tmem;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_ts(tm + T_Y, tm + T_S + 8 * kk, desc_kmajor(q, kBlk, kk), idesc_f16(128, C, false), kk > 0);
                    mma_commit(&sm.bar[B_OI]);
                }
            }
        } else if (c >= 0 && warp == 3 && c1 < sm.nc) {
            if (!warp_wait_for(&sm.bar[B_U], c & 1)) bad = 1;  // T is used
            if (!bad) {
                arm(B_T, c1 & 1);
                if (elect_one()) J.load_tile(c1, B_T, sm.T, 0);
            }
        } else if (warp == 2 && c + 2 < sm.nc) {
            if (elect_one()) J.prefetch(c + 2);
        }
        if (c1 < sm.nc) {
            // the next chunk's queries times e^c, in place, 16 bytes of a token each: tokens 16 apart, in both blocks
            // of 64 elements
            if (!warp_wait_for(&sm.bar[B_IN + (c1 & 1)], (c1 >> 1) & 1) || !warp_wait_for(&sm.bar[B_Q], c1 & 1)) bad = 1;
            const __half *g = sm.gates[c1 & 3].g + (tid >> 3);
            uint4 *ptr = reinterpret_cast<uint4 *>(sm.q[c1 & 1]) + tid;
            uint4 u[8];
            __half2 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __half2half2(g[16 * i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = ptr[128 * i];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                __half2 *hp = reinterpret_cast<__half2 *>(&u[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) hp[e] = __hmul2(hp[e], w[i & 3]);
                ptr[128 * i] = u[i];
            }
            fence_async_smem();
            if (warp == 1 && c + 2 < sm.nc) {
                if (!warp_wait_for(&sm.bar[B_TAKEN], c1 & 1)) bad = 1;  // the next values are in registers
                if (!bad) {
                    arm(B_IN + (c & 1), (c + 2) >> 1 & 1);
                    if (elect_one()) J.load_values(c + 2);
                }
            }
        }
        // this chunk's outputs, over its queries and from there to memory
        if (c >= 0) {
            const float *oq = sm.gates[c & 3].oq + (lane & 3) * 2;
            float2 w[8];
            float un[4];
#pragma unroll
            for (int n = 0; n < 8; ++n) w[n] = *reinterpret_cast<const float2 *>(oq + 8 * n);
            if (!warp_wait_for(&sm.bar[B_Y], c & 1)) bad = 1;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 4; ++i) un[i] = sm.unscale[c & 1][32 * warp + 8 * i + (lane >> 2)];
            if (warp == 2 && !bad) {
                if (c1 < sm.nc) arm(B_A, c1 & 1);
                if (c + 2 < sm.nc) arm(B_IN + (c & 1), (c + 2) >> 1 & 1);
                if (elect_one()) {
                    if (c1 < sm.nc) J.load_tile(c1, B_A, sm.A, kBlk);
                    if (c + 2 < sm.nc) J.load_keys(c + 2);
                }
            }
            if (live) {
#pragma unroll
                for (int n = 0; n < 8; n += 2) {
                    float y[2][8];
                    tmem_frag2(lanes + T_Y + 8 * n, y);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint64_t w2 = pair(w[n + m].x, w[n + m].y);
                        uint32_t pk[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float *yi = &y[i >> 1][4 * m + 2 * (i & 1)];
                            float lo, hi;
                            unpair(mul2(pair(yi[0], yi[1]), mul2(w2, pair(un[i], un[i]))), lo, hi);
                            const __nv_bfloat162 o = __floats2bfloat162_rn(lo, hi);
                            pk[i] = *reinterpret_cast<const uint32_t *>(&o);
                        }
                        stmatrix4_trans(token_row(sm.q[c & 1], n + m), pk);
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
        }
        if (half_sync_or(2, bad)) return true;  // Y is taken, the outputs are staged, the next queries scaled
        const bool whole = c >= 0 && (c + 1) * C <= sm.len;
        if (c >= 0 && !whole) {  // the sequence's last tokens: the rows after them are another's
            constexpr int CH = P / 8;  // 16-byte pieces of a token's outputs; a thread takes every 128 / CH-th token
            const int L = sm.len - c * C, ch = tid % CH;
            bf16 *dst = static_cast<bf16 *>(p.y) + ((int64_t)(sm.t0 + c * C) * p.H + sm.h) * P + ch * 8;
            const unsigned char *src = sm.q[c & 1] + (ch >> 3) * kBlk;
            for (int t = tid / CH; t < L; t += 128 / CH)
                *reinterpret_cast<uint4 *>(dst + (int64_t)t * p.H * P) = *reinterpret_cast<const uint4 *>(src + swz128_chunk(t, ch & 7));
        }
        if (warp == 3) {
            if (c + 2 < sm.nc) arm(B_Q, c & 1);
            if (elect_one()) {
                if (whole) {
                    for (int i = 0; i < P / 64; ++i) tma_store_2d(&J.ymap, sm.q[c & 1] + i * kBlk, sm.h * P + 64 * i, sm.t0 + c * C);
                    bulk_commit();
                    bulk_wait_read<0>();
                }
                if (c + 2 < sm.nc) J.load_queries(c + 2);  // (a chunk with two after it is whole, or there is none: the place is free)
            }
        }
    }
    // the copies out of shared memory have read it (bulk_wait_read, above); their writes complete with the grid
    return half_sync_or(2, bad);
}

// Block (sequence in the plan's order, head).  What bounds it is the chain itself, 2.8 us for 64 tokens (one prompt of
// 8192 tokens, 32 blocks: 358 us).  Three products that wait for one another take 370 to 510 cycles each from issue
// to completion, together a quarter of that; the rest are the four warps that may reach their tensor-memory lanes,
// which scale, round and write back the 128 rows' R, U and state, a row a thread, one warp on each of the SM's
// schedulers.  The writes' scaling in fp32, the row's largest value and its power of two in every chunk are an eighth
// of the time.  Two blocks share an SM: 8 ragged prompts of 32768 tokens in all, 256 blocks, take 355 us for the 104
// chunks of the longest, 3.4 us each, a fifth more than alone.  Heads of 64 values leave half of the rows idle:
// tcgen05's 64-row form puts its accumulator's rows elsewhere, and the chain's length would be the same.
template <int P>
__global__ void __launch_bounds__(kChainThreads, 2) k_gdn_chain(const ScanParams p, const WsLayout ws,
                                                                const __grid_constant__ CUtensorMap vmap,
                                                                const __grid_constant__ CUtensorMap ymap) {
    extern __shared__ __align__(1024) unsigned char chain_smem[];
    ChainSmem &sm = *align1024<ChainSmem>(chain_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    if (p.meta[0] == 0) return;  // bad cu_seqlens (flagged): nothing is done
    {
        const int s = meta_order(p)[blockIdx.x / p.H], h = blockIdx.x % p.H, len = p.cu[s + 1] - p.cu[s];
        const int32_t slot = p.slot[s];
        if (len <= 0 || slot < -1 || slot >= p.num_slots) return;  // empty, or bad slot (flagged)
        if (threadIdx.x == 160) {
            sm.s = s, sm.h = h, sm.t0 = p.cu[s], sm.len = len, sm.nc = (len + C - 1) / C;
            const int first = meta_chunks(p)[s];
            sm.head0 = ws.head(first, h);
            sm.kq0 = ws.kq(first, h / p.HG);
        }
    }
    const ChainJob<P> J = {p, ws, vmap, ymap, sm};
    const int warp = threadIdx.x >> 5;
    __syncwarp();
    if (warp == 5 && elect_one()) {
        for (int i = 0; i < kBars; ++i) mbar_init(&sm.bar[i], i == B_TAKEN ? 4 : i < B_Q ? 2 : 1);
        fence_mbar_init();
        tma_prefetch_desc(&vmap);
        J.load_keys(0);
        J.load_values(0);
        J.load_queries(0);
        J.load_tile(0, B_T, sm.T, 0);
        J.load_tile(0, B_A, sm.A, kBlk);
        if (sm.nc > 1) J.load_keys(1);
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    bool failed;
    if (warp < 4) {
        more_registers<kChainRegs>();
        Armed arm;
        failed = chain_warps(J, arm);
        if ((threadIdx.x & 31) == 0) sm.armed[warp] = arm.bars, sm.parity[warp] = arm.parity;
    } else {
        fewer_registers<kSideRegs>();
        Armed arm;
        arm(B_IN, 0), arm(B_Q, 0), arm(B_T, 0), arm(B_A, 0);
        failed = side_warps(J, arm);
        if ((threadIdx.x & 31) == 0) sm.armed[warp] = arm.bars, sm.parity[warp] = arm.parity;
    }
    if (__syncthreads_or(failed)) {
        // an operation did not complete in time: report it, and give what this block still has in flight
        // the same bounded time to finish before its memory is released
        if (warp == 4 && elect_one()) {
            flag_error(p.err, MAMBA_ERR_TIMEOUT);
            for (int w = 0; w < 8; ++w)
                for (int i = 0; i < kBars; ++i)
                    if (sm.armed[w] >> i & 1) wait_for(&sm.bar[i], sm.parity[w] >> i & 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tm, 256);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// Rows of tokens x (heads * head_dim) values, in boxes of 64 tokens: of a head's values each token after the
// other to load, of 64 values swizzled to store.  Rows past the end read as zero.
bool value_map(CUtensorMap *m, const void *ptr, uint64_t cols, uint64_t rows, int head_dim, bool store) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
    cuuint32_t box[2] = {store ? 64u : (cuuint32_t)head_dim, C}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, store ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool chunked_eligible(const mamba_layer_desc *d) {
    return d->act_dtype == MAMBA_BF16 && d->state_dtype == MAMBA_BF16 && (d->head_dim == 64 || d->head_dim == 128) &&
           d->d_state == TN;
}

size_t chunked_workspace_bytes(const mamba_layer_desc *d, int T, int nseq) {
    const WsLayout ws(nullptr, d->nheads, d->n_groups);
    return (size_t)(scan_max_chunks(T, nseq) * ws.chunk_bytes());
}

int chunked_launch(const ScanParams &p, int head_dim, cudaStream_t st) {
    const WsLayout ws(p.ws, p.H, p.G);
    CUtensorMap vmap, ymap;
    if (!value_map(&vmap, p.v, (uint64_t)p.H * head_dim, (uint64_t)p.T, head_dim, false) ||
        !value_map(&ymap, p.y, (uint64_t)p.H * head_dim, (uint64_t)p.T, head_dim, true))
        return MAMBA_ECUDA;
    const bool pairs = p.HG % 2 == 0;  // heads of a group share its products, two a block
    auto prep = pairs ? k_gdn_prep<2> : k_gdn_prep<1>;
    auto chain = head_dim == 128 ? k_gdn_chain<128> : k_gdn_chain<64>;
    const size_t prep_smem = (pairs ? sizeof(PrepSmem<2>) : sizeof(PrepSmem<1>)) + 1024, chain_smem = sizeof(ChainSmem) + 1024;
    if (cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem) != cudaSuccess ||
        cudaFuncSetAttribute(chain, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chain_smem) != cudaSuccess)
        return MAMBA_ECUDA;
    const dim3 grid((unsigned)scan_max_chunks(p.T, p.nseq), (unsigned)(pairs ? p.H / 2 : p.H));
    if (launch_pdl(prep, grid, dim3(kPrepThreads), prep_smem, st, p, ws) != cudaSuccess) return MAMBA_ECUDA;
    if (launch_pdl(chain, dim3((unsigned)((int64_t)p.nseq * p.H)), dim3(kChainThreads), chain_smem, st, p, ws, vmap, ymap) !=
        cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}

}  // namespace gdn
}  // namespace ms
