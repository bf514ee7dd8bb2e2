// gdn_scan_tc.cu -- the chunked gated delta rule on the tcgen05 tensor cores.
//
// For a chunk of 64 tokens and a head with the state S (P x N) before it, with c_i the running sum
// of the log decays, unit keys and queries k_i, q_i of lengths |k_i|, |q_i| (after any scaling):
//   (I + L) U = diag(b) R,   L_ij = b_i |k_i||k_j| (k_i . k_j) e^(c_i - c_j), j < i
//   R = V - diag(e^c |k|) K S^T            the values, less what the decayed state already returns
//   U = T R,  T = (I + L)^-1 diag(b)       what is written
//   Y = |q| (diag(e^c) Q S^T + A U),       A_ij = |k_j| (q_i . k_j) e^(c_i - c_j), j <= i
//   S <- e^(c_64) S + (diag(e^(c_64 - c) |k|) U)^T K
// T and A need no state, so k_gdn_prep forms them for all chunks of the batch at once; the chain
// from chunk to chunk, k_gdn_chain, has four products left, all of them transposed so that the
// value index is the row: its left operands S, R^T, U^T are the accumulators of the product
// before, rounded to 16 bits, and never leave tensor memory; T, A, K, Q are tiles in shared
// memory in the form the products read them.
//
// Number formats: the products run on fp16 operands (11 bits; bf16's 8 would put four times the
// output's own rounding into y), sums in fp32, and the state itself stays in fp32 in registers.
// Keys and queries are of unit length before they are rounded.  Values have bf16's range, so every
// row of the state (one value index) has a power of two that brings its values and state to a few
// units, taken anew every 16 chunks and whenever a value outgrows it; the rule cannot grow the state
// past sqrt(tokens) times the largest value, far inside the 2^12 left.
#include <mutex>

#include <cuda_fp16.h>

#include "gdn_scan_tc.h"
#include "umma.cuh"

namespace ms {
namespace gdn {

using namespace umma;

namespace {

constexpr int C = kChunk, TN = 128, TP = 128;
constexpr uint32_t kPolls = umma::kWaitPolls;
constexpr float LOG2E = 1.4426950408889634f;

// Workspace of one chunk.  Per group the tiles of unit keys and queries, 64 rows x 128 fp16 in two
// 128-byte-swizzled blocks each, interleaved [K 0..63 | Q 0..63 | K 64..127 | Q 64..127] so that keys
// and queries stacked are one operand of 128 rows; per head T, A (64 x 64, swizzled) and the gates.
constexpr uint32_t kBlk = 64 * 128;          // one swizzled block of 64 rows
constexpr uint32_t kKqBytes = 4 * kBlk;
struct HeadGates {
    float rk[C];   // e^c |k|
    float ek[C];   // e^(c_64 - c) |k|
    float g[C];    // e^c
    float oq[C];   // |q| * scale
    float last, pad[3];  // e^(c_64)
};
constexpr uint32_t kGateBytes = sizeof(HeadGates);
constexpr uint32_t kHeadBytes = 2 * kBlk + kGateBytes;
static_assert(kGateBytes % 16 == 0, "bulk copy size");

struct WsLayout {
    unsigned char *base;
    int H, G;
    __host__ __device__ int64_t chunk_bytes() const { return (int64_t)G * kKqBytes + (int64_t)H * kHeadBytes; }
    __device__ unsigned char *kq(int chunk, int g) const { return base + chunk * chunk_bytes() + (int64_t)g * kKqBytes; }
    __device__ unsigned char *head(int chunk, int h) const {
        return base + chunk * chunk_bytes() + (int64_t)G * kKqBytes + (int64_t)h * kHeadBytes;
    }
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return idesc_bf16(M, N, false, b_mn_major) & ~((7u << 7) | (7u << 10));  // A and B format: fp16
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
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
constexpr float kSpan = 96.0f;  // largest base-2 exponent span of a block whose decays are factored

// T of one head on the way: L's diagonal 16 x 16 blocks in fp32 (two blocks start 16 banks apart), the
// rest of L and (I + L)^-1 in fp16, rows 144 bytes apart so that eight rows' 16 bytes miss one another's
// banks.
struct Inverse {
    float diag[4][16 * 20 + 16];
    __half L[C][72], t[C][72];
};
// Decays within a 32-token half of the chunk and from the first half to the second, as a factor of the
// row times one of the column (with the key's length); see decay_factors.
struct Decays {
    float cum[C], b[C], near[C], far[32];
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
    float nk[C];
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
    for (int k = 0; k < K; ++k) ldmatrix4(a[k], block16(v.t, row, mid + 16 * k, lane));
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
            ldmatrix4_trans(b, block16(v.t, left + 16 * k, left + 16 * n, lane));
            mma16(out[2 * n], xa, b[0], b[1]);
            mma16(out[2 * n + 1], xa, b[2], b[3]);
        }
    }
}

// T = (I + L)^-1 diag(b) of one head by a pair of warps (w = 0, 1 of the pair).  The diagonal blocks of
// 16 by forward substitution in fp32, a column a thread; the blocks below them by products.
__device__ __forceinline__ void invert(Inverse &v, unsigned char *T, const float *b, int w, int lane, int pair) {
    const int d = 2 * w + (lane >> 4), c = lane & 15;  // diagonal block and its column
    {
        float x[16];
        const float bc = b[16 * d + c];
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
            v.t[row][col] = __float2half_rn(x[r]);
            *reinterpret_cast<__half *>(T + swz128_offset(row, col)) = __float2half_rn(x[r] * bc);
        }
        // the block right of the first of the pair's two diagonal blocks
        *reinterpret_cast<uint4 *>(&v.t[32 * w + c][32 * w + 16 + (lane >> 4) * 8]) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    const int fr = lane >> 2, fc = (lane & 3) * 2;
    auto put = [&](int row, int col, float v0, float v1) {
        const float2 w2 = *reinterpret_cast<const float2 *>(b + col);
        *reinterpret_cast<uint32_t *>(T + swz128_offset(row, col)) = pack_f16x2(v0 * w2.x, v1 * w2.y);
    };
    {
        float o[2][4];
        const int left = 32 * w, mid = left + 16;
        lower_left<1>(v, mid, mid, left, o, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = mid + fr + 8 * e, col = left + 8 * n + fc;
                *reinterpret_cast<uint32_t *>(&v.t[row][col]) = pack_f16x2(o[n][2 * e], o[n][2 * e + 1]);
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

// Block (chunk, group and share of its heads).
template <int HEADS>
__global__ void __launch_bounds__(kPrepThreads, 2) k_gdn_prep(const ScanParams p, const WsLayout ws) {
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
            if (col == 0) sm.ss[row] = ss;
        }
    }
    // running sums of the log decays (base 2) over each head's two warps of tokens
    if (hh < HEADS) {
        if (tok < L) {
            run = log_decay(p.gates, run, h0 + hh) * LOG2E;
            b = write_gate(p.gates, b);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (tok == 31) sm.half_sum[hh] = run;
        sm.dec[hh].b[tok] = b;
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
        const float nk = sqrtf(kk) * unit_factor(p.gates, kk);
        HeadGates &gt = sm.gates[hh];
        gt.rk[tok] = e * nk;
        gt.ek[tok] = exp2f(last - run) * nk;
        gt.g[tok] = e;
        gt.oq[tok] = sqrtf(qq) * unit_factor(p.gates, qq) * p.gates.scale;
        if (tok == 0) gt.last = exp2f(last);
        dec.near[tok] = exp2f(fminf(dec.cum[tok & 32] - run, kSpan)) * nk;
        if (tok < 32) dec.far[tok] = exp2f(dec.cum[31] - run) * nk;
        if (hh == 0) sm.nk[tok] = nk;
    }
    const int bad = mbar_wait(&sm.bar, 0, kPolls) ? 0 : 1;
    tc_fence_after();
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            flag_error(p.err, MAMBA_ERR_TIMEOUT);
            mbar_wait(&sm.bar, 0, kPolls);
        }
    } else {
        const int q = warp & 3, hf = warp >> 2, i = (q & 1) * 32 + lane;  // row i of K K^T (q < 2) or Q K^T
        float dots[32];
        tmem_ld32(tm + ((uint32_t)(q * 32) << 16) + hf * 32, dots);
        // L (what T needs of it) and A of this thread's 32 columns
#pragma unroll 1
        for (int x = 0; x < HEADS; ++x) {
            const Decays &dec = sm.dec[x];
            const float ci = dec.cum[i], wi = q < 2 ? dec.b[i] * sm.nk[i] : 1.0f;
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
                        const float v = dots[j] * wi * sm.nk[hf * 32 + j] * exp2_approx(ci - dec.cum[hf * 32 + j]);
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
            invert(sm.inv[x], sm.out[x], sm.dec[x].b, warp & 1, lane, x);
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

constexpr int kChainThreads = 512;
constexpr int kRescale = 16;  // chunks between two choices of the rows' powers of two

// What the block waits for: keys with gates (two stages), queries, T, A, the values; the products X, U,
// Q S^T, the increment and Y.
enum { B_K = 0, B_Q = 2, B_T, B_A, B_V, B_X, B_U, B_OI, B_S, B_Y, kBars };

struct ChainSmem {
    // q: a chunk's queries, and once they are used its outputs on their way to memory; v: values, 64 of
    // them in a swizzled block of 64 tokens
    unsigned char k[2][2 * kBlk], q[2][2 * kBlk], T[kBlk], A[kBlk], v[2 * kBlk];
    HeadGates gates[4];
    float row_max[4][TP];
    uint64_t bar[kBars];
    uint32_t tmem;
};

// Tensor-memory columns: the state's 16-bit copy and X (or R^T over X) make way for the new state's
// increment, which is as wide as both.
constexpr uint32_t T_S = 0, T_X = 64, T_D = 0, T_U = 128, T_Y = 192;

// The accumulators' 32 lanes of a warp as matrix fragments: two loads of 16 lanes each, 8 NC fp32
// columns; element [half][4 n + 2 r + e] is lane 16 half + 8 r + T / 4, column 8 n + 2 (T % 4) + e.
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
// Their 16-bit counterpart: element [half][2 n + r] holds columns 8 n + 2 (T % 4) and the next.
__device__ __forceinline__ void tmem_put2(uint32_t a, const uint32_t (&v)[2][4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%2,%3,%4,%5};\n\t"
        "tcgen05.st.sync.aligned.16x128b.x2.b32 [%1], {%6,%7,%8,%9};\n\t" ::"r"(a),
        "r"(a + (16u << 16)), "r"(v[0][0]), "r"(v[0][1]), "r"(v[0][2]), "r"(v[0][3]), "r"(v[1][0]), "r"(v[1][1]),
        "r"(v[1][2]), "r"(v[1][3])
        : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}

// Keys and gates of chunk c of the sequence.
__device__ __forceinline__ void load_keys(ChainSmem &sm, const WsLayout &ws, int first, int c, int g, int h) {
    uint64_t *bar = &sm.bar[B_K + (c & 1)];
    mbar_arrive_expect_tx(bar, 2 * kBlk + kGateBytes);
    const unsigned char *kq = ws.kq(first + c, g);
    bulk_g2s(sm.k[c & 1], kq, kBlk, bar);
    bulk_g2s(sm.k[c & 1] + kBlk, kq + 2 * kBlk, kBlk, bar);
    bulk_g2s(&sm.gates[c & 3], ws.head(first + c, h) + 2 * kBlk, kGateBytes, bar);
}
__device__ __forceinline__ void load_queries(ChainSmem &sm, const WsLayout &ws, int first, int c, int g) {
    mbar_arrive_expect_tx(&sm.bar[B_Q], 2 * kBlk);
    const unsigned char *kq = ws.kq(first + c, g);
    bulk_g2s(sm.q[c & 1], kq + kBlk, kBlk, &sm.bar[B_Q]);
    bulk_g2s(sm.q[c & 1] + kBlk, kq + 3 * kBlk, kBlk, &sm.bar[B_Q]);
}
__device__ __forceinline__ void load_tile(void *dst, const unsigned char *src, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, kBlk);
    bulk_g2s(dst, src, kBlk, bar);
}
__device__ __forceinline__ void load_values(ChainSmem &sm, const CUtensorMap *map, int h, int t) {
    mbar_arrive_expect_tx(&sm.bar[B_V], 2 * kBlk);
    tma_load_2d(sm.v, map, h * TP, t, &sm.bar[B_V]);
    tma_load_2d(sm.v + kBlk, map, h * TP + 64, t, &sm.bar[B_V]);
}

// Block (sequence in the plan's order, head) of 16 warps.  Warp w works on tensor-memory lanes
// 32 (w % 4) .. + 31, the value indices, and on quarter w / 4 of the columns: 16 tokens, or 32 of the
// state's.  A thread holds its rows 8 i + T / 4 and columns 8 n + 2 (T % 4) + {0, 1} as fragments, which
// is how ldmatrix and stmatrix turn values and outputs between (token, value) and (value, token).
__global__ void __launch_bounds__(kChainThreads, 2) k_gdn_chain(const ScanParams p, const WsLayout ws,
                                                                const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char chain_smem[];
    ChainSmem &sm = *align1024<ChainSmem>(chain_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    if (p.meta[0] == 0) return;  // bad cu_seqlens (flagged): nothing is done
    const int s = meta_order(p)[blockIdx.x / p.H], h = blockIdx.x % p.H, g = h / p.HG;
    const int t0 = p.cu[s], len = p.cu[s + 1] - t0, first = meta_chunks(p)[s];
    const int32_t slot = p.slot[s];
    if (len <= 0 || slot < -1 || slot >= p.num_slots) return;  // empty, or bad slot (flagged)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = warp & 3, Q = warp >> 2;
    const int fr = lane >> 2, fc = (lane & 3) * 2;
    const int nc = (len + C - 1) / C;
    bf16 *pool = static_cast<bf16 *>(p.pool);
    const int64_t off = ((int64_t)h * TP + 32 * q + fr) * TN + 32 * Q + fc;  // of this thread's first state element

    if (warp == 0 && elect_one()) {
        for (int i = 0; i < kBars; ++i) mbar_init(&sm.bar[i], 1);
        fence_mbar_init();
        tma_prefetch_desc(&vmap);
        load_keys(sm, ws, first, 0, g, h);
        load_values(sm, &vmap, h, t0);
        load_queries(sm, ws, first, 0, g);
        load_tile(sm.T, ws.head(first, h), &sm.bar[B_T]);
        load_tile(sm.A, ws.head(first, h) + kBlk, &sm.bar[B_A]);
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem, 256);
        tmem_relinquish();
    }
    // this thread's part of the state, each row times its power of two: S[i / 2][4 n + 2 (i % 2) + e]
    float S[2][16];
    if (slot >= 0 && p.has_init && p.has_init[s]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(pool + slot * p.stride + off + i * 8 * TN + 8 * n);
                S[i >> 1][4 * n + 2 * (i & 1)] = __uint_as_float(w << 16);
                S[i >> 1][4 * n + 2 * (i & 1) + 1] = __uint_as_float(w & 0xffff0000u);
            }
    } else {
#pragma unroll
        for (int n = 0; n < 32; ++n) S[n >> 4][n & 15] = 0.0f;
    }
    // row i's power of two, 2^(128 - E_i), by the byte E_i: its inverse 2^(E_i - 128)
    uint32_t powers = 0x80808080u;
    auto scale_of = [&](int i) { return __uint_as_float((255u - (powers >> (8 * i) & 0xffu)) << 23); };
    auto unscale_of = [&](int i) { return __uint_as_float(((powers >> (8 * i) & 0xffu) - 1u) << 23); };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem, lanes = tm + ((uint32_t)(q * 32) << 16);
    bool failed = false;
    uint32_t x_phase = 0;
    uint32_t armed = 0, parity = 0;  // of the issuing thread: the barriers with something in flight, ever, and its phase
    auto arm = [&](int i, uint32_t phase) {
        armed |= 1u << i;
        parity = (parity & ~(1u << i)) | phase << i;
    };
    arm(B_K, 0), arm(B_Q, 0), arm(B_T, 0), arm(B_A, 0), arm(B_V, 0);

    auto store_state16 = [&] {  // the state's copy for the products; the lanes' increment is consumed
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t pk[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                pk[i >> 2][i & 3] = pack_f16x2(S[i >> 2][8 * n + 2 * (i & 3)], S[i >> 2][8 * n + 2 * (i & 3) + 1]);
            tmem_put2(lanes + T_S + Q * 16 + n * 8, pk);
        }
        tmem_put_wait();
    };
    auto issue_x = [&](int c) {  // X = S K^T
        const uint32_t k = smem_u32(sm.k[c & 1]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tm + T_X, tm + T_S + 8 * kk, desc_kmajor(k, kBlk, kk), idesc_f16(128, C, false), kk > 0);
        mma_commit(&sm.bar[B_X]);
        arm(B_X, x_phase);
    };
    // this lane's row of 16 bytes (8 values of a token) in a swizzled tile of tokens, for the fragments of
    // 8 tokens from 16 Q + 8 n and this warp's 32 values
    auto value_row = [&](const unsigned char *tile, int n) {
        return smem_u32(tile) + (q >> 1) * kBlk + swz128_chunk(16 * Q + 8 * n + (lane & 7), 4 * (q & 1) + (lane >> 3));
    };
    // outputs of chunk c into its queries' place
    auto stage_outputs = [&](int c) {
        float y[2][8];
        tmem_frag2(lanes + T_Y + Q * 16, y);
        const float *oq = sm.gates[c & 3].oq + 16 * Q + fc;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 w = *reinterpret_cast<const float2 *>(oq + 8 * n);
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = unscale_of(i);
                const __nv_bfloat162 v = __floats2bfloat162_rn(y[i >> 1][4 * n + 2 * (i & 1)] * (w.x * u),
                                                               y[i >> 1][4 * n + 2 * (i & 1) + 1] * (w.y * u));
                pk[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
            stmatrix4_trans(value_row(sm.q[c & 1], n), pk[0], pk[1], pk[2], pk[3]);
        }
    };
    auto write_outputs = [&](int c) {  // from there to memory, 16 bytes a thread
        const int L = min(C, len - c * C);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = (tid >> 4) + 32 * i, ch = tid & 15;
            if (t < L)
                *reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.y) + ((int64_t)(t0 + c * C + t) * p.H + h) * TP + ch * 8) =
                    *reinterpret_cast<const uint4 *>(sm.q[c & 1] + (ch >> 3) * kBlk + swz128_chunk(t, ch & 7));
        }
    };
    auto write_state = [&](int32_t to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = unscale_of(i);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(S[i >> 1][4 * n + 2 * (i & 1)] * u,
                                                               S[i >> 1][4 * n + 2 * (i & 1) + 1] * u);
                *reinterpret_cast<__nv_bfloat162 *>(pool + to * p.stride + off + i * 8 * TN + 8 * n) = v;
            }
        }
    };

    for (int c = 0; c < nc; ++c) {
        const uint32_t ph = c & 1;
        const int L = min(C, len - c * C);
        int bad = 0;
        const bool fresh = c % kRescale == 0;  // this chunk starts from new powers of two
        const HeadGates &gt = sm.gates[c & 3];
        // 1. X = S K^T, while the last chunk's outputs leave tensor memory
        if (!mbar_wait(&sm.bar[B_K + ph], (c >> 1) & 1, kPolls)) bad = 1;
        if (warp == 0 && elect_one() && !bad) {
            tc_fence_after();
            if (!fresh) issue_x(c);
            if (c + 1 < nc) {
                load_keys(sm, ws, first, c + 1, g, h);
                arm(B_K + (ph ^ 1), ((c + 1) >> 1) & 1);
            }
        }
        if (c > 0) {
            if (!mbar_wait(&sm.bar[B_Y], ph ^ 1, kPolls)) bad = 1;
            tc_fence_after();
            if (warp == 0 && elect_one() && !bad) {
                load_tile(sm.A, ws.head(first + c, h) + kBlk, &sm.bar[B_A]);
                arm(B_A, ph);
            }
            stage_outputs(c - 1);
        }
        // 2. queries times e^c in place; this thread's values
        if (!mbar_wait(&sm.bar[B_Q], ph, kPolls)) bad = 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cidx = tid + kChainThreads * i;  // 16-byte chunk of the tile: row of 128 bytes = token
            uint4 *ptr = reinterpret_cast<uint4 *>(sm.q[ph] + cidx * 16);
            const __half2 w = __float2half2_rn(gt.g[(cidx >> 3) & (C - 1)]);
            uint4 u = *ptr;
            __half2 *hp = reinterpret_cast<__half2 *>(&u);
#pragma unroll
            for (int e = 0; e < 4; ++e) hp[e] = __hmul2(hp[e], w);
            *ptr = u;
        }
        fence_async_smem();
        if (!mbar_wait(&sm.bar[B_V], ph, kPolls)) bad = 1;
        uint32_t vals[2][4];  // [n][i]: two tokens of row i
#pragma unroll
        for (int n = 0; n < 2; ++n) ldmatrix4_trans(vals[n], value_row(sm.v, n));
        if (L < C) {  // rows past the sequence's end hold another sequence's values
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int t = 16 * Q + 8 * n + fc;
#pragma unroll
                for (int i = 0; i < 4; ++i) vals[n][i] = t + 1 < L ? vals[n][i] : (t < L ? vals[n][i] & 0xffffu : 0u);
            }
        }
        uint32_t vmax[4], over = 0;  // largest magnitudes as bf16 bits; whether one outgrew 2^4 units of its row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            vmax[i] = __vmaxu2(vals[0][i] & 0x7fff7fffu, vals[1][i] & 0x7fff7fffu);
            const uint32_t lim = ((powers >> (8 * i) & 0xffu) + 3u) << 7;
            over |= __vcmpgtu2(vmax[i], lim | lim << 16);
        }
        // (a wait that gave up goes the same way and ends the block below)
        if (__syncthreads_or(bad || over) || fresh) {
            if (!fresh) {  // X of the old powers is not used
                if (!mbar_wait(&sm.bar[B_X], x_phase, kPolls)) bad = 1;
                x_phase ^= 1;
            }
            // the largest magnitude in each row of the state (unscaled) and of the values
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = __uint_as_float(max(vmax[i] & 0xffffu, vmax[i] >> 16) << 16);
                const float u = unscale_of(i);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    top = fmaxf(top, u * fmaxf(fabsf(S[i >> 1][4 * n + 2 * (i & 1)]), fabsf(S[i >> 1][4 * n + 2 * (i & 1) + 1])));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (fc == 0) sm.row_max[Q][32 * q + 8 * i + fr] = top;
            }
            __syncthreads();
            uint32_t next = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 32 * q + 8 * i + fr;
                const float top = fmaxf(fmaxf(sm.row_max[0][row], sm.row_max[1][row]), fmaxf(sm.row_max[2][row], sm.row_max[3][row]));
                // the power that brings the largest to [2, 4); values may grow to 16 before the next choice
                int E = (int)(__float_as_uint(top) >> 23);
                E = top < INFINITY ? max(7, min(247, E)) : 127;
                next |= (uint32_t)E << (8 * i);
                const float ratio = __uint_as_float((255u - E) << 23) * unscale_of(i);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    S[i >> 1][4 * n + 2 * (i & 1)] *= ratio;
                    S[i >> 1][4 * n + 2 * (i & 1) + 1] *= ratio;
                }
            }
            powers = next;
            store_state16();
            tc_fence_before();
            if (__syncthreads_or(bad)) {
                failed = true;
                break;
            }
            tc_fence_after();
            if (warp == 0 && elect_one()) issue_x(c);
        }
        // 3. R = V - e^c |k| X, rounded, over X; then U^T = R^T T^T and the state's part of Y
        if (!mbar_wait(&sm.bar[B_X], x_phase, kPolls)) bad = 1;
        x_phase ^= 1;
        tc_fence_after();
        {
            float x[2][8];
            tmem_frag2(lanes + T_X + Q * 16, x);
            uint32_t pk[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 w = *reinterpret_cast<const float2 *>(gt.rk + 16 * Q + 8 * n + fc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // (past the end the values, the keys and so X are zero)
                    const float sc = scale_of(i);
                    const float *xi = &x[i >> 1][4 * n + 2 * (i & 1)];
                    pk[i >> 1][2 * n + (i & 1)] = pack_f16x2(fmaf(-w.x, xi[0], __uint_as_float(vals[n][i] << 16) * sc),
                                                             fmaf(-w.y, xi[1], __uint_as_float(vals[n][i] & 0xffff0000u) * sc));
                }
            }
            tmem_put2(lanes + T_X + Q * 16, pk);
            tmem_put_wait();
        }
        if (!mbar_wait(&sm.bar[B_T], ph, kPolls)) bad = 1;
        tc_fence_before();
        if (__syncthreads_or(bad)) {
            failed = true;
            break;
        }
        tc_fence_after();
        if (warp == 0 && elect_one()) {
            const uint32_t T = smem_u32(sm.T), qq = smem_u32(sm.q[ph]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ts(tm + T_U, tm + T_X + kk * 16, desc_kmajor(T, kBlk, kk), idesc_f16(128, C, false), kk > 0);
            mma_commit(&sm.bar[B_U]);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ts(tm + T_Y, tm + T_S + 8 * kk, desc_kmajor(qq, kBlk, kk), idesc_f16(128, C, false), kk > 0);
            mma_commit(&sm.bar[B_OI]);
            arm(B_U, ph), arm(B_OI, ph);
            if (c + 1 < nc) {
                load_values(sm, &vmap, h, t0 + (c + 1) * C);
                arm(B_V, ph ^ 1);
            }
        }
        if (c > 0) write_outputs(c - 1);
        // 4. U^T rounded, as it is and times e^(c_64 - c) |k|; then the state's increment and A's part of Y
        if (!mbar_wait(&sm.bar[B_U], ph, kPolls)) bad = 1;
        tc_fence_after();
        {
            float u[2][8];
            tmem_frag2(lanes + T_U + Q * 16, u);
            uint32_t pk[2][4], pe[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 w = *reinterpret_cast<const float2 *>(gt.ek + 16 * Q + 8 * n + fc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *ui = &u[i >> 1][4 * n + 2 * (i & 1)];
                    pk[i >> 1][2 * n + (i & 1)] = pack_f16x2(ui[0], ui[1]);
                    pe[i >> 1][2 * n + (i & 1)] = pack_f16x2(ui[0] * w.x, ui[1] * w.y);
                }
            }
            tmem_put2(lanes + T_U + Q * 16, pk);
            tmem_put2(lanes + T_U + Q * 16 + 8, pe);
            tmem_put_wait();
        }
        if (!mbar_wait(&sm.bar[B_OI], ph, kPolls)) bad = 1;  // the state's copy is read: its columns are free
        if (!mbar_wait(&sm.bar[B_A], ph, kPolls)) bad = 1;
        tc_fence_before();
        if (__syncthreads_or(bad)) {
            failed = true;
            break;
        }
        tc_fence_after();
        if (warp == 0 && elect_one()) {
            const uint32_t A = smem_u32(sm.A), k = smem_u32(sm.k[ph]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ts(tm + T_D, tm + T_U + kk * 16 + 8, desc_mnmajor(k, kBlk, kk), idesc_f16(128, TN, true), kk > 0);
            mma_commit(&sm.bar[B_S]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ts(tm + T_Y, tm + T_U + kk * 16, desc_kmajor(A, kBlk, kk), idesc_f16(128, C, false), 1);
            mma_commit(&sm.bar[B_Y]);
            arm(B_S, ph), arm(B_Y, ph);
            if (c + 1 < nc) {
                load_queries(sm, ws, first, c + 1, g);
                load_tile(sm.T, ws.head(first + c + 1, h), &sm.bar[B_T]);
                arm(B_Q, ph ^ 1), arm(B_T, ph ^ 1);
            }
        }
        // 5. the new state, and its copy
        if (!mbar_wait(&sm.bar[B_S], ph, kPolls)) bad = 1;
        tc_fence_after();
        const float last = gt.last;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float d[2][8];
            tmem_frag2(lanes + T_D + Q * 32 + n * 16, d);
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i >> 3][8 * n + (i & 7)] = fmaf(last, S[i >> 3][8 * n + (i & 7)], d[i >> 3][i & 7]);
        }
        const int32_t cs = ckpt_slot(p, s, c * C + L, tid == 0 && h == 0);
        if (cs >= 0) write_state(cs);
        if (c + 1 < nc && (c + 1) % kRescale != 0) {
            tc_fence_before();
            asm volatile("bar.sync %0, 128;" ::"r"(q + 1) : "memory");  // these lanes' increment has been read
            tc_fence_after();
            store_state16();
        }
        tc_fence_before();
        if (__syncthreads_or(bad)) {
            failed = true;
            break;
        }
        tc_fence_after();
    }
    if (!failed) {
        if (slot >= 0) write_state(slot);
        failed = !mbar_wait(&sm.bar[B_Y], (nc - 1) & 1, kPolls);
        tc_fence_after();
        stage_outputs(nc - 1);
    }
    if (__syncthreads_or(failed)) {
        // an operation did not complete in time: report it, and give what this block still has in flight
        // the same bounded time to finish before its memory is released
        if (warp == 0 && elect_one()) {
            flag_error(p.err, MAMBA_ERR_TIMEOUT);
            for (int i = 0; i < kBars; ++i)
                if (armed >> i & 1) mbar_wait(&sm.bar[i], parity >> i & 1, kPolls);
        }
    } else {
        write_outputs(nc - 1);
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

// Rows of tokens x (heads * 128) values, in swizzled boxes of 64 tokens x 64 values; rows past the end
// read as zero.
bool value_map(CUtensorMap *m, const void *ptr, uint64_t cols, uint64_t rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * 2};
    cuuint32_t box[2] = {64, C}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool chunked_eligible(const mamba_layer_desc *d) {
    return d->act_dtype == MAMBA_BF16 && d->state_dtype == MAMBA_BF16 && d->head_dim == TP && d->d_state == TN;
}

size_t chunked_workspace_bytes(const mamba_layer_desc *d, int T, int nseq) {
    const WsLayout ws = {nullptr, d->nheads, d->n_groups};
    return (size_t)(scan_max_chunks(T, nseq) * ws.chunk_bytes());
}

int chunked_launch(const ScanParams &p, cudaStream_t st) {
    const WsLayout ws = {p.ws, p.H, p.G};
    CUtensorMap vmap;
    if (!value_map(&vmap, p.v, (uint64_t)p.H * TP, (uint64_t)p.T)) return MAMBA_ECUDA;
    const bool pairs = p.HG % 2 == 0;  // heads of a group share its products, two a block
    auto prep = pairs ? k_gdn_prep<2> : k_gdn_prep<1>;
    const size_t prep_smem = (pairs ? sizeof(PrepSmem<2>) : sizeof(PrepSmem<1>)) + 1024, chain = sizeof(ChainSmem) + 1024;
    if (cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem) != cudaSuccess ||
        cudaFuncSetAttribute(k_gdn_chain, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chain) != cudaSuccess)
        return MAMBA_ECUDA;
    const dim3 grid((unsigned)scan_max_chunks(p.T, p.nseq), (unsigned)(pairs ? p.H / 2 : p.H));
    if (launch_pdl(prep, grid, dim3(kPrepThreads), prep_smem, st, p, ws) != cudaSuccess) return MAMBA_ECUDA;
    if (launch_pdl(k_gdn_chain, dim3((unsigned)((int64_t)p.nseq * p.H)), dim3(kChainThreads), chain, st, p, ws, vmap) != cudaSuccess)
        return MAMBA_ECUDA;
    return launch_status();
}

}  // namespace gdn
}  // namespace ms
