// la_scan_tc.cu -- the chunked form of linear attention on the tcgen05 tensor cores.
//
// For a chunk of L <= 128 tokens i = 0..L-1 and a head with the decay d = e^log_decay and the state S (P x N)
// before it:
//   A = (Q K^T) . D,  D_ij = d^(i-j) for j <= i, else 0
//   Y = A V + diag(d^(i+1)) Q S^T
//   S <- d^L S + V^T K',  K'_j = d^(L-1-j) k_j
// Four products of 128 x 128 x 128, none of which waits for another one's result but A V for A, and Q S^T for
// the state before: only the state's own update, elementwise, follows from chunk to chunk.  Everything else of the next
// chunk is under way meanwhile, in warps of its own: loads, products, A's decays, the keys' decays, the state, and the outputs.
// The state stands in registers in fp32, a key index a thread, and takes each chunk's product with one rounding to nearest: the
// tensor cores' own sums cut bits off, in one direction, and would add up over the chunks.  Its copy for the queries, and A, are rounded to bf16, the type of the V, K and Q that they meet: an output is off by about
// as much as its own rounding to bf16 takes.  K', whose rounding would stay in the state, is held as the sum of two bf16 numbers
// (16 bits) under a bf16 pool and of three (24) under an fp32 pool, in as many products.
//
// A sequence's state is linear in what came before, so a long sequence of few heads is cut into segments that are
// worked on side by side: k_la_segment forms what each but the last adds to the state, and a segment's block
// starts from the decayed sum of those before it.
#include "la_scan.h"
#include "tensor_map.h"
#include "umma.cuh"

namespace ms {
namespace la {

using namespace umma;

namespace {

constexpr int C = kChunk;
constexpr int kWhole = 1 << 30;               // tokens of a segment where sequences are not cut
constexpr uint32_t kPolls = umma::kWaitPolls;
constexpr float LOG2E = 1.4426950408889634f;
constexpr uint32_t kBlk = 128 * 128;          // bytes of a swizzled block: 128 tokens, 64 values each
constexpr uint32_t kTile = 2 * kBlk;          // of a tile of 128 tokens x 128 (or 64, in its first block)

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// d^m from log2(d) <= 0, also where that is minus infinity.
__device__ __forceinline__ float power(float l2, int m) { return m == 0 ? 1.0f : exp2f(l2 * (float)m); }

// Waits with one outcome for the whole warp, which takes part in collective instructions afterwards; gives up
// after the poll limit, or once another warp has.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *failed) {
    bool ok = false;
#pragma unroll 1
    for (uint32_t i = 0; i < kPolls; ++i) {
        if (mbar_try_wait(bar, parity)) {
            ok = true;
            break;
        }
        if (*failed) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *failed = 1;
    return ok;
}
// The same bounded wait for what is still in flight after a failure.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < kPolls; ++i)
        if (mbar_try_wait(bar, parity)) return;
}

template <int REGS>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <typename T>
__device__ __forceinline__ T *align1024(unsigned char *p) {
    return reinterpret_cast<T *>(p + (-smem_u32(p) & 1023u));  // (an offset, so that accesses stay shared-memory ones)
}

// What a block works on.
struct Job {
    int seq, index, last, t0, len, nc, entry;  // entry: of the sequence's first in the workspace, if it has several segments
    int32_t slot;
    bool ok;
};
__device__ __forceinline__ Job find_job(const ScanParams &p, int b) {
    Job j;
    j.ok = b < p.meta[0];
    if (!j.ok) return j;
    const Segment g = meta_segments(p)[b];
    const int a = p.cu[g.seq], len = p.cu[g.seq + 1] - a;
    j.seq = g.seq, j.index = g.index, j.slot = p.slot[g.seq];
    j.last = (len - 1) / p.seg_tokens;
    j.t0 = a + g.index * p.seg_tokens;
    j.len = min(p.seg_tokens, len - g.index * p.seg_tokens);
    j.nc = (j.len + C - 1) / C;
    j.entry = g.first + g.seq;
    j.ok = j.slot >= -1 && j.slot < p.num_slots;  // (else flagged by the plan)
    return j;
}
// Entries of the workspace: of each sequence, its initial state and what each segment but the last adds; a head's
// state each, transposed like tensor memory's lanes: value p of key n at p * 128 + n.
__device__ __forceinline__ float *entry_at(const ScanParams &p, int e, int h, int P) {
    return p.ws + ((int64_t)e * p.H + h) * (128 * P);
}

// A row of 64 * BLOCKS bf16 values of a swizzled tile, times f, as a sum of 1 + MORE bf16 numbers: the first back in
// place, the others into the tiles at rest.
template <int BLOCKS, int MORE>
__device__ __forceinline__ void scale_row(unsigned char *tile, unsigned char *rest, int row, float f) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t at = b * kBlk + swz128_chunk(row, c);
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + at);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[1 + MORE][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = __uint_as_float(in[e] << 16) * f, y = __uint_as_float(in[e] & 0xffff0000u) * f;
#pragma unroll
                for (int m = 0; m < MORE; ++m) {  // (cut off, not rounded: what is left is exact, and goes to the next)
                    out[m][e] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
                    x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
                    y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
                }
                out[MORE][e] = MORE == 2 ? __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632) : pack2(x, y);  // (8 bits are left)
            }
            *reinterpret_cast<uint4 *>(tile + at) = make_uint4(out[0][0], out[0][1], out[0][2], out[0][3]);
#pragma unroll
            for (int m = 0; m < MORE; ++m)
                *reinterpret_cast<uint4 *>(rest + m * kTile + at) = make_uint4(out[m + 1][0], out[m + 1][1], out[m + 1][2], out[m + 1][3]);
        }
}
template <int BLOCKS>
__device__ __forceinline__ void clear_row(unsigned char *tile, int row) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(tile + b * kBlk + swz128_chunk(row, c)) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------------------
// the chain: a segment of a sequence, one head
// ---------------------------------------------------------------------------------------

// Each barrier's phase c is chunk c's (of a stage: the c-th use of the stage).
enum {
    B_QF = 0, B_KF = 2, B_VF = 4,   // loaded, by stage
    B_QE = 6, B_KE = 8, B_VE = 10,  // the products have read it
    B_P = 12,  // Q K^T is there
    B_A,       // A is in tensor memory
    B_K2,      // K' is in place of K
    B_Y,       // A V and Q S^T are there
    B_YE,      // ... and read
    B_S,       // V^T K' is there
    B_SB,      // ... and added, and the state's copy is written (phase 0: before the first chunk)
    B_END,     // every product has finished
    kBars
};
// Groups of 4 warps: for A, for outputs, for the state, for the keys' decays, and one of which a warp loads and another issues the
// products.  The state's group takes registers from the others, within what the launch gave the block: 5 warps a scheduler
// leave 96 a thread (launch() checks that the compiler made it so).
constexpr int kThreads = 5 * 128, kRegs = 96, kStateRegs = 176, kOtherRegs = 88, kIssueRegs = 40;
static_assert(kStateRegs + 3 * kOtherRegs + kIssueRegs <= 5 * kRegs, "registers of the launch");

template <int P, bool F32S>
struct ChainSmem {
    // Parts of K' past the first, and stages of queries and values: what the parts leave room for.  Keys are needed first and
    // read last, so that they always have two.
    static constexpr int MORE = F32S ? 2 : 1, NQ = P == 64 && !F32S ? 2 : 1, NV = P == 128 && F32S ? 1 : 2;
    unsigned char q[NQ][kTile], k[2][kTile], v[NV][P * 256], sb[P * 256], rest[MORE][kTile];
    float diag[32], col[32];  // d^m; d^(31-m)
    uint64_t bar[kBars];
    uint32_t tmem;
    int failed;
};

constexpr uint32_t T_P = 0, T_Y = 128, T_Y2 = 256, T_D = 384;  // tensor memory columns; A takes the first half of Q K^T's

template <int P, int N, bool F32S>
__global__ void __launch_bounds__(kThreads, 1) k_la_chain(const ScanParams p, const __grid_constant__ CUtensorMap qmap,
                                                          const __grid_constant__ CUtensorMap kmap,
                                                          const __grid_constant__ CUtensorMap vmap) {
    using Smem = ChainSmem<P, F32S>;
    using StateT = typename std::conditional<F32S, float, bf16>::type;
    constexpr int NQ = Smem::NQ, NV = Smem::NV, MORE = Smem::MORE, NB = N / 64, PB = P / 64;
    extern __shared__ __align__(1024) unsigned char chain_smem[];
    Smem &sm = *align1024<Smem>(chain_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int h = blockIdx.x % p.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Job job = find_job(p, blockIdx.x / p.H);
    if (!job.ok) return;
    const float l2 = p.log_decay[h] * LOG2E;
    if (tid < 32) sm.diag[tid] = power(l2, tid);
    else if (tid < 64) sm.col[tid - 32] = power(l2, 63 - tid);
    if (N == 64)  // the keys' lanes without keys: products read them
        for (int i = tid; i < (int)kBlk / 16; i += kThreads) {
#pragma unroll
            for (int s = 0; s < 2; ++s) reinterpret_cast<uint4 *>(sm.k[s] + kBlk)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < MORE; ++m) reinterpret_cast<uint4 *>(sm.rest[m] + kBlk)[i] = make_uint4(0, 0, 0, 0);
        }
    if (warp == 16 && elect_one()) {
        for (int i = 0; i < kBars; ++i) mbar_init(&sm.bar[i], i == B_A || i == B_K2 || i == B_YE || i == B_SB ? 4 : 1);
        fence_mbar_init();
        sm.failed = 0;
    }
    if (warp == 17) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    volatile int *failed = &sm.failed;
    const int nc = job.nc;
    auto wait = [&](int b, uint32_t use) { return warp_wait(&sm.bar[b], use & 1, failed); };
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int row = tid & 127;
    int loaded = 0;

    if (warp < 4) {
        fewer_registers<kOtherRegs>();
        // A: row i a thread, in pieces of 32 columns j.  Left of the diagonal's piece d^(i-j) is
        // d^(i-j0-31) * d^(31-(j-j0)), neither of which can overflow.
        float rf[3];
#pragma unroll
        for (int b = 0; b < 3; ++b) rf[b] = row >= 32 * b + 32 ? power(l2, row - 32 * b - 31) : 0.0f;
        for (int c = 0; c < nc; ++c) {
            if (!wait(B_P, c)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t pk[16];
                if (b < warp) {
                    float x[32];
                    tmem_ld32(lanes + T_P + 32 * b, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&sm.col[e]);
                        pk[e / 2] = pack2(x[e] * (f.x * rf[b < 3 ? b : 0]), x[e + 1] * (f.y * rf[b < 3 ? b : 0]));
                        pk[e / 2 + 1] = pack2(x[e + 2] * (f.z * rf[b < 3 ? b : 0]), x[e + 3] * (f.w * rf[b < 3 ? b : 0]));
                    }
                } else if (b == warp) {
                    float x[32];
                    tmem_ld32(lanes + T_P + 32 * b, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        pk[e / 2] = pack2(e <= lane ? x[e] * sm.diag[max(lane - e, 0)] : 0.0f,
                                          e + 1 <= lane ? x[e + 1] * sm.diag[max(lane - e - 1, 0)] : 0.0f);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0u;
                }
                tmem_st16(lanes + T_P + 16 * b, pk);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[B_A]);
        }
    } else if (warp < 8) {
        fewer_registers<kOtherRegs>();
        // the outputs: row i a thread
        const float f2 = p.scale * power(l2, row + 1);
        bf16 *y = static_cast<bf16 *>(p.y) + ((int64_t)(job.t0 + row) * p.H + h) * P;
        for (int c = 0; c < nc; ++c, y += (int64_t)C * p.H * P) {
            if (!wait(B_Y, c)) break;
            tc_fence_after();
            const bool live = c * C + row < job.len;
#pragma unroll
            for (int b = 0; b < P / 32; ++b) {
                float a[32], s[32];
                tmem_ld32(lanes + T_Y + 32 * b, a);
                tmem_ld32(lanes + T_Y2 + 32 * b, s);
                if (b == P / 32 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(&sm.bar[B_YE]);
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = fmaf(f2, s[e + i], p.scale * a[e + i]);
                        *reinterpret_cast<uint4 *>(y + 32 * b + e) = pack16(o);
                    }
                }
            }
        }
    } else if (warp < 12) {
        // the state: key index n a thread (with N 64 the upper half hold zeros)
        more_registers<kStateRegs>();
        const int n = row;
        StateT *pool = static_cast<StateT *>(p.pool) + (int64_t)h * P * N + n;
        const bool seeded = n < N && job.slot >= 0 && p.has_init && p.has_init[job.seq];
        float S[P];
        {
            const float *from = entry_at(p, job.entry, h, P) + n;
            if (!seeded) {
#pragma unroll
                for (int e = 0; e < P; ++e) S[e] = 0.0f;
            } else if (job.last) {  // several segments: from the copy, since the last one's block writes the slot
#pragma unroll
                for (int e = 0; e < P; ++e) S[e] = from[e * 128];
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e) S[e] = to_f32(pool[job.slot * p.stride + e * N]);
            }
            if (n < N && job.index) {
                const float over = power(l2, p.seg_tokens);
#pragma unroll 1
                for (int r = 1; r <= job.index; ++r) {
                    from += (int64_t)p.H * (128 * P);
#pragma unroll
                    for (int e = 0; e < P; ++e) S[e] = fmaf(over, S[e], from[e * 128]);
                }
            }
        }
        const float whole = power(l2, C), part = power(l2, job.len - (nc - 1) * C);  // over a chunk, and the last one
        for (int c = -1; c < nc; ++c) {  // (from -1: only the copy for the first chunk)
            if (c >= 0) {
                if (!wait(B_S, c)) break;
                tc_fence_after();
                const float over = c + 1 == nc ? part : whole;
#pragma unroll
                for (int b = 0; b < P / 32; ++b) {
                    float d[32];
                    tmem_ld32(lanes + T_D + 32 * b, d);
#pragma unroll
                    for (int e = 0; e < 32; ++e) S[32 * b + e] = fmaf(over, S[32 * b + e], d[e]);
                }
            }
            if (c + 1 < nc) {
                if (n < N) {
#pragma unroll
                    for (int e = 0; e < P; e += 8) {
                        const float f[8] = {S[e], S[e + 1], S[e + 2], S[e + 3], S[e + 4], S[e + 5], S[e + 6], S[e + 7]};
                        *reinterpret_cast<uint4 *>(sm.sb + (e >> 6) * (N * 128) + swz128_chunk(n, (e >> 3) & 7)) = pack16(f);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sm.bar[B_SB]);
            }
            if (c >= 0) {
                const bool end = c + 1 == nc && job.index == job.last;
                const int32_t ckpt = ckpt_slot(p, job.seq, job.index * p.seg_tokens + min(job.len, (c + 1) * C), row == 0 && h == 0);
                auto write = [&](int32_t slot) {
                    if (slot < 0 || n >= N) return;
                    StateT *to = pool + slot * p.stride;
#pragma unroll
                    for (int e = 0; e < P; ++e) to[e * N] = from_f32<StateT>(S[e]);
                };
                if (ckpt >= 0) write(ckpt);
                if (end) write(job.slot);
            }
        }
    } else if (warp < 16) {
        fewer_registers<kOtherRegs>();
        // K' in place of K, token j a thread; past the segment's end zeros, in V as well: the tiles hold another's tokens there
        const float f = power(l2, C - 1 - row);
        for (int c = 0; c < nc; ++c) {
            if (!wait(B_P, c)) break;  // the scores have read K
            const int L = min(C, job.len - c * C);
            if (L == C) {
                scale_row<NB, MORE>(sm.k[c & 1], sm.rest[0], row, f);
            } else {
                if (!wait(B_VF + c % NV, c / NV)) break;
                if (row < L) {
                    scale_row<NB, MORE>(sm.k[c & 1], sm.rest[0], row, power(l2, L - 1 - row));
                } else {
                    clear_row<NB>(sm.k[c & 1], row);
#pragma unroll
                    for (int m = 0; m < MORE; ++m) clear_row<NB>(sm.rest[m], row);
                    clear_row<PB>(sm.v[c % NV], row);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[B_K2]);
        }
    } else if (warp == 16) {
        fewer_registers<kIssueRegs>();
        const int g = h / p.HG;
        int c = 0;
        for (; c < nc; ++c) {
            const int st = c & 1, use = c >> 1, qs = c % NQ, quse = c / NQ, vs = c % NV, vuse = c / NV, t = job.t0 + c * C;
            if (use && !wait(B_KE + st, use - 1)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.bar[B_KF + st], NB * kBlk);
#pragma unroll
                for (int b = 0; b < NB; ++b) tma_load_2d(sm.k[st] + b * kBlk, &kmap, g * N + 64 * b, t, &sm.bar[B_KF + st]);
            }
            __syncwarp();
            if (quse && !wait(B_QE + qs, quse - 1)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.bar[B_QF + qs], NB * kBlk);
#pragma unroll
                for (int b = 0; b < NB; ++b) tma_load_2d(sm.q[qs] + b * kBlk, &qmap, g * N + 64 * b, t, &sm.bar[B_QF + qs]);
            }
            __syncwarp();
            if (vuse && !wait(B_VE + vs, vuse - 1)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.bar[B_VF + vs], PB * kBlk);
#pragma unroll
                for (int b = 0; b < PB; ++b) tma_load_2d(sm.v[vs] + b * kBlk, &vmap, h * P + 64 * b, t, &sm.bar[B_VF + vs]);
            }
            __syncwarp();
        }
        loaded = c;
    } else if (warp == 17) {
        fewer_registers<kIssueRegs>();
        constexpr uint32_t ID_P = idesc_bf16(128, 128, false, false), ID_S = idesc_bf16(128, P, true, true),
                           ID_Y = idesc_bf16(128, P, false, true);
        for (int c = 0; c < nc; ++c) {
            const int st = c & 1, use = c >> 1, qs = c % NQ, vs = c % NV;
            const uint32_t q = smem_u32(sm.q[qs]), k = smem_u32(sm.k[st]), v = smem_u32(sm.v[vs]), sb = smem_u32(sm.sb);
            if (!wait(B_KF + st, use) || !wait(B_QF + qs, c / NQ)) break;
            if (c && !wait(B_Y, c - 1)) break;  // A, which lies where the scores go, is read
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk) mma_bf16(tm + T_P, desc_kmajor(q, kBlk, kk), desc_kmajor(k, kBlk, kk), ID_P, kk > 0);
                mma_commit(&sm.bar[B_P]);
            }
            __syncwarp();
            if (!wait(B_SB, c) || (c && !wait(B_YE, c - 1))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    mma_bf16(tm + T_Y2, desc_kmajor(q, kBlk, kk), desc_mnmajor(sb, N * 128, kk), ID_Y, kk > 0);
                mma_commit(&sm.bar[B_QE + qs]);
            }
            __syncwarp();
            if (!wait(B_K2, c) || !wait(B_VF + vs, c / NV)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int m = MORE; m >= 0; --m) {  // (the smallest first: their sums cut off less)
                    const uint32_t part = m ? smem_u32(sm.rest[m - 1]) : k;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16(tm + T_D, desc_mnmajor(part, kBlk, kk), desc_mnmajor(v, kBlk, kk), ID_S, m < MORE || kk > 0);
                }
                mma_commit(&sm.bar[B_S]);
                mma_commit(&sm.bar[B_KE + st]);
            }
            __syncwarp();
            if (!wait(B_A, c)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_bf16_ts(tm + T_Y, tm + T_P + 8 * kk, desc_mnmajor(v, kBlk, kk), ID_Y, kk > 0);
                mma_commit(&sm.bar[B_Y]);
                mma_commit(&sm.bar[B_VE + vs]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&sm.bar[B_END]);
        __syncwarp();
        drain(&sm.bar[B_END], 0);
    } else {
        fewer_registers<kIssueRegs>();  // (a group's registers go together)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sm.failed) {  // loads that nothing has waited for end before the block does: those of the last chunks
        if (warp == 16)
            for (int i = max(0, loaded - 2); i <= min(loaded, nc - 1); ++i) {
                drain(&sm.bar[B_KF + (i & 1)], (i >> 1) & 1);
                drain(&sm.bar[B_QF + i % NQ], (i / NQ) & 1);
                drain(&sm.bar[B_VF + i % NV], (i / NV) & 1);
            }
        if (tid == 0) flag_error(p.err, MAMBA_ERR_TIMEOUT);
        __syncthreads();
    }
    if (warp == 17) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------------------
// what a segment adds to the state
// ---------------------------------------------------------------------------------------

enum { G_F = 0, G_E = 2, G_K2 = 4, G_D = 6, G_DE = 8, G_END = 10, kSegBars };  // by stage: loaded, read, scaled, the product is there, added
// Two groups of 4 warps for the keys' decays, one for the sum, and one of which a warp loads and another issues the products.
constexpr int kSegThreads = 4 * 128, kSegRegs = 128, kSumRegs = 192, kScaleRegs = 112, kSegIssueRegs = 40;
static_assert(kSumRegs + 2 * kScaleRegs + kSegIssueRegs <= 4 * kSegRegs, "registers of the launch");

template <int P, bool F32S>
struct SegSmem {
    static constexpr int MORE = F32S ? 2 : 1, GROUPS = P == 128 && F32S ? 1 : 2;  // groups: of warps for the keys' decays
    unsigned char k[2][kTile], v[2][P * 256], rest[GROUPS][MORE][kTile];
    uint64_t bar[kSegBars];
    uint32_t tmem;
    int failed;
};

// One segment but a sequence's last, one head: sum of d^(tokens behind it in the segment) k_j v_j^T.  The first one's block
// also keeps the sequence's initial state.
template <int P, int N, bool F32S>
__global__ void __launch_bounds__(kSegThreads, 1) k_la_segment(const ScanParams p, const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap) {
    using Smem = SegSmem<P, F32S>;
    using StateT = typename std::conditional<F32S, float, bf16>::type;
    constexpr int MORE = Smem::MORE, GROUPS = Smem::GROUPS, NB = N / 64, PB = P / 64;
    extern __shared__ __align__(1024) unsigned char seg_smem[];
    Smem &sm = *align1024<Smem>(seg_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int h = blockIdx.x % p.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = tid & 127;
    const Job job = find_job(p, blockIdx.x / p.H);
    if (!job.ok || job.index == job.last) return;
    const float l2 = p.log_decay[h] * LOG2E;
    if (N == 64)
        for (int i = tid; i < (int)kBlk / 16; i += kSegThreads) {
#pragma unroll
            for (int s = 0; s < 2; ++s) reinterpret_cast<uint4 *>(sm.k[s] + kBlk)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int s = 0; s < GROUPS * MORE; ++s) reinterpret_cast<uint4 *>(sm.rest[s / MORE][s % MORE] + kBlk)[i] = make_uint4(0, 0, 0, 0);
        }
    if (warp == 12 && elect_one()) {
        for (int i = 0; i < kSegBars; ++i) mbar_init(&sm.bar[i], (i >= G_K2 && i < G_D) || (i >= G_DE && i < G_END) ? 4 : 1);
        fence_mbar_init();
        sm.failed = 0;
    }
    if (warp == 13) {
        tmem_alloc(&sm.tmem, 256);
        tmem_relinquish();
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    volatile int *failed = &sm.failed;
    const int nc = job.nc;  // (whole chunks: the segment is not the sequence's last)
    int loaded = 0;
    auto wait = [&](int b, uint32_t use) { return warp_wait(&sm.bar[b], use & 1, failed); };
    if (warp < 8) {
        fewer_registers<kScaleRegs>();
        const int group = warp >> 2;
        for (int c = group; c < nc && group < GROUPS; c += GROUPS) {
            const int st = c & 1;
            const float f = power(l2, job.len - 1 - (c * C + row));
            if (!wait(G_F + st, c >> 1)) break;
            // The other parts' place is the group's: free once the product of its last chunk is done.  Where groups take
            // turns that was two chunks ago, and the load of this chunk has waited for it.
            if (GROUPS == 1 && c && !wait(G_E + (c - 1 & 1), (c - 1) >> 1)) break;
            scale_row<NB, MORE>(sm.k[st], sm.rest[group % GROUPS][0], row, f);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[G_K2 + st]);
        }
    } else if (warp < 12) {
        more_registers<kSumRegs>();
        if (job.index == 0 && row < N && job.slot >= 0 && p.has_init && p.has_init[job.seq]) {
            float *to = entry_at(p, job.entry, h, P) + row;
            const StateT *from = static_cast<const StateT *>(p.pool) + job.slot * p.stride + (int64_t)h * P * N + row;
#pragma unroll 16
            for (int e = 0; e < P; ++e) to[e * 128] = to_f32(from[e * N]);
        }
        float S[P];
#pragma unroll
        for (int e = 0; e < P; ++e) S[e] = 0.0f;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        int c = 0;
        for (; c < nc; ++c) {
            const int st = c & 1;
            if (!wait(G_D + st, c >> 1)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < P / 32; ++b) {
                float d[32];
                tmem_ld32(lanes + 128 * st + 32 * b, d);
#pragma unroll
                for (int e = 0; e < 32; ++e) S[32 * b + e] += d[e];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[G_DE + st]);
        }
        if (c == nc) {
            float *to = entry_at(p, job.entry + 1 + job.index, h, P) + row;
#pragma unroll
            for (int e = 0; e < P; ++e) to[e * 128] = S[e];
        }
    } else if (warp == 12) {
        fewer_registers<kSegIssueRegs>();
        const int g = h / p.HG;
        int c = 0;
        for (; c < nc; ++c) {
            const int st = c & 1, use = c >> 1, t = job.t0 + c * C;
            if (use && !wait(G_E + st, use - 1)) break;
            if (elect_one()) {
                uint64_t *bar = &sm.bar[G_F + st];
                mbar_arrive_expect_tx(bar, (NB + PB) * kBlk);
#pragma unroll
                for (int b = 0; b < NB; ++b) tma_load_2d(sm.k[st] + b * kBlk, &kmap, g * N + 64 * b, t, bar);
#pragma unroll
                for (int b = 0; b < PB; ++b) tma_load_2d(sm.v[st] + b * kBlk, &vmap, h * P + 64 * b, t, bar);
            }
            __syncwarp();
        }
        loaded = c;
    } else if (warp == 13) {
        fewer_registers<kSegIssueRegs>();
        constexpr uint32_t ID_S = idesc_bf16(128, P, true, true);
        for (int c = 0; c < nc; ++c) {
            const int st = c & 1, use = c >> 1;
            const uint32_t k = smem_u32(sm.k[st]), v = smem_u32(sm.v[st]);
            if (!wait(G_K2 + st, use) || !wait(G_F + st, use) || (use && !wait(G_DE + st, use - 1))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int m = MORE; m >= 0; --m) {
                    const uint32_t part = m ? smem_u32(sm.rest[c % GROUPS][m - 1]) : k;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16(tm + 128 * st, desc_mnmajor(part, kBlk, kk), desc_mnmajor(v, kBlk, kk), ID_S, m < MORE || kk > 0);
                }
                mma_commit(&sm.bar[G_E + st]);
                mma_commit(&sm.bar[G_D + st]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&sm.bar[G_END]);
        __syncwarp();
        drain(&sm.bar[G_END], 0);
    } else {
        fewer_registers<kSegIssueRegs>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sm.failed) {
        if (warp == 12)
            for (int i = max(0, loaded - 2); i < loaded; ++i) drain(&sm.bar[G_F + (i & 1)], (i >> 1) & 1);
        if (tid == 0) flag_error(p.err, MAMBA_ERR_TIMEOUT);
        __syncthreads();
    }
    if (warp == 13) tmem_dealloc(tm, 256);
}

// Rows of tokens, `stride` elements apart, of `cols` values, in boxes of 128 tokens x 64 values, 128-byte swizzle.  Rows
// past the end read as zero.
bool tile_map(CUtensorMap *m, const void *ptr, int64_t cols, int64_t rows, int64_t stride) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {64, C}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Readies a kernel for its launch: its shared memory, and whether it was compiled to the registers that its groups share
// out (with fewer, the group that asks for more would wait for ever).
bool ready(const void *kern, size_t smem, int regs) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs >= regs &&
           cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
}

template <int P, int N, bool F32S>
int launch(const ScanParams &p, cudaStream_t st) {
    CUtensorMap qmap, kmap, vmap;
    if (!tile_map(&qmap, p.q, (int64_t)p.G * N, p.T, p.qs) || !tile_map(&kmap, p.k, (int64_t)p.G * N, p.T, p.ks) ||
        !tile_map(&vmap, p.v, (int64_t)p.H * P, p.T, p.vs))
        return MAMBA_ECUDA;
    const dim3 grid((unsigned)((int64_t)p.max_segs * p.H));
    if (p.seg_tokens < kWhole) {
        auto kern = k_la_segment<P, N, F32S>;
        constexpr size_t smem = sizeof(SegSmem<P, F32S>) + 1024;
        static_assert(smem <= 232448, "shared memory of a block");
        if (!ready(reinterpret_cast<const void *>(kern), smem, kSegRegs)) return MAMBA_ECUDA;
        if (launch_pdl(kern, grid, dim3(kSegThreads), smem, st, p, kmap, vmap) != cudaSuccess) return MAMBA_ECUDA;
    }
    auto kern = k_la_chain<P, N, F32S>;
    constexpr size_t smem = sizeof(ChainSmem<P, F32S>) + 1024;
    static_assert(smem <= 232448, "shared memory of a block");
    if (!ready(reinterpret_cast<const void *>(kern), smem, kRegs)) return MAMBA_ECUDA;
    if (launch_pdl(kern, grid, dim3(kThreads), smem, st, p, qmap, kmap, vmap) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <bool F32S>
int dispatch(const ScanParams &p, int P, int N, cudaStream_t st) {
    if (P == 128) return N == 128 ? launch<128, 128, F32S>(p, st) : launch<128, 64, F32S>(p, st);
    return N == 128 ? launch<64, 128, F32S>(p, st) : launch<64, 64, F32S>(p, st);
}

}  // namespace

bool chunked_eligible(const mamba_layer_desc *d) {
    return d->act_dtype == MAMBA_BF16 && (d->head_dim == 64 || d->head_dim == 128) && (d->d_state == 64 || d->d_state == 128);
}

// Sequences are cut where their heads alone are fewer than the SMs: into as many segments as make one block an SM, at
// least 4 chunks each (what a segment adds to the state costs about half of its pass).
int chunked_segment_tokens(int H, int T, int nseq) {
    const int64_t blocks = 152 / H;
    if (blocks < 2 * (int64_t)nseq) return kWhole;
    const int64_t chunks = ((int64_t)T + C - 1) / C, spare = blocks - nseq / 2;
    const int64_t per = (chunks + spare - 1) / spare;
    return (int)((per < 4 ? 4 : per) * C);
}

size_t chunked_workspace_bytes(const mamba_layer_desc *d, int64_t max_segs, int nseq, int seg_tokens) {
    return seg_tokens == kWhole ? 0 : (size_t)(max_segs + nseq) * d->nheads * 128 * d->head_dim * sizeof(float);
}

int chunked_launch(const ScanParams &p, const mamba_layer_desc *d, cudaStream_t st) {
    return d->state_dtype == MAMBA_F32 ? dispatch<true>(p, d->head_dim, d->d_state, st)
                                       : dispatch<false>(p, d->head_dim, d->d_state, st);
}

}  // namespace la
}  // namespace ms
