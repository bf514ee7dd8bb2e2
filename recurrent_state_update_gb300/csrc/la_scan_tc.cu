// la_scan_tc.cu -- the chunked form of linear attention on the tcgen05 tensor cores.
//
// For a chunk of L <= 128 tokens i = 0..L-1 and a head with the decay d = e^log_decay and the state S (P x N)
// before it:
//   A = (Q K^T) . D,  D_ij = d^(i-j) for j <= i, else 0
//   Y = A V + diag(d^(i+1)) Q S^T
//   S <- d^L S + V^T K',  K'_j = d^(L-1-j) k_j   (or V'^T K with the weights on V, which heads of 64 values do)
// Four products, none of which waits for another one's result but A V for A, and Q S^T for the state before: only the state's
// own update, elementwise, follows from chunk to chunk.  Everything else of the next chunk is under way meanwhile, in warps
// of its own: loads, products, A's decays, the weights, the state, and the outputs.
// The state stands in registers in fp32, a key index a thread, and takes each chunk's product with a rounding to nearest: the
// tensor cores' own sums cut bits off, in one direction, and would add up over the chunks.  Heads that remember 1 to 500 tokens
// hold a state to 1.8e-7 after 8192 tokens so, and to 1.3e-6 otherwise; one that remembers 1e4 tokens and more holds it to 5.6e-7
// after 65536.  Its copy for the queries, and A, are rounded to bf16, the type of the V, K and Q that they meet: an output is
// off by about as much as its own rounding to bf16 takes (2.3e-3 rms together, 1.7e-3 for that rounding alone).  K', whose
// rounding would stay in the state, is held as the sum of two bf16 numbers (16 bits) under a bf16 pool, without which outputs
// are 2.7e-3 off, and of three (24) under an fp32 pool, in as many products.
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
constexpr int kSMs = 152;
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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

// The warp's index, in a form that the compiler knows to be the same of all lanes: what the warps of one group do apart then
// needs no copies in registers of what stays the same (at most 20 bytes of spills in any form; without, up to 500, and 140 us
// instead of 115 for 8192 tokens of 128 heads of 64 x 128).
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

template <typename T>
__device__ __forceinline__ T *align1024(unsigned char *p) {
    return reinterpret_cast<T *>(p + (-smem_u32(p) & 1023u));  // (an offset, so that accesses stay shared-memory ones)
}

// Entries of the workspace: of each sequence, its initial state and what each segment but the last adds; a head's
// state each, transposed like tensor memory's lanes: value p of key n at p * 128 + n.
__device__ __forceinline__ float *entry_at(const ScanParams &p, int e, int h, int P) {
    return p.ws + ((int64_t)e * p.H + h) * (128 * P);
}

// A token's weight in the state: w, and as bf16 numbers, twice each, w1 of it and w2 of what is left.
struct Weight {
    float w;
    __nv_bfloat162 w1, w2;
    __device__ __forceinline__ explicit Weight(float f) : w(f) {
        w1 = __float2bfloat162_rn(f);
        w2 = __float2bfloat162_rn(f - __low2float(w1));
    }
};
__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// Offset of the 16-byte piece i (8 a block) of a row of a swizzled tile.
__device__ __forceinline__ uint32_t piece_at(int row, int i) { return (i >> 3) * kBlk + swz128_chunk(row, i & 7); }
// K' = w k of 8 values as a sum of 1 + MORE bf16 numbers.  The first is k w1, rounded, two values an instruction.
__device__ __forceinline__ uint4 first_part(const uint4 &k, const Weight &w) {
    auto one = [&](uint32_t x) { return as_u32(__hmul2(as_bf16x2(x), w.w1)); };
    return make_uint4(one(k.x), one(k.y), one(k.z), one(k.w));
}
// The others.  What rounding took from k w1 is a bf16 number itself, which a fused multiply-add gives; with k w2 it makes
// 16 bits.  Three parts take the product in fp32, and the second cuts off, so that 8 bits are left.
template <int MORE>
__device__ __forceinline__ void other_parts(const uint4 &k, const uint4 &first, const Weight &w, uint4 (&out)[MORE]) {
    const uint32_t in[4] = {k.x, k.y, k.z, k.w}, hi[4] = {first.x, first.y, first.z, first.w};
    uint32_t o[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (MORE == 1) {
            const __nv_bfloat162 x = as_bf16x2(in[e]);
            o[0][e] = as_u32(__hfma2(x, w.w2, __hfma2(x, w.w1, __hneg2(as_bf16x2(hi[e])))));
        } else {
            const uint64_t less = pair(-__uint_as_float(hi[e] << 16), -__uint_as_float(hi[e] & 0xffff0000u));
            float lo, up;
            unpair(fma2(pair(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xffff0000u)), pair(w.w, w.w), less), lo, up);
            o[0][e] = __byte_perm(__float_as_uint(lo), __float_as_uint(up), 0x7632);
            lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
            up -= __uint_as_float(__float_as_uint(up) & 0xffff0000u);
            o[1][e] = pack2(lo, up);
        }
    }
#pragma unroll
    for (int m = 0; m < MORE; ++m) out[m] = make_uint4(o[m][0], o[m][1], o[m][2], o[m][3]);
}
// The other parts of blocks B0 .. B1 - 1 of a row of K (or V) into the tiles at rest, REST bytes apart, and the first parts to
// registers.  Four pieces are read before the first is worked on.
template <int MORE, int B0, int B1, uint32_t REST>
__device__ __forceinline__ void other_parts(const unsigned char *k, unsigned char *rest, int row, const Weight &w, uint4 *first) {
#pragma unroll
    for (int i = 8 * B0; i < 8 * B1; i += 4) {
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const uint4 *>(k + piece_at(row, i + c));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t at = piece_at(row, i + c);
            const uint4 hi = first_part(x[c], w);
            uint4 out[MORE];
            other_parts<MORE>(x[c], hi, w, out);
            first[i - 8 * B0 + c] = hi;
#pragma unroll
            for (int m = 0; m < MORE; ++m) *reinterpret_cast<uint4 *>(rest + m * REST + at) = out[m];
        }
    }
}
__device__ __forceinline__ void clear_row(unsigned char *tile, int row, int b0, int b1) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b)
#pragma unroll 1
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(tile + b * kBlk + swz128_chunk(row, c)) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------------------
// the chain: a segment of a sequence, one head
// ---------------------------------------------------------------------------------------

// Each barrier's phase c is chunk c's (of a stage: the c-th use of the stage).
enum {
    B_QF = 0, B_KF = 2, B_VF = 4,   // loaded, by stage
    B_QE = 6, B_KE = 8, B_VE = 10,  // the products have read it
    B_P = 12,  // Q K^T is there, by place
    B_A = 14,  // A is in tensor memory
    B_K2,      // K' is in place of K, or V' beside V
    B_Y2,      // Q S^T is there
    B_M,       // ... scaled, and in the place where A V adds to it
    B_Y,       // the outputs are there
    B_S,       // the state's update is there
    B_SB,      // ... and added, and the state's copy is written (phase 0: before the first chunk)
    B_END,     // every product has finished
    B_U,       // a unit is given out, by turn
    kBars = B_U + 8
};
constexpr int kRing = 8;
// Groups of 4 warps: for A, for outputs, for the state, for the keys' decays, and one of which a warp loads and another issues the
// products.  The state's group takes registers from the others, within what the launch gave the block: 5 warps a scheduler
// leave 96 a thread (launch() checks that the compiler made it so).
constexpr int kThreads = 5 * 128, kRegs = 96, kScoreRegs = 88, kOutRegs = 88, kStateRegs = 168, kKeyRegs = 104,
              kIssueRegs = 32;
static_assert(kScoreRegs + kOutRegs + kStateRegs + kKeyRegs + kIssueRegs <= 5 * kRegs, "registers of the launch");

// Barrier of the outputs' group; whether any of its threads passed true.
__device__ __forceinline__ bool outputs_sync_or(bool v) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(any)
        : "r"((uint32_t)v)
        : "memory");
    return any != 0;
}
// A tile to memory, tracked in the issuing thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}

template <int P, int N, bool F32S>
struct ChainSmem {
    static_assert(N == 128 || P == 64, "compiled state shapes");
    // The weights of a chunk's tokens in the state meet its keys (K', in place of K) or its values (V', beside V): these, where
    // they are half as many and leave room.
    static constexpr bool ON_V = P == 64;
    // Parts of K' past the first, or of V' past V; stages of queries and values: what the parts leave room for.  Keys are needed
    // first and read last, so that they always have two.
    static constexpr int MORE = F32S ? 2 : 1, NQ = P == 64 && !F32S ? 2 : 1, NV = P == 128 && F32S ? 1 : 2;
    static constexpr int RESTS = ON_V ? MORE + 1 : MORE;
    static constexpr uint32_t kRest = ON_V ? kBlk : kTile;
    // Where the outputs stand on their way to memory: in a place of their own, where there is room for one, or over the chunk's
    // values, which are used by then, or its K' where values have one stage.  (Over K' the next keys come late: a ragged batch
    // took 209 us so.)
    static constexpr bool OWN_OUT = P == 64, OUT_ON_V = !OWN_OUT && NV == 2, OUT_ON_K = !OWN_OUT && !OUT_ON_V;
    static constexpr uint32_t kQ = N * 256, kSb = P * N * 2, kOut = OWN_OUT ? P * 256 : 1024;
    unsigned char q[NQ][kQ], k[2][kTile], v[NV][P * 256], sb[kSb], rest[RESTS][kRest], out[kOut];
    float diag[4][32];  // d^m, for each of the scores' warps
    int32_t ring[kRing];   // units given out, by turn
    uint64_t bar[kBars];
    uint32_t tmem;
    int failed;
};


// The segments and heads that a block works on, the longest first: the first by the block's index, each further one taken from
// the grid's counter by the warp that loads keys with the last of its loads for the unit before, and passed on through shared
// memory.  (Given out beforehand, in turn there and back, they took 512 sequences of narrow heads 148 us; taken a unit ahead,
// 256 ragged ones 238 us instead of 190.)
struct Units {
    const ScanParams &p;
    const int32_t *ring;
    uint64_t *bar;
    volatile int *failed;
    int total, k, h;  // h: the head of the last one given
    __device__ __forceinline__ Units(const ScanParams &q, const int32_t *ring, uint64_t *bar, volatile int *failed)
        : p(q), ring(ring), bar(bar), failed(failed), total(q.meta[0] * q.H), k(0), h(0) {}
    __device__ __forceinline__ bool at(int i, Segment &job) {
        if ((uint32_t)i >= (uint32_t)total) return false;
        job = meta_segments(p)[i / p.H];
        h = i % p.H;
        return true;
    }
    __device__ __forceinline__ bool next(Segment &job) {
        const int at_ring = k % kRing, use = k / kRing;  // (the first is not passed on: the k-th after it is the ring's k - 1st)
        ++k;
        return warp_wait(&bar[at_ring], use & 1, failed) && at(ring[at_ring], job);
    }
};

// A block an SM, each with one segment of one head after the other.  What bounds a chunk in bf16 is shared memory: of 128 x 128
// heads the products read 288 KB of operands from it, the warps move 160 KB through it, loads and outputs 128 KB, 4600 cycles at
// 128 bytes a cycle, and a chunk takes about 5000; of 64 x 128 heads 368 KB, 2900 cycles, in about 3300 (3600 with a product for
// each part of V', 4100 with the weights on K).  Under an fp32 pool it is 5300 of 6200 cycles, and a chunk's steps follow one another:
// the keys' three parts, of which the scores' warps make half before they turn to the scores (2700 cycles), A (1400), A V (900)
// and the outputs (1600).  Where all SMs work on heads of 128 x 128 device memory is as slow: 8 ragged prompts of 32768 tokens of 32
// heads, 1.11 GB, take 193 to 197 us, 0.84 to 0.86 of a copy's rate.  29 seeded sequences of 4001 tokens, a chunk or two each, take 68 us (their
// states alone are 122 MB), 8192 tokens of 128 heads of 64 x 128 115 us, one prompt of 8192 tokens 105 us: 8 for the plan and the
// launches, 34 for its segments' sums, 2 to 9 until a block has the state before its segment, 53 for 16 chunks of 128 blocks.
template <int P, int N, bool F32S>
__global__ void __launch_bounds__(kThreads, 1) k_la_chain(const ScanParams p, const __grid_constant__ CUtensorMap qmap,
                                                          const __grid_constant__ CUtensorMap kmap,
                                                          const __grid_constant__ CUtensorMap vmap,
                                                          const __grid_constant__ CUtensorMap ymap) {
    using Smem = ChainSmem<P, N, F32S>;
    using StateT = typename std::conditional<F32S, float, bf16>::type;
    constexpr int NQ = Smem::NQ, NV = Smem::NV, MORE = Smem::MORE, NB = N / 64, PB = P / 64;
    // Tensor memory columns: scores (of two chunks, where there is room), the state's part of the outputs, the outputs, the
    // state's update.  A takes the second half of its scores' columns.
    constexpr int NP = P == 64 && NQ == 2 ? 2 : 1;
    constexpr uint32_t T_P = 0, T_Y2 = NP * 128, T_Y = T_Y2 + P, T_D = T_Y + P;
    constexpr bool ON_V = Smem::ON_V;
    constexpr int PARTS = ON_V ? MORE + 1 : 1;  // of the state's update, side by side: those of V' meet K in one product
    static_assert(T_D + PARTS * P <= 512, "tensor memory");
    constexpr bool HELP = MORE == 2 && !ON_V;  // HELP: whether the scores' group takes half of the other parts
    extern __shared__ __align__(1024) unsigned char chain_smem[];
    Smem &sm = *align1024<Smem>(chain_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    volatile int *failed = &sm.failed;
    Units units(p, sm.ring, &sm.bar[B_U], failed);
    Segment job;
    if (!units.at(blockIdx.x, job)) return;
    if (N == 64)  // the keys' lanes without keys: products read them
        for (int i = tid; i < (int)kBlk / 16; i += kThreads) {
#pragma unroll
            for (int s = 0; s < 2; ++s) reinterpret_cast<uint4 *>(sm.k[s] + kBlk)[i] = make_uint4(0, 0, 0, 0);
        }
    if (warp == 16 && elect_one()) {
        tma_prefetch_desc(&qmap), tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap), tma_prefetch_desc(&ymap);
        for (int i = 0; i < kBars; ++i) mbar_init(&sm.bar[i], i == B_K2 && HELP ? 8 : i == B_A || i == B_K2 || i == B_M || i == B_SB ? 4 : 1);
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
    auto wait = [&](int b, uint32_t use) { return warp_wait(&sm.bar[b], use & 1, failed); };
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int row = tid & 127;
    int loaded = 0, in_flight = -1, of = 1;  // what this warp has loaded, and the first barrier of its stages
    int g = 0;                               // chunks before this one, of all the block's segments
    bool ok = true;                          // no wait has given up

    if (warp < 4) {
        fewer_registers<kScoreRegs>();
        // A: row i a thread, in pieces of 16 columns j, from the diagonal's two to the left.  There d^(i-j) is
        // d^(i-j0-15) * d^(15-(j-j0)), neither of which can overflow.  A lies from column 64 on, where scores stood that have
        // been read by the time.
        do {
            const float l2 = p.log_decay[units.h] * LOG2E;
            sm.diag[warp][lane] = power(l2, lane);
            __syncwarp();
            const float *diag = sm.diag[warp];
            uint64_t col[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) col[e] = pair(power(l2, 15 - 2 * e), power(l2, 14 - 2 * e));
            const float step = power(l2, 16), first = power(l2, lane + 1);
            for (int left = job.len; left > 0; left -= C, ++g) {
                if (HELP) {  // (three parts of K' take the keys' group longer than the scores take to come: half is done here)
                    if (!(ok = wait(B_KF + (g & 1), g >> 1) && (!g || wait(B_S, g - 1)))) break;
                    const int L = min(C, left);
                    uint4 part[8];
                    if (row < L) {
                        other_parts<MORE, NB / 2, NB, kTile>(sm.k[g & 1], sm.rest[0], row, Weight(power(l2, L - 1 - row)), part);
                    } else {
#pragma unroll
                        for (int m = 0; m < MORE; ++m) clear_row(sm.rest[m], row, NB / 2, NB);
#pragma unroll
                        for (int i = 0; i < 8; ++i) part[i] = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    if (!(ok = wait(B_P + g % NP, g / NP))) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(sm.k[g & 1] + piece_at(row, 8 * (NB / 2) + i)) = part[i];
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(&sm.bar[B_K2]);
                } else if (!(ok = wait(B_P + g % NP, g / NP))) {
                    break;
                }
                tc_fence_after();
                const uint32_t T_c = lanes + T_P + (NP == 2 ? (g & 1) * 128 : 0), T_A = T_c + 64;
                uint32_t x[2][16], pk[8];
                tmem_get(T_c + 32 * warp + 16, x[0]);
                if (warp < 3) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = 0u;
#pragma unroll 1
                    for (int i = 2 * warp + 2; i < 8; ++i) tmem_put8(T_A + 8 * i, pk);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {  // columns 16 .. 31 of the diagonal's 32, then 0 .. 15
                    tmem_got(x[u]);
                    if (u == 0) tmem_get(T_c + 32 * warp, x[1]);
                    else if (warp) tmem_get(T_c + 32 * warp - 16, x[0]);
                    const int at = lane - (u ? 0 : 16);
#pragma unroll
                    for (int e = 0; e < 16; e += 2)
                        pk[e / 2] = pack2(e <= at ? __uint_as_float(x[u][e]) * diag[max(at - e, 0)] : 0.0f,
                                          e + 1 <= at ? __uint_as_float(x[u][e + 1]) * diag[max(at - e - 1, 0)] : 0.0f);
                    tmem_put8(T_A + 8 * (2 * warp + 1 - u), pk);
                }
                float rf = first;
#pragma unroll 1
                for (int i = 2 * warp - 1; i > 0; i -= 2) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_got(x[u]);
                        if (u == 0 || i > 1) tmem_get(T_c + 16 * (i - u - 1), x[u ^ 1]);
                        const uint64_t r2 = pair(rf, rf);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float lo, hi;
                            unpair(mul2(pair(__uint_as_float(x[u][2 * e]), __uint_as_float(x[u][2 * e + 1])), mul2(col[e], r2)), lo, hi);
                            pk[e] = pack2(lo, hi);
                        }
                        tmem_put8(T_A + 8 * (i - u), pk);
                        rf *= step;
                    }
                }
                tmem_put_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sm.bar[B_A]);
            }
        } while (ok && units.next(job));
    } else if (warp < 8) {
        fewer_registers<kOutRegs>();
        // The outputs, row i a thread: the state's part, decayed, to where A V adds to it (so that it leaves its place for the next
        // chunk's long before the outputs are done, and the queries theirs), and the sum through shared memory, whence whole
        // chunks go as tiles.  (Stored from here, 32 rows apart in every instruction, they took 2000 cycles of the load and store
        // unit a chunk.)
        const uint64_t scale = pair(p.scale, p.scale);
        do {
            const int h = units.h;
            const float f = power(p.log_decay[h] * LOG2E, row + 1);
            const uint64_t f2 = pair(f, f);
            int t = job.t0;
            for (int left = job.len; left > 0; left -= C, t += C, ++g) {
                unsigned char *out = Smem::OWN_OUT ? sm.out : Smem::OUT_ON_V ? sm.v[g % NV] : sm.k[g & 1];
                if (outputs_sync_or(!wait(B_Y2, g))) {  // (all four warps leave together: they meet below)
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t a[2][16];
                tmem_get(lanes + T_Y2, a[0]);
#pragma unroll 1
                for (int b = 0; b < P / 16; b += 2) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_got(a[u]);
                        if (u == 0 || b + 2 < P / 16) tmem_get(lanes + T_Y2 + 16 * (b + u + 1), a[u ^ 1]);
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float lo, hi;
                            unpair(mul2(f2, pair(__uint_as_float(a[u][e]), __uint_as_float(a[u][e + 1]))), lo, hi);
                            o[e] = __float_as_uint(lo), o[e + 1] = __float_as_uint(hi);
                        }
                        tmem_put16(lanes + T_Y + 16 * (b + u), o);
                    }
                }
                tmem_put_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sm.bar[B_M]);
                if (Smem::OWN_OUT && warp == 4) bulk_wait_read<0>();  // (by the thread that issued the last tile)
                if (!(ok = !outputs_sync_or(!wait(B_Y, g)))) break;
                tc_fence_after();
                tmem_get(lanes + T_Y, a[0]);
#pragma unroll 1
                for (int b = 0; b < P / 16; b += 2) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_got(a[u]);
                        if (u == 0 || b + 2 < P / 16) tmem_get(lanes + T_Y + 16 * (b + u + 1), a[u ^ 1]);
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float lo, hi;
                            unpair(mul2(scale, pair(__uint_as_float(a[u][e]), __uint_as_float(a[u][e + 1]))), lo, hi);
                            o[e / 2] = pack2(lo, hi);
                        }
                        unsigned char *to = out + ((b + u) >> 2) * kBlk;
                        *reinterpret_cast<uint4 *>(to + swz128_chunk(row, ((b + u) & 3) * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(to + swz128_chunk(row, ((b + u) & 3) * 2 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                tc_fence_before();
                fence_async_smem();
                outputs_sync_or(false);
                if (left >= C) {
                    if (warp == 4 && elect_one()) {
#pragma unroll
                        for (int b = 0; b < PB; ++b) tma_store_2d(&ymap, out + b * kBlk, h * P + 64 * b, t);
                        bulk_commit();
                        if (!Smem::OWN_OUT) {
                            bulk_wait_read<0>();
                            arrive(&sm.bar[Smem::OUT_ON_V ? B_VE + g % NV : B_KE + (g & 1)]);
                        }
                    }
                    __syncwarp();
                } else {  // the sequence's last tokens: the rows after them are another's
                    constexpr int CH = P / 8;  // 16-byte pieces of a token's outputs; a thread takes every 128 / CH-th token
                    const int ch = row % CH;
                    bf16 *dst = static_cast<bf16 *>(p.y) + ((int64_t)t * p.H + h) * P + ch * 8;
                    for (int i = row / CH; i < left; i += 128 / CH)
                        *reinterpret_cast<uint4 *>(dst + (int64_t)i * p.H * P) =
                            *reinterpret_cast<const uint4 *>(out + (ch >> 3) * kBlk + swz128_chunk(i, ch & 7));
                    if (!Smem::OWN_OUT) {  // the place is the next segment's
                        outputs_sync_or(false);
                        if (row == 0) arrive(&sm.bar[Smem::OUT_ON_V ? B_VE + g % NV : B_KE + (g & 1)]);
                        __syncwarp();
                    }
                }
            }
        } while (ok && units.next(job));
        if (Smem::OWN_OUT && warp == 4) bulk_wait_read<0>();
    } else if (warp < 12) {
        // the state: key index n a thread (with N 64 the upper half hold zeros)
        more_registers<kStateRegs>();
        const int n = row;
        do {
            const int h = units.h, nc = (job.len + C - 1) / C;
            const float l = p.log_decay[h];
            StateT *pool = static_cast<StateT *>(p.pool) + (int64_t)h * P * N + n;
            const bool seeded = n < N && job.seeded;
            uint64_t S[P / 2];  // values 2 e and 2 e + 1
            {
                const float *from = entry_at(p, job.entry, h, P) + n;
                if (!seeded) {
#pragma unroll
                    for (int e = 0; e < P / 2; ++e) S[e] = 0;
                } else if (job.last) {  // several segments: from the copy, since the last one's block writes the slot
#pragma unroll
                    for (int e = 0; e < P / 2; ++e) S[e] = pair(from[2 * e * 128], from[(2 * e + 1) * 128]);
                } else {
#pragma unroll
                    for (int e = 0; e < P / 2; ++e)
                        S[e] = pair(to_f32(pool[job.slot * p.stride + 2 * e * N]), to_f32(pool[job.slot * p.stride + (2 * e + 1) * N]));
                }
                if (n < N && job.index) {
                    const float2 over = decay_of(l * (float)p.seg_tokens);
                    const uint64_t over2 = pair(over.x, over.x), rest2 = pair(over.y, over.y);
#pragma unroll 1
                    for (int r = 1; r <= job.index; ++r) {
                        from += (int64_t)p.H * (128 * P);
#pragma unroll
                        for (int e = 0; e < P / 2; ++e)
                            S[e] = decayed(over2, rest2, S[e], pair(from[2 * e * 128], from[(2 * e + 1) * 128]));
                    }
                }
            }
            // Over a chunk, and over the last one: two numbers, since what one loses to rounding is lost anew every chunk (up to
            // 2^-25 each, 1.5e-5 of a state after 512, and all of a decay of less than that).
            const float2 whole = decay_of(l * (float)C), part = decay_of(l * (float)(job.len - (nc - 1) * C));
            for (int c = -1; c < nc; ++c) {  // (from -1: only the copy for the first chunk)
                if (c >= 0) {
                    if (!(ok = wait(B_S, g))) break;
                    ++g;
                    tc_fence_after();
                    const float2 over = c + 1 == nc ? part : whole;
                    const uint64_t over2 = pair(over.x, over.x), rest2 = pair(over.y, over.y);
                    if constexpr (PARTS == 1) {
                        tmem_pieces<P / 16>(lanes + T_D, [&](int i, const uint32_t (&d)[16]) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                S[8 * i + e] = decayed(over2, rest2, S[8 * i + e],
                                                       pair(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
                        });
                    } else {
#pragma unroll
                        for (int i = 0; i < P / 16; ++i) {
                            uint32_t d[PARTS][16];
#pragma unroll
                            for (int m = 0; m < PARTS; ++m) tmem_get(lanes + T_D + m * P + 16 * i, d[m]);
#pragma unroll
                            for (int m = 0; m < PARTS; ++m) tmem_got(d[m]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                uint64_t sum = pair(__uint_as_float(d[MORE][2 * e]), __uint_as_float(d[MORE][2 * e + 1]));
#pragma unroll
                                for (int m = MORE - 1; m >= 0; --m)  // (the smallest first)
                                    sum = add2(sum, pair(__uint_as_float(d[m % PARTS][2 * e]), __uint_as_float(d[m % PARTS][2 * e + 1])));
                                S[8 * i + e] = decayed(over2, rest2, S[8 * i + e], sum);
                            }
                        }
                    }
                }
                if (c + 1 < nc) {
                    if (n < N) {
#pragma unroll
                        for (int e = 0; e < P / 2; e += 4) {
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float lo, hi;
                                unpair(S[e + i], lo, hi);
                                o[i] = pack2(lo, hi);
                            }
                            *reinterpret_cast<uint4 *>(sm.sb + (e >> 5) * (N * 128) + swz128_chunk(n, (e >> 2) & 7)) =
                                make_uint4(o[0], o[1], o[2], o[3]);
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
                        for (int e = 0; e < P / 2; ++e) {
                            float lo, hi;
                            unpair(S[e], lo, hi);
                            to[2 * e * N] = from_f32<StateT>(lo);
                            to[(2 * e + 1) * N] = from_f32<StateT>(hi);
                        }
                    };
                    if (ckpt >= 0) write(ckpt);
                    if (end) write(job.slot);
                }
            }
        } while (ok && units.next(job));
    } else if (warp < 16) {
        more_registers<kKeyRegs>();
        // K', token j a thread: its other parts (with the scores' group, see there) once the chunk before is through with theirs,
        // while the scores are formed, and the first in place of K when these have read it.  Or V', all parts beside V, which waits
        // for no scores.  Past the segment's end zeros, in V and K as well: the tiles hold another's tokens there (whose scores
        // nothing reads).
        do {
            const float l2 = p.log_decay[units.h] * LOG2E;
            for (int left = job.len; left > 0; left -= C, ++g) {
                const int L = min(C, left);
                unsigned char *tile = sm.k[g & 1];
                const Weight w(power(l2, max(L - 1 - row, 0)));
                if (!(ok = wait(B_KF + (g & 1), g >> 1) && (!g || wait(B_S, g - 1)))) break;
                if constexpr (ON_V) {
                    if (!(ok = wait(B_VF + g % NV, g / NV))) break;
                    unsigned char *values = sm.v[g % NV];
                    if (row < L) {
                        uint4 first[8];
                        other_parts<MORE, 0, 1, kBlk>(values, sm.rest[1], row, w, first);
#pragma unroll
                        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(sm.rest[0] + piece_at(row, i)) = first[i];
                    } else {
#pragma unroll
                        for (int m = 0; m <= MORE; ++m) clear_row(sm.rest[m], row, 0, 1);
                        clear_row(values, row, 0, 1);
                        clear_row(tile, row, 0, NB);
                    }
                } else {
                    constexpr int OWN = HELP ? NB / 2 : NB;
                    uint4 first[8 * OWN];
                    if (row < L) {
                        other_parts<MORE, 0, OWN, kTile>(tile, sm.rest[0], row, w, first);
                    } else {
#pragma unroll
                        for (int m = 0; m < MORE; ++m) clear_row(sm.rest[m], row, 0, OWN);
#pragma unroll
                        for (int i = 0; i < 8 * OWN; ++i) first[i] = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    if (!(ok = wait(B_P + g % NP, g / NP))) break;
#pragma unroll
                    for (int i = 0; i < 8 * OWN; ++i) *reinterpret_cast<uint4 *>(tile + piece_at(row, i)) = first[i];
                    if (L < C) {
                        if (!(ok = wait(B_VF + g % NV, g / NV))) break;
                        if (row >= L) clear_row(sm.v[g % NV], row, 0, PB);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&sm.bar[B_K2]);
            }
        } while (ok && units.next(job));
    } else {
        fewer_registers<kIssueRegs>();  // (before the group's warps part: all of them have to execute the same one)
        if (warp != 17) {
            // loads: of queries, keys and values, a warp each
            const int stages = warp == 16 ? NQ : warp == 18 ? 2 : NV, full = warp == 16 ? B_QF : warp == 18 ? B_KF : B_VF,
                      empty = warp == 16 ? B_QE : warp == 18 ? B_KE : B_VE, blocks = warp == 19 ? PB : NB;
            unsigned char *tiles = warp == 16 ? sm.q[0] : warp == 18 ? sm.k[0] : sm.v[0];
            const uint32_t size = warp == 16 ? Smem::kQ : warp == 18 ? kTile : P * 256;
            const CUtensorMap *map = warp == 16 ? &qmap : warp == 18 ? &kmap : &vmap;
            int st = 0, use = 0;
            do {
                const int x = warp == 19 ? units.h * P : units.h / p.HG * N;
                for (int t = job.t0; t < job.t0 + job.len; t += C, ++loaded) {
                    if (use && !(ok = wait(empty + st, use - 1))) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&sm.bar[full + st], blocks * kBlk);
                        for (int b = 0; b < blocks; ++b)
                            tma_load_2d(tiles + st * size + b * kBlk, map, x + 64 * b, t, &sm.bar[full + st]);
                    }
                    __syncwarp();
                    if (++st == stages) st = 0, ++use;
                    if (warp == 18 && t + C >= job.t0 + job.len) {  // the next unit, for all warps (none is kRing units behind)
                        const int k = units.k % kRing;
                        if (elect_one()) {
                            const int i = gridDim.x + atomicAdd(&p.meta[1], 1);
                            sm.ring[k] = i;
                            arrive(&sm.bar[B_U + k]);
                            if (i < units.total) {  // and its state on the way into L2
                                const Segment &next = meta_segments(p)[i / p.H];
                                if (next.seeded && !next.last)
                                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                                     static_cast<const StateT *>(p.pool) + next.slot * p.stride + (int64_t)(i % p.H) * P * N),
                                                 "r"((uint32_t)(P * N * sizeof(StateT)))
                                                 : "memory");
                            }
                        }
                        __syncwarp();
                    }
                }
            } while (ok && units.next(job));
            in_flight = full, of = stages;
        } else {
            constexpr uint32_t ID_P = idesc_bf16(128, 128, false, false), ID_S = idesc_bf16(128, PARTS * P, true, true),
                               ID_Y = idesc_bf16(128, P, false, true);
            constexpr bool AHEAD = NP == 2;  // whether the next chunk's scores go before this one's outputs
            auto scores = [&](int c) {
                const int st = c & 1, qs = c % NQ;
                if (!wait(B_KF + st, c >> 1) || !wait(B_QF + qs, c / NQ)) return false;
                if (c >= NP && !wait(B_Y, c - NP)) return false;  // A, which lies where the scores go, is read
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t q = smem_u32(sm.q[qs]), k = smem_u32(sm.k[st]), to = tm + T_P + (NP == 2 ? (c & 1) * 128 : 0);
    #pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) mma_bf16(to, desc_kmajor(q, kBlk, kk), desc_kmajor(k, kBlk, kk), ID_P, kk > 0);
                    mma_commit(&sm.bar[B_P + c % NP]);
                }
                __syncwarp();
                return true;
            };
            ok = scores(0);
            for (bool more = true; ok && more;) {
                for (int left = job.len; left > 0; left -= C, ++g) {
                    const int st = g & 1, qs = g % NQ, vs = g % NV;
                    const uint32_t q = smem_u32(sm.q[qs]), k = smem_u32(sm.k[st]), v = smem_u32(sm.v[vs]), sb = smem_u32(sm.sb);
                    if (!(ok = wait(B_SB, g) && (!g || wait(B_M, g - 1)))) break;
                    tc_fence_after();
                    if (elect_one()) {
    #pragma unroll
                        for (int kk = 0; kk < N / 16; ++kk)
                            mma_bf16(tm + T_Y2, desc_kmajor(q, kBlk, kk), desc_mnmajor(sb, N * 128, kk), ID_Y, kk > 0);
                        mma_commit(&sm.bar[B_QE + qs]);
                        mma_commit(&sm.bar[B_Y2]);
                    }
                    __syncwarp();
                    if (!(ok = wait(B_K2, g) && wait(B_VF + vs, g / NV))) break;
                    tc_fence_after();
                    if (elect_one()) {
    #pragma unroll
                        for (int m = ON_V ? 0 : MORE; m >= 0; --m) {  // (the smallest first: their sums cut off less)
                            const uint32_t keys = m ? smem_u32(sm.rest[m - 1]) : k, values = ON_V ? smem_u32(sm.rest[0]) : v;
    #pragma unroll
                            for (int kk = 0; kk < C / 16; ++kk)
                                mma_bf16(tm + T_D, desc_mnmajor(keys, kBlk, kk), desc_mnmajor(values, kBlk, kk), ID_S,
                                         (!ON_V && m < MORE) || kk > 0);
                        }
                        mma_commit(&sm.bar[B_S]);
                        if (!Smem::OUT_ON_K) mma_commit(&sm.bar[B_KE + st]);  // (else the outputs go there first)
                    }
                    __syncwarp();
                    if (left <= C) more = units.next(job);  // (given out when the chunk's keys were loaded)
                    if (AHEAD && (left > C || more) && !(ok = scores(g + 1))) break;
                    if (!(ok = wait(B_A, g) && wait(B_M, g))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t a = tm + T_P + (NP == 2 ? (g & 1) * 128 : 0) + 64;
    #pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk) mma_bf16_ts(tm + T_Y, a + 8 * kk, desc_mnmajor(v, kBlk, kk), ID_Y, 1);
                        mma_commit(&sm.bar[B_Y]);
                        if (!Smem::OUT_ON_V) mma_commit(&sm.bar[B_VE + vs]);
                    }
                    __syncwarp();
                    if (!AHEAD && (left > C || more) && !(ok = scores(g + 1))) break;
                }
            }
            if (elect_one()) mma_commit(&sm.bar[B_END]);
            __syncwarp();
            drain(&sm.bar[B_END], 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sm.failed) {  // loads that nothing has waited for end before the block does
        if (in_flight >= 0)
            for (int i = max(0, loaded - of); i < loaded; ++i) drain(&sm.bar[in_flight + i % of], (i / of) & 1);
        if (tid == 0) flag_error(p.err, MAMBA_ERR_TIMEOUT);
        __syncthreads();
    }
    if (warp == 17) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------------------
// what a segment adds to the state
// ---------------------------------------------------------------------------------------

// By stage: loaded, read, the product is there, added; scaled, by group and stage; other parts read, by group.
enum { G_F = 0, G_E = 2, G_D = 4, G_DE = 6, G_K2 = 8, G_R = 12, G_END = 14, kSegBars };
// Two groups of 4 warps for the keys' decays, one for the sum, and one of which a warp loads and another issues the products.
constexpr int kSegThreads = 4 * 128, kSegRegs = 128, kSumRegs = 192, kScaleRegs = 112, kSegIssueRegs = 40;
static_assert(kSumRegs + 2 * kScaleRegs + kSegIssueRegs <= 4 * kSegRegs, "registers of the launch");

template <int P, bool F32S>
struct SegSmem {
    static constexpr int MORE = F32S ? 2 : 1;
    unsigned char k[2][kTile], v[2][P * 256], rest[2][MORE][kTile / 2];  // rest: the other parts of half a chunk, by group
    uint64_t bar[kSegBars];
    uint32_t tmem;
    int failed;
};

// One segment but a sequence's last, one head: sum of d^(tokens behind it in the segment) k_j v_j^T.  The first one's block
// also keeps the sequence's initial state.  Each group of warps readies half of every chunk's tokens, and one half's product
// runs while the other half is readied.
template <int P, int N, bool F32S>
__global__ void __launch_bounds__(kSegThreads, 1) k_la_segment(const ScanParams p, const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap) {
    using Smem = SegSmem<P, F32S>;
    using StateT = typename std::conditional<F32S, float, bf16>::type;
    constexpr int MORE = Smem::MORE, NB = N / 64, PB = P / 64;
    extern __shared__ __align__(1024) unsigned char seg_smem[];
    Smem &sm = *align1024<Smem>(seg_smem);
    pdl_wait();  // see pdl_wait: no global access before the previous grid is complete
    pdl_launch_dependents();
    const int h = blockIdx.x % p.H, tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31, row = tid & 127;
    const int which = blockIdx.x / p.H;
    const Segment job = meta_segments(p)[min(which, p.max_segs - 1)];
    if (which >= p.meta[0] || job.index == job.last) return;
    const float l2 = p.log_decay[h] * LOG2E;
    if (N == 64)
        for (int i = tid; i < (int)kBlk / 16; i += kSegThreads) {
#pragma unroll
            for (int s = 0; s < 2; ++s) reinterpret_cast<uint4 *>(sm.k[s] + kBlk)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int s = 0; s < 2 * MORE; ++s)
                if (i < (int)kBlk / 32) reinterpret_cast<uint4 *>(sm.rest[s / MORE][s % MORE] + kBlk / 2)[i] = make_uint4(0, 0, 0, 0);
        }
    if (warp == 12 && elect_one()) {
        for (int i = 0; i < kSegBars; ++i) mbar_init(&sm.bar[i], (i >= G_DE && i < G_R) ? 4 : 1);
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
    const int nc = job.len / C;  // (whole chunks: the segment is not the sequence's last)
    int loaded = 0;
    auto wait = [&](int b, uint32_t use) { return warp_wait(&sm.bar[b], use & 1, failed); };
    if (warp < 8) {
        fewer_registers<kScaleRegs>();
        constexpr int PC = 4 * NB;  // 16-byte pieces a thread: half of a token's
        const int group = warp >> 2, j = group * 64 + (tid & 63), i0 = (row >> 6) * PC;
        for (int c = 0; c < nc; ++c) {
            const int st = c & 1;
            const Weight w(power(l2, job.len - 1 - (c * C + j)));
            if (!wait(G_F + st, c >> 1) || (c && !wait(G_R + group, c - 1))) break;
#pragma unroll
            for (int i = 0; i < PC; i += 4) {
                uint4 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const uint4 *>(sm.k[st] + piece_at(j, i0 + i + e));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = i0 + i + e;
                    const uint4 hi = first_part(x[e], w);
                    uint4 out[MORE];
                    other_parts<MORE>(x[e], hi, w, out);
                    *reinterpret_cast<uint4 *>(sm.k[st] + piece_at(j, at)) = hi;
#pragma unroll
                    for (int m = 0; m < MORE; ++m)  // (blocks of 64 tokens)
                        *reinterpret_cast<uint4 *>(sm.rest[group][m] + (at >> 3) * (kBlk / 2) + swz128_chunk(j & 63, at & 7)) = out[m];
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[G_K2 + 2 * group + st]);
        }
    } else if (warp < 12) {
        more_registers<kSumRegs>();
        if (job.index == 0 && row < N && job.seeded) {
            float *to = entry_at(p, job.entry, h, P) + row;
            const StateT *from = static_cast<const StateT *>(p.pool) + job.slot * p.stride + (int64_t)h * P * N + row;
#pragma unroll 16
            for (int e = 0; e < P; ++e) to[e * 128] = to_f32(from[e * N]);
        }
        uint64_t S[P / 2];  // values 2 e and 2 e + 1
#pragma unroll
        for (int e = 0; e < P / 2; ++e) S[e] = 0;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        int c = 0;
        for (; c < nc; ++c) {
            const int st = c & 1;
            if (!wait(G_D + st, c >> 1)) break;
            tc_fence_after();
            tmem_pieces<P / 16>(lanes + 128 * st, [&](int i, const uint32_t (&d)[16]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) S[8 * i + e] = add2(S[8 * i + e], pair(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
            });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&sm.bar[G_DE + st]);
        }
        if (c == nc) {
            float *to = entry_at(p, job.entry + 1 + job.index, h, P) + row;
#pragma unroll
            for (int e = 0; e < P / 2; ++e) unpair(S[e], to[2 * e * 128], to[(2 * e + 1) * 128]);
        }
    } else {
        fewer_registers<kSegIssueRegs>();
        if (warp == 12) {
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
            constexpr uint32_t ID_S = idesc_bf16(128, P, true, true);
            for (int c = 0; c < nc; ++c) {
                const int st = c & 1, use = c >> 1;
                const uint32_t k = smem_u32(sm.k[st]), v = smem_u32(sm.v[st]);
                if (!wait(G_F + st, use) || (use && !wait(G_DE + st, use - 1))) break;
                bool ok = true;
    #pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = wait(G_K2 + 2 * half + st, use))) break;
                    tc_fence_after();
                    if (elect_one()) {
    #pragma unroll
                        for (int m = MORE; m >= 0; --m)  // (the smallest first: their sums cut off less)
    #pragma unroll
                            for (int kk = 0; kk < C / 32; ++kk)
                                mma_bf16(tm + 128 * st,
                                         m ? desc_mnmajor(smem_u32(sm.rest[half][m - 1]), kBlk / 2, kk) : desc_mnmajor(k, kBlk, 4 * half + kk),
                                         desc_mnmajor(v, kBlk, 4 * half + kk), ID_S, half > 0 || m < MORE || kk > 0);
                        mma_commit(&sm.bar[G_R + half]);
                        if (half == 1) {
                            mma_commit(&sm.bar[G_E + st]);
                            mma_commit(&sm.bar[G_D + st]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (elect_one()) mma_commit(&sm.bar[G_END]);
            __syncwarp();
            drain(&sm.bar[G_END], 0);
        }
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
    CUtensorMap qmap, kmap, vmap, ymap;
    if (!tile_map(&qmap, p.q, (int64_t)p.G * N, p.T, p.qs) || !tile_map(&kmap, p.k, (int64_t)p.G * N, p.T, p.ks) ||
        !tile_map(&vmap, p.v, (int64_t)p.H * P, p.T, p.vs) || !tile_map(&ymap, p.y, (int64_t)p.H * P, p.T, (int64_t)p.H * P))
        return MAMBA_ECUDA;
    const int64_t units = (int64_t)p.max_segs * p.H;
    if (p.seg_tokens < kWhole) {
        auto kern = k_la_segment<P, N, F32S>;
        constexpr size_t smem = sizeof(SegSmem<P, F32S>) + 1024;
        static_assert(smem <= 232448, "shared memory of a block");
        if (!ready(reinterpret_cast<const void *>(kern), smem, kSegRegs)) return MAMBA_ECUDA;
        if (launch_pdl(kern, dim3((unsigned)units), dim3(kSegThreads), smem, st, p, kmap, vmap) != cudaSuccess) return MAMBA_ECUDA;
    }
    auto kern = k_la_chain<P, N, F32S>;
    constexpr size_t smem = sizeof(ChainSmem<P, N, F32S>) + 1024;
    static_assert(smem <= 232448, "shared memory of a block");
    if (!ready(reinterpret_cast<const void *>(kern), smem, kRegs)) return MAMBA_ECUDA;
    const dim3 grid((unsigned)(units < kSMs ? units : kSMs));
    if (launch_pdl(kern, grid, dim3(kThreads), smem, st, p, qmap, kmap, vmap, ymap) != cudaSuccess) return MAMBA_ECUDA;
    return launch_status();
}

template <bool F32S>
int dispatch(const ScanParams &p, int P, int N, cudaStream_t st) {
    if (P == 128) return launch<128, 128, F32S>(p, st);
    return N == 128 ? launch<64, 128, F32S>(p, st) : launch<64, 64, F32S>(p, st);
}

}  // namespace

bool chunked_eligible(const mamba_layer_desc *d) {
    return d->act_dtype == MAMBA_BF16 && (d->head_dim == 64 || d->head_dim == 128);  // (of the compiled shapes)
}

// Sequences are cut where twice their heads are no more than the SMs: into as many segments as make one block an SM, at least 4
// chunks each (what a segment adds to the state costs about half of its pass).  The host knows how many tokens and sequences there
// are (those of padding among them), not a sequence's length: with more than 152 / (2 H) sequences a long prompt among short ones
// is not cut (8192 tokens of 32 heads beside two sequences of 64 tokens 200 us, alone 105).
constexpr int kLeastChunks = 4;
int64_t spare_blocks(int H, int nseq) {  // segments that sequences are cut into, but for one each; 0: they are not
    const int64_t blocks = kSMs / H;
    return nseq == 0 || blocks < 2 * (int64_t)nseq ? 0 : blocks - nseq / 2;
}
int chunked_segment_tokens(int H, int T, int nseq) {
    const int64_t chunks = ((int64_t)T + C - 1) / C, spare = spare_blocks(H, nseq);
    if (spare == 0) return kWhole;
    const int64_t even = (chunks + spare - 1) / spare, per = even < kLeastChunks ? kLeastChunks : even;
    return per < chunks ? (int)(per * C) : kWhole;
}
// Segments make T / (per C) + nseq, and per is at least chunks / spare and kLeastChunks whatever T.
int64_t chunked_most_segments(int H, int T, int nseq) {
    const int64_t spare = spare_blocks(H, nseq), least = T / (kLeastChunks * C);
    return (spare < least ? spare : least) + nseq;
}

size_t chunked_workspace_bytes(const mamba_layer_desc *d, int64_t max_segs, int nseq) {
    return max_segs == nseq ? 0 : (size_t)(max_segs + nseq) * d->nheads * 128 * d->head_dim * sizeof(float);
}

int chunked_launch(const ScanParams &p, const mamba_layer_desc *d, cudaStream_t st) {
    return d->state_dtype == MAMBA_F32 ? dispatch<true>(p, d->head_dim, d->d_state, st)
                                       : dispatch<false>(p, d->head_dim, d->d_state, st);
}

}  // namespace la
}  // namespace ms
