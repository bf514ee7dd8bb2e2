// gdn_scan.h -- internal interface between the gated delta rule's scan paths.
#pragma once

#include "gdn.cuh"

namespace ms {
namespace gdn {

constexpr int kChunk = 64;  // tokens of one chunk of the chunked form

struct ScanParams {
    void *pool;
    int64_t stride, num_slots;  // elements
    const int32_t *cu, *slot;
    const uint8_t *has_init;
    const int32_t *ckpt_slots;
    int max_ckpt, ckpt_interval;
    int nseq, T, H, G, HG;
    const void *v, *k, *q, *dt, *beta;
    Gates gates;
    void *y;
    int32_t *err;
    int32_t *meta;  // workspace: [valid, chunks, pad x2, (first token, tokens) of each chunk, order[nseq], first chunk of each
                    // sequence[nseq + 1]]
    unsigned char *ws;  // workspace of the chunked form, past meta
};

// Chunks of the whole batch, at most.
__host__ __device__ inline int64_t scan_max_chunks(int T, int nseq) { return (int64_t)T / kChunk + nseq; }
inline size_t scan_meta_bytes(int T, int nseq) {
    return ((size_t)(5 + 2 * (int64_t)nseq + 2 * scan_max_chunks(T, nseq)) * sizeof(int32_t) + 1023) / 1024 * 1024;
}
__device__ __forceinline__ int2 *meta_table(const ScanParams &p) { return reinterpret_cast<int2 *>(p.meta + 4); }
__device__ __forceinline__ int32_t *meta_order(const ScanParams &p) { return p.meta + 4 + 2 * scan_max_chunks(p.T, p.nseq); }
__device__ __forceinline__ int32_t *meta_chunks(const ScanParams &p) { return meta_order(p) + p.nseq; }

// Slot of the checkpoint due after `done` tokens of sequence s, or -1 (an id outside the pool is
// flagged by the one thread that passes flag).
__device__ __forceinline__ int32_t ckpt_slot(const ScanParams &p, int s, int done, bool flag) {
    if (!p.ckpt_slots || done % p.ckpt_interval != 0) return -1;
    const int m = done / p.ckpt_interval;
    if (m < 1 || m > p.max_ckpt) return -1;
    const int32_t cs = p.ckpt_slots[(int64_t)s * p.max_ckpt + m - 1];
    if (cs < -1 || cs >= p.num_slots) {
        if (flag) flag_error(p.err, MAMBA_ERR_SLOT_RANGE);
        return -1;
    }
    return cs;
}

}  // namespace gdn
}  // namespace ms
