// la_scan.h -- internal interface between the linear attention scan's paths.
#pragma once

#include "la.cuh"

namespace ms {
namespace la {

constexpr int kChunk = 128;  // tokens of one chunk of the chunked form
// Tokens of a segment where sequences are not cut, and the most of a call: a whole chunk below 2^31, since loops step that far past
// the last token.
constexpr int kWhole = 0x7fffff80;

// A run of whole chunks of a sequence (the sequence's last one ends with it), worked on from start to end by one block a head: all
// that its block has to know, in one load.
struct __align__(16) Segment {
    int32_t seq, index, last;  // of which sequence, which one of it, and the sequence's last one's index
    int32_t entry;             // the sequence's first entry in the workspace
    int32_t t0, len;           // first token, tokens
    int32_t slot;              // the sequence's
    int32_t seeded;            // whether the sequence starts from its slot's state
};

struct ScanParams {
    void *pool;
    int64_t stride, num_slots;  // elements
    const int32_t *cu, *slot;
    const uint8_t *has_init;
    const int32_t *ckpt_slots;
    int max_ckpt, ckpt_interval;
    int nseq, T, H, G, HG;
    const void *v, *k, *q;
    int64_t vs, ks, qs;  // token strides, elements
    const float *log_decay;
    float scale;
    void *y;
    int32_t *err;
    int seg_tokens;  // tokens of a whole segment, a multiple of kChunk
    int max_segs;    // segments of the batch, at most
    int32_t *meta;   // workspace: [segments, units given out past the first of each block, pad x2, Segment[max_segs]]
    float *ws;       // workspace of the chunked form, past meta
};

// Segments of a batch, at most: a sequence's last one, and one for each whole one that more tokens follow.
__host__ __device__ inline int64_t scan_max_segments(int T, int nseq, int seg_tokens) {
    return (int64_t)((T > 0 ? T - 1 : 0) / seg_tokens) + nseq;
}
inline size_t scan_meta_bytes(int64_t max_segs) {
    return ((size_t)(4 * sizeof(int32_t)) + (size_t)max_segs * sizeof(Segment) + 1023) / 1024 * 1024;
}
__device__ __forceinline__ Segment *meta_segments(const ScanParams &p) { return reinterpret_cast<Segment *>(p.meta + 4); }

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

// Whether a layer of a compiled shape runs in chunks: bf16 activations, head_dim 64 or 128.
bool chunked_eligible(const mamba_layer_desc *d);
// Tokens of a segment of the chunked form for a batch of these sizes.
int chunked_segment_tokens(int H, int T, int nseq);
// The most segments of a batch of T tokens or fewer.
int64_t chunked_most_segments(int H, int T, int nseq);
// Workspace past the plan.
size_t chunked_workspace_bytes(const mamba_layer_desc *d, int64_t max_segs, int nseq);
// Launches the chunked form after the plan; MAMBA_OK or a negative status.
int chunked_launch(const ScanParams &p, const mamba_layer_desc *d, cudaStream_t stream);

}  // namespace la
}  // namespace ms
