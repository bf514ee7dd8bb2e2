// int8_entry.h -- layout of one entry of the int8 checkpoint store (host side).
#pragma once

#include "common.cuh"

namespace ms {

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

struct EntryLayout {
    size_t q, scales, conv, total;  // section offsets and entry size in bytes
};

inline EntryLayout entry_layout(const mamba_layer_desc *d) {
    EntryLayout L;
    const size_t q = (size_t)d->nheads * d->head_dim * d->d_state;
    const size_t sc = (size_t)d->nheads * d->d_state * sizeof(float);
    const size_t cv = (size_t)mamba_conv_dim(d) * (d->conv_kernel - 1 + d->num_spec) * dtype_bytes(d->conv_dtype);
    L.q = 0;
    L.scales = align256(q);
    L.conv = L.scales + align256(sc);
    L.total = L.conv + align256(cv);
    return L;
}

}  // namespace ms
