// gdn_scan_tc.h -- internal interface of the chunked gated delta rule on the tensor cores.
#pragma once

#include "gdn_scan.h"

namespace ms {
namespace gdn {

// Whether the layer runs in chunks: bf16 activations and state, head_dim 64 or 128,
// d_state 128.
bool chunked_eligible(const mamba_layer_desc *d);
// Workspace past the plan.
size_t chunked_workspace_bytes(const mamba_layer_desc *d, int T, int nseq);
// Launches the chunked form after the plan; MAMBA_OK or a negative status.
int chunked_launch(const ScanParams &p, int head_dim, cudaStream_t stream);

}  // namespace gdn
}  // namespace ms
