#include "la_scan.h"
namespace ms {
namespace la {
bool chunked_eligible(const mamba_layer_desc *d) { return false; }
int chunked_segment_tokens(int H, int T, int nseq) { return 1 << 30; }
size_t chunked_workspace_bytes(const mamba_layer_desc *d, int64_t max_segs, int nseq) { return 0; }
int chunked_launch(const ScanParams &p, const mamba_layer_desc *d, cudaStream_t stream) { return MAMBA_EUNSUPPORTED; }
}  // namespace la
}  // namespace ms
