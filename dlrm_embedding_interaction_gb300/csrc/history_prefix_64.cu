// history_prefix_attention's kernels for head_dim 64.
#include "history_prefix.cuh"

namespace dlrm {
namespace prefix {
cudaError_t launch_64(Params& p, cudaStream_t stream) { return launch_d<64>(p, stream); }
}  // namespace prefix
}  // namespace dlrm
