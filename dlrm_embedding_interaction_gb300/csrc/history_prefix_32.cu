// history_prefix_attention's kernels for head_dim 32.
#include "history_prefix.cuh"

namespace dlrm {
namespace prefix {
cudaError_t launch_32(Params& p, cudaStream_t stream) { return launch_d<32>(p, stream); }
}  // namespace prefix
}  // namespace dlrm
