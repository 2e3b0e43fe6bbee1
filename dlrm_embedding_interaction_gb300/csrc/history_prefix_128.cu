// history_prefix_attention's kernels for head_dim 128.
#include "history_prefix.cuh"

namespace dlrm {
namespace prefix {
cudaError_t launch_128(Params& p, cudaStream_t stream) { return launch_d<128>(p, stream); }
}  // namespace prefix
}  // namespace dlrm
