// history_attention on the tensor cores: bf16 queries, many rows a request
// (attention_tc.cuh; history_attention.cu takes every other call).
#include "attention_tc.cuh"

namespace dlrm {

// Rows of a request and kv head, on average, from which this kernel is taken.
constexpr int kManyRows = 64;

bool history_tc_takes(const dlrm_history_t& h, const dlrm_attention_t& a) {
  return a.dtype == DLRM_DTYPE_BF16 && a.scale > 0.f &&
         vector_rows(a.q, a.ld_q, a.ld_q_head, a.n_heads) &&
         a.q_rows * (a.n_heads / h.n_heads) >= static_cast<int64_t>(a.batch) * kManyRows;
}

cudaError_t launch_history_attention_tc(const dlrm_history_t& h, const dlrm_attention_t& call,
                                        int32_t* counters, float* partials, cudaStream_t stream) {
  dlrm_attention_t a = call;
  a.n_kv_heads = h.n_heads;
  a.head_dim = h.head_dim;
  TcParams p{};
  alignas(64) CUtensorMap mq{};
  if (!fill_params(p, mq, a)) return cudaErrorInvalidValue;
  p.h = h;
  p.counters = counters;
  p.partials = partials;
  const unsigned grid = static_cast<unsigned>(std::min(device_sm_count(), kAttnTcCtas));
  if (h.head_dim == 32) return launch_tc<32, DLRM_DTYPE_BF16, true>(mq, mq, mq, p, grid, stream);
  if (h.head_dim == 64) return launch_tc<64, DLRM_DTYPE_BF16, true>(mq, mq, mq, p, grid, stream);
  return launch_tc<128, DLRM_DTYPE_BF16, true>(mq, mq, mq, p, grid, stream);
}

}  // namespace dlrm
