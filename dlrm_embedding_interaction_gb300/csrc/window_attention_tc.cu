// window_attention on the tensor cores: bf16 and fp16 rows that TMA can read
// (attention_tc.cuh; window_attention.cu takes every other call).
//
// What bounds it: the softmax warps. A step of 128 rows x 64 events takes a warp
// about 2070 cycles, of which the exponentials are 700 and the rest latency, and
// two warps a sub-partition do not hide it; the tensor core is 47% busy at
// head_dim 128.
#include "attention_tc.cuh"

namespace dlrm {

bool window_tc_takes(const dlrm_attention_t& a) {
  return a.dtype != DLRM_DTYPE_FP32 && a.scale > 0.f && a.k_rows > 0 &&
         vector_rows(a.q, a.ld_q, a.ld_q_head, a.n_heads) &&
         tma_rows(a.k, a.ld_k, a.ld_k_head, a.n_kv_heads, a.head_dim) &&
         tma_rows(a.v, a.ld_v, a.ld_v_head, a.n_kv_heads, a.head_dim);
}

cudaError_t launch_window_attention_tc(const dlrm_attention_t& call, cudaStream_t stream) {
  dlrm_attention_t a = call;
  a.causal = 1;
  TcParams p{};
  alignas(64) CUtensorMap mq{}, mk, mv;
  if (!fill_params(p, mq, a) ||
      !encode_rows(&mk, a.k, a.k_rows, a.n_kv_heads, a.head_dim, a.ld_k, a.ld_k_head, a.dtype, kBox, 1) ||
      !encode_rows(&mv, a.v, a.k_rows, a.n_kv_heads, a.head_dim, a.ld_v, a.ld_v_head, a.dtype, kBox, 1))
    return cudaErrorInvalidValue;
  const int64_t units = (a.q_rows * p.w.group / kUnit + a.batch) * a.n_kv_heads;
  const int ctas = a.head_dim == 128 ? kCtas<128, false> : kCtas<64, false>;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, device_sm_count() * ctas));
  const bool bf16 = a.dtype == DLRM_DTYPE_BF16;
  if (a.head_dim == 32)
    return bf16 ? launch_tc<32, DLRM_DTYPE_BF16, false>(mq, mk, mv, p, grid, stream)
                : launch_tc<32, DLRM_DTYPE_FP16, false>(mq, mk, mv, p, grid, stream);
  if (a.head_dim == 64)
    return bf16 ? launch_tc<64, DLRM_DTYPE_BF16, false>(mq, mk, mv, p, grid, stream)
                : launch_tc<64, DLRM_DTYPE_FP16, false>(mq, mk, mv, p, grid, stream);
  return bf16 ? launch_tc<128, DLRM_DTYPE_BF16, false>(mq, mk, mv, p, grid, stream)
              : launch_tc<128, DLRM_DTYPE_FP16, false>(mq, mk, mv, p, grid, stream);
}

}  // namespace dlrm
