// window_attention on the tensor cores: bf16 and fp16 rows that TMA can read
// (attention_tc.cuh; window_attention.cu takes every other call).
//
#include "attention_tc.cuh"

namespace dlrm {

// From this many rows of a request on average this kernel is faster than
// window_attention.cu's up to head_dim 64; at 128 it always is. us in bf16, 4 heads,
// this kernel against that one, head_dim 32 (64, 128):
//   32 users x 64 events: 5.2 against 6.1 (5.7 against 11, 6.3 against 20)
//   32 users x 16 events: 4.9 against 4.2 (5.3 against 4.9, 6.1 against 7.9)
//   256 users x 64 events: 13 against 14 (14 against 30, 25 against 75)
//   256 users x 8 events: 12 against 8.1 (13 against 9.7, 24 against 23)
//   64 users x 512 events, window 64: 23 against 39 (24 against 66, 37 against 203)
constexpr int kFewRows = 32;

bool window_tc_takes(const dlrm_attention_t& a) {
  const int64_t rows = a.q_rows * (a.n_heads / a.n_kv_heads);
  return a.dtype != DLRM_DTYPE_FP32 && a.scale > 0.f && a.k_rows > 0 &&
         (a.head_dim == 128 || rows >= static_cast<int64_t>(a.batch) * kFewRows) &&
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
  const int ctas = a.head_dim == 128 ? kCtas<128, false> : kCtas<64, false>;
  const unsigned grid = static_cast<unsigned>(std::min(p.most, device_sm_count() * ctas));
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
