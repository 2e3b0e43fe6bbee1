// history_attention on the tensor cores: bf16 queries, many rows a request
// (attention_tc.cuh; history_attention.cu takes every other call).
//
// (A code times its page's scale is exact in bf16; fp16 has not the exponents.) Weights
// have 8 bits here and 11 in history_attention.cu, so a bf16 query's rounding depends on the
// rows of its call: an error of 1.9e-3 of the values against 1.6e-3, of which the output's
// own rounding is 1.6e-3.
// What bounds it: the softmax, and with few units the time of one key tile after
// another.
#include "attention_tc.cuh"

namespace dlrm {

// From this many rows of a request and kv head on average, and of all together,
// this kernel is faster than history_attention.cu's. us at head_dim 64 (128), two
// kv heads, this kernel against that one:
//   64 users x 1024 events, 64 rows each: 23 against 29 (35 against 52);
//     32 rows: 23 against 24 (35 against 34)
//   16 users x 4096 events, 128 rows: 33 against 39 (47 against 61);
//     64 rows (2048 in all): 32 against 28 (46 against 43)
//   16 users x 256 events, 128 rows: 10.9 against 10.4 (15.2 against 14.6)
//   1 user x 4096 events, 1024 rows (2048 in all): 35 against 28 (50 against 43)
constexpr int kManyRows = 64, kManyInAll = 4096;

bool history_tc_takes(const dlrm_history_t& h, const dlrm_attention_t& a) {
  const int64_t rows = a.q_rows * (a.n_heads / h.n_heads);
  return a.dtype == DLRM_DTYPE_BF16 && a.scale > 0.f &&
         vector_rows(a.q, a.ld_q, a.ld_q_head, a.n_heads) &&
         rows >= static_cast<int64_t>(a.batch) * kManyRows && rows * h.n_heads >= kManyInAll;
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
