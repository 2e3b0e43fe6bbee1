// What the two kernels of window_attention share: a request's rows, and a row
// done from the definition. window_attention.cu takes any strides and types,
// window_attention_tc.cu (tcgen05) the bf16 and fp16 rows that TMA can read.
#pragma once

#include "attention.cuh"

namespace dlrm {

struct WindowParams {
  dlrm_attention_t a;
  int group;
  int vec;                                       // rows can be loaded 16 bytes at a time
};

struct WindowSpan {
  int q0, k0, rows, len, tiles;
};

__device__ __forceinline__ WindowSpan window_span(const WindowParams& p, int b, int tile_rows, bool report) {
  WindowSpan s;
  const int q0 = p.a.q_starts[b], q1 = p.a.q_starts[b + 1];
  const int k0 = p.a.k_starts[b], k1 = p.a.k_starts[b + 1];
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.a.q_rows || k0 < 0 || k1 < k0 || k1 > p.a.k_rows;
  if (bad && report) flag(p.a.err, DLRM_ERRBIT_OFFSETS);
  s.q0 = q0;
  s.k0 = k0;
  s.rows = bad ? 0 : (q1 - q0) * p.group;
  s.len = bad ? 0 : k1 - k0;
  s.tiles = (s.rows + tile_rows - 1) / tile_rows;
  return s;
}

// One row from the definition, event by event, by one warp: for a row whose
// output is not finite (0 * a masked event's infinity or NaN), or that sees events
// but found no weights (scores of -infinity).
template <int D, int DT>
__device__ __noinline__ void window_careful_row(const WindowParams& p, const WindowSpan& s, int head, int row) {
  const int lane = threadIdx.x % kWarp;
  const int i = row / p.group, hq = head * p.group + row % p.group;
  const Visible v = visible(s.len - s.rows / p.group + i, s.len, p.a.window, p.a.sinks);
  const int64_t q_at = (s.q0 + static_cast<int64_t>(i)) * p.a.ld_q + hq * p.a.ld_q_head;
  constexpr int N = D / kWarp;
  float q[N], acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = load_element<DT>(p.a.q, q_at + lane + 32 * e) * (p.a.scale * kLog2e);
    acc[e] = 0.f;
  }
  float top = -INFINITY, sum = 0.f;
  bool any = false;                               // there are events to see
  for (int t = 0; t < v.end; ++t) {
    if (!sees(v, t)) {
      t = v.gap1 - 1;
      continue;
    }
    const int64_t kt = s.k0 + static_cast<int64_t>(t);
    any = true;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e)
      x = fmaf(q[e], load_element<DT>(p.a.k, kt * p.a.ld_k + head * p.a.ld_k_head + lane + 32 * e), x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float m = (x > top || x != x) ? x : top;              // a NaN stays
    const float base = m == -INFINITY ? 0.f : m;
    const float f = exp2f(top - base), w = exp2f(x - base);
    top = m;
    sum = fmaf(sum, f, w);
    if (sum != sum) {                                           // so is every output, whatever follows
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = sum;
      break;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      acc[e] = fmaf(acc[e], f, w * load_element<DT>(p.a.v, kt * p.a.ld_v + head * p.a.ld_v_head + lane + 32 * e));
  }
  const int64_t o = (s.q0 + static_cast<int64_t>(i)) * p.a.ld_out + hq * p.a.ld_out_head;
#pragma unroll
  for (int e = 0; e < N; ++e) store_element<DT>(p.a.out, o + lane + 32 * e, any ? acc[e] / sum : 0.f);
  if (lane == 0 && p.a.lse)
    p.a.lse[(s.q0 + static_cast<int64_t>(i)) * p.a.n_heads + hq] =
        any ? (top == -INFINITY ? 0.f : top) * kLn2 + logf(sum) : -INFINITY;
}

// The tcgen05 kernel: whether it takes this call, and its launch.
bool window_tc_takes(const dlrm_attention_t& a);
cudaError_t launch_window_attention_tc(const dlrm_attention_t& a, cudaStream_t stream);

}  // namespace dlrm
