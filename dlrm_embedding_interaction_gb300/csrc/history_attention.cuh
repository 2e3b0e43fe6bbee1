// What the kernels of attention over cached histories share
// (history_attention.cu, history_prefix.cu): queries as loaded, the layout of a block
// of 32 events in shared memory, and a row from the definition.
#pragma once

#include "attention.cuh"

namespace dlrm {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * kWarp;
constexpr int kBlock = 32;                       // events of a warp's step

// Four consecutive query elements.
template <int DT>
__device__ __forceinline__ void load_four(float (&x)[4], const void* q, int64_t at, int vec) {
  if (vec) {
    if (DT == DLRM_DTYPE_FP32) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(q) + at));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at));
      if (DT == DLRM_DTYPE_BF16) {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
      } else {
        const float2 a = f16x2_to_float2(v.x), b = f16x2_to_float2(v.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = load_element<DT>(q, at + e);
  }
}

// Element of a thread's key or query word: part j, step ks, pair element e.
template <int D>
__device__ __forceinline__ int key_element(int c, int word) {
  if (D == 32) return 8 * c + 4 * word;
  return 64 * (word / 4) + 16 * c + 4 * (word % 4);
}

// One row from the definition, event by event, for a row whose output is not
// finite (0 * NaN of a masked event's value must not reach it), or that sees
// events but found no weights: query head hq at q_at, kv head `head` of the slot, the
// events in v. One CTA of kThreads, every thread.
template <int DT>
__device__ __noinline__ void careful_row(const dlrm_history_t& h, const dlrm_attention_t& a, int slot,
                                         const Visible& v, int head, int64_t q_at, int64_t o_at,
                                         int64_t lse_at, float* sm) {
  const int G = h.page_tokens, D = h.head_dim, M = h.max_pages, H = h.n_heads;
  const int32_t* row_pages = h.table + static_cast<int64_t>(slot) * M;
  float* prob = sm;                               // one per thread
  float* red = sm + kThreads;
  auto code = [](uint8_t c) { return f16x2_to_float2(e4m3x2_to_f16x2(c)).x; };
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  bool any = false;                               // there are events to see
  const int d = threadIdx.x;
  for (int pass = 0; pass < 2; ++pass) {
    for (int t0 = 0; t0 < v.end; t0 += kThreads) {
      const int t = t0 + static_cast<int>(threadIdx.x);
      float x = -INFINITY;
      bool there = false;
      if (t < v.end && sees(v, t)) {
        const int page = row_pages[t / G];
        if (page >= 0 && page < h.n_pages) {
          there = true;
          const int64_t place = static_cast<int64_t>(page) * H + head;
          const uint8_t* k = h.k_codes + (place * G + t % G) * D;
          float dot = 0.f;
          for (int e = 0; e < D; ++e) dot = fmaf(load_element<DT>(a.q, q_at + e), code(k[e]), dot);
          x = dot * (h.k_scales[place] * a.scale * kLog2e);
        }
      }
      if (pass == 0) {
        top = (x > top || x != x) ? x : top;      // a NaN stays
      } else {
        __syncthreads();
        prob[threadIdx.x] = there ? exp2f(x - top) : -1.f;
        __syncthreads();
        const int n = min(kThreads, v.end - t0);
        for (int u = 0; u < n; ++u) {
          const float pr = prob[u];
          if (pr == -1.f) continue;
          any = true;
          sum += pr;
          if (d < D) {
            const int page = row_pages[(t0 + u) / G];
            const int64_t place = static_cast<int64_t>(page) * H + head;
            acc = fmaf(pr * h.v_scales[place], code(h.v_codes[(place * G + (t0 + u) % G) * D + d]), acc);
          }
        }
      }
    }
    if (pass == 0) {
      __syncthreads();
      red[threadIdx.x] = top;
      __syncthreads();
      for (int u = 0; u < kThreads; ++u) {
        const float y = red[u];
        top = (y > top || y != y) ? y : top;
      }
      if (top == -INFINITY) top = 0.f;
    }
  }
  if (d < D) store_element<DT>(a.out, o_at + d, any ? acc / sum : 0.f);
  if (d == 0 && a.lse) a.lse[lse_at] = any ? top * kLn2 + logf(sum) : -INFINITY;
  __syncthreads();
}

// Offset of 16-byte chunk `ch` of event t in a block of keys or values. Reads:
// keys, 8 events x 64 bytes; values, 4 events (t / 2 = 0..3 mod 4) x a few chunks.
template <int D>
__device__ __forceinline__ int key_offset(int t, int ch) {
  return D == 128 ? t * 128 + ((ch ^ ((t & 1) << 2)) << 4) : t * D + (ch << 4);
}
template <int D>
__device__ __forceinline__ int value_offset(int t, int ch) {
  if (D == 128) return t * 128 + ((ch ^ (((t >> 1) & 3) << 1)) << 4);
  if (D == 64) return (t >> 1) * 128 + ((((t & 1) * 4 + ch) ^ (((t >> 1) & 3) << 1)) << 4);
  return (t >> 2) * 128 + ((((t & 3) * 2 + ch) ^ (((t >> 2) & 1) << 1)) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

}  // namespace dlrm
