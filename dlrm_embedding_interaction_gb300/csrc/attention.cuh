// What the attention kernels share: which events a row sees, where a CTA's
// work lies in a ragged batch, and the fragments of the warp-level MMA.
#pragma once

#include "history.cuh"

namespace dlrm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// m16n8k16, f16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same, c = A B (+ c with `add`, a constant).
__device__ __forceinline__ void mma_f16_from(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1, bool add) {
  if (add) {
    mma_f16(c, a, b0, b1);
    return;
  }
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// m16n8k8, tf32 operands, fp32 sums.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// The events that the row at position pos sees: [0, end) less the gap
// [gap0, gap1) between the sinks and the window.
struct Visible {
  int end, gap0, gap1;
};
__device__ __forceinline__ Visible visible(int pos, int len, int window, int sinks) {
  Visible v;
  v.end = max(min(len, pos + 1), 0);
  v.gap0 = v.gap1 = 0;
  if (window > 0) {
    // (a row before the first event, of more queries than events, has no gap, and its
    // window may begin below -2^31)
    v.gap1 = max(max(pos, 0) - window + 1, 0);
    v.gap0 = min(sinks, v.gap1);
  }
  return v;
}
__device__ __forceinline__ bool sees(const Visible& v, int t) {
  return t < v.end && (t < v.gap0 || t >= v.gap1);
}
// Any event at all: a row without weights is zeros if it sees none, else 0 / 0 (all its
// scores are -infinity).
__device__ __forceinline__ bool sees_any(const Visible& v) {
  return v.end > 0 && (v.gap0 > 0 || v.gap1 < v.end);
}

// Finds where a CTA's work lies: request b has units(b) >= 0 units, and the
// CTA wants the request that holds unit `target` of all of them, or wants the
// total (target < 0). Block-wide; every thread gets the answer. `shared` has
// 40 int64.
template <int THREADS, class F>
__device__ __forceinline__ void locate(int batch, const F& units, int64_t target, int64_t* shared,
                                       int& request, int64_t& first, int64_t& total) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  constexpr int kWarps = THREADS / kWarp;
  const int per = (batch + THREADS - 1) / THREADS;
  const int b0 = min(batch, static_cast<int>(threadIdx.x) * per), b1 = min(batch, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += units(b);
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < kWarp; d *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == kWarp - 1) shared[warp] = inc;
  if (threadIdx.x == 0) {
    shared[36] = batch;
    shared[37] = 0;
  }
  __syncthreads();
  int64_t at = inc - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t s = shared[w];
    at += w < warp ? s : 0;
    total += s;
  }
  if (target >= 0 && target >= at && target < at + mine) {
    for (int b = b0; b < b1; ++b) {
      const int64_t n = units(b);
      if (target < at + n) {
        shared[36] = b;
        shared[37] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  request = static_cast<int>(shared[36]);
  first = shared[37];
}

// Sum of two counts, INT_MAX from there on.
__device__ __forceinline__ int add_counts(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7fffffffu));
}

// Cuts a batch's units evenly over the CTAs: request b has units(span(b)) >= 0
// of them, fewer than 2^31 in all, in pieces(span) pieces, `most` at most in all. (Starts
// that decrease can claim rows many times over and make more of either: then nothing is
// done.) CTA c of up to
// gridDim.x takes [cut(c), cut(c + 1)): `least` units at least, or about a piece,
// because a piece that is cut in many parts takes long to join. Block-wide; the spans and first units of the requests
// that hold both cuts come back in shared memory (the last request's where the
// cut is the total).
struct Cuts {
  int total, ctas, each, extra;                  // the first `extra` CTAs take each + 1
  __device__ __forceinline__ void set(int n, int pieces, int least) {
    total = n;
    ctas = min(static_cast<int>(gridDim.x), min(n, max(n / least, pieces)));
    each = ctas > 0 ? n / ctas : 0;
    extra = n - each * ctas;
  }
  __device__ __forceinline__ int cut(int c) const {
    c = min(c, ctas);
    return c * each + min(c, extra);
  }
  __device__ __forceinline__ int owner(int unit) const {
    const int long_ones = extra * (each + 1);
    return unit < long_ones ? unit / (each + 1) : extra + (unit - long_ones) / each;
  }
};
template <class Span>
struct Found {
  int request[2], first[2];
  Span span[2];
};
// sums: two ints a warp.
template <int THREADS, class Span, class S, class U, class P>
__device__ __forceinline__ Cuts locate_cuts(int batch, int least, int most, const S& span,
                                            const U& units, const P& pieces, int* sums,
                                            Found<Span>& found) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  constexpr int kWarps = THREADS / kWarp;
  const int per = (batch + THREADS - 1) / THREADS;
  const int b0 = min(batch, static_cast<int>(threadIdx.x) * per), b1 = min(batch, b0 + per);
  unsigned mine = 0;
  int parts = 0;
  Span s{};
  for (int b = b0; b < b1; ++b) {
    s = span(b);
    mine += units(s);
    parts = add_counts(parts, pieces(s));
  }
  // of a warp: 2^31 and more stay that
  const int high = __reduce_add_sync(0xffffffffu, parts >> 16);
  parts = add_counts(min(high, 0x7fff) << 16, __reduce_add_sync(0xffffffffu, parts & 0xffff));
  unsigned inc = mine;
#pragma unroll
  for (int d = 1; d < kWarp; d *= 2) {
    const unsigned v = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += v;
  }
  if (lane == kWarp - 1) {
    sums[warp] = inc;
    sums[kWarps + warp] = parts;
  }
  __syncthreads();
  unsigned before = inc - mine, sum = 0;
  int all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const unsigned x = sums[w];
    before += w < warp ? x : 0;
    sum += x;
    all = add_counts(all, sums[kWarps + w]);
  }
  const int at = static_cast<int>(before), total = all > most ? 0 : static_cast<int>(sum);
  Cuts cuts;
  cuts.set(total, all, least);
  for (int i = 0; i < 2; ++i) {
    const int target = min(cuts.cut(blockIdx.x + i), total - 1);
    if (target < at || target >= at + static_cast<int>(mine)) continue;
    int here = at;
    for (int b = b0; b < b1; ++b) {
      if (per > 1) s = span(b);
      const int n = units(s);
      if (target < here + n) {
        found.request[i] = b;
        found.first[i] = here;
        found.span[i] = s;
        break;
      }
      here += n;
    }
  }
  __syncthreads();
  return cuts;
}

}  // namespace dlrm
