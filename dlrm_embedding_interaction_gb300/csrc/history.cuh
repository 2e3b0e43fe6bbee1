// Event histories: what the page operators (history_pages.cu), the attention
// over a pool (history_attention.cu) and the windowed attention over plain
// rows (window_attention.cu) share. include/dlrm.h defines the pool, the
// codes and the operators.
#pragma once

#include "common.cuh"

namespace dlrm {

// Codes: e4m3 times a power of two. Limits of the exponent, so that
// products of a code, a scale and a query stay far inside fp32's range.
constexpr int kScaleExpMax = 60;

// The least e in [-60, 60] with amax <= 448 * 2^e, amax finite and >= 0:
// 448 = 1.75 * 2^8, so e is amax's exponent less 8, plus one past 1.75.
__host__ __device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 135 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return e < -kScaleExpMax ? -kScaleExpMax : e > kScaleExpMax ? kScaleExpMax : e;
}

__device__ __forceinline__ float pow2f(int e) {   // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two e4m3 codes (low byte first) as two halves: exact, NaN included.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(two_codes));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(four_codes));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_lo_to_f16x2(uint32_t four_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(four_codes));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Rounds to nearest even; past 448 and infinities become +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Weights that are rounded to f16 are made larger by a power of two (2^kLift of the
// row's largest), as f16 has no normal numbers below 2^-14: the weights of a long history's
// many events beside one that outweighs them would lose their bits there, or vanish. The
// sums are those of the larger weights. A row's reference is a whole number, so that its
// difference to kLift has no rounding.
constexpr int kLift = 15;

template <int DT>
__device__ __forceinline__ float load_element(const void* p, int64_t i) {
  if (DT == DLRM_DTYPE_FP32) return static_cast<const float*>(p)[i];
  const uint16_t u = static_cast<const uint16_t*>(p)[i];
  if (DT == DLRM_DTYPE_BF16) return __uint_as_float(static_cast<uint32_t>(u) << 16);
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(u));
  return f;
}

template <int DT>
__device__ __forceinline__ void store_element(void* p, int64_t i, float x) {
  if (DT == DLRM_DTYPE_FP32) {
    static_cast<float*>(p)[i] = x;
  } else if (DT == DLRM_DTYPE_BF16) {
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16(x, 0.f));
  } else {
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_f16x2(x, 0.f));
  }
}

inline int dtype_bytes(int dtype) { return dtype == DLRM_DTYPE_FP32 ? 4 : 2; }

__device__ __forceinline__ void flag(int32_t* err, uint32_t bits) {
  if (err) atomicOr(reinterpret_cast<unsigned int*>(err), bits);
}

__device__ __forceinline__ bool finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
}

// The parts of a pool's scratch (byte offsets; every part 16-byte aligned).
struct HistoryWork {
  int64_t head, mark_slot, mark_page, request, items, stash, remap, holes, movers, tiles, counters,
      partials, total;
};

// CTAs of one attention launch that can hold an unfinished row tile, and the
// floats of one (kRows rows of D sums, a maximum and a sum, at D = 128).
constexpr int kAttnMaxCtas = 152 * 8;
constexpr int kAttnRows = 16;
constexpr int kAttnPartial = kAttnRows * (128 + 2);
// The same of the tensor-core kernel: a CTA per SM, units of 256 rows, a counter
// for each of 8 warps.
constexpr int kAttnTcCtas = 152;
constexpr int kAttnTcPartial = 256 * (128 + 2);
static_assert(kAttnTcCtas * 8 <= kAttnMaxCtas, "counters");

inline HistoryWork history_work(const dlrm_history_t& h) {
  HistoryWork w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 16);
    return here;
  };
  const int64_t slots = h.n_slots, pages = h.n_pages, entries = slots * h.max_pages;
  w.head = take(64);
  w.mark_slot = take(4 * slots);
  w.mark_page = take(4 * pages);
  w.request = take(32 * slots);
  // items of one call: copies (at most every page, as each is a new one) or
  // touched pages (at most the new pages and one old page a slot)
  w.items = take(8 * (pages + slots));
  w.stash = take(4 * entries);
  w.remap = take(4 * pages);
  w.holes = take(4 * pages);
  w.movers = take(4 * pages);
  w.tiles = take(8 * (pages / 1024 + 1));
  w.counters = take(4 * kAttnMaxCtas);
  w.partials = take(int64_t(4) * 2 * std::max(kAttnMaxCtas * kAttnPartial, kAttnTcCtas * kAttnTcPartial));
  w.total = at;
  return w;
}

template <class T>
inline T* work_part(const dlrm_history_t& h, int64_t offset) {
  return reinterpret_cast<T*>(static_cast<char*>(h.work) + offset);
}

cudaError_t launch_history_reset(const dlrm_history_t& h, cudaStream_t stream);
cudaError_t launch_history_append(const dlrm_history_t& h, const int32_t* slots,
                                  const int32_t* starts, int batch, const void* k, int64_t ld_k,
                                  int64_t ld_k_head, const void* v, int64_t ld_v,
                                  int64_t ld_v_head, int64_t rows, int dtype, cudaStream_t stream);
cudaError_t launch_history_fork(const dlrm_history_t& h, const int32_t* src, const int32_t* dst,
                                int batch, bool share, cudaStream_t stream);
cudaError_t launch_history_free(const dlrm_history_t& h, const int32_t* slots, int batch,
                                int window, int sinks, cudaStream_t stream);
cudaError_t launch_history_compact(const dlrm_history_t& h, cudaStream_t stream);
cudaError_t launch_history_attention(const dlrm_history_t& h, const dlrm_attention_t& a,
                                     cudaStream_t stream);
bool history_tc_takes(const dlrm_history_t& h, const dlrm_attention_t& a);
cudaError_t launch_history_attention_tc(const dlrm_history_t& h, const dlrm_attention_t& a,
                                        int32_t* counters, float* partials, cudaStream_t stream);
cudaError_t launch_window_attention(const dlrm_attention_t& a, cudaStream_t stream);
WaitCfg attention_wait();                        // attention_test_stall's

}  // namespace dlrm
