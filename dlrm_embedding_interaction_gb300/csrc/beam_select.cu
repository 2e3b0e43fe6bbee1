// The best continuations of each group of beams (include/dlrm.h, beam_select): of all
// (row, token) pairs of a group, the `width` with the largest
//   score[row] + logit[row][token] - log sum over allowed t of exp(logit[row][t]).
//
// Large vocabularies take two launches. beam_scan_kernel reads the logits once, a CTA for
// each chunk of a row, and leaves the chunk's maximum, its sum of exponentials and a short
// list that holds the chunk's `width` largest logits (within a row their order is that of
// the scores). beam_join_kernel, a CTA a group, adds up the rows' sums and selects among
// the lists. Small vocabularies take one launch that does both, a CTA a group.
//
// Selection never sorts the data. The k-th largest of the maxima of k or more disjoint
// subsets (a thread's elements each) is a lower bound of the k-th largest element, found
// bit by bit with counting barriers; few elements reach it, and those are ranked by
// comparison with one another. Where many do (ties, adverse orders) the bound is bisected
// to the exact value, and ties to the exact index.
//
// The order hangs by differences of the rows' logarithms, so these are held more
// precisely than fp32: the sums' terms have rounding errors of their own (2^-23 each, not
// of one sign), their sums are exact to 2^-40 or so, and scores are compared in 64 bits.
#include <float.h>

#include "history.cuh"

namespace dlrm {

namespace {

constexpr int kScanThreads = 256;
constexpr int kJoinThreads = 512;
constexpr int kVectors = 4;                      // 16-byte vectors of a thread and tile
constexpr int kSubsets = 64;                     // widths up to here: one subset a thread will do
constexpr int kFinal = 2048;                     // candidates that are ranked at most
static_assert(kBeamMaxWidth <= kScanThreads && kBeamMaxWidth <= kFinal, "a subset for each place");

struct Part {                                    // of a chunk of a row
  float top;                                     // reference of the sum; -infinity: nothing allowed
  int32_t count;                                 // entries of its list
  double sum;                                    // of exp(logit - top)
};
struct Entry {
  float logit;
  int32_t token;
};
struct RowState {
  double lse;
  float offset;                                  // score - lse; -infinity: the row has no candidates
  int32_t pad;
};
static_assert(sizeof(Part) == 16 && sizeof(Entry) == 8 && sizeof(RowState) == 16, "scratch sizes");

struct Params {
  dlrm_beam_select_t a;
  int chunks;                                    // of a row
  int tiles;                                     // of a chunk
  int cap;                                       // entries of a list at most
  RowState* rows;
  Part* parts;
  Entry* entries;
};

// Floats as integers of the same order.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// The bound that a key stands for: at least the least finite number, as -infinity is none.
__device__ __forceinline__ float bound_of(uint32_t k) {
  return k <= key_of(-FLT_MAX) ? -FLT_MAX : of_key(k);
}

// exp(x - ref): log2(e) in two parts, the larger one rounded down so that an infinite
// difference stays one; rounding errors of the arguments then have no common sign.
__device__ __forceinline__ float exp_from(float x, float ref) {
  constexpr float kHigh = 1.44269490242004394531f, kLow = 1.38468919e-7f;
  const float d = x - ref;
  return exp2_approx(fmaf(d, kHigh, d * kLow));
}

// Largest key with kBits bits past the first that not all threads' keys have in common
// which k or more of the keys reach; a thread has N. Block-wide. red: 2 ints a warp.
template <int THREADS, int N>
__device__ __forceinline__ uint32_t block_bound(const uint32_t (&key)[N], int k, uint32_t* red) {
  constexpr int kBits = 12, kWarps = THREADS / kWarp;
  uint32_t hi = key[0], lo = key[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    hi = max(hi, key[i]);
    lo = min(lo, key[i]);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (threadIdx.x % kWarp == 0) {
    red[threadIdx.x / kWarp] = hi;
    red[kWarps + threadIdx.x / kWarp] = lo;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    hi = max(hi, red[w]);
    lo = min(lo, red[kWarps + w]);
  }
  __syncthreads();
  if (hi == lo) return hi;
  const int first = 31 - __clz(hi ^ lo);
  uint32_t bound = first == 31 ? 0u : hi & (0xffffffffu << (first + 1));
  for (int bit = first; bit >= max(first - kBits + 1, 0); --bit) {
    const uint32_t trial = bound | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __syncthreads_count(key[i] >= trial);
    if (n >= k) bound = trial;
  }
  return bound;
}

// ------------------------------------------------------------------ rows as loaded

// kVec consecutive logits (16 bytes) from element e0 of a row on, as words. A row may begin
// at any element: then two aligned vectors are shifted together. Aligned vectors that
// hold an element of the row are read whole.
template <int DT>
struct Row {
  static constexpr int kVec = DT == DLRM_DTYPE_FP32 ? 4 : 8;
  static constexpr int kBytes = DT == DLRM_DTYPE_FP32 ? 4 : 2;
};

template <int DT, bool ALIGNED>
__device__ __forceinline__ uint4 load_vector(const char* row, int64_t e0, int64_t n) {
  const char* at = row + e0 * Row<DT>::kBytes;
  if (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(at));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
  const uint4* base = reinterpret_cast<const uint4*>(at - off);
  const uint4 a = __ldg(base);
  uint4 b = make_uint4(0, 0, 0, 0);
  if (reinterpret_cast<const char*>(base + 1) < row + n * Row<DT>::kBytes) b = __ldg(base + 1);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int bits = (off & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}
// The same of the bytes that allow tokens: kVec of them.
template <int VEC, bool ALIGNED>
__device__ __forceinline__ uint2 load_allowed(const uint8_t* row, int64_t e0, int64_t n) {
  const uint8_t* at = row + e0;
  if (VEC == 4) {
    if (ALIGNED) return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(at)), 0);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 3);
    const uint32_t* base = reinterpret_cast<const uint32_t*>(at - off);
    const uint32_t a = __ldg(base);
    const uint32_t b = reinterpret_cast<const uint8_t*>(base + 1) < row + n ? __ldg(base + 1) : 0;
    return make_uint2(__funnelshift_r(a, b, off * 8), 0);
  }
  if (ALIGNED) return __ldg(reinterpret_cast<const uint2*>(at));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 7);
  const uint2* base = reinterpret_cast<const uint2*>(at - off);
  const uint2 a = __ldg(base);
  uint2 b = make_uint2(0, 0);
  if (reinterpret_cast<const uint8_t*>(base + 1) < row + n) b = __ldg(base + 1);
  uint32_t w[4] = {a.x, a.y, b.x, b.y};
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i] = w[i + 1];
  }
  const int bits = (off & 3) * 8;
  return make_uint2(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits));
}
// Element e of a vector, -infinity where it is not allowed.
template <int DT>
__device__ __forceinline__ float element_of(const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (DT == DLRM_DTYPE_FP32) return __uint_as_float(w[e]);
  const uint32_t x = w[e / 2];
  if (DT == DLRM_DTYPE_BF16) return __uint_as_float(e % 2 ? x & 0xffff0000u : x << 16);
  const float2 f = f16x2_to_float2(x);
  return e % 2 ? f.y : f.x;
}
__device__ __forceinline__ bool byte_of(const uint2& m, int e) {
  return ((e < 4 ? m.x : m.y) >> (8 * (e % 4)) & 0xff) != 0;
}

// ------------------------------------------------------------------ scan

// The `width` largest logits of [e0, e1) of a row, when the quick way found too many: the
// exact bound, then the exact index among its ties, by bisection. Every thread.
template <int DT>
__device__ __noinline__ int exact_chunk(const Params& p, int64_t row, int64_t e0, int64_t e1, Entry* list,
                                        int* counter) {
  const auto logit = [&](int64_t e) {
    const float x = load_element<DT>(p.a.logits, row * p.a.ld + e);
    return p.a.allowed && !p.a.allowed[row * p.a.ld_allowed + e] ? -INFINITY : x;
  };
  // (a NaN reaches no bound)
  const auto reach = [&](float bound, int64_t last) {   // logits above it, and those at it up to an index
    int n = 0;
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kScanThreads) {
      const float x = logit(e);
      n += x > bound || (x == bound && e <= last);
    }
    __syncthreads();
    if (threadIdx.x == 0) *counter = 0;
    __syncthreads();
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x % kWarp == 0) atomicAdd(counter, n);
    __syncthreads();
    return *counter;
  };
  uint32_t k = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = k | (1u << bit);
    const float x = of_key(trial);
    if (x == x && trial > key_of(-INFINITY) && reach(x, e1) >= p.a.width) k = trial;
    // (keys below -infinity's and above infinity's stand for NaN)
    if (trial <= key_of(-INFINITY)) k = trial;
  }
  const float bound = bound_of(k);
  int64_t lo = e0 - 1, hi = e1;                  // the last index whose tie is taken
  while (hi - lo > 1) {
    const int64_t mid = lo + (hi - lo) / 2;
    if (reach(bound, mid) >= p.a.width) hi = mid; else lo = mid;
  }
  __syncthreads();
  if (threadIdx.x == 0) *counter = 0;
  __syncthreads();
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kScanThreads) {
    const float x = logit(e);
    if (x > bound || (x == bound && e <= hi)) list[atomicAdd(counter, 1)] = Entry{x, static_cast<int>(e)};
  }
  __syncthreads();
  return *counter;
}

// Drops what is below the k-th largest of a list of n >= k entries (to 12 bits past what all
// have in common); returns how many stay. One warp.
__device__ __forceinline__ int tighten(Entry* list, int n, int k) {
  const int lane = threadIdx.x % kWarp;
  uint32_t hi = 0, lo = 0xffffffffu;
  for (int i = lane; i < n; i += kWarp) {
    const uint32_t x = key_of(list[i].logit);
    hi = max(hi, x);
    lo = min(lo, x);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (hi == lo) return n;
  const int first = 31 - __clz(hi ^ lo);
  uint32_t bound = first == 31 ? 0u : hi & (0xffffffffu << (first + 1));
  for (int bit = first; bit >= max(first - 11, 0); --bit) {
    const uint32_t trial = bound | (1u << bit);
    int c = 0;
    for (int i = lane; i < n; i += kWarp) c += key_of(list[i].logit) >= trial;
    if (__reduce_add_sync(0xffffffffu, c) >= k) bound = trial;
  }
  const float least = of_key(bound);
  int kept = 0;
  for (int i0 = 0; i0 < n; i0 += kWarp) {
    Entry x{};
    const bool in = i0 + lane < n;
    if (in) x = list[i0 + lane];
    const bool keep = in && x.logit >= least;
    const unsigned who = __ballot_sync(0xffffffffu, keep);
    if (keep) list[kept + __popc(who & ((1u << lane) - 1))] = x;
    kept += __popc(who);
    __syncwarp();
  }
  return kept;
}

template <int DT, bool MASK, bool ALIGNED>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ Params p) {
  constexpr int kVec = Row<DT>::kVec, kWarps = kScanThreads / kWarp;
  constexpr int kTile = kScanThreads * kVec * kVectors;
  extern __shared__ __align__(16) unsigned char smem[];
  Entry* list = reinterpret_cast<Entry*>(smem);
  __shared__ uint32_t red[2 * kWarps];
  __shared__ double sums[kWarps];
  __shared__ int count_s, other_s;
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp;
  const int64_t row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks, vocab = p.a.vocab;
  const int64_t e0 = chunk * p.tiles * kTile, e1 = min(vocab, e0 + static_cast<int64_t>(p.tiles) * kTile);
  const char* logits = static_cast<const char*>(p.a.logits) + row * p.a.ld * Row<DT>::kBytes;
  const uint8_t* allowed = MASK ? p.a.allowed + row * p.a.ld_allowed : nullptr;
  const int width = p.a.width;
  if (t == 0) count_s = 0;
  pdl_wait();
  pdl_trigger();

  uint4 raw[kVectors];
  uint2 may[kVectors];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      const int64_t e = at + (v * kScanThreads + t) * kVec;
      if (e < e1) {
        raw[v] = load_vector<DT, ALIGNED>(logits, e, vocab);
        if (MASK) may[v] = load_allowed<kVec, ALIGNED>(allowed, e, vocab);
      }
    }
  };
  load(e0);
  float ref = -INFINITY, sum = 0.f, rest = 0.f;   // the sum in two parts
  float bound = -FLT_MAX;
  bool many = false;                              // the list overflowed
  for (int64_t at = e0; at < e1; at += kTile) {
    float x[kVectors][kVec], top[kVectors];
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      const int64_t e = at + (v * kScanThreads + t) * kVec;
      top[v] = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        x[v][i] = element_of<DT>(raw[v], i);
        if (e + i >= e1 || (MASK && !byte_of(may[v], i))) x[v][i] = -INFINITY;
        top[v] = fmaxf(top[v], x[v][i]);
      }
    }
    if (at + kTile < e1) load(at + kTile);
    float most = top[0];
#pragma unroll
    for (int v = 1; v < kVectors; ++v) most = fmaxf(most, top[v]);
    if (at == e0) {
      // the bound; and one reference for all threads, so that sums need no factors
      uint32_t key;
      if (width <= kSubsets) {
        const uint32_t mine[1] = {key_of(most)};
        key = block_bound<kScanThreads>(mine, width, red);
      } else {
        uint32_t mine[kVectors];
#pragma unroll
        for (int v = 0; v < kVectors; ++v) mine[v] = key_of(top[v]);
        key = block_bound<kScanThreads>(mine, width, red);
      }
      bound = bound_of(key);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, key_of(most));
      if (lane == 0) red[warp] = hi;
      __syncthreads();
      uint32_t all = red[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) all = max(all, red[w]);
      ref = of_key(all);
    } else if (most > ref + 20.f) {
      const float f = exp_from(ref, most);
      sum *= f;
      rest *= f;
      ref = most;
    }
    const float base = ref == -INFINITY ? 0.f : ref;
    float part[kVectors];
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      part[v] = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) part[v] += exp_from(x[v][i], base);
    }
    // sum + rest, the rounding errors of sum in rest
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      const float s = sum + part[v], z = s - sum;
      rest += (sum - (s - z)) + (part[v] - z);
      sum = s;
    }
    if (!many && most >= bound) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        if (top[v] < bound) continue;
        const int64_t e = at + (v * kScanThreads + t) * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (x[v][i] >= bound) {
            const int place = atomicAdd(&count_s, 1);
            if (place < p.cap) list[place] = Entry{x[v][i], static_cast<int>(e + i)};
          }
      }
    }
    __syncthreads();
    const int count = count_s;
    many |= count > p.cap;
    if (!many && count > 2 * width + 32) {
      __syncthreads();                            // `count_s` is read
      if (warp == 0) {
        const int n = tighten(list, count, width);
        if (lane == 0) count_s = n;
      }
      __syncthreads();
      if (count_s > p.cap / 2) {
        many = true;                              // ties: the exact way, at the end
      } else {
        // the least that is left
        float least = INFINITY;
        for (int i = lane; i < count_s; i += kWarp) least = fminf(least, list[i].logit);
        bound = of_key(__reduce_min_sync(0xffffffffu, key_of(least)));
      }
    }
    __syncthreads();
  }
  // ---- the chunk's sum, in 64 bits
  const uint32_t hi = __reduce_max_sync(0xffffffffu, key_of(ref));
  __syncthreads();
  if (lane == 0) red[warp] = hi;
  __syncthreads();
  uint32_t all = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) all = max(all, red[w]);
  const float common = of_key(all);
  double mine = static_cast<double>(sum) + static_cast<double>(rest);
  if (ref != common) mine *= ref == -INFINITY ? 0.0 : static_cast<double>(exp_from(ref, common));
#pragma unroll
  for (int d = kWarp / 2; d > 0; d /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  if (lane == 0) sums[warp] = mine;
  Entry* out = p.entries + static_cast<int64_t>(blockIdx.x) * p.cap;
  int count = many ? exact_chunk<DT>(p, row, e0, e1, out, &other_s) : count_s;
  __syncthreads();
  if (!many)
    for (int i = t; i < count; i += kScanThreads) out[i] = list[i];
  if (t == 0) {
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    p.parts[blockIdx.x] = Part{common, count, total};
  }
}

// ------------------------------------------------------------------ join

struct Candidate {
  double score;
  int32_t row, token;
};
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | (uint64_t(1) << 63));
}
__device__ __forceinline__ uint64_t index_of(int row, int token) {
  return static_cast<uint64_t>(static_cast<uint32_t>(row)) << 32 | static_cast<uint32_t>(token);
}

// What the rows' scores and sums make of them; returns whether the row is bad.
__device__ __forceinline__ bool row_state(const Params& p, int64_t row, float top, double sum, RowState& s) {
  const float score = p.a.scores ? p.a.scores[row] : 0.f;
  s.pad = 0;
  s.lse = top == -INFINITY ? -INFINITY : static_cast<double>(top) + log(sum);
  const bool bad = !(score < INFINITY) || !(sum < INFINITY) || top == INFINITY;
  s.offset = bad || top == -INFINITY || score == -INFINITY ? -INFINITY
                                                           : static_cast<float>(static_cast<double>(score) - s.lse);
  return bad;
}

// Selects among the candidates that each(f) calls f(row, token, logit, offset) for, every
// thread for its own, and writes the group's outputs. Block-wide.
template <class Each>
__device__ __forceinline__ void select_of(const Params& p, int group, float widest, const Each& each,
                                          Candidate* found, uint32_t* red, int* count_s) {
  const int t = threadIdx.x, width = p.a.width;
  const auto score_of = [&](int row, float logit) {
    return static_cast<double>(p.a.scores ? p.a.scores[row] : 0.f) + (static_cast<double>(logit) - p.rows[row].lse);
  };
  float most = -INFINITY;
  each([&](int, int, float logit, float offset) { most = fmaxf(most, offset + logit); });
  const uint32_t key[1] = {key_of(most)};
  float bound = bound_of(block_bound<kJoinThreads>(key, width, red));
  // an fp32 score is off by at most half an ulp of its own and of the offset's
  if (bound > -FLT_MAX) bound -= 2.4e-7f * (fabsf(bound) + widest) + 1e-30f;
  if (t == 0) *count_s = 0;
  __syncthreads();
  each([&](int row, int token, float logit, float offset) {
    if (!(offset + logit >= bound)) return;
    const int at = atomicAdd(count_s, 1);
    if (at < kFinal) found[at] = Candidate{score_of(row, logit), row, token};
  });
  __syncthreads();
  int n = *count_s;
  if (n > kFinal) {
    // too many at the bound: the exact score, then the exact index among its ties
    const auto reach = [&](uint64_t k, uint64_t last) {
      int c = 0;
      each([&](int row, int token, float logit, float offset) {
        if (!(offset + logit >= bound)) return;
        const uint64_t x = key_of(score_of(row, logit));
        c += x > k || (x == k && index_of(row, token) <= last);
      });
      __syncthreads();
      if (t == 0) *count_s = 0;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, c);
      if (t % kWarp == 0) atomicAdd(count_s, c);
      __syncthreads();
      return *count_s;
    };
    uint64_t k = 0, last = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t trial = k | (uint64_t(1) << bit);
      if (reach(trial, ~uint64_t(0)) >= width) k = trial;
    }
    // the least index up to which the ties fill the places
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t trial = last | (uint64_t(1) << bit);
      if (reach(k, trial - 1) < width) last = trial;
    }
    __syncthreads();
    if (t == 0) *count_s = 0;
    __syncthreads();
    each([&](int row, int token, float logit, float offset) {
      if (!(offset + logit >= bound)) return;
      const double s = score_of(row, logit);
      const uint64_t x = key_of(s);
      if (!(x > k || (x == k && index_of(row, token) <= last))) return;
      const int at = atomicAdd(count_s, 1);
      if (at < kFinal) found[at] = Candidate{s, row, token};
    });
    __syncthreads();
    n = min(*count_s, kFinal);
  }
  // ---- ranks
  const int64_t out = static_cast<int64_t>(group) * width;
  for (int i = t; i < n; i += kJoinThreads) {
    const Candidate c = found[i];
    const uint64_t mine = index_of(c.row, c.token);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const Candidate d = found[j];
      rank += d.score > c.score || (d.score == c.score && index_of(d.row, d.token) < mine);
    }
    if (rank < width) {
      p.a.out_scores[out + rank] = static_cast<float>(c.score);
      p.a.out_rows[out + rank] = c.row;
      p.a.out_tokens[out + rank] = c.token;
    }
  }
  for (int i = n + t; i < width; i += kJoinThreads) {
    p.a.out_scores[out + i] = -INFINITY;
    p.a.out_rows[out + i] = -1;
    p.a.out_tokens[out + i] = -1;
  }
}

// The rows [s0, s1) of a group; none, and the error bit, where starts are bad.
__device__ __forceinline__ void group_rows(const Params& p, int group, int64_t& s0, int64_t& s1) {
  s0 = p.a.starts[group];
  s1 = p.a.starts[group + 1];
  if (s0 < 0 || s1 < s0 || s1 > p.a.rows) {
    if (threadIdx.x == 0) flag(p.a.err, DLRM_ERRBIT_OFFSETS);
    s0 = s1 = 0;
  }
}

// Largest magnitude of the rows' offsets, in every thread.
__device__ __forceinline__ float widest_of(float mine, uint32_t* red) {
  uint32_t x = __reduce_max_sync(0xffffffffu, __float_as_uint(mine));
  __syncthreads();
  if (threadIdx.x % kWarp == 0) red[threadIdx.x / kWarp] = x;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / kWarp; ++w) x = max(x, red[w]);
  __syncthreads();
  return __uint_as_float(x);
}

__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ Params p) {
  __shared__ Candidate found[kFinal];
  __shared__ uint32_t red[2 * kJoinThreads / kWarp];
  __shared__ int count_s;
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp;
  pdl_wait();
  pdl_trigger();
  int64_t s0, s1;
  group_rows(p, blockIdx.x, s0, s1);
  // ---- the rows' sums
  float widest = 0.f;
  for (int64_t row = s0 + warp; row < s1; row += kJoinThreads / kWarp) {
    const Part* parts = p.parts + row * p.chunks;
    uint32_t hi = 0;
    for (int c = lane; c < p.chunks; c += kWarp) hi = max(hi, key_of(parts[c].top));
    const float top = of_key(__reduce_max_sync(0xffffffffu, hi));
    double sum = 0.0;
    for (int c = lane; c < p.chunks; c += kWarp) {
      const Part x = parts[c];
      // (nothing allowed: zero, or NaN)
      sum += x.top == top || x.top == -INFINITY ? x.sum : x.sum * exp(static_cast<double>(x.top) - top);
    }
#pragma unroll
    for (int d = kWarp / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    RowState s;
    if (row_state(p, row, top, sum, s) && lane == 0) flag(p.a.err, DLRM_ERRBIT_INVALID_ARG);
    if (lane == 0) p.rows[row] = s;
    if (s.offset != -INFINITY) widest = fmaxf(widest, fabsf(s.offset));
  }
  widest = widest_of(widest, red);
  // ---- the lists, a warp each
  const int64_t lists = (s1 - s0) * p.chunks;
  select_of(p, blockIdx.x, widest, [&](const auto& f) {
    for (int64_t l = warp; l < lists; l += kJoinThreads / kWarp) {
      const int row = static_cast<int>(s0 + l / p.chunks);
      const int64_t at = s0 * p.chunks + l;
      const float offset = p.rows[row].offset;
      const int n = offset == -INFINITY ? 0 : p.parts[at].count;
      const Entry* entries = p.entries + at * p.cap;
      for (int i = lane; i < n; i += kWarp) f(row, entries[i].token, entries[i].logit, offset);
    }
  }, found, red, &count_s);
}

// Everything of a group in one CTA: its rows stay in L1 between the passes.
template <int DT>
__global__ void __launch_bounds__(kJoinThreads) beam_small_kernel(const __grid_constant__ Params p) {
  __shared__ Candidate found[kFinal];
  __shared__ uint32_t red[2 * kJoinThreads / kWarp];
  __shared__ int count_s;
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp, vocab = p.a.vocab;
  pdl_wait();
  pdl_trigger();
  int64_t s0, s1;
  group_rows(p, blockIdx.x, s0, s1);
  const auto logit_of = [&](int64_t row, int e) {
    const float x = load_element<DT>(p.a.logits, row * p.a.ld + e);
    return p.a.allowed && !p.a.allowed[row * p.a.ld_allowed + e] ? -INFINITY : x;
  };
  float widest = 0.f;
  for (int64_t row = s0 + warp; row < s1; row += kJoinThreads / kWarp) {
    float top = -INFINITY;
    for (int e = lane; e < vocab; e += kWarp) top = fmaxf(top, logit_of(row, e));
    top = of_key(__reduce_max_sync(0xffffffffu, key_of(top)));
    const float base = top == -INFINITY ? 0.f : top;
    double sum = 0.0;
    for (int e0 = lane; e0 < vocab; e0 += 32 * kWarp) {
      float part = 0.f;
      for (int e = e0; e < min(vocab, e0 + 32 * kWarp); e += kWarp) part += exp_from(logit_of(row, e), base);
      sum += part;
    }
#pragma unroll
    for (int d = kWarp / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    RowState s;
    if (row_state(p, row, top, sum, s) && lane == 0) flag(p.a.err, DLRM_ERRBIT_INVALID_ARG);
    if (lane == 0) p.rows[row] = s;
    if (s.offset != -INFINITY) widest = fmaxf(widest, fabsf(s.offset));
  }
  widest = widest_of(widest, red);
  // a warp takes 256 tokens of a row at a time
  const int pieces = (vocab + 255) / 256;
  const int64_t all = (s1 - s0) * pieces;
  select_of(p, blockIdx.x, widest, [&](const auto& f) {
    for (int64_t u = warp; u < all; u += kJoinThreads / kWarp) {
      const int row = static_cast<int>(s0 + u / pieces), first = static_cast<int>(u % pieces) * 256 + lane;
      const float offset = p.rows[row].offset;
      if (offset == -INFINITY) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int token = first + i * kWarp;
        const float x = token < vocab ? logit_of(row, token) : -INFINITY;
        if (x > -INFINITY) f(row, token, x, offset);
      }
    }
  }, found, red, &count_s);
}

// ------------------------------------------------------------------ launches

// One launch for groups of at most this many logits, on average.
constexpr int64_t kSmallGroup = 32768;
constexpr int kSmallVocab = 4096;
// CTAs of the scan that chunks are made for: rows are cut until there are so many.
constexpr int64_t kScanCtas = 152 * 8 * 2;
constexpr int kMostTiles = 8;                    // of a chunk

struct Plan {
  bool small;
  int chunks, tiles, cap;
  int64_t parts, entries, bytes;                 // offsets of the scratch, and its size
};
Plan plan_of(const dlrm_beam_select_t& a) {
  Plan s{};
  s.bytes = round_up(a.rows * static_cast<int64_t>(sizeof(RowState)), 16);
  s.small = a.rows == 0 || (a.vocab <= kSmallVocab && a.rows * a.vocab <= kSmallGroup * a.groups);
  if (s.small) return s;
  const int64_t tile = kScanThreads * kVectors * (a.dtype == DLRM_DTYPE_FP32 ? 4 : 8);
  const int64_t tiles = (a.vocab + tile - 1) / tile;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(tiles, kScanCtas / std::max<int64_t>(a.rows, 1)));
  s.tiles = static_cast<int>(std::min<int64_t>((tiles + want - 1) / want, kMostTiles));
  s.chunks = static_cast<int>((tiles + s.tiles - 1) / s.tiles);
  s.cap = 8 * a.width + 256;
  s.parts = s.bytes;
  s.entries = s.parts + a.rows * s.chunks * static_cast<int64_t>(sizeof(Part));
  s.bytes = s.entries + a.rows * s.chunks * s.cap * static_cast<int64_t>(sizeof(Entry));
  return s;
}

template <int DT, bool MASK>
cudaError_t launch_scan(const Params& p, bool aligned, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.a.rows * p.chunks);
  const size_t smem = p.cap * sizeof(Entry);
  return aligned ? launch_pdl(beam_scan_kernel<DT, MASK, true>, dim3(grid), dim3(kScanThreads), smem, stream, p)
                 : launch_pdl(beam_scan_kernel<DT, MASK, false>, dim3(grid), dim3(kScanThreads), smem, stream, p);
}

template <int DT>
cudaError_t launch(const Params& p, bool small, cudaStream_t stream) {
  if (small)
    return launch_pdl(beam_small_kernel<DT>, dim3(p.a.groups), dim3(kJoinThreads), 0, stream, p);
  constexpr int kVec = Row<DT>::kVec;
  const bool aligned = aligned_to(p.a.logits, 16) && (p.a.rows == 1 || p.a.ld % kVec == 0) &&
                       (!p.a.allowed || (aligned_to(p.a.allowed, kVec) && (p.a.rows == 1 || p.a.ld_allowed % kVec == 0)));
  const cudaError_t e = p.a.allowed ? launch_scan<DT, true>(p, aligned, stream) : launch_scan<DT, false>(p, aligned, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_join_kernel, dim3(p.a.groups), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace

int64_t beam_select_work(const dlrm_beam_select_t& a) { return plan_of(a).bytes; }

bool beam_select_fits(const dlrm_beam_select_t& a) {
  const Plan s = plan_of(a);
  return s.small || a.rows * s.chunks < (int64_t(1) << 31);
}

cudaError_t launch_beam_select(const dlrm_beam_select_t& a, cudaStream_t stream) {
  const Plan s = plan_of(a);
  char* work = static_cast<char*>(a.work);
  const Params p{a, s.chunks, s.tiles, s.cap, reinterpret_cast<RowState*>(work),
                 reinterpret_cast<Part*>(work + s.parts), reinterpret_cast<Entry*>(work + s.entries)};
  if (a.dtype == DLRM_DTYPE_FP32) return launch<DLRM_DTYPE_FP32>(p, s.small, stream);
  if (a.dtype == DLRM_DTYPE_BF16) return launch<DLRM_DTYPE_BF16>(p, s.small, stream);
  return launch<DLRM_DTYPE_FP16>(p, s.small, stream);
}

}  // namespace dlrm
