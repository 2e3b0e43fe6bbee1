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
// comparison with one another. Where many do (ties, adverse orders) the bound is made
// the exact value, and ties at it go by their index.
//
// The order hangs by differences of the rows' logarithms, so these are held more
// precisely than fp32: the sums' terms have rounding errors of their own (2^-22 each, not
// of one sign), sums and logarithms are kept in two floats (64-bit arithmetic has few
// units: a logarithm in it took the join of 64 users 2.4 us, the sums 13), and the scores of
// the few that are ranked are compared in 64 bits.
#include <float.h>

#include "history.cuh"

namespace dlrm {

namespace {

constexpr int kScanThreads = 128;
constexpr int kJoinThreads = 1024;
constexpr int kSmallThreads = 512;
constexpr int kVectors = 4;                      // 16-byte vectors of a thread and tile
constexpr int kSubsets = 64;                     // widths up to here: one subset a thread will do
constexpr int kFinal = 2048;                     // candidates that shared memory holds
// Candidates that are ranked at most, by comparison with one another: a call that ranked 1792
// took 407 us, and takes 35 with an exact bound that leaves 512 or fewer.
constexpr int kRanked = 512;
constexpr int kLists = 1024;                     // lists of a group that shared memory knows
constexpr int kRowsHere = 256;                   // rows of a group whose states lie in shared memory,
constexpr int kRowsJoin = 128;                   // and of the join's
static_assert(kSubsets <= kScanThreads && kBeamMaxWidth <= kScanThreads * kVectors && kBeamMaxWidth <= kSmallThreads &&
                  kSmallThreads <= kJoinThreads && kBeamMaxWidth <= kRanked && kRanked <= kFinal, "a subset for each place");

// A sum in two floats: the rounding errors of `sum` in `rest`.
struct Sum {
  float sum, rest;
  __device__ __forceinline__ void add(float x) {
    const float s = sum + x, z = s - sum;
    rest += (sum - (s - z)) + (x - z);
    sum = s;
  }
};
struct Part {                                    // of a chunk of a row
  Sum sum;                                       // of exponentials, times 2^-power(ref), or e^-ref if it is far
  float ref;                                     // near the largest logit; -infinity: nothing allowed
  float top;                                     // largest logit
  int32_t count;                                 // entries of its list
  int32_t pad;
};
struct Entry {
  float logit;
  int32_t token;
};
struct RowState {
  Sum lse;                                       // (first the sum of exponentials, and its reference in offset)
  float offset;                                  // score - lse; -infinity: the row has no candidates
  float score;
};
static_assert(sizeof(Part) == 24 && sizeof(Entry) == 8 && sizeof(RowState) == 16, "scratch sizes");

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

// Exponentials of a row are powers of two of x log2(e) - power(ref), in one FMA: the power is a
// whole number, so sums with other references differ by powers of two. log2(e) in fp32 is
// short of kLow: x kLow is left out of the powers, ref kLow (nearly all of it) comes back with the
// logarithm. References that are far from zero are subtracted instead.
constexpr float kLog2E = 1.4426950408889634f, kLow = 1.92596299e-8f;
constexpr float kLn2 = 0.693147180559945309f, kLn2Low = -1.90465430e-9f;
constexpr float kFar = 65536.f;
__device__ __forceinline__ float power(float ref) { return ceilf(ref * kLog2E); }
__device__ __forceinline__ float exp_from(float x, float ref) {
  return fabsf(ref) < kFar ? exp2_approx(fmaf(x, kLog2E, -power(ref))) : exp2_approx((x - ref) * kLog2E);
}
// Two at a time.
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 z;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(z.x), "=f"(z.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return z;
}
// Over the warp, the same in every lane.
__device__ __forceinline__ Sum warp_sum(Sum s) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d /= 2) {
    const float x = __shfl_xor_sync(0xffffffffu, s.sum, d);
    s.rest += __shfl_xor_sync(0xffffffffu, s.rest, d);
    s.add(x);
  }
  return s;
}
// What a sum with reference `from` is with reference `to` (>= from). A near reference scales by
// 2^-power(ref), a far one by 2^-(ref kLog2E); where one is near and one far, the power between
// the two scales is one FMA, too (e^(from - to) there left out what power() rounds up: a sum up
// to twice too small or large).
__device__ __forceinline__ Sum moved(Sum s, float from, float to) {
  if (from == to) return s;
  if (from == -INFINITY) return Sum{s.sum, 0.f};  // zero, or NaN
  const bool near_from = fabsf(from) < kFar, near_to = fabsf(to) < kFar;
  float f;
  if (near_from && near_to)
    f = pow2f(static_cast<int>(fmaxf(power(from) - power(to), -126.f)));
  else if (near_from)
    f = exp2_approx(fmaf(-to, kLog2E, power(from)));
  else if (near_to)
    f = exp2_approx(fmaf(from, kLog2E, -power(to)));
  else
    f = exp2_approx((from - to) * kLog2E);
  return Sum{s.sum * f, s.rest * f};              // (a power of two is exact)
}
// log(s) with its reference, in two floats: s = m 2^k with m around 1, log m = 2 artanh z,
// z = (m - 1) / (m + 1), by the series 2 z (1 + z^2 / 3 + z^4 / 5 + ...), |z| <= 0.172.
__device__ __forceinline__ Sum log_sum(const Sum& s, float ref) {
  const int k = (static_cast<int>(__float_as_uint(s.sum) - 0x3f3504f3u)) >> 23;   // m from sqrt(1/2) on
  const float scale = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  const float m = s.sum * scale, low = s.rest * scale;
  const float p = m - 1.f, q = m + 1.f, q_low = (m - (q - 1.f)) + low;   // p is exact
  const float z = p / q;
  const float z_low = (fmaf(-z, q, p) + low - z * q_low) / q;
  const float z2 = z * z;
  float t = fmaf(z2, 1.f / 11, 1.f / 9);
  t = fmaf(t, z2, 1.f / 7);
  t = fmaf(t, z2, 1.f / 5);
  t = fmaf(t, z2, 1.f / 3) * z2 * z;
  Sum y{2.f * z, 2.f * z_low};
  y.rest = fmaf(2.f, t, y.rest);
  const bool far = !(fabsf(ref) < kFar);
  const float n = static_cast<float>(k) + (far ? 0.f : power(ref));
  const float high = n * kLn2;
  y.rest += fmaf(n, kLn2, -high) + n * kLn2Low;
  y.add(high);
  if (far)
    y.add(ref);
  else
    y.rest += ref * (kLow * kLn2);
  const float sum = y.sum + y.rest;
  return Sum{sum, (y.sum - sum) + y.rest};
}

// Of counts of kValues values: the largest value that k (or more) of those counted reach, and how
// many do. Every warp for itself; there are k.
constexpr int kValues = 256;
__device__ __forceinline__ void reached(const int* values, int k, int& value, int& there) {
  constexpr int kEach = kValues / kWarp;
  const int lane = threadIdx.x % kWarp;
  int mine[kEach], from = 0;                      // keys of the lane's values, and with those of later lanes
#pragma unroll
  for (int i = 0; i < kEach; ++i) from += mine[i] = values[lane * kEach + i];
  const int own = from;
#pragma unroll
  for (int d = 1; d < kWarp; d *= 2) {
    const int x = __shfl_down_sync(0xffffffffu, from, d);
    if (lane + d < kWarp) from += x;
  }
  const int last = 31 - __clz(__ballot_sync(0xffffffffu, from >= k));   // (lane 0 has all)
  int reach = from - own, at = 0;                 // of the largest value that k reach
  value = 0;
#pragma unroll
  for (int i = kEach - 1; i >= 0; --i) {
    reach += mine[i];
    if (at < k) {
      at = reach;
      value = lane * kEach + i;
    }
  }
  value = __shfl_sync(0xffffffffu, value, last);
  there = __shfl_sync(0xffffffffu, at, last);
}

// A lower bound of the k-th largest of the threads' keys: the first eight bits that they do not
// have in common by a count of each value, then bit by bit, until few more than k
// reach it (keys of -infinity do not count, and are the bound where there are fewer than k
// others). Block-wide; between two calls the caller has a barrier. red: kRed words a warp.
constexpr int kRed = 19;
template <int THREADS>
__device__ __forceinline__ uint32_t block_bound(uint32_t key, int k, uint32_t* red) {
  constexpr int kWarps = THREADS / kWarp;
  static_assert(kWarps <= kWarp, "a warp's lanes hold what all warps found");
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const uint32_t none = key_of(-INFINITY);
  uint32_t hi = __reduce_max_sync(0xffffffffu, key), lo = __reduce_min_sync(0xffffffffu, key > none ? key : 0xffffffffu);
  int there = __popc(__ballot_sync(0xffffffffu, key > none));
  if (lane == 0) {
    red[warp] = hi;
    red[kWarps + warp] = lo;
    red[2 * kWarps + warp] = there;
  }
  static_assert(16 * kWarps >= kValues && THREADS >= kValues, "room");
  int* values = reinterpret_cast<int*>(red + 3 * kWarps);
  if (threadIdx.x < kValues) values[threadIdx.x] = 0;
  __syncthreads();
  const bool one = lane < kWarps;
  hi = __reduce_max_sync(0xffffffffu, one ? red[lane] : 0);
  lo = __reduce_min_sync(0xffffffffu, one ? red[kWarps + lane] : 0xffffffffu);
  there = __reduce_add_sync(0xffffffffu, one ? red[2 * kWarps + lane] : 0);
  if (there < k) return none;
  if (hi == lo) return hi;
  const int first = 31 - __clz(hi ^ lo);
  uint32_t bound = first == 31 ? 0u : hi & (0xffffffffu << (first + 1));
  const int low = max(first - 7, 0);
  if (there > k + k / 4 + 8) {
    if (key > none) atomicAdd(&values[key >> low & (kValues - 1)], 1);
    __syncthreads();
    int value;
    reached(values, k, value, there);
    bound |= static_cast<uint32_t>(value) << low;
  }
  for (int bit = low - 1; bit >= 0 && there > k + k / 4 + 8; --bit) {
    const uint32_t trial = bound | (1u << bit);
    const int n = __syncthreads_count(key >= trial);
    if (n >= k) {
      bound = trial;
      there = n;
    }
  }
  return bound;
}

// ------------------------------------------------------------------ rows as loaded

// Rows are read as aligned 16-byte vectors, of which each lane has its own and, from the next
// lane, what a row that begins between two vectors needs of the following one. So a row is
// grouped by its tokens wherever it lies, and rows that are alike get sums that are alike. Vectors
// are moved into place when they are used, not when they are asked for.
template <int DT>
struct Row {
  static constexpr int kVec = DT == DLRM_DTYPE_FP32 ? 4 : 8;
  static constexpr int kBytes = DT == DLRM_DTYPE_FP32 ? 4 : 2;
};

// The lane's vectors, Q words and `bits` on; `tail` is what follows the last lane's last one.
template <int DT, int Q>
__device__ __forceinline__ void move_vectors(uint4 (&now)[kVectors], const uint4 (&raw)[kVectors], const uint4& tail, int bits) {
  const int lane = threadIdx.x % kWarp;
  const uint32_t last[4] = {tail.x, tail.y, tail.z, tail.w};
#pragma unroll
  for (int v = 0; v < kVectors; ++v) {
    const uint4 a = raw[v], b = raw[v + 1 < kVectors ? v + 1 : v];
    const uint32_t mine[4] = {a.x, a.y, a.z, a.w}, first[4] = {b.x, b.y, b.z, b.w};
    uint32_t w[8] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < Q + (DT != DLRM_DTYPE_FP32); ++i) {
      const uint32_t x = v + 1 < kVectors && lane == 0 ? first[i] : mine[i];
      w[4 + i] = __shfl_sync(0xffffffffu, x, (lane + 1) % kWarp);
      if (v + 1 == kVectors && lane == kWarp - 1) w[4 + i] = last[i];
    }
    if (DT != DLRM_DTYPE_FP32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i + Q], w[i + Q + 1], bits);
      now[v] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      now[v] = make_uint4(w[Q], w[Q + 1], w[Q + 2], w[Q + 3]);
    }
  }
}

// The bytes that allow a vector's elements begin at any byte: as aligned words, of which the last
// is needed only where they do not begin with a word.
template <int DT>
struct May {
  uint32_t w[Row<DT>::kVec / 4 + 1];
  __device__ __forceinline__ uint2 bytes(int shift) const {
    return make_uint2(__funnelshift_r(w[0], w[1], shift),
                      Row<DT>::kVec == 8 ? __funnelshift_r(w[1], w[Row<DT>::kVec / 4], shift) : 0);
  }
};
// The vector with -infinity where a byte of `may` is zero.
template <int DT>
__device__ __forceinline__ void hide(uint4& v, const uint2& may) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (DT == DLRM_DTYPE_FP32) {
    const uint32_t m = __vcmpne4(may.x, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = __byte_perm(m, 0, 0x1111 * i);
      w[i] = (w[i] & k) | (0xff800000u & ~k);
    }
  } else {
    constexpr uint32_t kNone = DT == DLRM_DTYPE_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    const uint32_t m[2] = {__vcmpne4(may.x, 0), __vcmpne4(may.y, 0)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = __byte_perm(m[i / 2], 0, i % 2 ? 0x3322 : 0x1100);
      w[i] = (w[i] & k) | (kNone & ~k);
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}
// Bytes that allow the first n of a vector's elements.
__device__ __forceinline__ uint2 first_bytes(int n) {
  const uint64_t m = n >= 8 ? ~uint64_t(0) : n <= 0 ? 0 : (uint64_t(1) << (8 * n)) - 1;
  return make_uint2(static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32));
}
// Pair i of a vector's elements.
template <int DT>
__device__ __forceinline__ float2 pair_of(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (DT == DLRM_DTYPE_FP32) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  if (DT == DLRM_DTYPE_BF16) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return f16x2_to_float2(w[i]);
}
// Largest element (NaN passed over).
template <int DT>
__device__ __forceinline__ float largest(const uint4& v) {
  if (DT == DLRM_DTYPE_FP32)
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  uint32_t m, n;
  if (DT == DLRM_DTYPE_BF16) {
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(n));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
  asm("max.f16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
  asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(n));
  const float2 f = f16x2_to_float2(m);
  return fmaxf(f.x, f.y);
}

// ------------------------------------------------------------------ scan

// The `width` largest logits of [e0, e1) of a row, when too many reached `bound`, which `width` or
// more reach; `highest` is the largest. Those above it are few where the rest are ties (a head
// that saturates, tokens masked by a value of their own), of which the first are taken; else the
// bound is found eight bits at a time, until no more reach it than the list has places. Every
// thread; values: kValues words. (1024 rows of 32,768 bf16 logits, all but one in a thousand
// alike: 85 us; with a pass over the chunk for each bit of the value and of the index 1385.)
template <int DT>
__device__ __noinline__ int exact_chunk(const Params& p, int64_t row, int64_t e0, int64_t e1, float bound, float highest,
                                        Entry* list, int* counter, int* values) {
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp, width = p.a.width;
  const auto logit = [&](int64_t e) {
    const float x = load_element<DT>(p.a.logits, row * p.a.ld + e);
    return p.a.allowed && !p.a.allowed[row * p.a.ld_allowed + e] ? -INFINITY : x;
  };
  // (a NaN reaches no bound)
  const auto collect = [&](bool ties) {           // those above the bound, and those at it
    __syncthreads();
    if (t == 0) *counter = 0;
    __syncthreads();
#pragma unroll 8
    for (int64_t e = e0 + t; e < e1; e += kScanThreads) {
      const float x = logit(e);
      if (!(x > bound || (ties && x == bound))) continue;
      const int place = atomicAdd(counter, 1);
      if (place < p.cap) list[place] = Entry{x, static_cast<int>(e)};
    }
    __syncthreads();
    return *counter;
  };
  bound += 0.f;                                   // (zeros have one key)
  int n = collect(false);
  if (n > p.cap) {
    const uint32_t hi = key_of(highest + 0.f);
    int low = 32 - __clz(hi ^ key_of(bound)), above = 0, reach = INT_MAX;   // bits from `low` on are found
    uint32_t key = low == 32 ? 0u : hi >> low << low;
    while (low > 0) {
      const int next = max(low - 8, 0);
      for (int i = t; i < kValues; i += kScanThreads) values[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int64_t e = e0 + t; e < e1; e += kScanThreads) {
        const float x = logit(e);
        const uint32_t k = key_of(x + 0.f);
        if (x > bound && (k ^ key) >> next >> (low - next) == 0) atomicAdd(&values[(k >> next) & ((1 << (low - next)) - 1)], 1);
      }
      __syncthreads();
      int value, there;
      reached(values, width - above, value, there);
      key |= static_cast<uint32_t>(value) << next;
      reach = above + there;
      if (reach <= p.cap) break;
      above += there - values[value];
      low = next;
      __syncthreads();                            // `values` are read
    }
    bound = bound_of(key);
    n = collect(reach <= p.cap);
  }
  if (n >= width) return n;
  // ties, in order, as far as there are places
  for (int64_t first = e0; first < e1 && n < width; first += 8 * kScanThreads) {
    const int64_t mine = first + 8 * t;
    uint32_t tie = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) tie |= static_cast<uint32_t>(mine + i < e1 && logit(mine + i) == bound) << i;
    int before = __popc(tie);
#pragma unroll
    for (int d = 1; d < kWarp; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += y;
    }
    if (lane == kWarp - 1) values[warp] = before;
    __syncthreads();
    int place = n + before - __popc(tie);
#pragma unroll
    for (int w = 0; w < kScanThreads / kWarp; ++w) {
      place += w < warp ? values[w] : 0;
      n += values[w];
    }
    __syncthreads();                              // `values` are read
    for (; tie && place < width; tie &= tie - 1, ++place)
      list[place] = Entry{bound, static_cast<int>(mine) + __ffs(tie) - 1};
  }
  return min(n, width);
}

// Drops entries below a lower bound of the k-th largest of a list of n >= k, until few more than k
// are left (or ties); returns how many stay, and the bound. One warp.
__device__ __forceinline__ int tighten(Entry* list, int n, int k, float& least) {
  const int lane = threadIdx.x % kWarp;
  uint32_t hi = 0, lo = 0xffffffffu;
  for (int i = lane; i < n; i += kWarp) {
    const uint32_t x = key_of(list[i].logit);
    hi = max(hi, x);
    lo = min(lo, x);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  least = of_key(lo);
  if (hi == lo) return n;
  const int first = 31 - __clz(hi ^ lo);
  uint32_t bound = first == 31 ? 0u : hi & (0xffffffffu << (first + 1));
  int there = n;
  for (int bit = first; bit >= 0 && there > k + k / 4 + 1; --bit) {
    const uint32_t trial = bound | (1u << bit);
    int c = 0;
#pragma unroll 4
    for (int i = lane; i < n; i += kWarp) c += key_of(list[i].logit) >= trial;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= k) {
      bound = trial;
      there = c;
    }
  }
  least = bound_of(bound);
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

// A lower bound of the k-th largest of a warp's keys, N a lane, as block_bound.
template <int N>
__device__ __forceinline__ uint32_t warp_bound(const uint32_t (&key)[N], int k) {
  const uint32_t none = key_of(-INFINITY);
  uint32_t hi = none, lo = 0xffffffffu;
  int there = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    hi = max(hi, key[i]);
    lo = key[i] > none ? min(lo, key[i]) : lo;
    there += __popc(__ballot_sync(0xffffffffu, key[i] > none));
  }
  if (there < k) return none;
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (hi == lo) return hi;
  const int first = 31 - __clz(hi ^ lo);
  uint32_t bound = first == 31 ? 0u : hi & (0xffffffffu << (first + 1));
  for (int bit = first; bit >= 0 && there > k + k / 4 + 1; --bit) {
    const uint32_t trial = bound | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popc(__ballot_sync(0xffffffffu, key[i] >= trial));
    if (n >= k) {
      bound = trial;
      there = n;
    }
  }
  return bound;
}

// What bounds it: instructions (a conversion, half an FMA, one exponential and half a sum a
// logit; issue slots are 66% busy) and what each CTA begins and ends with, then HBM: 1643 rows of
// 32,768 bf16 logits 34 us (3.2 TB/s), 33 of 1,000,003 masked fp16 ones 41 us (2.5 TB/s).
// Warps meet twice, after the first tile and at the end: each has a list of its own, of vectors
// by their largest element; their elements are looked at once more at the end.
template <int DT, bool MASK>
__global__ void __launch_bounds__(kScanThreads, MASK ? 6 : 8) beam_scan_kernel(const __grid_constant__ Params p) {
  constexpr int kVec = Row<DT>::kVec, kWarps = kScanThreads / kWarp, kWords = kVec / 4;
  constexpr int kTile = kScanThreads * kVec * kVectors;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t red[2 * kWarps];
  __shared__ Sum sums[kWarps];
  __shared__ int counts[kWarps], other_s;
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp;
  const int64_t row = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks, vocab = p.a.vocab;
  const int64_t e0 = chunk * p.tiles * kTile, e1 = min(vocab, e0 + static_cast<int64_t>(p.tiles) * kTile);
  const char* logits = static_cast<const char*>(p.a.logits) + row * p.a.ld * Row<DT>::kBytes;
  const uint8_t* allowed = MASK ? p.a.allowed + row * p.a.ld_allowed : nullptr;
  const int width = p.a.width, room = p.cap / kWarps;   // of a warp's list
  Entry* every = reinterpret_cast<Entry*>(smem);  // largest logit, first token (of the chunk's) of vectors
  Entry* list = every + warp * room;
  if (t == 0) other_s = 0;
  pdl_wait();
  pdl_trigger();

  const int n = static_cast<int>(e1 - e0);        // of the chunk
  const int first = (warp * kVectors * kWarp + lane) * kVec;   // the thread's of a tile; the others kWarp vectors apart
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(logits) & 15);
  const char* at_logits = logits - off + (e0 + first) * Row<DT>::kBytes;
  const int shift = MASK ? static_cast<int>(reinterpret_cast<uintptr_t>(allowed) & 3) * 8 : 0;
  const uint8_t* at_allowed = MASK ? allowed - shift / 8 + e0 + first : nullptr;
  uint4 raw[kVectors], tail = make_uint4(0, 0, 0, 0);
  May<DT> may[kVectors];
  auto load = [&](int at) {
    if (at + kTile <= n) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        raw[v] = __ldg(reinterpret_cast<const uint4*>(at_logits) + v * kWarp);
        if (MASK) {
          const uint32_t* words = reinterpret_cast<const uint32_t*>(at_allowed + v * kWarp * kVec);
#pragma unroll
          for (int i = 0; i < kWords; ++i) may[v].w[i] = __ldg(words + i);
          may[v].w[kWords] = shift ? __ldg(words + kWords) : 0;
        }
      }
      if (off && lane == kWarp - 1) tail = __ldg(reinterpret_cast<const uint4*>(at_logits) + (kVectors - 1) * kWarp + 1);
    } else {
      // vectors and words that hold something of the row
      const char* end_logits = logits + vocab * Row<DT>::kBytes;
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        const uint4* vector = reinterpret_cast<const uint4*>(at_logits) + v * kWarp;
        if (reinterpret_cast<const char*>(vector) < end_logits) raw[v] = __ldg(vector);
        if (MASK) {
          const uint32_t* words = reinterpret_cast<const uint32_t*>(at_allowed + v * kWarp * kVec);
#pragma unroll
          for (int i = 0; i <= kWords; ++i)
            may[v].w[i] = reinterpret_cast<const uint8_t*>(words + i) < allowed + vocab ? __ldg(words + i) : 0;
        }
      }
      const uint4* vector = reinterpret_cast<const uint4*>(at_logits) + (kVectors - 1) * kWarp + 1;
      if (lane == kWarp - 1 && reinterpret_cast<const char*>(vector) < end_logits) tail = __ldg(vector);
    }
    at_logits += kTile * Row<DT>::kBytes;
    if (MASK) at_allowed += kTile;
  };
  load(0);
  float ref = -INFINITY;
  Sum sum{0.f, 0.f};
  float bound = -FLT_MAX, peak = -INFINITY;
  int count = 0;                                  // of the warp's list
  bool many = false;                              // it overflowed
#pragma unroll 1
  for (int at = 0; at < n; at += kTile) {
    uint4 now[kVectors];
    float top[kVectors];
    if (off == 0) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) now[v] = raw[v];
    } else if (off < 8) {
      if (off < 4) move_vectors<DT, 0>(now, raw, tail, off * 8); else move_vectors<DT, 1>(now, raw, tail, off % 4 * 8);
    } else {
      if (off < 12) move_vectors<DT, 2>(now, raw, tail, off % 4 * 8); else move_vectors<DT, 3>(now, raw, tail, off % 4 * 8);
    }
    if (MASK) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) hide<DT>(now[v], may[v].bytes(shift));
    }
    if (at + kTile > n) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) hide<DT>(now[v], first_bytes(n - (at + first + v * kWarp * kVec)));
    }
#pragma unroll
    for (int v = 0; v < kVectors; ++v) top[v] = largest<DT>(now[v]);
    if (at + kTile < n) load(at + kTile);
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    peak = fmaxf(peak, most);
    static_assert(kVectors == 4, "largest of a thread");
    if (at == 0) {
      // each warp has its share of `width` maxima, as many as it has of all, at the least of the
      // warps' bounds or above (equal shares would leave no bound where few warps have tokens: the
      // end of a row, or a mask that allows a range); and one reference for all threads, so that
      // sums need no factors
      const bool few = width <= kSubsets;         // one subset a thread
      int have = 0;
      if (few) {
        have = __popc(__ballot_sync(0xffffffffu, most > -INFINITY));
      } else {
#pragma unroll
        for (int v = 0; v < kVectors; ++v) have += __popc(__ballot_sync(0xffffffffu, top[v] > -INFINITY));
      }
      const uint32_t hi = __reduce_max_sync(0xffffffffu, key_of(most));
      if (lane == 0) {
        red[warp] = hi;
        counts[warp] = have;
      }
      __syncthreads();
      uint32_t all = red[0];
      int maxima = counts[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        all = max(all, red[w]);
        maxima += counts[w];
      }
      ref = of_key(all);
      uint32_t key = maxima < width ? 0u : 0xffffffffu;
      if (have > 0 && maxima >= width) {
        const int share = static_cast<unsigned>(width * have + maxima - 1) / static_cast<unsigned>(maxima);
        if (few) {
          const uint32_t mine[1] = {key_of(most)};
          key = warp_bound(mine, share);
        } else {
          uint32_t mine[kVectors];
#pragma unroll
          for (int v = 0; v < kVectors; ++v) mine[v] = key_of(top[v]);
          key = warp_bound(mine, share);
        }
      }
      if (lane == 0) red[kWarps + warp] = key;
      __syncthreads();
      key = red[kWarps];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) key = min(key, red[kWarps + w]);
      bound = bound_of(key);
    } else if (most > ref + 20.f) {
      sum = moved(sum, ref, most);
      ref = most;
    }
    // (sums two at a time; powers, too, would have their factors moved into pairs: 2.5% longer)
    float2 part[kVectors];
    if (fabsf(ref) < kFar || ref == -INFINITY) {
      const float less = ref == -INFINITY ? 0.f : -power(ref);
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        part[v] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
          const float2 x = pair_of<DT>(now[v], i);
          const float2 y = make_float2(exp2_approx(fmaf(x.x, kLog2E, less)), exp2_approx(fmaf(x.y, kLog2E, less)));
          part[v] = i == 0 ? y : add2(part[v], y);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        part[v] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
          const float2 x = pair_of<DT>(now[v], i);
          part[v].x += exp_from(x.x, ref);
          part[v].y += exp_from(x.y, ref);
        }
      }
    }
    const float2 y = add2(add2(part[0], part[1]), add2(part[2], part[3]));
    sum.add(y.x + y.y);
    // ---- the warp's list
    unsigned who[kVectors];
    int more;
    const auto look = [&] {
      more = 0;
#pragma unroll
      for (int v = 0; v < kVectors; ++v) {
        who[v] = __ballot_sync(0xffffffffu, top[v] >= bound);
        more += __popc(who[v]);
      }
    };
    look();
    if (more > 0) {
      if (count + more > room && !many) {
        // what is not among the warp's largest is not among the chunk's
        __syncwarp();
        if (count > width) {
          float least;
          count = tighten(list, count, width, least);
          bound = fmaxf(bound, least);
          look();
        }
        many = count + more > room;
      }
      if (!many) {
#pragma unroll
        for (int v = 0; v < kVectors; ++v) {
          if (top[v] >= bound)
            list[count + __popc(who[v] & ((1u << lane) - 1))] =
                Entry{top[v], at + first + v * kWarp * kVec};
          count += __popc(who[v]);
        }
      }
    }
  }
  // ---- the chunk's sum, and the warps' lists as one
  const uint32_t hi = __reduce_max_sync(0xffffffffu, key_of(ref)), most = __reduce_max_sync(0xffffffffu, key_of(peak));
  __syncthreads();                                // (of one tile: `red` is read)
  if (lane == 0) {
    red[warp] = hi;
    red[kWarps + warp] = most;
    counts[warp] = many ? -1 : count;
  }
  __syncthreads();
  uint32_t all = red[0], highest = red[kWarps];
  int before = 0, total = 0;
  many = false;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    all = max(all, red[w]);
    highest = max(highest, red[kWarps + w]);
    many |= counts[w] < 0;
    before += w < warp ? counts[w] : 0;
    total += counts[w];
  }
  const float common = of_key(all);
  sum = warp_sum(moved(sum, ref, common));
  if (lane == 0) sums[warp] = sum;
  Entry* joined = every + p.cap;
  if (!many)
    for (int i = lane; i < count; i += kWarp) joined[before + i] = list[i];
  __syncthreads();
  if (!many && total > width + width / 4 + 8) {
    if (warp == 0) {                              // (all warps would meet at every bit)
      float least;
      total = tighten(joined, total, width, least);
      if (lane == 0) {
        counts[0] = total;
        red[0] = key_of(fmaxf(bound, least));
      }
    }
    __syncthreads();
    total = counts[0];
    bound = of_key(red[0]);
  }
  // ---- the list's elements
  Entry* out = p.entries + static_cast<int64_t>(blockIdx.x) * p.cap;
  int written = 0;
  if (!many) {
    for (int i = t; i < total * kVec; i += kScanThreads) {
      const int e = static_cast<int>(e0) + joined[i / kVec].token + i % kVec;
      if (e >= e1 || (MASK && !allowed[e])) continue;
      const float x = load_element<DT>(logits, e);
      if (!(x >= bound)) continue;
      const int place = atomicAdd(&other_s, 1);
      if (place < p.cap) out[place] = Entry{x, e};
    }
    __syncthreads();
    written = other_s;
    many = written > p.cap;                       // ties
    __syncthreads();
  }
  if (many) {
    if (lane == 0) red[warp] = key_of(bound);     // (each warp's is one of the chunk)
    __syncthreads();
    uint32_t least = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) least = max(least, red[w]);
    written = exact_chunk<DT>(p, row, e0, e1, of_key(least), of_key(highest), out, &other_s, reinterpret_cast<int*>(smem));
  }
  if (t == 0) {
    Sum total_sum = sums[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      total_sum.rest += sums[w].rest;
      total_sum.add(sums[w].sum);
    }
    p.parts[blockIdx.x] = Part{total_sum, common, of_key(highest), written, 0};
  }
}

// ------------------------------------------------------------------ join

struct Candidate {
  uint64_t key;                                  // of the score (first the logit's bits)
  int32_t row, token;
};
// 64-bit floats as integers of the same order: compared as such, as 64-bit arithmetic has
// few units.
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | (uint64_t(1) << 63));
}
__device__ __forceinline__ double of_key(uint64_t k) {
  return __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ (uint64_t(1) << 63) : ~k));
}
__device__ __forceinline__ uint64_t index_of(int row, int token) {
  return static_cast<uint64_t>(static_cast<uint32_t>(row)) << 32 | static_cast<uint32_t>(token);
}

// A row's state from its sum (in lse), reference (in offset) and score; a thread a row.
__device__ __forceinline__ void row_state(const Params& p, RowState& s) {
  const float score = s.score, ref = s.offset, sum = s.lse.sum;
  const bool bad = !(score < INFINITY) || !(sum < INFINITY) || ref == INFINITY;
  if (bad) flag(p.a.err, DLRM_ERRBIT_INVALID_ARG);
  if (bad || ref == -INFINITY || score == -INFINITY) {
    s.offset = -INFINITY;
    return;
  }
  s.lse = log_sum(s.lse, ref);
  s.offset = (score - s.lse.sum) - s.lse.rest;
}

// Scores in fp32 only decide which candidates are looked at. offset + logit is off by two
// roundings of the offset and one of the sum. Lowered or raised by four half ulps, of which one is
// for its own rounding, the offset leaves the sum's alone: bounds are those of lowered
// scores, and raised ones have to reach them. So a row that is far from the others (a beam that is
// not in use, at -1e9) makes no margin but its own wide: with one for all rows 128 beams of 4096
// tokens, 16 of them in use, took 5600 us, and take 27.
__device__ __forceinline__ float lowered(float offset) { return fmaf(fabsf(offset), -0x1p-22f, offset); }
__device__ __forceinline__ float raised(float offset) { return fmaf(fabsf(offset), 0x1p-22f, offset); }

// Below the k-th largest of the threads' lowered scores by the rounding of that sum, of the
// raised one that is to reach it and of the bound itself: three half ulps, and 5 are taken.
template <int THREADS>
__device__ __forceinline__ float score_bound(float most, int k, uint32_t* red) {
  const float bound = bound_of(block_bound<THREADS>(key_of(most), k, red));
  return bound > -FLT_MAX ? fmaxf(bound - (3e-7f * fabsf(bound) + 1e-30f), -FLT_MAX) : bound;
}

// Selects among the candidates that each(bound, most, f) calls f(row, token, logit, offset)
// for, every thread for its own, and writes the group's outputs; it may pass over what lies below
// the bound. No place's raised score lies below `bound`. Rows count from the group's first, s0,
// whose states are `state`. LISTS: candidates come in lists, of which each looks at `most` entries;
// the first bound is that of a part of them. Block-wide.
template <int THREADS, bool LISTS, class Each>
__device__ __forceinline__ void select_of(const Params& p, int64_t s0, const RowState* state, float bound,
                                          const Each& each, Candidate* found, uint32_t* red, int* count_s) {
  const int t = threadIdx.x, width = p.a.width;
  const auto score_of = [&](int row, float logit) {
    const RowState s = state[row];
    return static_cast<double>(s.score) +
           ((static_cast<double>(logit) - static_cast<double>(s.lse.sum)) - static_cast<double>(s.lse.rest));
  };
  const auto better = [&](int entries) {         // the bound, by the threads' largest
    float most = -INFINITY;
    each(bound, entries, [&](int, int, float logit, float offset) { most = fmaxf(most, lowered(offset) + logit); });
    bound = fmaxf(bound, score_bound<THREADS>(most, width, red));
  };
  const auto put = [&](const Candidate& c) {
    const int at = atomicAdd(count_s, 1);
    if (at < kFinal) found[at] = c;
  };
  const auto collect = [&] {
    if (t == 0) *count_s = 0;
    __syncthreads();
    each(bound, INT_MAX, [&](int row, int token, float logit, float offset) {
      if (raised(offset) + logit >= bound) put(Candidate{__float_as_uint(logit), row, token});
    });
    __syncthreads();
    return *count_s;
  };
  better(LISTS ? kWarp : INT_MAX);
  int n = collect();
  if (LISTS && n > kFinal) {
    better(INT_MAX);
    n = collect();
  } else if (LISTS && n > width + width / 4 + 64) {
    // the best of those that are here
    constexpr int kMine = kFinal / THREADS;
    Candidate mine[kMine];
    float score[kMine], most = -INFINITY;         // (raised)
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      score[i] = -INFINITY;
      if (t + i * THREADS >= n) continue;
      mine[i] = found[t + i * THREADS];
      const float offset = state[mine[i].row].offset, logit = __uint_as_float(static_cast<uint32_t>(mine[i].key));
      score[i] = raised(offset) + logit;
      most = fmaxf(most, lowered(offset) + logit);
    }
    bound = fmaxf(bound, score_bound<THREADS>(most, width, red));
    if (t == 0) *count_s = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (t + i * THREADS < n && score[i] >= bound) put(mine[i]);
    __syncthreads();
    n = *count_s;
  }
  if (n > kRanked) {
    // too many at the bound: a bound of the exact scores that few enough reach, or, where
    // ties at it are too many, one of their places, too
    auto* range = reinterpret_cast<unsigned long long*>(found);
    int* values = reinterpret_cast<int*>(found + 1);
    // the largest bound that `need` keys reach, as far as it takes until no more than `room` do, by
    // counts of eight bits at a time, each from the first that differs among those left; `reach`
    // do, and `above` lie above it
    const auto bound_of_keys = [&](const auto& keys, int need, int room, int& reach, int& above) {
      uint64_t bound = 0;
      reach = INT_MAX;
      above = 0;
      for (int low = 64; low > 0;) {              // bits from `low` on are found
        uint64_t hi = 0, lo = ~uint64_t(0);
        keys([&](uint64_t x) {
          if ((x ^ bound) >> (low - 1) >> 1 != 0) return;
          hi = max(hi, x);
          lo = min(lo, x);
        });
#pragma unroll
        for (int d = kWarp / 2; d > 0; d /= 2) {
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, d));
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        }
        __syncthreads();                          // (what `found` held before is read)
        if (t == 0) {
          range[0] = 0;
          range[1] = ~0ull;
        }
        for (int i = t; i < kValues; i += THREADS) values[i] = 0;
        __syncthreads();
        if (t % kWarp == 0) {
          atomicMax(&range[0], hi);
          atomicMin(&range[1], lo);
        }
        __syncthreads();
        hi = range[0];
        lo = range[1];
        // (none: bad starts let another group write the rows' states meanwhile; both agree with
        // `bound` from `low` on, so `low` falls whatever they hold)
        if (hi < lo) break;
        bound = hi;
        if (hi == lo) break;
        low = 64 - __clzll(hi ^ lo);
        bound = hi >> (low - 1) >> 1 << 1 << (low - 1);
        const int next = max(low - 8, 0);
        keys([&](uint64_t x) {
          if ((x ^ bound) >> (low - 1) >> 1 == 0) atomicAdd(&values[(x >> next) & ((1 << (low - next)) - 1)], 1);
        });
        __syncthreads();
        int value, there;
        reached(values, need - above, value, there);
        bound |= static_cast<uint64_t>(value) << next;
        reach = above + there;
        if (reach <= room) break;
        above += there - values[value];
        low = next;
        __syncthreads();                          // `values` and `range` are read
      }
      return bound;
    };
    const auto exact = [&](const auto& f) {
      each(bound, INT_MAX, [&](int row, int token, float logit, float offset) {
        if (raised(offset) + logit >= bound) f(key_of(score_of(row, logit)), row, token, logit);
      });
    };
    const auto place_of = [&](int row, int token) {   // later ones less
      return ~(static_cast<uint64_t>(row) * static_cast<uint64_t>(p.a.vocab) + static_cast<uint64_t>(token));
    };
    int reach, above;
    const uint64_t k = bound_of_keys(
        [&](const auto& f) { exact([&](uint64_t x, int, int, float) { f(x); }); }, width, kRanked, reach, above);
    uint64_t first = 0;
    if (reach > kRanked) {
      int more, before;
      first = bound_of_keys(
          [&](const auto& f) {
            exact([&](uint64_t x, int row, int token, float) {
              if (x == k) f(place_of(row, token));
            });
          },
          width - above, kRanked - above, more, before);
    }
    __syncthreads();
    if (t == 0) *count_s = 0;
    __syncthreads();
    exact([&](uint64_t x, int row, int token, float logit) {
      if (x > k || (x == k && place_of(row, token) >= first)) put(Candidate{__float_as_uint(logit), row, token});
    });
    __syncthreads();
    n = min(*count_s, kRanked);
  }
  for (int i = t; i < n; i += THREADS) {
    const Candidate c = found[i];
    found[i].key = key_of(score_of(c.row, __uint_as_float(static_cast<uint32_t>(c.key))));
  }
  __syncthreads();
  // ---- ranks: a candidate by several threads, where there are few
  const int64_t out = static_cast<int64_t>(blockIdx.x) * width;
  int share = 1;
  while (2 * share <= kWarp && 2 * share * n <= THREADS) share *= 2;
  for (int i0 = 0; i0 < n; i0 += THREADS / share) {
    const int i = i0 + t / share;
    const Candidate c = found[min(i, n - 1)];
    const uint64_t mine = index_of(c.row, c.token);
    int rank = 0;
#pragma unroll 4
    for (int j = t % share; j < n; j += share) {
      const Candidate d = found[j];
      rank += d.key > c.key || (d.key == c.key && index_of(d.row, d.token) < mine);
    }
    for (int d = 1; d < share; d *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, d);
    if (i < n && t % share == 0 && rank < width) {
      p.a.out_scores[out + rank] = static_cast<float>(of_key(c.key));
      p.a.out_rows[out + rank] = static_cast<int>(s0) + c.row;
      p.a.out_tokens[out + rank] = c.token;
    }
  }
  for (int i = n + t; i < width; i += THREADS) {
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

// What bounds it: a chain of loads and barriers: sums, tops of the lists, a part of the lists,
// the lists, ranks (64 groups of 26 lists 12 us, 4 groups of 206 lists of 100 20 us).
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ Params p) {
  __shared__ Candidate found[kFinal];
  __shared__ uint32_t red[kRed * kJoinThreads / kWarp];
  __shared__ int count_s, n_open, open[kLists], list_count[kLists];   // open: lists to look at
  __shared__ float list_top[kLists];             // largest (raised) score of each
  __shared__ RowState here[kRowsJoin];
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp;
  pdl_wait();
  pdl_trigger();
  int64_t s0, s1;
  group_rows(p, blockIdx.x, s0, s1);
  const int chunks = p.chunks;
  RowState* state = s1 - s0 <= kRowsJoin ? here : p.rows + s0;
  const auto score_of_row = [&](int64_t row) { return p.a.scores && row < s1 - s0 ? p.a.scores[s0 + row] : 0.f; };
  const float mine = score_of_row(t);
  // ---- the rows' sums, a warp each, then their logarithms, a thread each
  for (int64_t row = warp; row < s1 - s0; row += kJoinThreads / kWarp) {
    const Part* parts = p.parts + (s0 + row) * chunks;
    const Part first = lane < chunks ? parts[lane] : Part{Sum{0.f, 0.f}, -INFINITY, -INFINITY, 0, 0};
    uint32_t hi = key_of(first.ref);
    for (int c = lane + kWarp; c < chunks; c += kWarp) hi = max(hi, key_of(parts[c].ref));
    const float ref = of_key(__reduce_max_sync(0xffffffffu, hi));
    Sum sum = moved(first.sum, first.ref, ref);
    for (int c = lane + kWarp; c < chunks; c += kWarp) {
      const Sum x = moved(parts[c].sum, parts[c].ref, ref);
      sum.rest += x.rest;
      sum.add(x.sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) state[row] = RowState{sum, ref, 0.f};
  }
  __syncthreads();
  for (int64_t row = t; row < s1 - s0; row += kJoinThreads) {
    RowState s = state[row];
    s.score = row == t ? mine : score_of_row(row);
    row_state(p, s);
    state[row] = s;
  }
  __syncthreads();
  // ---- the lists, a warp each; those whose largest logit lies below the bound are passed over
  // (below 2^31, as all rows' chunks are)
  const unsigned lists = static_cast<unsigned>((s1 - s0) * chunks), per_row = chunks;
  const bool few = lists <= kLists;
  const auto score_of_list = [&](unsigned l) { return raised(state[l / per_row].offset) + p.parts[s0 * chunks + l].top; };
  float most = -INFINITY;
  for (unsigned l = t; l < lists; l += kJoinThreads) {
    const float offset = state[l / per_row].offset;
    const Part& part = p.parts[s0 * chunks + l];
    const float top = part.top;
    if (few) {
      list_top[l] = raised(offset) + top;
      list_count[l] = part.count;
    }
    most = fmaxf(most, lowered(offset) + top);
  }
  // where there are lists enough, one of their largest logits bounds the places
  const float bound = lists >= static_cast<unsigned>(p.a.width) ? score_bound<kJoinThreads>(most, p.a.width, red) : -FLT_MAX;
  const auto each = [&](float least, int entries_each, const auto& f) {
    __syncthreads();                              // `open` and its count are read
    if (t == 0) n_open = 0;
    __syncthreads();
    for (unsigned l = t; l < lists; l += kJoinThreads) {
      if (!((few ? list_top[l] : score_of_list(l)) >= least)) continue;
      const int at = atomicAdd(&n_open, 1);
      if (at < kLists) open[at] = static_cast<int>(l);
    }
    __syncthreads();
    const bool known = n_open <= kLists;          // else all of them are gone through
    const unsigned n_lists = known ? n_open : lists;
    // kAtOnce lists at a time, kOfEach times 32 entries of each
    constexpr int kAtOnce = 2, kOfEach = 2, kWarps = kJoinThreads / kWarp;
    for (unsigned i0 = warp; i0 < n_lists; i0 += kAtOnce * kWarps) {
      const Entry* entries[kAtOnce];
      int row[kAtOnce], n[kAtOnce], longest = 0;
      float offset[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const unsigned i = i0 + k * kWarps;
        n[k] = 0;
        if (i >= n_lists) continue;
        const unsigned l = known ? open[i] : i;
        row[k] = static_cast<int>(l / per_row);
        offset[k] = state[row[k]].offset;
        n[k] = offset[k] == -INFINITY ? 0 : min(few ? list_count[l] : p.parts[s0 * chunks + l].count, entries_each);
        entries[k] = p.entries + (s0 * chunks + l) * p.cap;
        longest = max(longest, n[k]);
      }
      for (int j = lane; j < longest; j += kOfEach * kWarp) {
        Entry x[kAtOnce][kOfEach];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int u = 0; u < kOfEach; ++u)
            if (j + u * kWarp < n[k]) x[k][u] = entries[k][j + u * kWarp];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int u = 0; u < kOfEach; ++u)
            if (j + u * kWarp < n[k]) f(row[k], x[k][u].token, x[k][u].logit, offset[k]);
      }
    }
  };
  select_of<kJoinThreads, true>(p, s0, state, bound, each, found, red, &count_s);
}

// Everything of a group in one CTA: its rows stay in L1 between the passes. What bounds it: the
// chain of its passes (4 rows of 256 logits 9 to 10 us, 256 groups of 32 such rows 14).
template <int DT>
__global__ void __launch_bounds__(kSmallThreads, 2) beam_small_kernel(const __grid_constant__ Params p) {
  __shared__ Candidate found[kFinal];
  __shared__ RowState here[kRowsHere];
  __shared__ uint32_t red[kRed * kSmallThreads / kWarp];
  __shared__ int count_s;
  const int t = threadIdx.x, lane = t % kWarp, warp = t / kWarp, vocab = static_cast<int>(p.a.vocab);
  pdl_wait();
  pdl_trigger();
  int64_t s0, s1;
  group_rows(p, blockIdx.x, s0, s1);
  RowState* state = s1 - s0 <= kRowsHere ? here : p.rows + s0;
  // eight logits of a row, kWarp apart
  const auto load8 = [&](float (&x)[8], int64_t row, int first) {
    uint8_t may[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = first + i * kWarp;
      x[i] = e < vocab ? load_element<DT>(p.a.logits, row * p.a.ld + e) : -INFINITY;
      may[i] = p.a.allowed && e < vocab ? p.a.allowed[row * p.a.ld_allowed + e] : 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = may[i] ? x[i] : -INFINITY;
  };
  // up to kHeld rows a warp of up to 256 logits stay in registers, and are read once
  constexpr int kWarps = kSmallThreads / kWarp, kHeld = 2;
  const bool holds = s1 - s0 <= kHeld * kWarps && vocab <= 256;
  float held[kHeld][8];
  const auto sums = [&](int64_t row, float (&x)[8], bool loaded) {
    float top = -INFINITY;
    for (int e = lane; e < vocab; e += 8 * kWarp) {
      if (!loaded) load8(x, row, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
    }
    top = of_key(__reduce_max_sync(0xffffffffu, key_of(top)));
    const float ref = top == -INFINITY ? 0.f : top;
    Sum sum{0.f, 0.f};
    for (int e = lane; e < vocab; e += 8 * kWarp) {
      if (vocab > 8 * kWarp) load8(x, row, e);    // (else they are there)
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) part += exp_from(x[i], ref);
      sum.add(part);
    }
    sum = warp_sum(sum);
    if (lane == 0) state[row - s0] = RowState{sum, top, 0.f};
  };
  if (holds) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (warp + k * kWarps < s1 - s0) load8(held[k], s0 + warp + k * kWarps, lane);
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (warp + k * kWarps < s1 - s0) sums(s0 + warp + k * kWarps, held[k], true);
  } else {
    for (int64_t row = s0 + warp; row < s1; row += kWarps) {
      float x[8];
      sums(row, x, false);
    }
  }
  __syncthreads();
  for (int64_t row = t; row < s1 - s0; row += kSmallThreads) {
    RowState s = state[row];
    s.score = p.a.scores ? p.a.scores[s0 + row] : 0.f;
    row_state(p, s);
    state[row] = s;
  }
  __syncthreads();
  // a warp takes 256 tokens of a row at a time
  const int pieces = (vocab + 255) / 256;
  const int64_t all = (s1 - s0) * pieces;
  const auto divided = [&](int64_t u) {           // by the pieces of a row
    return all >> 32 ? u / pieces : static_cast<int64_t>(static_cast<uint32_t>(u) / static_cast<uint32_t>(pieces));
  };
  const auto each = [&](float, int, const auto& f) {
    if (holds) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int row = warp + k * kWarps;
        const float offset = row < s1 - s0 ? state[row].offset : -INFINITY;
        if (offset == -INFINITY) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (held[k][i] > -INFINITY) f(row, lane + i * kWarp, held[k][i], offset);
      }
      return;
    }
    for (int64_t u = warp; u < all; u += kWarps) {
      const int row = static_cast<int>(divided(u)), first = static_cast<int>(u - static_cast<int64_t>(row) * pieces) * 256 + lane;
      const float offset = state[row].offset;
      if (offset == -INFINITY) continue;
      float x[8];
      load8(x, s0 + row, first);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x[i] > -INFINITY) f(row, first + i * kWarp, x[i], offset);
    }
  };
  select_of<kSmallThreads, false>(p, s0, state, -FLT_MAX, each, found, red, &count_s);
}

// ------------------------------------------------------------------ launches

// One launch for groups of at most this many logits, on average: the host does not know more of the
// groups. Where one of them holds all rows, its CTA does all the work: 64 groups of 16 x 256
// fp32 logits 22 us, one of 1024 x 256 among 63 without rows 134; 256 groups of 4 x 4096 25, one of
// 1024 x 4096 2190.
constexpr int64_t kSmallGroup = 32768;
constexpr int kSmallVocab = 4096;
// CTAs of the scan that chunks are made for: one for each place that the SMs have for masked
// rows (33 of 1,000,003 with 825 CTAs took 60 us, with 1155 68, 1650 65; 8 places without a mask).
constexpr int64_t kScanCtas = 152 * 6;
constexpr int kLeastTiles = 2, kMostTiles = 16;  // of a chunk

struct Plan {
  bool small;
  int chunks, tiles, cap;
  int64_t parts, entries, bytes;                 // offsets of the scratch, and its size
};
Plan plan_of(const dlrm_beam_select_t& a) {
  Plan s{};
  s.small = a.rows == 0 || (a.vocab <= kSmallVocab && a.rows * a.vocab <= kSmallGroup * a.groups);
  if (s.small && a.rows <= kRowsHere) return s;
  s.bytes = a.rows * static_cast<int64_t>(sizeof(RowState));
  if (s.small) return s;
  const int vec = a.dtype == DLRM_DTYPE_FP32 ? 4 : 8;
  const int64_t tile = kScanThreads * kVectors * vec, tiles = (a.vocab + tile - 1) / tile;
  const int64_t chunks = std::max((tiles + kMostTiles - 1) / kMostTiles,
                                  std::min(kScanCtas / a.rows, (tiles + kLeastTiles - 1) / kLeastTiles));
  s.tiles = static_cast<int>((tiles + chunks - 1) / chunks);
  s.chunks = static_cast<int>((tiles + s.tiles - 1) / s.tiles);
  s.cap = 8 * a.width + 256;
  s.parts = s.bytes;
  s.entries = s.parts + a.rows * s.chunks * static_cast<int64_t>(sizeof(Part));
  s.bytes = s.entries + a.rows * s.chunks * s.cap * static_cast<int64_t>(sizeof(Entry));
  return s;
}

template <int DT>
cudaError_t launch(const Params& p, bool small, cudaStream_t stream) {
  if (small)
    return launch_pdl(beam_small_kernel<DT>, dim3(p.a.groups), dim3(kSmallThreads), 0, stream, p);
  const dim3 grid(static_cast<unsigned>(p.a.rows * p.chunks));
  const size_t smem = 2 * p.cap * sizeof(Entry);
  const cudaError_t e = launch_pdl(p.a.allowed ? beam_scan_kernel<DT, true> : beam_scan_kernel<DT, false>, grid,
                                   dim3(kScanThreads), smem, stream, p);
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
