// Attention on the 5th-generation tensor cores: the kernel that
// window_attention_tc.cu (rows of keys and values, by TMA) and
// history_attention_tc.cu (8-bit pages, converted on the way) instantiate.
//
// A work unit is 256 rows, as two tiles of 128 (the MMA's M), of one kv head of
// a request; rows are (query, head of the group) pairs. Persistent CTAs, one
// per SM, or two where tensor and shared memory have room (plain rows, head_dim up
// to 64: the ragged batch below 58 us against 64). Per unit the keys that any of its rows sees flow by in key tiles of at
// most 64 events: the sinks that lie apart from the window first (a narrow
// tile), then the window from its first event on.
//   warp 11: finds the units and writes what the others need of them into a
//     ring in shared memory;
//   warp 10, one lane: TMA of key and value tiles (boxes of 32 events x 64
//     elements, 128-byte swizzle) through rings of four stages each. PAGED:
//     warps 12-15 load codes instead, a tile ahead in registers, and write them
//     as bf16 with their page's scale, which is exact (a code has 4 bits, the
//     scale is a power of two);
//   warps 8 and 9, one lane each: the products of tile 0 and 1: S_t = Q_t K^T
//     (operands from shared memory), then, when the weights are there, O_t += P_t V
//     (P from tensor memory, V as stored: the MN-major operand form). One lane's
//     waits and issues take about as long as a tile's softmax, hence two warps.
//     They also load their tile's queries, by TMA where the group divides 128
//     (else the softmax warps do);
//   warps 0-3 and 4-7: softmax of tile 0 and 1. A thread owns a row: it reads
//     its 64 scores from tensor memory, masks, takes the maximum, writes the
//     weights in the input's type (8 bits of them in bf16, 11 in fp16) over the scores,
//     and keeps their sum as it was before the rounding. The
//     output is only corrected when a row's maximum has grown by more than 2^8
//     over the reference in use (weights up to 2^8 are as exact, and the sum is
//     fp32), which real scores do in the first tiles only. 32 columns that none
//     of a warp's rows sees are neither read nor exponentiated. The outputs' sums are
//     the tensor core's fp32, which cuts off what it adds: a sum loses up to 2^-24 of
//     itself for every 16 events (fp16, one CTA: 1.3e-4 measured over 65,000, 5.2e-4 over
//     131,072), as much as one weight's rounding at 65,000 events in fp16, 500,000 in bf16.
// Tensor memory: two score buffers of 64 columns a tile, two of weights (32) and
// the output. The scores of the next key tile are made while the softmax works on
// this one's. At head_dim 128 there is no room for the weights: they lie over
// their scores, whose buffer is then only free when the weights have been used.
// Two CTAs an SM have one score buffer a tile, weights over it, and overlap each
// other instead.
//
// PAGED: candidates of few users make few units, so the key tiles of all units
// are cut evenly over the CTAs, as in history_attention.cu; a unit that is split
// leaves partial outputs, and of each tile's warps the one that arrives last
// joins its 32 rows, in the order of the events.
//
// What bounds it: the steps of the softmax between the two products. A step of 64 keys
// takes its warps, two a scheduler, about 2000 cycles, 700 of them the exponentials; most
// of the others are waits of one role for another (scores, tensor memory, weights). The
// tensor pipe is 48% active at head_dim 128. More softmax warps leave each too
// few registers (16 warps 298 us against 254; moving registers between the roles is not
// tried), and powers by a polynomial on the FMA pipe cost more issue slots than the
// special function unit saves (269).
// Measured: 2 x 16384 events, 8 heads of 128, window 2048, fp16: 258 us, 1.0
// PFLOP/s of visible products (52% of the bf16 rate); 64 users of 100 to 1024 events,
// 8 heads of 64 over 2, window 256, bf16: 58 us, of which the first loads and the last
// products of short units are 10K of 26K cycles a unit; PAGED, 16 users x up to 500
// candidates over 1000 to 4096 events, 4 heads of 64 over 2: 63 us, 0.28 PFLOP/s.
//
// Every wait is bounded (WaitCfg); on expiry DLRM_ERRBIT_TIMEOUT is set, every
// role leaves its loop, work in flight is waited for and the tensor memory freed. PAGED:
// the CTA still counts for the units that it shares, so that the counters end at zero.
// (How the code of the roles falls into the instruction cache is worth up to 6% of the
// ragged batch: a branch more in the loop of warp 10, or a call after it, took 58 us to 61.)
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "tc.cuh"
#include "window_attention.cuh"

namespace dlrm {

using namespace tc;

namespace {

template <bool PAGED>
constexpr int kThreadsOf = PAGED ? 512 : 384;
constexpr int kUnit = 256;                       // rows of a work unit
constexpr int kKeys = 64;                        // events of a key tile
constexpr int kBox = 32;                         // events of one TMA box
constexpr int kQBlock = 128 * 128;               // 128 rows of 128 bytes (64 elements)
constexpr int kBlockBytes = kKeys * 128;         // the same of a key tile
constexpr int kStages = 4;                       // of keys, and of values
constexpr uint64_t kLandNs = 10000000;           // limit of a wait for work in flight
constexpr float kSlack = 8.f;                    // log2 of the largest weight
// ... and f16 weights are 2^kRaise times larger, as in kLift
template <int DT>
constexpr int kRaise = DT == DLRM_DTYPE_FP16 ? kLift - 8 : 0;

// Resident CTAs of an SM, score buffers of a tile, tensor memory columns.
template <int D, bool PAGED>
constexpr int kCtas = D == 128 || PAGED ? 1 : 2;
template <int D, bool PAGED>
constexpr int kBufs = 3 - kCtas<D, PAGED>;

template <int D, bool PAGED>
struct Layout {
  static constexpr int kBlocks = (D + 63) / 64;  // 64-element column blocks
  static constexpr int kTile = kBlocks * kBlockBytes;
  static constexpr int kQTile = kBlocks * kQBlock;
  static constexpr int kQ = 0;                   // two query tiles
  static constexpr int kK = 2 * kQTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kBars = kV + kStages * kTile;
  // a lone CTA takes all of the tensor memory, so it asks for more than half an
  // SM's shared memory
  static constexpr int kNeed = kBars + 1024 + 1024;
  static constexpr bool kAlone = kCtas<D, PAGED> == 1;
  static constexpr int kSmem = kAlone && kNeed < 120 * 1024 ? 120 * 1024 : kNeed;
  static_assert(kSmem <= (kAlone ? 232448 : 115712), "shared memory of an SM");
  // tensor memory columns: scores of tile t in buffer i, its weights, its output.
  // Where there is no room for the weights they lie over their scores: with two
  // CTAs an SM, and at head_dim 128.
  static constexpr int kB = kBufs<D, PAGED>;
  static constexpr bool kOver = D == 128 || kB == 1;
  static constexpr int kColumns = kB == 1 ? 256 : 512;
  static __device__ __forceinline__ int s_col(int t, int i) { return (t * kB + i) * kKeys; }
  static __device__ __forceinline__ int o_col(int t) {
    return 2 * kB * kKeys + t * (D == 128 ? 128 : 64);
  }
  static __device__ __forceinline__ int p_col(int t, int i) {
    return kOver ? s_col(t, i) : 384 + t * 64 + i * 32;
  }
};

// n / d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d) and
// mul = floor(2^32 (2^s - d) / d) + 1, n / d = (hi32(n mul) + n) >> s (the
// method of Granlund and Montgomery for invariant divisors).
struct FastDiv {
  uint32_t mul, shift, d;
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};
FastDiv fast_div(int d) {
  FastDiv f{};
  f.d = static_cast<uint32_t>(d);
  while ((uint64_t(1) << f.shift) < f.d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - f.d)) / f.d + 1);
  return f;
}

struct TcParams {
  WindowParams w;
  dlrm_history_t h;                              // PAGED
  int32_t* counters;
  float* partials;
  FastDiv group, heads;
  int most;                                      // units that starts which never decrease make
  int vec_out;
  int q_tma;                                     // queries by TMA: boxes of group x 128 / group
  WaitCfg wait;
};

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(
                   smem_addr(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Not inline: a copy at every wait costs instruction cache (batch 66 -> 80 us).
// Bounded wait for a phase; false once this or another thread gave up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                       int32_t* err, uint64_t limit) {
  const uint32_t a = smem_addr(bar);
  const uint64_t t0 = now_ns();
  for (uint32_t i = 1;; ++i) {
    if (try_wait(a, parity)) return true;
    if ((i & 15) == 0) {
      if (*abort_flag) return false;
      if (now_ns() - t0 > limit) {
        *abort_flag = 1;
        flag(err, DLRM_ERRBIT_TIMEOUT);
        return false;
      }
    }
  }
}
struct Waiter {
  volatile int* abort_flag;
  int32_t* err;
  uint64_t limit;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (try_wait(smem_addr(bar), parity)) return true;
    return wait_slow(bar, parity, abort_flag, err, limit);
  }
  // regardless of the abort flag and the limit: work in flight, which takes microseconds
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    const uint64_t t0 = now_ns();
    while (!try_wait(smem_addr(bar), parity)) {
      if (now_ns() - t0 > kLandNs) {
        flag(err, DLRM_ERRBIT_TIMEOUT);
        return;
      }
    }
  }
};

// Shared-memory descriptors: the low word holds the start address (and the
// leading byte offset), the high word is the same for all operands here:
// 8-row groups 1024 bytes apart, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// rows of the inner dimension (queries, keys): K-major
__device__ __forceinline__ uint32_t rows_desc(uint32_t addr) { return (addr >> 4) | (1u << 16); }
// values, as the B operand of P V: MN-major, an event's 64 elements are a row
// of 128 bytes, 64-element column blocks kBlockBytes apart
__device__ __forceinline__ uint32_t values_desc(uint32_t addr) {
  return (addr >> 4) | (static_cast<uint32_t>(kBlockBytes >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// A in tensor memory: the weights.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
      "%27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
      "%27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// A request's rows; PAGED: over the history of a slot, which k0 holds.
template <bool PAGED>
__device__ __forceinline__ WindowSpan tc_span(const TcParams& p, int b, bool report) {
  if (!PAGED) return window_span(p.w, b, kUnit, report);
  const dlrm_attention_t& a = p.w.a;
  const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1], slot = a.slots[b];
  const bool bad = q0 < 0 || q1 < q0 || q1 > a.q_rows;
  const bool known = slot >= 0 && slot < p.h.n_slots;
  if (report && bad) flag(p.h.err, DLRM_ERRBIT_OFFSETS);
  if (report && !known) flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);
  WindowSpan s;
  s.q0 = q0;
  s.k0 = slot;
  s.rows = bad ? 0 : (q1 - q0) * p.w.group;
  s.len = 0;
  if (known) {
    const int64_t cap = static_cast<int64_t>(p.h.max_pages) * p.h.page_tokens;
    s.len = static_cast<int>(min(static_cast<int64_t>(max(p.h.lengths[slot], 0)), cap));
  }
  s.tiles = (s.rows + kUnit - 1) / kUnit;
  return s;
}

// One work unit, in shared memory.
struct Unit {
  int valid, head, row0;                         // row0: first row of tile 0
  WindowSpan s;
  int pos0;                                      // position of the request's first query
  int rows[2];                                   // rows of each tile
  int end1[2], gap0[2], gap1[2];                 // of a tile's last row: end, gap0; of its first: gap1
  int last[2];                                   // last key tile that a tile needs, -1: none
  int sink, lo, end, sink_tiles;                 // keys [0, sink) and [lo, end)
  int begin, tiles;                              // key tiles [begin, tiles) are this CTA's
  int parts, part0, place;                       // CTAs that share the unit, the first; partial's place

  // Key tile k: events [key0, key0 + n).
  __device__ __forceinline__ void tile(int k, int& key0, int& n) const {
    if (k < sink_tiles) {
      key0 = k * kKeys;
      n = min(kKeys, sink - key0);
    } else {
      key0 = lo + (k - sink_tiles) * kKeys;
      n = min(kKeys, end - key0);
    }
  }
  __device__ __forceinline__ bool needs(int t, int key0, int n) const {
    return rows[t] > 0 && key0 < end1[t] && !(key0 >= gap0[t] && key0 + n <= gap1[t]);
  }
};
constexpr int kUnits = 3;                        // units known ahead
template <bool PAGED>
constexpr int kReaders = PAGED ? 14 : 11;        // warps that read a unit

// What a loop over key tiles needs of a unit, in registers.
struct Keys {
  int lo, end, sink, sink_tiles, begin, tiles;
  bool have[2];
  int end1[2], gap0[2], gap1[2];
  __device__ __forceinline__ explicit Keys(const Unit& x)
      : lo(x.lo), end(x.end), sink(x.sink), sink_tiles(x.sink_tiles), begin(x.begin), tiles(x.tiles) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      have[t] = x.rows[t] > 0;
      end1[t] = x.end1[t];
      gap0[t] = x.gap0[t];
      gap1[t] = x.gap1[t];
    }
  }
  __device__ __forceinline__ void tile(int k, int& key0, int& n) const {
    const bool s = k < sink_tiles;
    key0 = s ? k * kKeys : lo + (k - sink_tiles) * kKeys;
    n = min(kKeys, (s ? sink : end) - key0);
  }
  template <int T>
  __device__ __forceinline__ bool needs(int key0, int n) const {
    return have[T] && key0 < end1[T] && !(key0 >= gap0[T] && key0 + n <= gap1[T]);
  }
};

struct Bars {
  uint64_t q_full[2], k_full[kStages], k_empty[kStages], v_full[kStages],
      v_empty[kStages], s_full[2][2], p_full[2][2], pv_done[2][2], o_empty[2], u_full[kUnits],
      u_empty[kUnits], drain[2];
  uint32_t tmem;
  int abort;
  Unit units[kUnits];
};
static_assert(sizeof(Bars) <= 1024, "space behind the tiles");

// Unit i of the request with rows s, by one thread: all its key tiles.
template <bool PAGED>
__device__ __forceinline__ Unit make_unit(const TcParams& tp, int i, const WindowSpan& s) {
  const WindowParams& p = tp.w;
  Unit x;
  x.valid = 1;
  x.s = s;
  // the last rows of a request first: without a window they see the most
  const int tile = tp.heads(i);
  x.head = i - tile * p.a.n_kv_heads;
  x.row0 = (s.tiles - 1 - tile) * kUnit;
  x.pos0 = p.a.causal ? s.len - tp.group(s.rows) : s.len - 1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    x.rows[t] = max(0, min(128, s.rows - x.row0 - 128 * t));
    const int r0 = min(x.row0 + 128 * t, s.rows - 1), r1 = max(r0, r0 + x.rows[t] - 1);
    const int step = p.a.causal ? 1 : 0;
    const Visible first = visible(x.pos0 + step * tp.group(r0), s.len, p.a.window, p.a.sinks);
    const Visible last = visible(x.pos0 + step * tp.group(r1), s.len, p.a.window, p.a.sinks);
    x.end1[t] = last.end;
    x.gap0[t] = last.gap0;
    x.gap1[t] = first.gap1;
  }
  const int u = x.rows[1] > 0 ? 1 : 0;
  x.end = x.end1[u];
  const bool apart = x.gap1[0] > x.gap0[u];
  x.lo = apart ? min(x.gap1[0], x.end) : 0;
  x.sink = apart ? min(x.gap0[u], x.end) : 0;
  if (PAGED) {
    // a box of 32 events lies in one page; events before the window are masked,
    // and must not be sinks again
    x.lo &= ~(kBox - 1);
    x.sink = min(x.sink, x.lo);
  }
  x.sink_tiles = (x.sink + kKeys - 1) / kKeys;
  x.begin = 0;
  x.tiles = x.sink_tiles + (x.end - x.lo + kKeys - 1) / kKeys;
  x.parts = 1;
  x.part0 = x.place = 0;
  return x;
}

// The last key tile of the unit's that each of its tiles needs.
__device__ __forceinline__ void find_last(Unit& x) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    x.last[t] = -1;
    for (int k = x.tiles - 1; k >= x.begin; --k) {
      int key0, n;
      x.tile(k, key0, n);
      if (x.needs(t, key0, n)) {
        x.last[t] = k;
        break;
      }
    }
  }
}

// Finds a CTA's units in order, by one warp.
struct Walk {
  int b = 0;
  int before = 0;                                // units of the requests before b

  __device__ __forceinline__ void find(const TcParams& tp, int u, Unit& x) {
    const WindowParams& p = tp.w;
    const int lane = threadIdx.x % kWarp;
    const int heads = p.a.n_kv_heads;
    WindowSpan s{};
    for (;;) {
      // (starts that decrease can claim rows many times over: not without end)
      if (b >= p.a.batch || u >= tp.most) {
        if (lane == 0) x.valid = 0;
        return;
      }
      int n = 0;
      if (b + lane < p.a.batch) {
        s = window_span(p, b + lane, kUnit, false);
        n = s.tiles * heads;
      }
      int inc = n;
#pragma unroll
      for (int d = 1; d < kWarp; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + inc > u);
      if (past) {
        const int at = __ffs(past) - 1;
        before += __shfl_sync(0xffffffffu, inc - n, at);
        if (lane == at) {
          x = make_unit<false>(tp, u - before, s);
          find_last(x);
        }
        b += at;
        return;
      }
      before += __shfl_sync(0xffffffffu, inc, kWarp - 1);
      b += kWarp;
    }
  }
};

// PAGED: key tiles that the rows of a request see, one at least: what a unit
// counts when the work is cut. Units of up to kWhole are not split, and of longer
// ones a CTA takes kLeast at least: one user x 4096 events x 128 rows takes 31 us in
// parts of 16 key tiles, 121 in parts of one.
constexpr int kWhole = 8, kLeast = 16;
__device__ __forceinline__ int key_tiles(const TcParams& p, const WindowSpan& s) {
  const dlrm_attention_t& a = p.w.a;
  const int queries = p.group(s.rows);
  const Visible first = visible(a.causal ? s.len - queries : s.len - 1, s.len, a.window, a.sinks);
  const int sink = min(first.gap0, s.len), lo = first.gap1;
  return max((sink + kKeys - 1) / kKeys + max(s.len - lo + kKeys - 1, 0) / kKeys, 1);
}

// PAGED: the units of a CTA's part of all key tiles in order, by one thread.
struct PagedWalk {
  int u = 0, end = 0, b = 0, first = 0, each = 1;
  WindowSpan s{};

  __device__ __forceinline__ PagedWalk(const TcParams& p, const Cuts& cuts, const Found<WindowSpan>& found) {
    if (cuts.total == 0) return;
    // a cut inside a short unit moves to the unit's start
    auto snap = [&](int u, int i) {
      const int each = key_tiles(p, found.span[i]);
      return u >= cuts.total || each > kWhole ? u : u - (u - found.first[i]) % each;
    };
    u = snap(cuts.cut(blockIdx.x), 0);
    end = snap(cuts.cut(blockIdx.x + 1), 1);
    b = found.request[0];
    first = found.first[0];
    s = found.span[0];
    each = key_tiles(p, s);
  }
  // false: no more
  __device__ __forceinline__ bool next(const TcParams& p, const Cuts& cuts, Unit& x) {
    if (u >= end) return false;
    const int heads = p.w.a.n_kv_heads;
    while (u - first >= s.tiles * heads * each) {
      first += s.tiles * heads * each;
      s = tc_span<true>(p, ++b, false);
      each = key_tiles(p, s);
    }
    const int i = (u - first) / each, from = u - first - i * each;
    const int to = min(each, from + end - u);
    x = make_unit<true>(p, i, s);
    // its part of the unit's own key tiles
    const int64_t all = x.tiles;
    x.begin = static_cast<int>(from * all / each);
    x.tiles = static_cast<int>(to * all / each);
    find_last(x);
    const int unit0 = first + i * each;
    x.part0 = cuts.owner(unit0);
    x.parts = from > 0 || to < each ? cuts.owner(unit0 + each - 1) - x.part0 + 1 : 1;
    x.place = from > 0 ? 0 : 1;
    u += to - from;
    return true;
  }
};

// PAGED: a CTA that gave up still counts for the units that it shares, from the first that
// each softmax warp has not finished on: counters are zero after every call. One thread.
__device__ __noinline__ void count_given_up(const TcParams& p, const Cuts& cuts, const Found<WindowSpan>& found,
                                            const int* finished) {
  PagedWalk walk(p, cuts, found);
  Unit x;
  for (int n = 0; walk.next(p, cuts, x); ++n) {
    if (x.parts == 1) continue;
    for (int w = 0; w < 8; ++w) {
      if (n < finished[w] || x.rows[w / 4] == 0) continue;
      int32_t* counter = &p.counters[x.part0 * 8 + w];
      if (atomicAdd(counter, 1) == x.parts - 1) *counter = 0;
    }
  }
}

// A warp's place in the ring of units; one lane of it may walk alone.
struct Units {
  Bars& bars;
  const Waiter& wait;
  int it = 0;
  __device__ __forceinline__ const Unit* next() {
    const int slot = it % kUnits;
    const bool ok = wait(&bars.u_full[slot], (it / kUnits) & 1);
    const Unit* x = &bars.units[slot];
    return ok && x->valid ? x : nullptr;
  }
  __device__ __forceinline__ void done() { bar_arrive(&bars.u_empty[it++ % kUnits]); }
  // by all lanes
  __device__ __forceinline__ const Unit* next_warp() {
    const Unit* x = next();
    return __all_sync(0xffffffffu, x != nullptr) ? x : nullptr;
  }
  __device__ __forceinline__ void done_warp() {
    __syncwarp();
    if (threadIdx.x % kWarp == 0) bar_arrive(&bars.u_empty[it % kUnits]);
    ++it;
  }
};

// 32 values as pairs, for the packed fp32 instructions.
__device__ __forceinline__ void fma2(float& x, float& y, float f, float c) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mov.b64 c, {%3, %3};\n\tfma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// Bits [0, n) of a word, n any integer.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// PAGED: one row from the definition, by one warp, as window_careful_row.
template <int D, int DT>
__device__ __noinline__ void paged_careful_row(const TcParams& p, const WindowSpan& s, int head,
                                               int row) {
  const dlrm_attention_t& a = p.w.a;
  const int lane = threadIdx.x % kWarp, group = p.w.group, G = p.h.page_tokens;
  const int i = row / group, hq = head * group + row % group;
  const Visible v = visible(a.causal ? s.len - s.rows / group + i : s.len - 1, s.len, a.window, a.sinks);
  const int64_t q_at = (s.q0 + static_cast<int64_t>(i)) * a.ld_q + hq * a.ld_q_head;
  const int32_t* pages = p.h.table + static_cast<int64_t>(s.k0) * p.h.max_pages;
  auto code = [](uint8_t c) { return f16x2_to_float2(e4m3x2_to_f16x2(c)).x; };
  constexpr int N = D / kWarp;
  float q[N], acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = load_element<DT>(a.q, q_at + lane + 32 * e) * (a.scale * kLog2e);
    acc[e] = 0.f;
  }
  float top = -INFINITY, sum = 0.f;
  bool any = false;                               // there are events to see
  for (int t = 0; t < v.end; ++t) {
    if (!sees(v, t)) {
      t = v.gap1 - 1;
      continue;
    }
    const int page = pages[t / G];
    if (page < 0 || page >= p.h.n_pages) continue;
    any = true;
    const int64_t at = static_cast<int64_t>(page) * p.h.n_heads + head;
    const int64_t c = (at * G + t % G) * D + lane;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) x = fmaf(q[e], code(p.h.k_codes[c + 32 * e]), x);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= p.h.k_scales[at];
    const float m = (x > top || x != x) ? x : top;              // a NaN stays
    const float off = m == -INFINITY ? 0.f : m;
    const float f = exp2f(top - off), w = exp2f(x - off);
    top = m;
    sum = fmaf(sum, f, w);
    if (sum != sum) {                                           // so is every output, whatever follows
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = sum;
      break;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      acc[e] = fmaf(acc[e], f, w * p.h.v_scales[at] * code(p.h.v_codes[c + 32 * e]));
  }
  const int64_t o = (s.q0 + static_cast<int64_t>(i)) * a.ld_out + hq * a.ld_out_head;
#pragma unroll
  for (int e = 0; e < N; ++e) store_element<DT>(a.out, o + lane + 32 * e, any ? acc[e] / sum : 0.f);
  if (lane == 0 && a.lse)
    a.lse[(s.q0 + static_cast<int64_t>(i)) * a.n_heads + hq] =
        any ? (top == -INFINITY ? 0.f : top) * kLn2 + logf(sum) : -INFINITY;
}

// The products of tile T of every unit, by one lane. T is no template argument:
// one copy of the code for both tiles keeps more of the kernel in the instruction
// cache (16384 events 265 -> 260 us, the ragged batch 66 -> 63). Returns the phase of
// q_full in which queries may still be landing, -1 for none.
template <int D, int DT, bool PAGED>
__device__ __forceinline__ int products(const int T, const TcParams& p, const CUtensorMap* map_q, Bars& bars,
                                        const Waiter& wait, unsigned char* base, uint32_t tmem) {
  using L = Layout<D, PAGED>;
  constexpr int kFormat = DT == DLRM_DTYPE_BF16 ? 1 : 0;
  // D fp32; A, B formats; M = 128; B of the second product is MN-major
  constexpr uint32_t kIdescS = (1u << 4) | (kFormat << 7) | (kFormat << 10) | (8u << 24);
  constexpr uint32_t kIdescO = kIdescS | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17);
  const uint32_t q_desc = rows_desc(smem_addr(base + L::kQ + T * L::kQTile));
  const uint32_t k_desc = rows_desc(smem_addr(base + L::kK));
  const uint32_t v_desc = values_desc(smem_addr(base + L::kV));
  const uint32_t o = tmem + L::o_col(T);
  uint32_t kv = 0, it = 0, units_done = 0;       // key tiles of the CTA, of this tile; its units
  int landing = -1;
  Units units{bars, wait};
  for (const Unit* x; (x = units.next()); units.done()) {
    const Keys keys(*x);
    // the queries: every score of the unit before has been read, so the tile
    // may be replaced
    if (p.q_tma && x->last[T] >= 0) {
      bar_expect(&bars.q_full[T], L::kQTile);
#pragma unroll
      for (int c = 0; c < L::kBlocks; ++c)
        tma_load_3d(smem_addr(base + L::kQ + T * L::kQTile + c * kQBlock), map_q, c * 64,
                    x->head * p.w.group, x->s.q0 + p.group(x->row0 + 128 * T), &bars.q_full[T]);
      landing = units_done & 1;
    }
    bool due = false, begun = false, used_before = false, queried = false;
    int due_width = 0;
    for (int k = keys.begin; k <= keys.tiles; ++k) {
      int key0 = 0, n = 0;
      bool need = false, used = false;
      if (k < keys.tiles) {
        keys.tile(k, key0, n);
        const bool n0 = keys.needs<0>(key0, n), n1 = keys.needs<1>(key0, n);
        need = T ? n1 : n0;
        used = n0 || n1;
      }
      // scores of this tile, into the buffer of the tile before last (of the tile
      // before, with one buffer)
      auto scores = [&]() -> bool {
        if (!used) return true;
        const uint32_t st = kv % kStages;
        if (!wait(&bars.k_full[st], (kv / kStages) & 1)) return false;
        if (need && !queried) {
          if (!wait(&bars.q_full[T], units_done & 1)) return false;
          landing = -1;
          queried = true;
        }
        if (need) {
          // the old scores have been read: their weights have arrived. Where those
          // lie over them they must have been used too: products of different shapes
          // are not ordered among themselves.
          // (Product i completes phase i / kB of barrier i % kB. Whoever waits for it
          // knows that i - kB is complete, by this wait or by the commit that scores
          // i came with, and that i + kB is not issued: the phase's parity says enough.)
          if (L::kOver && it >= L::kB &&
              !wait(&bars.pv_done[T][it % L::kB], ((it - L::kB) / L::kB) & 1))
            return false;
          fence_after();
          const uint32_t idesc = kIdescS | (n > 32 ? 8u << 17 : 4u << 17);
          const uint32_t sa = tmem + L::s_col(T, it % L::kB), kd = k_desc + st * (L::kTile >> 4);
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            mma_ss(sa, q_desc + (((j / 4) * kQBlock + (j % 4) * 32) >> 4),
                   kd + (((j / 4) * kBlockBytes + (j % 4) * 32) >> 4), idesc, j > 0 ? 1u : 0u);
          mma_commit(smem_addr(&bars.s_full[T][it % L::kB]));
          mma_commit(smem_addr(&bars.k_empty[st]));
        } else {
          bar_arrive(&bars.k_empty[st]);
        }
        return true;
      };
      // products with the values of the tile before
      auto outputs = [&]() -> bool {
        if (!used_before) return true;
        const uint32_t vi = kv - 1, st = vi % kStages;
        if (!wait(&bars.v_full[st], (vi / kStages) & 1)) return false;
        if (due) {
          const uint32_t of = it - 1;
          if (!begun && units_done > 0 && !wait(&bars.o_empty[T], (units_done - 1) & 1)) return false;
          if (!wait(&bars.p_full[T][of % L::kB], (of / L::kB) & 1)) return false;
          fence_after();
          const uint32_t vd = v_desc + st * (L::kTile >> 4), pa = tmem + L::p_col(T, of % L::kB);
          mma_ts(o, pa, vd, kIdescO, begun ? 1u : 0u);
          mma_ts(o, pa + 8, vd + (2048 >> 4), kIdescO, 1u);
          if (due_width > 32) {
            mma_ts(o, pa + 16, vd + 2 * (2048 >> 4), kIdescO, 1u);
            mma_ts(o, pa + 24, vd + 3 * (2048 >> 4), kIdescO, 1u);
          }
          mma_commit(smem_addr(&bars.pv_done[T][of % L::kB]));
          mma_commit(smem_addr(&bars.v_empty[st]));
          begun = true;
        } else {
          bar_arrive(&bars.v_empty[st]);
        }
        return true;
      };
      if (L::kB == 1) {
        if (!outputs() || !scores()) return landing;
      } else {
        if (!scores() || !outputs()) return landing;
      }
      kv += used ? 1 : 0;
      it += need ? 1 : 0;
      used_before = used;
      due = need;
      due_width = n;
    }
    units_done += begun ? 1 : 0;
  }
  return landing;
}

template <int D, int DT, bool PAGED>
__global__ void __launch_bounds__(kThreadsOf<PAGED>, kCtas<D, PAGED>)
attention_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TcParams p) {
  using L = Layout<D, PAGED>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(base + L::kBars);
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const WindowParams& w = p.w;
  const Waiter wait{&bars.abort, PAGED ? p.h.err : w.a.err, wait_limit_ns(p.wait)};

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&bars.tmem)),
                 "n"(L::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      bar_init(&bars.q_full[t], p.q_tma ? 1 : 4);
      for (int i = 0; i < 2; ++i) {
        bar_init(&bars.s_full[t][i], 1);
        bar_init(&bars.p_full[t][i], 4);
        bar_init(&bars.pv_done[t][i], 1);
      }
      bar_init(&bars.o_empty[t], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      bar_init(&bars.k_full[i], PAGED ? 4 : 1);
      bar_init(&bars.k_empty[i], 2);
      bar_init(&bars.v_full[i], PAGED ? 4 : 1);
      bar_init(&bars.v_empty[i], 2);
    }
    for (int i = 0; i < kUnits; ++i) {
      bar_init(&bars.u_full[i], 1);
      bar_init(&bars.u_empty[i], kReaders<PAGED>);
    }
    for (int t = 0; t < 2; ++t) bar_init(&bars.drain[t], 1);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_trigger();

  // PAGED: this CTA's part [begin, end) of all units' key tiles. A request's
  // units count as if each had all the key tiles that any of its rows sees.
  __shared__ Found<WindowSpan> found;
  __shared__ int sums[kThreadsOf<PAGED> / kWarp * 2];
  __shared__ int finished[8];                     // units that a softmax warp has finished
  Cuts cuts{};
  if (PAGED)
    cuts = locate_cuts<kThreadsOf<PAGED>>(
        w.a.batch, kLeast, p.most, [&](int i) { return tc_span<PAGED>(p, i, false); },
        [&](const WindowSpan& s) { return s.tiles * w.a.n_kv_heads * key_tiles(p, s); },
        [&](const WindowSpan& s) { return s.tiles * w.a.n_kv_heads; }, sums, found);

  Units units{bars, wait};
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // all 64 scores of a row in registers, or 32 at a time, read twice: with 16 warps
    // (PAGED) a thread has 128 registers, and the spills cost more (ranking 67 us
    // against 61; with 12 warps the reverse, 270 against 265 at 16384 events)
    constexpr bool kKeep = !PAGED && L::kB == 2;
    const int t = warp / 4;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_at = tmem + lanes + L::o_col(t);
    const float f = w.a.scale * kLog2e;
    uint32_t it = 0;                              // key tiles so far
    bool ok = true;
    for (const Unit* x; ok && (x = units.next_warp()); units.done_warp()) {
      const int rows = x->rows[t];
      if (rows == 0) continue;
      const Keys keys(*x);
      const int r = (warp & 3) * 32 + lane;
      const int row = min(x->row0 + 128 * t + r, x->s.rows - 1);
      const bool in = r < rows;
      const int i = p.group(row);
      const Visible v =
          visible(x->pos0 + (!PAGED || w.a.causal ? i : 0), x->s.len, w.a.window, w.a.sinks);
      if (!p.q_tma && x->last[t] >= 0) {
        // this row's queries; zeros past the last row
        unsigned char* dst = base + L::kQ + t * L::kQTile;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(w.a.q) + (x->s.q0 + static_cast<int64_t>(i)) * w.a.ld_q +
            (x->head * w.group + row - i * w.group) * w.a.ld_q_head);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c / 8) * kQBlock + swz_offset(r, c % 8)) =
              in ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.q_full[t]);
      }
      float top = -INFINITY, sum = 0.f;
      bool any = false;
      const int tiles = x->last[t] + 1;
      for (int k = keys.begin; k < tiles; ++k) {
        int key0, n;
        keys.tile(k, key0, n);
        if (!(t ? keys.needs<1>(key0, n) : keys.needs<0>(key0, n))) continue;
        const uint32_t s_at = tmem + lanes + L::s_col(t, it % L::kB);
        const uint32_t p_at = tmem + lanes + L::p_col(t, it % L::kB);
        ok = __all_sync(0xffffffffu, wait(&bars.s_full[t][it % L::kB], (it / L::kB) & 1));
        if (!ok) break;
        fence_after();
        // a running maximum m (times f) of scores not seen before: keeps the
        // reference unless m passed it by more than the slack
        auto raise = [&](float m) {
          const bool grow = m > top + kSlack || (top == -INFINITY && m > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            if (kRaise<DT>) m = ceilf(m);
            const float alpha = grow ? exp2_approx(top - m) : 1.f;
            if (grow) top = m;
            sum *= alpha;
            if (any) {
              // the product before this tile's must be complete; the one before
              // that is (its weights lay where these scores are)
              ok = __all_sync(0xffffffffu,
                              wait(&bars.pv_done[t][(it - 1) % L::kB], ((it - 1) / L::kB) & 1));
              fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(o, o_at + c);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st16(o_at + c, o);
              }
            }
          }
          return top == -INFINITY ? 0.f : kRaise<DT> - top;
        };
        // 32 scores to 16 words of weights
        auto weigh = [&](uint32_t (&pw)[16], const uint32_t* s, float off) {
          float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a = __uint_as_float(s[2 * j]), b = __uint_as_float(s[2 * j + 1]);
            fma2(a, b, f, off);
            a = exp2_approx(a);
            b = exp2_approx(b);
            add2(add[2 * (j & 1)], add[2 * (j & 1) + 1], a, b);
            pw[j] = DT == DLRM_DTYPE_BF16 ? pack_bf16(a, b) : pack_f16x2(a, b);
          }
          sum += (add[0] + add[1]) + (add[2] + add[3]);
        };
        // columns [0, 32) and [32, 64): skipped where none of the warp's rows
        // sees any, masked where some do not see all
        uint32_t some = 3, part = 0;
        if (!__all_sync(0xffffffffu, n == kKeys && key0 + kKeys <= v.end &&
                                         (key0 >= v.gap1 || key0 + kKeys <= v.gap0))) {
          some = 0;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            const int c0 = key0 + 32 * c, c1 = c0 + 32;
            const bool all = 32 * c + 32 <= n && c1 <= v.end && (c0 >= v.gap1 || c1 <= v.gap0);
            const bool none = 32 * c >= n || c0 >= v.end || (c0 >= v.gap0 && c1 <= v.gap1);
            some |= __any_sync(0xffffffffu, !none) ? 1u << c : 0u;
            part |= __any_sync(0xffffffffu, !all) ? 1u << c : 0u;
          }
        }
        auto mask = [&](uint32_t (&s)[32], int c) {
          const int e = min(n, v.end - key0) - 32 * c;
          const uint32_t bits = low_bits(min(v.gap0 - key0 - 32 * c, e)) |
                                (low_bits(e) & ~low_bits(v.gap1 - key0 - 32 * c));
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(bits & (1u << j))) s[j] = 0xff800000u;
        };
        float big[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (kKeep) {
          uint32_t s[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (some & (1u << c)) tmem_ld32(s[c], s_at + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (some & (1u << c)) {
              if (part & (1u << c)) mask(s[c], c);
#pragma unroll
              for (int j = 0; j < 32; ++j) big[j & 3] = fmaxf(big[j & 3], __uint_as_float(s[c][j]));
            }
          const float off = raise(fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) * f);
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (c == 0 || n > 32) {
              uint32_t pw[16];
              if (some & (1u << c)) {
                weigh(pw, s[c], off);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pw[j] = 0;
              }
              tmem_st16(p_at + 16 * c, pw);       // over the scores, which are in registers
            }
        } else {
          // masked scores go back to tensor memory: one masking for both readings
#pragma unroll 1
          for (int c = 0; c < 2; ++c)
            if (some & (1u << c)) {
              uint32_t s[32];
              tmem_ld32(s, s_at + 32 * c);
              tmem_wait_ld();
              if (part & (1u << c)) {
                mask(s, c);
                tmem_st32(s_at + 32 * c, s);
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) big[j & 3] = fmaxf(big[j & 3], __uint_as_float(s[j]));
            }
          const float off = raise(fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) * f);
          if (!ok) break;
          if (part) tmem_wait_st();
#pragma unroll 1
          for (int c = 0; c < 2; ++c)
            if (c == 0 || n > 32) {
              uint32_t pw[16];
              if (some & (1u << c)) {
                uint32_t s[32];
                tmem_ld32(s, s_at + 32 * c);
                tmem_wait_ld();
                weigh(pw, s, off);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pw[j] = 0;
              }
              tmem_st16(p_at + 16 * c, pw);       // over scores that have been read
            }
        }
        any = true;
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.p_full[t][it % L::kB]);
        ++it;
      }
      if (!ok) break;
      // ---- output
      if (any) {
        // the last product, and with it all before it
        ok = __all_sync(0xffffffffu, wait(&bars.pv_done[t][(it - 1) % L::kB], ((it - 1) / L::kB) & 1));
        if (!ok) break;
        fence_after();
      }
      const int hq = x->head * w.group + row - i * w.group;
      const int64_t q = x->s.q0 + static_cast<int64_t>(i);
      const int64_t o_row = q * w.a.ld_out + hq * w.a.ld_out_head;
      bool odd = false;
      // 32 elements of the row, unnormalised, to the output
      auto put = [&](int c, const uint32_t (&o)[32], float inv) {
        uint32_t h[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float a = inv != 0.f ? __uint_as_float(o[2 * j]) * inv : 0.f;
          const float b = inv != 0.f ? __uint_as_float(o[2 * j + 1]) * inv : 0.f;
          odd |= !finite(a) || !finite(b);
          h[j] = DT == DLRM_DTYPE_BF16 ? pack_bf16(a, b) : pack_f16x2(a, b);
        }
        if (in) {
          uint16_t* out = static_cast<uint16_t*>(w.a.out) + o_row + c;
          if (p.vec_out) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              reinterpret_cast<uint4*>(out)[j] =
                  make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              out[2 * j] = static_cast<uint16_t>(h[j]);
              out[2 * j + 1] = static_cast<uint16_t>(h[j] >> 16);
            }
          }
        }
      };
      const bool whole = !PAGED || x->parts == 1;
      // partial outputs of a CTA's place: element d of row r at d * kUnit + r,
      // then the rows' maxima and sums
      auto place = [&](int cta, int which) {
        return p.partials + (static_cast<int64_t>(cta) * 2 + which) * (kUnit * (D + 2)) + 128 * t + r;
      };
      float* part = place(blockIdx.x, PAGED ? x->place : 0);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (any) {
          tmem_ld32(o, o_at + c);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        if (whole) {
          put(c, o, inv);
        } else if (in) {
#pragma unroll
          for (int j = 0; j < 32; ++j) part[(c + j) * kUnit] = __uint_as_float(o[j]);
        }
      }
      if (any) {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.o_empty[t]);
      }
      bool mine = whole;                          // this warp writes the rows
      if (PAGED && !whole) {
        if (in) {
          part[D * kUnit] = top;
          part[(D + 1) * kUnit] = sum;
        }
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(&p.counters[x->part0 * 8 + warp], 1);
        mine = __shfl_sync(0xffffffffu, before, 0) == x->parts - 1;
        if (mine) {
          if (lane == 0) p.counters[x->part0 * 8 + warp] = 0;
          __threadfence();
          top = -INFINITY;
          sum = 0.f;
          if (in)
            for (int k = 0; k < x->parts; ++k)
              top = fmaxf(top, __ldcg(place(x->part0 + k, k ? 0 : 1) + D * kUnit));
          const float off = top == -INFINITY ? 0.f : top;
          if (in)
            for (int k = 0; k < x->parts; ++k) {
              const float* y = place(x->part0 + k, k ? 0 : 1);
              sum = fmaf(exp2_approx(__ldcg(y + D * kUnit) - off), __ldcg(y + (D + 1) * kUnit), sum);
            }
          const float all = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
            if (in)
              for (int k = 0; k < x->parts; ++k) {
                const float* y = place(x->part0 + k, k ? 0 : 1);
                const float g = exp2_approx(__ldcg(y + D * kUnit) - off);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  o[j] = __float_as_uint(fmaf(g, __ldcg(y + (c + j) * kUnit), __uint_as_float(o[j])));
              }
            put(c, o, all);
          }
        }
      }
      if (mine && in && w.a.lse)
        w.a.lse[q * w.a.n_heads + hq] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum * pow2f(-kRaise<DT>));
      if (sum == 0.f)
        odd |= sees_any(visible(x->pos0 + (!PAGED || w.a.causal ? i : 0), x->s.len, w.a.window, w.a.sinks));
      for (unsigned who = __ballot_sync(0xffffffffu, odd && in && mine); who; who &= who - 1) {
        __syncwarp();
        const int again = x->row0 + 128 * t + (warp & 3) * 32 + __ffs(who) - 1;
        if (PAGED)
          paged_careful_row<D, DT>(p, x->s, x->head, again);
        else
          window_careful_row<D, DT>(w, x->s, x->head, again);
      }
    }
    if (PAGED && lane == 0) finished[warp] = units.it;
  } else if (warp < 10) {
    // ------------------------------------------------------------ products
    const int t = warp - 8;
    if (elect_one()) {
      const int landing = products<D, DT, PAGED>(t, p, &map_q, bars, wait, base, tmem);
      // neither queries nor anything of the tensor core's may be in flight when its
      // memory is freed
      if (landing >= 0) wait.drain(&bars.q_full[t], landing);
      mma_commit(smem_addr(&bars.drain[t]));
      wait.drain(&bars.drain[t], 0);
    }
    __syncwarp();
  } else if (PAGED && warp >= 12) {
    // ------------------------------------------------------------ keys and values: codes
    constexpr int kPer = D / 32;                  // 16-code chunks of a thread, tile and side
    struct Codes {
      uint4 k[kPer], v[kPer];
      float ks[kPer], vs[kPer];
    };
    const int tid = threadIdx.x - 384;
    const int G = p.h.page_tokens, shift = __ffs(G) - 1;   // a power of two
    uint32_t it = 0;
    bool ok = true;
    for (const Unit* x; ok && (x = units.next_warp()); units.done_warp()) {
      const Keys keys(*x);
      const int head = x->head, len = x->s.len;
      const int32_t* pages = p.h.table + static_cast<int64_t>(x->s.k0) * p.h.max_pages;
      auto after = [&](int k) {
        while (++k < keys.tiles) {
          int key0, n;
          keys.tile(k, key0, n);
          if (keys.needs<0>(key0, n) || keys.needs<1>(key0, n)) break;
        }
        return k;
      };
      auto load = [&](Codes& y, int k) {
        int key0, n;
        keys.tile(k, key0, n);
        const int width = n > kBox ? kKeys : kBox;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int id = i * 128 + tid, row = id / (D / 16), ch = id % (D / 16);
          const int e = key0 + row;
          y.k[i] = y.v[i] = make_uint4(0, 0, 0, 0);
          y.ks[i] = y.vs[i] = 1.f;
          if (row < width && e < len) {
            const int page = pages[e >> shift];
            if (page >= 0 && page < p.h.n_pages) {
              const int64_t at = static_cast<int64_t>(page) * p.h.n_heads + head;
              const int64_t code = (at * G + (e & (G - 1))) * D + ch * 16;
              y.k[i] = __ldg(reinterpret_cast<const uint4*>(p.h.k_codes + code));
              y.v[i] = __ldg(reinterpret_cast<const uint4*>(p.h.v_codes + code));
              y.ks[i] = __ldg(p.h.k_scales + at);
              y.vs[i] = __ldg(p.h.v_scales + at);
            } else if (row < n) {
              // trimmed, or a broken table: NaN values have the rows done again
              // from the definition, without these events
              flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);
              y.v[i] = make_uint4(0x7f7f7f7f, 0x7f7f7f7f, 0x7f7f7f7f, 0x7f7f7f7f);
            }
          }
        }
      };
      auto store = [&](unsigned char* dst, const uint4& codes, float scale, int i) {
        const int id = i * 128 + tid, row = id / (D / 16), ch = id % (D / 16);
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = f16x2_to_float2(e4m3x2_lo_to_f16x2(w[j]));
          const float2 b = f16x2_to_float2(e4m3x2_hi_to_f16x2(w[j]));
          h[2 * j] = pack_bf16(a.x * scale, a.y * scale);
          h[2 * j + 1] = pack_bf16(b.x * scale, b.y * scale);
        }
        unsigned char* block = dst + ch / 4 * kBlockBytes;
        *reinterpret_cast<uint4*>(block + swz_offset(row, ch % 4 * 2)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(block + swz_offset(row, ch % 4 * 2 + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
      };
      Codes now, next;
      int k = after(keys.begin - 1);
      if (k < keys.tiles) load(now, k);
      while (k < keys.tiles) {
        const int k2 = after(k);
        if (k2 < keys.tiles) load(next, k2);
        const uint32_t st = it % kStages, ph = ((it / kStages) & 1) ^ 1;
        ok = it < kStages || __all_sync(0xffffffffu, wait(&bars.k_empty[st], ph));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) store(base + L::kK + st * L::kTile, now.k[i], now.ks[i], i);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.k_full[st]);
        ok = it < kStages || __all_sync(0xffffffffu, wait(&bars.v_empty[st], ph));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) store(base + L::kV + st * L::kTile, now.v[i], now.vs[i], i);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.v_full[st]);
        ++it;
        now = next;
        k = k2;
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ keys and values
    if (!PAGED && lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (const Unit* x; ok && (x = units.next()); units.done()) {
        const Keys keys(*x);
        const int head = x->head, k0 = x->s.k0;
        for (int k = keys.begin; k < keys.tiles && ok; ++k) {
          int key0, n;
          keys.tile(k, key0, n);
          if (!keys.needs<0>(key0, n) && !keys.needs<1>(key0, n)) continue;
          const uint32_t st = it % kStages, ph = ((it / kStages) & 1) ^ 1;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            uint64_t* full = side ? &bars.v_full[st] : &bars.k_full[st];
            if (it >= kStages && !(ok = wait(side ? &bars.v_empty[st] : &bars.k_empty[st], ph))) break;
            bar_expect(full, (n > kBox ? 2u : 1u) * kBox * 128 * L::kBlocks);
            const uint32_t dst = smem_addr(base + (side ? L::kV : L::kK) + st * L::kTile);
#pragma unroll
            for (int r = 0; r < kKeys; r += kBox)
              if (r < n)
#pragma unroll
                for (int c = 0; c < L::kBlocks; ++c)
                  tma_load_3d(dst + c * kBlockBytes + r * 128, side ? &map_v : &map_k, c * 64, head,
                              k0 + key0 + r, full);
          }
          ++it;
        }
      }
      // loads in flight must land before the shared memory is released: the last of
      // every stage, and of the tile at which a wait gave up perhaps the keys (if they were
      // not asked for, this wait runs out too)
      const uint32_t to = ok ? it : it - 1;
      for (uint32_t q = to > kStages ? to - kStages : 0; q < it; ++q) {
        wait.drain(&bars.k_full[q % kStages], (q / kStages) & 1);
        if (q < to) wait.drain(&bars.v_full[q % kStages], (q / kStages) & 1);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ units
    // (failure tests: the first CTA never hears of its first one)
    auto withhold = [&](int it) { return it == 0 && p.wait.withhold_last && blockIdx.x == 0; };
    if (!PAGED) {
      Walk walk;
      for (int it = 0, u = blockIdx.x;; ++it, u += gridDim.x) {
        const int slot = it % kUnits;
        if (it >= kUnits &&
            !__all_sync(0xffffffffu, wait(&bars.u_empty[slot], ((it / kUnits) & 1) ^ 1)))
          break;
        walk.find(p, u, bars.units[slot]);
        __syncwarp();
        const bool valid = bars.units[slot].valid != 0;
        __syncwarp();
        if (lane == 0 && !withhold(it)) bar_arrive(&bars.u_full[slot]);
        if (!valid) break;
      }
    } else if (lane == 0) {
      PagedWalk walk(p, cuts, found);
      for (int it = 0;; ++it) {
        const int slot = it % kUnits;
        if (it >= kUnits && !wait(&bars.u_empty[slot], ((it / kUnits) & 1) ^ 1)) break;
        Unit x;
        const bool more = walk.next(p, cuts, x);
        if (more)
          bars.units[slot] = x;
        else
          bars.units[slot].valid = 0;
        if (!withhold(it)) bar_arrive(&bars.u_full[slot]);
        if (!more) break;
      }
    }
    __syncwarp();
    if (blockIdx.x == 0)
      for (int i = lane; i < w.a.batch; i += kWarp) tc_span<PAGED>(p, i, true);
  }
  fence_before();
  __syncthreads();
  if (PAGED && bars.abort && threadIdx.x == 0) count_given_up(p, cuts, found, finished);
  if (warp == 8) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kColumns)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// (rows, heads, D) with strides ld, ld_head: boxes of box_rows rows x box_heads
// heads x 64 elements; zeros past D and past the last row.
bool encode_rows(CUtensorMap* map, const void* x, int64_t rows, int heads, int dim, int64_t ld,
                 int64_t ld_head, int dtype, int box_rows, int box_heads) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  if (heads == 1) ld_head = dim;                  // not used
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld_head) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t steps[3] = {1, 1, 1};
  return enc(map,
             dtype == DLRM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             3, const_cast<void*>(x), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What TMA asks of (rows, heads, dim) in 16 bits: a 16-byte aligned base,
// strides that are multiples of 16 bytes, below 2^40, each a whole multiple of
// the one before.
bool tma_rows(const void* x, int64_t ld, int64_t ld_head, int heads, int dim) {
  if (reinterpret_cast<uintptr_t>(x) % 16 != 0 || ld % 8 != 0 || ld >= (int64_t(1) << 38)) return false;
  if (heads == 1) return ld >= dim && ld % dim == 0;
  return ld_head % 8 == 0 && ld_head >= dim && ld > 0 && ld % ld_head == 0;
}

// What both calls give the kernel; false where the driver refuses a tensor map.
bool fill_params(TcParams& p, CUtensorMap& map_q, const dlrm_attention_t& a) {
  p.wait = attention_wait();
  p.w.a = a;
  p.w.group = a.n_heads / a.n_kv_heads;
  p.w.vec = 1;
  p.group = fast_div(p.w.group);
  p.heads = fast_div(a.n_kv_heads);
  p.most = static_cast<int>((a.q_rows * p.w.group / kUnit + a.batch) * a.n_kv_heads);
  p.vec_out = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ld_out % 8 == 0 &&
              (a.n_heads == 1 || a.ld_out_head % 8 == 0);
  p.q_tma = 128 % p.w.group == 0 && tma_rows(a.q, a.ld_q, a.ld_q_head, a.n_heads, a.head_dim);
  return !p.q_tma || encode_rows(&map_q, a.q, a.q_rows, a.n_heads, a.head_dim, a.ld_q, a.ld_q_head,
                                 a.dtype, 128 / p.w.group, p.w.group);
}

// Rows that a thread can load 16 bytes at a time.
bool vector_rows(const void* x, int64_t ld, int64_t ld_head, int heads) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld % 8 == 0 && (heads == 1 || ld_head % 8 == 0);
}

template <int D, int DT, bool PAGED>
cudaError_t launch_tc(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TcParams& p, unsigned grid,
                   cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(attention_tc_kernel<D, DT, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<D, PAGED>::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(attention_tc_kernel<D, DT, PAGED>, dim3(grid), dim3(kThreadsOf<PAGED>), Layout<D, PAGED>::kSmem, stream,
                    mq, mk, mv, p);
}

}  // namespace

}  // namespace dlrm
