// Attention of queries over event histories kept in 8 bits (include/dlrm.h,
// history_attention).
//
// One launch. The unit of work is a chunk of events (kWarps blocks of 32
// events) of one row tile: one kv head of one request and up to kRows of its
// query rows (rows are (query, head of the group) pairs, so heads that share
// a kv head share its bytes). All chunks of the batch form one sequence,
// request by request; every CTA takes an equal, contiguous part of it,
// whatever the histories' lengths, so a long history is split over many CTAs
// and a short one costs one chunk. A tile that lies in one CTA is finished
// there; one that is split leaves partial results (maximum, sum, weighted
// values per row) in scratch, and the CTA that arrives last joins them, in the
// order of the events: results do not depend on timing.
//
// In a CTA, warp w takes block w of each chunk and keeps its own running
// maximum, sum and output in registers; the warps are joined once per tile.
// Every warp streams its blocks through a ring of its own in shared memory
// (cp.async, kStages deep, no block-wide barrier), with the page numbers and
// scales of 32 blocks ahead in one register of each lane. S = Q K^T and O += P V
// are m16n8k16 MMAs. The MMA does not care which element of the head (for S) or
// which event (for P V) an index of its inner dimension stands for, as long as
// both operands agree, so a thread reads 16 contiguous bytes of an event's key,
// and 4 to 16 of a value, and converts them (e4m3 to f16 is exact) in place.
//   keys: thread (g, c) = (lane / 4, lane % 4) holds event g of an 8-event
//     tile, elements 64 j + 16 c + 4 ks + e (j: 64-byte part, ks: k step);
//   values: thread (g, c) holds events 2c, 2c+1, 2c+8, 2c+9 of a 16-event
//     step, elements g D/8 .. (g+1) D/8 - 1; the bytes of a pair of events
//     are interleaved, then converted. Output column 2c + i of n tile nt is
//     element (2c + i) D/8 + nt.
// 16-byte chunks are swizzled in shared memory so that these reads meet no bank
// twice.
// Scales: a block lies in one page, so the page's key scale multiplies S and
// its value scale the block's P V, both in fp32 (one FMA per output, which
// also applies the running maximum's correction).
//
// Queries become f16 after a division by a power of two for each row. A bf16
// or fp16 query and P (11 bits) take one MMA row: 16 rows a tile. An fp32
// query is split into an f16 head and a rest of 11 more bits, which take two
// MMA rows, and so is P: 8 rows a tile, errors as of fp32 (2.2e-7 of the values against
// 4.2e-7 of fp32 products and sums: 256 users, 3 rows, window 256). Weights are relative to a
// whole number at or above the largest score, 2^15 times as large (kLift).
//
// What bounds it: reading the codes (2 D bytes an event and kv head). Measured, one
// query a user: 4 users of 65,000 to 100,001 events, 8 heads of 128, fp16, 124 us, 83%
// of the copy rate; 64 users of 37 to 4096 events, 8 heads of 64 over 2, bf16, 22 us,
// half of it the start (the lengths of all requests, then table, then codes, each a
// read that waits for the one before) and the join; one user of 150 events 5 us, all of
// it start.
#include <atomic>

#include "history_attention.cuh"

namespace dlrm {

namespace {

constexpr int kWhole = 4;                        // chunks of a tile that is never split
// Chunks of a CTA at least, where tiles are longer: 16 users x 4096 events x 8 rows
// 16.7 us against 20.0 with one chunk, one user x 4096 x 16 rows 16 against 21.
constexpr int kLeast = 4;

struct Params {
  dlrm_history_t h;
  dlrm_attention_t a;
  int group;                                     // query heads of a kv head
  int most;                                      // (head, tile)s that starts which never decrease make
  int vec_q;                                     // four query elements can be loaded at once
  int32_t* counters;
  float* partials;
  const int32_t* groups;                         // checked only, where there are any
  int n_groups;
};

// What a CTA needs to know of a request.
struct Span {
  int slot, queries, rows, len, q0, tiles;       // rows: queries * group
  int sink_blocks, block0, blocks, chunks;       // blocks of events: the sinks', then from block0 on
};

template <int ROWS>
__device__ __forceinline__ Span span_of(const Params& p, int b, bool report) {
  Span s;
  const int q0 = p.a.q_starts[b], q1 = p.a.q_starts[b + 1];
  s.slot = p.a.slots[b];
  s.q0 = q0;
  s.rows = 0;
  s.len = 0;
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.a.q_rows;
  s.queries = bad ? 0 : q1 - q0;
  s.rows = s.queries * p.group;
  if (s.slot >= 0 && s.slot < p.h.n_slots) {
    const int64_t cap = static_cast<int64_t>(p.h.max_pages) * p.h.page_tokens;
    s.len = static_cast<int>(min(static_cast<int64_t>(max(p.h.lengths[s.slot], 0)), cap));
  } else if (report) {
    flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);
  }
  if (bad && report) flag(p.h.err, DLRM_ERRBIT_OFFSETS);
  s.tiles = (s.rows + ROWS - 1) / ROWS;
  // the events that any row of the request sees
  const Visible first =
      visible(p.a.causal ? s.len - (q1 - q0) : s.len - 1, s.len, p.a.window, p.a.sinks);
  const int end = (s.len + kBlock - 1) / kBlock;
  const int sink = min(p.a.sinks, s.len);
  s.block0 = first.gap1 / kBlock;
  s.sink_blocks = first.gap1 > 0 ? (sink + kBlock - 1) / kBlock : 0;
  if (s.sink_blocks >= s.block0) s.sink_blocks = s.block0;   // no gap: blocks from 0 on
  s.blocks = s.sink_blocks + max(end - s.block0, 0);
  s.chunks = max((s.blocks + kWarps - 1) / kWarps, 1);        // an empty one writes zeros
  return s;
}

template <int D, int DT>
struct Shape {
  static constexpr bool kSplit = DT == DLRM_DTYPE_FP32;
  static constexpr int kRows = kSplit ? 8 : 16;
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kBytes = 2 * kBlock * D;   // keys and values of a block
  static constexpr int kStride = D + 2;           // a row's sums, maximum, sum of weights
  static constexpr int kRing = kWarps * kStages * kBytes;
  static constexpr int kJoin = kWarps * kRows * kStride * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

// Three CTAs an SM up to head_dim 64 (left to itself the compiler stops at 128 registers at
// 32: 256 users, window 256, 13.0 us against 12.2, and spills at 64: 64 users 26.7
// against 21.6), two at 128.
template <int D, int DT>
__global__ void __launch_bounds__(kThreads, D == 128 ? 1 : 3)
history_attention_kernel(const __grid_constant__ Params p) {
  using Sh = Shape<D, DT>;
  constexpr bool kSplit = Sh::kSplit;
  constexpr int kRows = Sh::kRows, kStages = Sh::kStages, kStride = Sh::kStride;
  constexpr int KW = D / 16;                      // key words of a thread and event tile
  constexpr int VW = D / 32;                      // value words of a thread and event
  constexpr int NT = D / 8;                       // n tiles of the output
  constexpr int kAcc = kSplit ? 2 : 4;            // output values of a thread and n tile
  extern __shared__ __align__(128) unsigned char smem[];
  float (*joined)[kRows][kStride] = reinterpret_cast<float (*)[kRows][kStride]>(smem);
  __shared__ int sums[2 * kWarps];
  __shared__ Found<Span> found;
  __shared__ float row_factor[kRows];
  __shared__ int odd[kRows + 1];

  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int g = lane / 4, c = lane % 4;
  const int G = p.h.page_tokens, H = p.h.n_heads, shift = __ffs(G) - 1;   // G: a power of two
  unsigned char* ring = smem + warp * kStages * Sh::kBytes;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  pdl_wait();
  pdl_trigger();

  auto units = [&](const Span& s) { return s.tiles * s.chunks * H; };
  const Cuts cuts = locate_cuts<kThreads>(
      p.a.batch, kLeast, p.most, [&](int i) { return span_of<kRows>(p, i, false); }, units,
      [&](const Span& s) { return s.tiles * H; }, sums, found);
  // a cut inside a short tile moves to the tile's start: finishing it in one
  // CTA is faster than joining parts
  auto snap = [&](int x, int i) {
    const int chunks = found.span[i].chunks;
    if (x >= cuts.total || chunks > kWhole) return x;
    const unsigned off = x - found.first[i];
    return static_cast<int>(x - off % static_cast<unsigned>(chunks));
  };
  const int begin = cuts.total ? snap(cuts.cut(blockIdx.x), 0) : 0;
  const int end = cuts.total ? snap(cuts.cut(blockIdx.x + 1), 1) : 0;
  int b = found.request[0], at = found.first[0];
  Span s = found.span[0];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.a.batch; i += kThreads) span_of<kRows>(p, i, true);
  if (p.groups && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.n_groups; i += kThreads)
      if (i < p.n_groups ? p.groups[i] < 0 || p.groups[i + 1] < p.groups[i] || (i == 0 && p.groups[0] != 0)
                         : p.groups[i] != p.a.batch)
        flag(p.h.err, DLRM_ERRBIT_OFFSETS);

  for (int u = begin; u < end;) {
    if (u >= at + units(s)) {
      at += units(s);
      s = span_of<kRows>(p, ++b, false);
      continue;
    }
    const int seg = static_cast<unsigned>(u - at) / static_cast<unsigned>(s.chunks);   // (head, tile)
    const int head = s.tiles == 1 ? seg : static_cast<unsigned>(seg) / static_cast<unsigned>(s.tiles);
    const int tile = seg - head * s.tiles;
    const int seg0 = at + seg * s.chunks, seg1 = seg0 + s.chunks;
    const int chunk0 = u - seg0, chunk1 = min(end, seg1) - seg0;
    const int rows = min(kRows, s.rows - tile * kRows);
    u = seg0 + chunk1;

    // ---- queries: the loads first, the arithmetic while the events are on their way
    float x[2][KW][4];
    int query[2];                                 // of the thread's rows
#pragma unroll
    for (int r2 = 0; r2 < 2; ++r2) {
      // rows past the last stand for it (their queries are zero), so that
      // they do not make blocks of events partly visible
      const int r = min(kSplit ? g : g + 8 * r2, rows - 1);
      const int row = tile * kRows + r;
      query[r2] = p.group == 1 ? row : static_cast<unsigned>(row) / static_cast<unsigned>(p.group);
      const bool in = r == g + 8 * r2;
      const int64_t q_at = (s.q0 + static_cast<int64_t>(query[r2])) * p.a.ld_q +
                           (head * p.group + row - query[r2] * p.group) * p.a.ld_q_head;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        if (in) {
          load_four<DT>(x[r2][w], p.a.q, q_at + key_element<D>(c, w), p.vec_q);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[r2][w][e] = 0.f;
        }
      }
    }

    // ---- blocks of this warp: n0, n0 + kWarps, ...; lane l knows block l of
    // the 32 at hand (info) and of the 32 after them (ahead)
    const int pos0 = p.a.causal ? s.len - s.queries : s.len - 1;
    const unsigned group = p.group;
    const int i_first = p.group == 1 ? tile * kRows : static_cast<unsigned>(tile * kRows) / group;
    const int i_last = p.group == 1 ? tile * kRows + rows - 1
                                    : static_cast<unsigned>(tile * kRows + rows - 1) / group;
    const Visible v_first = visible(pos0 + (p.a.causal ? i_first : 0), s.len, p.a.window, p.a.sinks);
    const Visible v_last = visible(pos0 + (p.a.causal ? i_last : 0), s.len, p.a.window, p.a.sinks);
    const int n0 = chunk0 * kWarps + warp, n1 = min(chunk1 * kWarps, s.blocks);
    const int count = n0 < n1 ? (n1 - n0 + kWarps - 1) / kWarps : 0;
    auto first_event = [&](int i) {
      const int n = n0 + i * kWarps;
      return (n < s.sink_blocks ? n : n - s.sink_blocks + s.block0) * kBlock;
    };
    struct Info {
      int page;                                   // -1: nothing to read
      float ks, vs;
    };
    const int32_t* pages = p.h.table + static_cast<int64_t>(s.slot) * p.h.max_pages;
    auto look = [&](int i) {
      Info x{-1, 0.f, 0.f};
      if (i < count) {
        const int t0 = first_event(i);
        // not what no row of the tile sees
        if (t0 < v_last.end && !(t0 >= v_last.gap0 && t0 + kBlock <= v_first.gap1)) {
          x.page = pages[t0 >> shift];
          if (x.page < 0 || x.page >= p.h.n_pages) {
            // trimmed, or a broken table: events that some row needs
            x.page = -1;
            flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);
          } else {
            const int64_t place = static_cast<int64_t>(x.page) * H + head;
            x.ks = p.h.k_scales[place];
            x.vs = p.h.v_scales[place];
          }
        }
      }
      return x;
    };
    Info info = look(lane), ahead = look(kWarp + lane);
    int base = 0;                                 // blocks [base, base + 32) are in info
    auto fetch = [&](int i) {
      if (i < count) {
        const int page = __shfl_sync(0xffffffffu, i - base < kWarp ? info.page : ahead.page, i % kWarp);
        if (page >= 0) {
          const int64_t codes = ((static_cast<int64_t>(page) * H + head) * G + (first_event(i) & (G - 1))) * D;
          const uint32_t dst = ring_at + (i % kStages) * Sh::kBytes;
#pragma unroll
          for (int x = 0; x < 2 * D / 32; ++x) {
            const int id = x * kWarp + lane, t = id / (D / 16), ch = id % (D / 16);
            copy16(dst + key_offset<D>(t, ch), p.h.k_codes + codes + id * 16);
          }
#pragma unroll
          for (int x = 0; x < 2 * D / 32; ++x) {
            const int id = x * kWarp + lane, t = id / (D / 16), ch = id % (D / 16);
            copy16(dst + kBlock * D + value_offset<D>(t, ch), p.h.v_codes + codes + id * 16);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ---- fragments of the queries, scaled to f16; a negative softmax scale is
    // theirs, so that the factors of the scores are positive
    uint32_t qa[KW][4];
    float qf[2];
    Visible vis[2];
    {
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        float big = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[r2][w][e]));
        big = quad_max(big);
        const int ex = max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100);
        const float f = copysignf(pow2f(min(8 - ex, 127)), p.a.scale);
        qf[r2] = pow2f(max(ex - 8, -126)) * fabsf(p.a.scale) * kLog2e;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[r2][w][e] *= f;
        vis[r2] = visible(pos0 + (p.a.causal ? query[r2] : 0), s.len, p.a.window, p.a.sinks);
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        qa[w][0] = pack_f16x2(x[0][w][0], x[0][w][1]);
        qa[w][2] = pack_f16x2(x[0][w][2], x[0][w][3]);
        if (kSplit) {
          const float2 h0 = f16x2_to_float2(qa[w][0]), h1 = f16x2_to_float2(qa[w][2]);
          qa[w][1] = pack_f16x2((x[0][w][0] - h0.x) * 2048.f, (x[0][w][1] - h0.y) * 2048.f);
          qa[w][3] = pack_f16x2((x[0][w][2] - h1.x) * 2048.f, (x[0][w][3] - h1.y) * 2048.f);
        } else {
          qa[w][1] = pack_f16x2(x[1][w][0], x[1][w][1]);
          qa[w][3] = pack_f16x2(x[1][w][2], x[1][w][3]);
        }
      }
      if (kSplit) {
        qf[1] = qf[0];
        vis[1] = vis[0];
      }
    }

    // ---- events
    float o[NT][kAcc];
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < kAcc; ++i) o[nt][i] = 0.f;
    for (int it = 0; it < count; ++it) {
      if (it - base == kWarp) {
        base += kWarp;
        info = ahead;
        ahead = look(base + kWarp + lane);
      }
      fetch(it + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const int page = __shfl_sync(0xffffffffu, info.page, it % kWarp);
      if (page < 0) continue;
      const float ks = __shfl_sync(0xffffffffu, info.ks, it % kWarp);
      const float vs = __shfl_sync(0xffffffffu, info.vs, it % kWarp);
      const int t0 = first_event(it);
      const unsigned char* kb = ring + (it % kStages) * Sh::kBytes;
      const unsigned char* vb = kb + kBlock * D;

      // S = Q K^T
      float sc[kBlock / 8][4];
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        uint32_t kw[KW];
        if (D == 32) {
          const uint2 x = *reinterpret_cast<const uint2*>(kb + (8 * j + g) * 32 + 8 * c);
          kw[0] = x.x;
          kw[1] = x.y;
        } else {
#pragma unroll
          for (int i = 0; i < KW / 4; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(kb + key_offset<D>(8 * j + g, 4 * i + c));
            kw[4 * i] = x.x;
            kw[4 * i + 1] = x.y;
            kw[4 * i + 2] = x.z;
            kw[4 * i + 3] = x.w;
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w)
          mma_f16_from(sc[j], qa[w], e4m3x2_lo_to_f16x2(kw[w]), e4m3x2_hi_to_f16x2(kw[w]), w > 0);
      }
      // weights: exp2 of the scores times f0, f1, less the running maximum
      // (not zero, even for a softmax scale of zero: a masked score is -infinity)
      const float f0 = fmaxf(qf[0] * ks, 1e-37f), f1 = fmaxf(qf[1] * ks, 1e-37f);
      const bool whole = t0 + kBlock <= min(vis[0].end, vis[1].end) &&
                         (t0 >= vis[0].gap1 || t0 + kBlock <= vis[0].gap0) &&
                         (t0 >= vis[1].gap1 || t0 + kBlock <= vis[1].gap0);
      if (kSplit) {
#pragma unroll
        for (int j = 0; j < kBlock / 8; ++j) {
          sc[j][0] = fmaf(sc[j][2], 1.f / 2048.f, sc[j][0]);
          sc[j][1] = fmaf(sc[j][3], 1.f / 2048.f, sc[j][1]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < kBlock / 8; ++j) {
          const int t = t0 + 8 * j + 2 * c;
          if (!sees(vis[0], t)) sc[j][0] = -INFINITY;
          if (!sees(vis[0], t + 1)) sc[j][1] = -INFINITY;
          if (!kSplit) {
            if (!sees(vis[1], t)) sc[j][2] = -INFINITY;
            if (!sees(vis[1], t + 1)) sc[j][3] = -INFINITY;
          }
        }
      }
      float big[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        big[0] = fmaxf(big[0], fmaxf(sc[j][0], sc[j][1]));
        if (!kSplit) big[1] = fmaxf(big[1], fmaxf(sc[j][2], sc[j][3]));
      }
      // running maximum and sum
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int r = 0; r < (kSplit ? 1 : 2); ++r) {
        const float f = r ? f1 : f0;
        const float m = fmaxf(top[r], ceilf(quad_max(big[r]) * f));
        const float base = m == -INFINITY ? 0.f : m, off = kLift - base;
        alpha[r] = exp2_approx(top[r] - base);
        top[r] = m;
        float add = 0.f;
#pragma unroll
        for (int j = 0; j < kBlock / 8; ++j) {
          sc[j][2 * r] = exp2_approx(fmaf(sc[j][2 * r], f, off));
          sc[j][2 * r + 1] = exp2_approx(fmaf(sc[j][2 * r + 1], f, off));
          add += sc[j][2 * r] + sc[j][2 * r + 1];
        }
        sum[r] = fmaf(sum[r], alpha[r], add);
      }
      // the output's correction, where the maximum of some row grew
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < kAcc; ++i) o[nt][i] *= alpha[i >> 1];
      }
      // O += vs P V
      uint32_t pa[kBlock / 16][4];
#pragma unroll
      for (int kt = 0; kt < kBlock / 16; ++kt) {
        pa[kt][0] = pack_f16x2(sc[2 * kt][0], sc[2 * kt][1]);
        pa[kt][2] = pack_f16x2(sc[2 * kt + 1][0], sc[2 * kt + 1][1]);
        if (kSplit) {
          const float2 h0 = f16x2_to_float2(pa[kt][0]), h1 = f16x2_to_float2(pa[kt][2]);
          pa[kt][1] = pack_f16x2((sc[2 * kt][0] - h0.x) * 2048.f, (sc[2 * kt][1] - h0.y) * 2048.f);
          pa[kt][3] =
              pack_f16x2((sc[2 * kt + 1][0] - h1.x) * 2048.f, (sc[2 * kt + 1][1] - h1.y) * 2048.f);
        } else {
          pa[kt][1] = pack_f16x2(sc[2 * kt][2], sc[2 * kt][3]);
          pa[kt][3] = pack_f16x2(sc[2 * kt + 1][2], sc[2 * kt + 1][3]);
        }
      }
      uint32_t vw[kBlock / 16][4][VW];
#pragma unroll
      for (int kt = 0; kt < kBlock / 16; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + value_offset<D>(t, g));
            vw[kt][i][0] = x.x;
            vw[kt][i][VW > 1 ? 1 : 0] = x.y;
            vw[kt][i][VW > 2 ? 2 : 0] = x.z;
            vw[kt][i][VW > 3 ? 3 : 0] = x.w;
          } else if (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2*>(vb + value_offset<D>(t, g >> 1) + 8 * (g & 1));
            vw[kt][i][0] = x.x;
            vw[kt][i][VW > 1 ? 1 : 0] = x.y;
          } else {
            vw[kt][i][0] = *reinterpret_cast<const uint32_t*>(vb + value_offset<D>(t, g >> 2) + 4 * (g & 3));
          }
        }
      if (t0 + kBlock > s.len) {
        // codes of events past the end are whatever an earlier history left there
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1) >= s.len)
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[kt][i][w] = 0;
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        float acc[4][4];
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt) {
          // bytes of a pair of events side by side: n tiles 4w, 4w+1 and 4w+2, 4w+3
          const uint32_t l0 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x5140);
          const uint32_t l1 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x7362);
          const uint32_t h0 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x5140);
          const uint32_t h1 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x7362);
          mma_f16_from(acc[0], pa[kt], e4m3x2_lo_to_f16x2(l0), e4m3x2_lo_to_f16x2(h0), kt > 0);
          mma_f16_from(acc[1], pa[kt], e4m3x2_hi_to_f16x2(l0), e4m3x2_hi_to_f16x2(h0), kt > 0);
          mma_f16_from(acc[2], pa[kt], e4m3x2_lo_to_f16x2(l1), e4m3x2_lo_to_f16x2(h1), kt > 0);
          mma_f16_from(acc[3], pa[kt], e4m3x2_hi_to_f16x2(l1), e4m3x2_hi_to_f16x2(h1), kt > 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* out = o[4 * w + i];
          if (kSplit) {
            out[0] = fmaf(vs, fmaf(acc[i][2], 1.f / 2048.f, acc[i][0]), out[0]);
            out[1] = fmaf(vs, fmaf(acc[i][3], 1.f / 2048.f, acc[i][1]), out[1]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = fmaf(vs, acc[i][j], out[j]);
          }
        }
      }
      __syncwarp();                               // the stage is read: it may be filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps
    __syncthreads();                              // every warp's ring is done with: `joined` lies there
#pragma unroll
    for (int r = 0; r < (kSplit ? 1 : 2); ++r) {
      const float l = quad_sum(sum[r]);
      float* out = joined[warp][g + 8 * r];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        out[2 * c * (D / 8) + nt] = o[nt][2 * r];
        out[(2 * c + 1) * (D / 8) + nt] = o[nt][2 * r + 1];
      }
      if (c == 0) {
        out[D] = top[r];
        out[D + 1] = l;
      }
    }
    __syncthreads();
    if (threadIdx.x < kRows) {
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, joined[w][threadIdx.x][D]);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_approx(joined[w][threadIdx.x][D] - base);
        l = fmaf(f, joined[w][threadIdx.x][D + 1], l);
        joined[w][threadIdx.x][D] = f;
      }
      joined[0][threadIdx.x][D + 1] = l;
      row_factor[threadIdx.x] = m;
    }
    __syncthreads();
    const bool split = chunk0 > 0 || chunk1 < s.chunks;
    float* mine = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (chunk0 > 0 ? 0 : 1)) * kAttnPartial;
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
      const int r = e / D, d = e % D;
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x = fmaf(joined[w][r][D], joined[w][r][d], x);
      if (split)
        mine[r * kStride + d] = x;
      else
        joined[0][r][d] = x;
    }
    if (split) {
      if (threadIdx.x < rows) {
        mine[threadIdx.x * kStride + D] = row_factor[threadIdx.x];
        mine[threadIdx.x * kStride + D + 1] = joined[0][threadIdx.x][D + 1];
      }
      // the CTAs that share this tile: first .. last, one part each. (A cut moves
      // out of short tiles only, so a split tile's cuts are where they were.)
      const int64_t first = cuts.owner(seg0);
      const int parts = cuts.owner(seg1 - 1) - static_cast<int>(first) + 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int before = atomicAdd(&p.counters[first], 1);
        odd[kRows] = before == parts - 1;
        if (before == parts - 1) p.counters[first] = 0;
      }
      __syncthreads();
      if (!odd[kRows]) continue;                  // (`joined` was read before the barrier)
      __threadfence();
      auto part = [&](int i) {
        return p.partials + ((first + i) * 2 + (i > 0 ? 0 : 1)) * kAttnPartial;
      };
      // maximum of each row over the parts, the parts' weights, then the weighted
      // sums: kWeights parts at a time, every thread with all its elements of four
      // parts under way
      for (int r = warp; r < rows; r += kWarps) {
        float m = -INFINITY;
        for (int i = lane; i < parts; i += kWarp) m = fmaxf(m, __ldcg(part(i) + r * kStride + D));
#pragma unroll
        for (int x = 16; x > 0; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (lane == 0) row_factor[r] = m;
      }
      constexpr int kWeights = 128, kPairs = kRows * D / 2 / kThreads;
      static_assert(kPairs * 2 * kThreads == kRows * D, "elements of a thread");
      static_assert((kRows * kStride + kWeights * kRows) * 4 <= Sh::kSmem, "space");
      float* weight = &joined[1][0][0];           // [part][row]
      float2 acc[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) acc[e] = make_float2(0.f, 0.f);
      float l = 0.f;
      for (int p0 = 0; p0 < parts; p0 += kWeights) {
        const int n = min(kWeights, parts - p0);
        __syncthreads();
        for (int e = threadIdx.x; e < n * kRows; e += kThreads) {
          const int i = e / kRows, r = e % kRows;
          const float m = r < rows ? row_factor[r] : -INFINITY;
          weight[e] = m == -INFINITY ? 0.f : exp2_approx(__ldcg(part(p0 + i) + r * kStride + D) - m);
        }
        __syncthreads();
        if (threadIdx.x < rows)
          for (int i = 0; i < n; ++i)
            l = fmaf(weight[i * kRows + threadIdx.x],
                     __ldcg(part(p0 + i) + threadIdx.x * kStride + D + 1), l);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const float* q = part(p0 + i);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const int at = 2 * (e * kThreads + threadIdx.x), r = at / D, d = at % D;
            if (r >= rows) continue;
            const float2 y = __ldcg(reinterpret_cast<const float2*>(q + r * kStride + d));
            const float f = weight[i * kRows + r];
            acc[e].x = fmaf(f, y.x, acc[e].x);
            acc[e].y = fmaf(f, y.y, acc[e].y);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const int at = 2 * (e * kThreads + threadIdx.x), r = at / D, d = at % D;
        joined[0][r][d] = acc[e].x;
        joined[0][r][d + 1] = acc[e].y;
      }
      if (threadIdx.x < rows) joined[0][threadIdx.x][D + 1] = l;
    }
    if (threadIdx.x <= kRows) odd[threadIdx.x] = 0;
    __syncthreads();

    // ---- outputs
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
      const int r = e / D, d = e % D;
      const int row = tile * kRows + r;
      const float l = joined[0][r][D + 1];
      const float x = l == 0.f ? 0.f : joined[0][r][d] / l;
      const int64_t i = s.q0 + static_cast<int64_t>(row / p.group);
      const int hq = head * p.group + row % p.group;
      store_element<DT>(p.a.out, i * p.a.ld_out + hq * p.a.ld_out_head + d, x);
      if (d == 0 && p.a.lse)
        p.a.lse[i * p.a.n_heads + hq] = l == 0.f ? -INFINITY : row_factor[r] * kLn2 + logf(l * pow2f(-kLift));
      if (!finite(x) || l == 0.f) odd[r] = odd[kRows] = l == 0.f ? 2 : 1;   // 2: sees nothing, or has no weights
    }
    __syncthreads();
    if (odd[kRows]) {
      for (int r = 0; r < rows; ++r) {
        const int row = tile * kRows + r, query = row / p.group, hq = head * p.group + row % p.group;
        const Visible v = visible(pos0 + (p.a.causal ? query : 0), s.len, p.a.window, p.a.sinks);
        const int64_t i = s.q0 + static_cast<int64_t>(query);
        if (odd[r] == 1 || (odd[r] == 2 && sees_any(v)))
          careful_row<DT>(p.h, p.a, s.slot, v, head, i * p.a.ld_q + hq * p.a.ld_q_head,
                          i * p.a.ld_out + hq * p.a.ld_out_head, i * p.a.n_heads + hq, &joined[0][0][0]);
      }
    }
    __syncthreads();                              // `joined` is read: the rings may be filled
  }
}

template <int D, int DT>
cudaError_t launch(Params& p, cudaStream_t stream) {
  using Sh = Shape<D, DT>;
  constexpr int kRows = Sh::kRows;
  // The shared memory that the kernel may take is set once on every device, by a bit
  // each; the CTAs of an SM are the same on every GB300.
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  int per_sm = 0;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(history_attention_kernel<D, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Sh::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, history_attention_kernel<D, DT>,
                                                      kThreads, Sh::kSmem);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, std::min(per_sm, kAttnMaxCtas / 152));
    resident.store(per_sm, std::memory_order_relaxed);
    done.fetch_or(bit, std::memory_order_acq_rel);
  } else {
    per_sm = resident.load(std::memory_order_relaxed);
  }
  // no more CTAs than chunks there can be
  const int64_t chunk = kWarps * kBlock;
  const int64_t events = static_cast<int64_t>(p.h.max_pages) * p.h.page_tokens;
  const int64_t tiles = p.a.q_rows * p.group / kRows + p.a.batch;
  const int64_t chunks = tiles * p.h.n_heads * ((events + chunk - 1) / chunk + 1);
  if (chunks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;   // history_attention has checked
  p.most = static_cast<int>(tiles * p.h.n_heads);
  const int64_t grid = std::min<int64_t>(
      {chunks, static_cast<int64_t>(device_sm_count()) * per_sm, int64_t(kAttnMaxCtas)});
  return launch_pdl(history_attention_kernel<D, DT>, dim3(static_cast<unsigned>(grid)),
                    dim3(kThreads), Sh::kSmem, stream, p);
}

template <int D>
cudaError_t launch_d(Params& p, cudaStream_t stream) {
  if (p.a.dtype == DLRM_DTYPE_FP32) return launch<D, DLRM_DTYPE_FP32>(p, stream);
  if (p.a.dtype == DLRM_DTYPE_BF16) return launch<D, DLRM_DTYPE_BF16>(p, stream);
  return launch<D, DLRM_DTYPE_FP16>(p, stream);
}

}  // namespace

cudaError_t launch_history_attention(const dlrm_history_t& h, const dlrm_attention_t& a,
                                     cudaStream_t stream, const int32_t* groups, int n_groups) {
  const HistoryWork w = history_work(h);
  Params p;
  p.h = h;
  p.a = a;
  p.group = a.n_heads / h.n_heads;
  const int64_t four = 4 * dtype_bytes(a.dtype);
  p.vec_q = reinterpret_cast<uintptr_t>(a.q) % four == 0 && a.ld_q % 4 == 0 && a.ld_q_head % 4 == 0;
  p.counters = work_part<int32_t>(h, w.counters);
  p.partials = work_part<float>(h, w.partials);
  p.groups = groups;
  p.n_groups = n_groups;
  if (history_tc_takes(h, a)) return launch_history_attention_tc(h, a, p.counters, p.partials, stream);
  if (h.head_dim == 32) return launch_d<32>(p, stream);
  if (h.head_dim == 64) return launch_d<64>(p, stream);
  return launch_d<128>(p, stream);
}

}  // namespace dlrm
