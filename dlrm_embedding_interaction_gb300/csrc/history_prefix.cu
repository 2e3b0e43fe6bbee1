// Attention of queries over cached histories that share a long prefix
// (include/dlrm.h, history_prefix_attention): the pages that all histories of a
// group of requests hold in common are read once for the group's rows.
//
// Two launches. The plan (a CTA a group) compares the page tables of a group's
// histories and lists the row tiles: up to kRows of the group's (query, head of the
// kv head) rows, which see the shared events together, then, one after another, the
// events that the tile's requests have of their own. The last CTA of the plan cuts all
// tiles of all kv heads, chunk by chunk, into equal parts for the second launch.
//
// The second launch is history_attention's method (history_attention.cu: layouts of
// keys and values, scales, splits of fp32, the join of parts) with more rows a block of
// events: WR warps share a ring of blocks and take MT MMA row tiles each, and a warp
// converts a block's codes once for its MT tiles. A block of one request's own events
// is multiplied with the row tiles that hold its rows alone, and masked for the others'.
#include <atomic>

#include "history_attention.cuh"

namespace dlrm {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kWholeBlocks = 16;                 // blocks of a tile that is never split
constexpr int kLeastBlocks = 16;                 // blocks of a CTA at least, where tiles are longer
constexpr int kWeights = 32;                     // parts whose weights lie in shared memory at once

// What the plan knows of a request with rows, and of the tiles.
struct Member {
  int32_t slot, len, queries;
  int32_t row0, rows;                            // among the group's rows
  int32_t first;                                 // blocks of the group's earlier requests
  int32_t sinks, block0;                         // blocks of its own events: the sinks', then from block0 on
};
static_assert(sizeof(Member) == kPrefixMember, "scratch size of a member");
struct Tile {
  int32_t first, chunks;                         // units of work (chunk of a kv head) before it; its chunks
  int32_t q0, row0, rows;                        // the group's first query row; rows among the group's
  int32_t member0, member1;                      // first and last request with rows in the tile
  int32_t slot;                                  // whose table gives the shared pages
  int32_t shared_sinks, shared0, shared_blocks;  // blocks of shared events: the sinks', then from shared0 on
  int32_t own0;                                  // first block that is not shared
};
static_assert(sizeof(Tile) == kPrefixTile, "scratch size of a tile");

struct Params {
  dlrm_history_t h;
  dlrm_attention_t a;
  const int32_t* groups;
  int n_groups;
  int group;                                     // query heads of a kv head
  int rows, split;                               // of a tile; warps that split a chunk's blocks
  int grid;                                      // CTAs of the second launch
  int vec_q;
  int32_t* head;                                 // arrived, units, CTAs with units
  Member* members;
  Tile* found;                                   // tiles, with gaps between the groups
  Tile* tiles;                                   // without
  int2* cuts;                                    // of each CTA: first unit, its tile
  int32_t* counters;
  float* partials;
};
enum { kHeadArrived = 0, kHeadUnits = 1, kHeadCtas = 2 };

// Exclusive prefix sum over the CTA; total in every thread.
__device__ __forceinline__ int scan(int x, int* sums, int& total) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  int inc = x;
#pragma unroll
  for (int d = 1; d < kWarp; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == kWarp - 1) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int s = sums[lane];
    int si = s;
#pragma unroll
    for (int d = 1; d < kWarp; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, si, d);
      if (lane >= d) si += y;
    }
    sums[lane] = si - s;
    if (lane == kWarp - 1) sums[kWarp] = si;
  }
  __syncthreads();
  total = sums[kWarp];
  return sums[warp] + inc - x;
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ Params p) {
  __shared__ int sums[kWarp + 1];
  __shared__ int ref_s, len_s, gap_s, shared_s, last_s;
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, t = threadIdx.x, lane = t % kWarp;
  const int32_t* starts = p.a.q_starts;
  if (t == 0) {
    ref_s = INT32_MAX;
    len_s = INT32_MAX;
    gap_s = INT32_MAX;
  }
  pdl_wait();
  pdl_trigger();
  // starts or groups that decrease or leave their range: nothing is done
  bool bad = false;
  for (int i = t; i <= p.a.batch; i += kPlanThreads) {
    const int x = starts[i];
    bad |= x < 0 || x > p.a.q_rows || (i < p.a.batch && starts[i + 1] < x);
  }
  for (int i = t; i <= p.n_groups; i += kPlanThreads) {
    const int x = p.groups[i];
    bad |= x < 0 || x > p.a.batch || (i < p.n_groups && p.groups[i + 1] < x);
  }
  bad = __syncthreads_or(bad);
  const int g = blockIdx.x;
  auto tile_base = [&](int group) {              // at least a group's tiles apart
    return static_cast<int>(static_cast<int64_t>(starts[p.groups[group]]) * p.group / p.rows) + group;
  };
  if (!bad) {
    const int b0 = p.groups[g], b1 = p.groups[g + 1], q0 = starts[b0];
    const int64_t cap = static_cast<int64_t>(M) * G;
    // ---- lengths; the events that every request with rows and events has
    auto first_seen = [&](int len, int queries) {   // of its first row
      return visible(p.a.causal ? len - queries : len - 1, len, p.a.window, p.a.sinks);
    };
    for (int b = b0 + t; b < b1; b += kPlanThreads) {
      Member m{};
      m.slot = p.a.slots[b];
      m.queries = starts[b + 1] - starts[b];
      m.row0 = (starts[b] - q0) * p.group;
      m.rows = m.queries * p.group;
      if (m.slot >= 0 && m.slot < h.n_slots) {
        m.len = static_cast<int>(min(static_cast<int64_t>(max(h.lengths[m.slot], 0)), cap));
      } else {
        flag(h.err, DLRM_ERRBIT_INDEX_OOB);
      }
      p.members[b] = m;
      if (m.rows > 0 && m.len > 0) {
        atomicMin(&ref_s, b);
        atomicMin(&len_s, m.len);
        atomicMin(&gap_s, first_seen(m.len, m.queries).gap1);
      }
    }
    __syncthreads();
    const int ref = ref_s;
    if (t == 0) shared_s = ref == INT32_MAX ? 0 : len_s / G;
    __syncthreads();
    // ---- shared pages: the first entry that differs, 8 x 32 entries of a request at a time
    const int pages = shared_s;
    int ref_slot = -1;
    if (pages > 0) {
      ref_slot = p.members[ref].slot;
      const int32_t* mine = h.table + static_cast<int64_t>(ref_slot) * M;
      const int pieces = (pages + 255) / 256;
      const int64_t work = static_cast<int64_t>(b1 - b0) * pieces;
      for (int64_t w = t / kWarp; w < work; w += kPlanThreads / kWarp) {
        const int b = b0 + static_cast<int>(w / pieces), j0 = static_cast<int>(w % pieces) * 256 + lane;
        const Member m = p.members[b];
        if (b == ref || m.rows == 0 || m.len == 0) continue;
        const int32_t* row = h.table + static_cast<int64_t>(m.slot) * M;
        int differ = INT32_MAX;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const int j = j0 + i * kWarp;
          if (j < pages && row[j] != mine[j]) differ = j;
        }
        differ = __reduce_min_sync(0xffffffffu, differ);
        if (lane == 0 && differ < pages) atomicMin(&shared_s, differ);
      }
    }
    __syncthreads();
    const int shared = shared_s * G;             // events
    // ---- every request's blocks of its own, and how many lie before them
    int before = 0;
    for (int c0 = b0; c0 < b1; c0 += kPlanThreads) {
      const int b = c0 + t;
      int n = 0;
      Member m{};
      if (b < b1) {
        m = p.members[b];
        if (m.rows > 0 && m.len > 0) {
          const Visible v = first_seen(m.len, m.queries);
          const int end = (m.len + kBlock - 1) / kBlock, low = shared / kBlock;
          m.block0 = max(v.gap1 / kBlock, low);
          m.sinks = v.gap1 > shared ? max((min(v.gap0, m.len) + kBlock - 1) / kBlock - low, 0) : 0;
          if (low + m.sinks >= m.block0) {       // no gap: blocks from `shared` on
            m.sinks = 0;
            m.block0 = low;
          }
          n = m.sinks + max(end - m.block0, 0);
        }
      }
      int total;
      m.first = before + scan(n, sums, total);
      before += total;
      if (b < b1) p.members[b] = m;
      __syncthreads();
    }
    __syncthreads();
    // ---- tiles
    const int rows = (starts[b1] - q0) * p.group, tiles = (rows + p.rows - 1) / p.rows;
    const int base = tile_base(g), next = tile_base(g + 1);
    const int gap1 = gap_s == INT32_MAX ? 0 : gap_s, gap0 = min(p.a.sinks, gap1);
    Tile x{};
    x.q0 = q0;
    x.slot = ref_slot;
    x.own0 = shared / kBlock;
    x.shared0 = min(gap1, shared) / kBlock;
    x.shared_sinks = min((min(gap0, shared) + kBlock - 1) / kBlock, x.shared0);
    if (x.shared_sinks == x.shared0) x.shared_sinks = x.shared0 = 0;
    x.shared_blocks = x.shared_sinks + x.own0 - x.shared0;
    auto holds = [&](int row) {                  // the request of a row
      int lo = b0, hi = b1;                      // the last one that begins at or before it
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if ((starts[mid] - q0) * p.group <= row) lo = mid; else hi = mid;
      }
      return lo;
    };
    for (int i = t; base + i < next; i += kPlanThreads) {
      Tile y = x;
      if (i < tiles) {
        y.row0 = i * p.rows;
        y.rows = min(p.rows, rows - y.row0);
        y.member0 = holds(y.row0);
        y.member1 = holds(y.row0 + y.rows - 1);
        const Member last = p.members[y.member1];
        int blocks = y.shared_blocks - p.members[y.member0].first + last.first;
        if (last.len > 0) blocks += last.sinks + max((last.len + kBlock - 1) / kBlock - last.block0, 0);
        y.chunks = max((blocks + p.split - 1) / p.split, 1);   // an empty one writes zeros
      }
      p.found[base + i] = y;
    }
  }
  // ---- the last CTA: units, and the CTAs' parts
  __threadfence();
  __syncthreads();
  if (t == 0) {
    const unsigned before = atomicInc(reinterpret_cast<unsigned*>(&p.head[kHeadArrived]), gridDim.x - 1);
    last_s = before == gridDim.x - 1;
  }
  __syncthreads();
  if (!last_s) return;
  __threadfence();
  if (bad && t == 0) flag(h.err, DLRM_ERRBIT_OFFSETS);
  const int t0 = bad ? 0 : tile_base(0), t1 = bad ? 0 : tile_base(p.n_groups);
  int units = 0, dense = 0, pieces = 0;
  const int per = (t1 - t0 + kPlanThreads - 1) / kPlanThreads;
  const int mine0 = min(t1, t0 + t * per), mine1 = min(t1, mine0 + per);
  for (int i = mine0; i < mine1; ++i) {
    const int chunks = __ldcg(&p.found[i].chunks);
    units += chunks * h.n_heads;
    dense += chunks > 0;
  }
  int total, n_tiles;
  int at = scan(units, sums, total);
  int place = scan(dense, sums, n_tiles);
  pieces = n_tiles * h.n_heads;
  Cuts cuts;
  cuts.total = total;
  cuts.ctas = min(p.grid, min(total, max(total / max(kLeastBlocks / p.split, 1), pieces)));
  cuts.each = cuts.ctas > 0 ? total / cuts.ctas : 0;
  cuts.extra = total - cuts.each * cuts.ctas;
  const int whole = kWholeBlocks / p.split;
  for (int i = mine0; i < mine1; ++i) {
    Tile y;
    const int4* from = reinterpret_cast<const int4*>(&p.found[i]);
    int4* to = reinterpret_cast<int4*>(&y);
#pragma unroll
    for (int w = 0; w < static_cast<int>(sizeof(Tile) / 16); ++w) to[w] = __ldcg(from + w);
    if (y.chunks == 0) continue;
    y.first = at;
    p.tiles[place] = y;
    // the CTAs that begin in this tile; a cut inside a short piece moves to its
    // start: finishing it in one CTA is faster than joining parts
    const int end = at + y.chunks * h.n_heads;
    int c = cuts.owner(at);
    if (cuts.cut(c) < at) ++c;
    for (; c < cuts.ctas && cuts.cut(c) < end; ++c) {
      int cut = cuts.cut(c);
      if (y.chunks <= whole) cut -= static_cast<unsigned>(cut - at) % static_cast<unsigned>(y.chunks);
      p.cuts[c] = make_int2(cut, place);
    }
    at = end;
    ++place;
  }
  for (int c = cuts.ctas + t; c <= p.grid; c += kPlanThreads) p.cuts[c] = make_int2(total, n_tiles);
  if (t == 0) {
    p.head[kHeadUnits] = total;
    p.head[kHeadCtas] = cuts.ctas;
  }
}

template <int D, int DT, int MT, int WR>
struct Shape {
  static constexpr bool kSplit = DT == DLRM_DTYPE_FP32;
  static constexpr int kTile = kSplit ? 8 : 16;   // rows of an MMA tile
  static constexpr int kRows = kTile * MT * WR;
  static constexpr int kSets = kWarps / WR;       // sets of warps, a ring and a block of each chunk each
  static constexpr int kStages = WR == 1 ? (D == 128 ? 3 : 4) : D == 128 ? 4 : 6;
  static constexpr int kBytes = 2 * kBlock * D;   // keys and values of a block
  static constexpr int kStride = D + 2;           // a row's sums, maximum, sum of weights
  static constexpr int kRing = kSets * kStages * kBytes;
  static constexpr int kJoin = (kSets * kRows * kStride + kWeights * kRows) * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

template <int D, int DT, int MT, int WR>
__global__ void __launch_bounds__(kThreads) prefix_attention_kernel(const __grid_constant__ Params p) {
  using Sh = Shape<D, DT, MT, WR>;
  constexpr bool kSplit = Sh::kSplit;
  constexpr int kTile = Sh::kTile, kRows = Sh::kRows, kSets = Sh::kSets, kStages = Sh::kStages;
  constexpr int kStride = Sh::kStride;
  constexpr int KW = D / 16;                      // key words of a thread and event tile
  constexpr int VW = D / 32;                      // value words of a thread and event
  constexpr int NT = D / 8;                       // n tiles of the output
  constexpr int kAcc = kSplit ? 2 : 4;            // output values of a thread and n tile
  constexpr int kR2 = kSplit ? 1 : 2;             // rows of a thread and row tile
  extern __shared__ __align__(128) unsigned char smem[];
  float (*joined)[kRows][kStride] = reinterpret_cast<float (*)[kRows][kStride]>(smem);
  float* weight = reinterpret_cast<float*>(smem) + kSets * kRows * kStride;   // [part][row]
  __shared__ float row_factor[kRows];
  __shared__ int odd[kRows + 1];
  __shared__ int see_end[kRows], see_gap0[kRows], see_gap1[kRows], row_member[kRows];
  __shared__ int hull_end, hull_gap0, hull_gap1, n_members;
  // requests with rows in the tile: their rows [lo, hi) of it, first block
  __shared__ int m_lo[kRows], m_hi[kRows], m_first[kRows], m_id[kRows];
  __shared__ Member m_of[kRows];

  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int set = warp / WR, wr = warp % WR;
  const int g = lane / 4, c = lane % 4;
  const int G = p.h.page_tokens, H = p.h.n_heads, shift = __ffs(G) - 1;   // G: a power of two
  unsigned char* ring = smem + set * kStages * Sh::kBytes;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  pdl_wait();
  pdl_trigger();
  Cuts cuts;
  cuts.total = p.head[kHeadUnits];
  cuts.ctas = p.head[kHeadCtas];
  cuts.each = cuts.ctas > 0 ? cuts.total / cuts.ctas : 0;
  cuts.extra = cuts.total - cuts.each * cuts.ctas;
  const int2 from = p.cuts[blockIdx.x];
  const int end = p.cuts[blockIdx.x + 1].x;
  int place = from.y - 1, at = from.x, at_end = at;
  Tile s{};

  for (int u = from.x; u < end;) {
    if (u >= at_end) {
      s = p.tiles[++place];
      at = s.first;
      at_end = at + s.chunks * H;
      // ---- the tile's requests and rows
      __syncthreads();
      if (warp == 0) {
        int n = 0, first = s.shared_blocks;
        for (int b0 = s.member0; b0 <= s.member1; b0 += kWarp) {
          const int b = b0 + lane;
          Member m{};
          if (b <= s.member1) m = p.members[b];
          const bool in = m.rows > 0;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          const int blocks = in && m.len > 0 ? m.sinks + max((m.len + kBlock - 1) / kBlock - m.block0, 0) : 0;
          int inc = blocks;
#pragma unroll
          for (int d = 1; d < kWarp; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
          }
          const int i = n + __popc(who & ((1u << lane) - 1));
          if (in && i < kRows) {                  // (each has a row of the tile)
            m_lo[i] = max(m.row0 - s.row0, 0);
            m_hi[i] = min(m.row0 + m.rows - s.row0, s.rows);
            m_first[i] = first + inc - blocks;
            m_id[i] = b;
            m_of[i] = m;
          }
          n += __popc(who);
          first += __shfl_sync(0xffffffffu, inc, kWarp - 1);
        }
        if (lane == 0) {
          n_members = min(n, kRows);
          hull_end = 0;
          hull_gap0 = 0;
          hull_gap1 = INT32_MAX;
        }
      }
      __syncthreads();
      for (int r = threadIdx.x; r < kRows; r += kThreads) {
        const int row = min(r, s.rows - 1);       // rows past the last stand for it
        int i = 0;                                // the last request that begins at or before it
        for (int d = n_members; d > 1;) {
          const int half = d / 2;
          if (m_lo[i + half] <= row) i += half;
          d -= half;
        }
        const Member& m = m_of[i];
        const int query = static_cast<unsigned>(s.row0 + row - m.row0) / static_cast<unsigned>(p.group);
        const Visible v = visible(p.a.causal ? m.len - m.queries + query : m.len - 1, m.len, p.a.window, p.a.sinks);
        see_end[r] = v.end;
        see_gap0[r] = v.gap0;
        see_gap1[r] = v.gap1;
        row_member[r] = i;
        atomicMax(&hull_end, v.end);
        atomicMax(&hull_gap0, v.gap0);
        atomicMin(&hull_gap1, v.gap1);
      }
      __syncthreads();
    }
    const int head = static_cast<unsigned>(u - at) / static_cast<unsigned>(s.chunks);
    const int seg0 = at + head * s.chunks, seg1 = seg0 + s.chunks;
    const int chunk0 = u - seg0, chunk1 = min(end, seg1) - seg0;
    const int rows = s.rows;
    u = seg0 + chunk1;

    // ---- queries: the loads first, the arithmetic while the events are on their way
    float x[MT][2][KW][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        const int r = (wr * MT + mt) * kTile + (kSplit ? g : g + 8 * r2);
        const bool in = r < rows;
        const int row = s.row0 + min(r, rows - 1);
        const int query = static_cast<unsigned>(row) / static_cast<unsigned>(p.group);
        const int64_t q_at = (s.q0 + static_cast<int64_t>(query)) * p.a.ld_q +
                             (head * p.group + row - query * p.group) * p.a.ld_q_head;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          if (in) {
            load_four<DT>(x[mt][r2][w], p.a.q, q_at + key_element<D>(c, w), p.vec_q);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][r2][w][e] = 0.f;
          }
        }
      }

    // ---- blocks of this set of warps: n0, n0 + kSets, ...; lane l knows block l of
    // the 32 at hand (info) and of the 32 after them (ahead)
    const int last = n_members - 1;
    const Member& m_last = m_of[last];
    const int blocks = m_first[last] +
        (m_last.len > 0 ? m_last.sinks + max((m_last.len + kBlock - 1) / kBlock - m_last.block0, 0) : 0);
    const int n0 = chunk0 * kSets + set, n1 = min(chunk1 * kSets, blocks);
    const int count = n0 < n1 ? (n1 - n0 + kSets - 1) / kSets : 0;
    struct Info {
      int page;                                   // -1: nothing to read
      int t0, member;                             // first event; whose own, or -1: shared
      float ks, vs;
    };
    auto look = [&](int i) {
      Info x{-1, 0, -1, 0.f, 0.f};
      if (i < count) {
        const int n = n0 + i * kSets;
        int slot = s.slot;
        bool seen;
        if (n < s.shared_blocks) {
          x.t0 = (n < s.shared_sinks ? n : n - s.shared_sinks + s.shared0) * kBlock;
          // not what no row of the tile sees
          seen = x.t0 < hull_end && !(x.t0 >= hull_gap0 && x.t0 + kBlock <= hull_gap1);
        } else {
          int k = 0;                              // the last request whose blocks begin at or before it
          for (int d = n_members; d > 1;) {
            const int half = d / 2;
            if (m_first[k + half] <= n) k += half;
            d -= half;
          }
          const Member& m = m_of[k];
          const int j = n - m_first[k];
          x.member = k;
          x.t0 = (j < m.sinks ? s.own0 + j : j - m.sinks + m.block0) * kBlock;
          slot = m.slot;
          seen = x.t0 < m.len;
        }
        if (seen) {
          x.page = p.h.table[static_cast<int64_t>(slot) * p.h.max_pages + (x.t0 >> shift)];
          if (x.page < 0 || x.page >= p.h.n_pages) {
            // trimmed, or a broken table: events that some row needs
            x.page = -1;
            flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);
          } else {
            const int64_t where = static_cast<int64_t>(x.page) * H + head;
            x.ks = p.h.k_scales[where];
            x.vs = p.h.v_scales[where];
          }
        }
      }
      return x;
    };
    Info info = look(lane), ahead = look(kWarp + lane);
    int base = 0;                                 // blocks [base, base + 32) are in info
    auto fetch = [&](int i) {
      if (i < count) {
        const bool here = i - base < kWarp;
        const int page = __shfl_sync(0xffffffffu, here ? info.page : ahead.page, i % kWarp);
        const int t0 = __shfl_sync(0xffffffffu, here ? info.t0 : ahead.t0, i % kWarp);
        if (page >= 0) {
          const int64_t codes = ((static_cast<int64_t>(page) * H + head) * G + (t0 & (G - 1))) * D;
          const uint32_t dst = ring_at + (i % kStages) * Sh::kBytes;
          constexpr int kSide = 2 * D;            // 16-byte chunks of a side
#pragma unroll
          for (int x = 0; x < 2 * kSide / (kWarp * WR); ++x) {
            const int both = (x * WR + wr) * kWarp + lane;   // (a warp's chunks lie on one side)
            const int id = both % kSide, t = id / (D / 16), ch = id % (D / 16);
            if (both < kSide)
              copy16(dst + key_offset<D>(t, ch), p.h.k_codes + codes + id * 16);
            else
              copy16(dst + kBlock * D + value_offset<D>(t, ch), p.h.v_codes + codes + id * 16);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto set_barrier = [&] {
      if (WR == 1)
        __syncwarp();
      else if (WR == kWarps)
        __syncthreads();
      else if (set == 0)
        asm volatile("bar.sync 1, %0;" ::"n"(WR * kWarp) : "memory");
      else
        asm volatile("bar.sync 2, %0;" ::"n"(WR * kWarp) : "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ---- fragments of the queries, scaled to f16; a negative softmax scale is
    // theirs, so that the factors of the scores are positive
    uint32_t qa[MT][KW][4];
    float qf[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        float big = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[mt][r2][w][e]));
        big = quad_max(big);
        const int ex = max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100);
        const float f = copysignf(pow2f(min(8 - ex, 127)), p.a.scale);
        qf[mt][r2] = pow2f(max(ex - 8, -126)) * fabsf(p.a.scale) * kLog2e;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[mt][r2][w][e] *= f;
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float (&x0)[4] = x[mt][0][w], (&x1)[4] = x[mt][1][w];
        qa[mt][w][0] = pack_f16x2(x0[0], x0[1]);
        qa[mt][w][2] = pack_f16x2(x0[2], x0[3]);
        if (kSplit) {
          const float2 h0 = f16x2_to_float2(qa[mt][w][0]), h1 = f16x2_to_float2(qa[mt][w][2]);
          qa[mt][w][1] = pack_f16x2((x0[0] - h0.x) * 2048.f, (x0[1] - h0.y) * 2048.f);
          qa[mt][w][3] = pack_f16x2((x0[2] - h1.x) * 2048.f, (x0[3] - h1.y) * 2048.f);
        } else {
          qa[mt][w][1] = pack_f16x2(x1[0], x1[1]);
          qa[mt][w][3] = pack_f16x2(x1[2], x1[3]);
        }
      }
    }

    // ---- events
    float o[MT][NT][kAcc];
    float top[MT][2], sum[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      top[mt][0] = top[mt][1] = -INFINITY;
      sum[mt][0] = sum[mt][1] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kAcc; ++i) o[mt][nt][i] = 0.f;
    }
    for (int it = 0; it < count; ++it) {
      if (it - base == kWarp) {
        base += kWarp;
        info = ahead;
        ahead = look(base + kWarp + lane);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      set_barrier();                              // block `it` is there, and block it - 1 done with
      fetch(it + kStages - 1);
      const int page = __shfl_sync(0xffffffffu, info.page, it % kWarp);
      const int member = __shfl_sync(0xffffffffu, info.member, it % kWarp);
      if (page < 0) continue;
      // rows of the tile that the block is for
      const int lo = member < 0 ? 0 : m_lo[member], hi = member < 0 ? kRows : m_hi[member];
      if (hi <= wr * MT * kTile || lo >= (wr + 1) * MT * kTile) continue;
      const float ks = __shfl_sync(0xffffffffu, info.ks, it % kWarp);
      const float vs = __shfl_sync(0xffffffffu, info.vs, it % kWarp);
      const int t0 = __shfl_sync(0xffffffffu, info.t0, it % kWarp);
      const unsigned char* kb = ring + (it % kStages) * Sh::kBytes;
      const unsigned char* vb = kb + kBlock * D;
      bool takes[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        takes[mt] = MT == 1 || (hi > (wr * MT + mt) * kTile && lo < (wr * MT + mt + 1) * kTile);

      // S = Q K^T
      float sc[MT][kBlock / 8][4];
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        uint32_t kw[KW];
        if (D == 32) {
          const uint2 y = *reinterpret_cast<const uint2*>(kb + (8 * j + g) * 32 + 8 * c);
          kw[0] = y.x;
          kw[1] = y.y;
        } else {
#pragma unroll
          for (int i = 0; i < KW / 4; ++i) {
            const uint4 y = *reinterpret_cast<const uint4*>(kb + key_offset<D>(8 * j + g, 4 * i + c));
            kw[4 * i] = y.x;
            kw[4 * i + 1] = y.y;
            kw[4 * i + 2] = y.z;
            kw[4 * i + 3] = y.w;
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t b0 = e4m3x2_lo_to_f16x2(kw[w]), b1 = e4m3x2_hi_to_f16x2(kw[w]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            if (takes[mt]) mma_f16_from(sc[mt][j], qa[mt][w], b0, b1, w > 0);
        }
      }
      // weights: exp2 of the scores times the factors, less the running maximum
      uint32_t pa[MT][kBlock / 16][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (!takes[mt]) continue;
        const int r0 = (wr * MT + mt) * kTile + g;
        if (kSplit) {
#pragma unroll
          for (int j = 0; j < kBlock / 8; ++j) {
            sc[mt][j][0] = fmaf(sc[mt][j][2], 1.f / 2048.f, sc[mt][j][0]);
            sc[mt][j][1] = fmaf(sc[mt][j][3], 1.f / 2048.f, sc[mt][j][1]);
          }
        }
        float alpha[2] = {1.f, 1.f};
#pragma unroll
        for (int r2 = 0; r2 < kR2; ++r2) {
          const int r = r0 + 8 * r2;
          const Visible v{see_end[r], see_gap0[r], see_gap1[r]};
          const int row = min(r, rows - 1);
          const bool mine = row >= lo && row < hi;
          if (!(mine && t0 + kBlock <= v.end && (t0 >= v.gap1 || t0 + kBlock <= v.gap0))) {
#pragma unroll
            for (int j = 0; j < kBlock / 8; ++j) {
              const int t = t0 + 8 * j + 2 * c;
              if (!mine || !sees(v, t)) sc[mt][j][2 * r2] = -INFINITY;
              if (!mine || !sees(v, t + 1)) sc[mt][j][2 * r2 + 1] = -INFINITY;
            }
          }
          float big = -INFINITY;
#pragma unroll
          for (int j = 0; j < kBlock / 8; ++j)
            big = fmaxf(big, fmaxf(sc[mt][j][2 * r2], sc[mt][j][2 * r2 + 1]));
          // (the factor is not zero, even for a softmax scale of zero: a masked score is -infinity)
          const float f = fmaxf(qf[mt][r2] * ks, 1e-37f);
          const float m = fmaxf(top[mt][r2], ceilf(quad_max(big) * f));
          const float ref = m == -INFINITY ? 0.f : m, off = kLift - ref;
          alpha[r2] = exp2_approx(top[mt][r2] - ref);
          top[mt][r2] = m;
          float add = 0.f;
#pragma unroll
          for (int j = 0; j < kBlock / 8; ++j) {
            sc[mt][j][2 * r2] = exp2_approx(fmaf(sc[mt][j][2 * r2], f, off));
            sc[mt][j][2 * r2 + 1] = exp2_approx(fmaf(sc[mt][j][2 * r2 + 1], f, off));
            add += sc[mt][j][2 * r2] + sc[mt][j][2 * r2 + 1];
          }
          sum[mt][r2] = fmaf(sum[mt][r2], alpha[r2], add);
        }
        // the output's correction, where the maximum of some row grew
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < kAcc; ++i) o[mt][nt][i] *= alpha[i >> 1];
        }
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt) {
          const float (&s0)[4] = sc[mt][2 * kt], (&s1)[4] = sc[mt][2 * kt + 1];
          uint32_t (&a)[4] = pa[mt][kt];
          a[0] = pack_f16x2(s0[0], s0[1]);
          a[2] = pack_f16x2(s1[0], s1[1]);
          if (kSplit) {
            const float2 h0 = f16x2_to_float2(a[0]), h1 = f16x2_to_float2(a[2]);
            a[1] = pack_f16x2((s0[0] - h0.x) * 2048.f, (s0[1] - h0.y) * 2048.f);
            a[3] = pack_f16x2((s1[0] - h1.x) * 2048.f, (s1[1] - h1.y) * 2048.f);
          } else {
            a[1] = pack_f16x2(s0[2], s0[3]);
            a[3] = pack_f16x2(s1[2], s1[3]);
          }
        }
      }
      // O += vs P V
      uint32_t vw[kBlock / 16][4][VW];
#pragma unroll
      for (int kt = 0; kt < kBlock / 16; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1);
          if (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(vb + value_offset<D>(t, g));
            vw[kt][i][0] = y.x;
            vw[kt][i][VW > 1 ? 1 : 0] = y.y;
            vw[kt][i][VW > 2 ? 2 : 0] = y.z;
            vw[kt][i][VW > 3 ? 3 : 0] = y.w;
          } else if (D == 64) {
            const uint2 y = *reinterpret_cast<const uint2*>(vb + value_offset<D>(t, g >> 1) + 8 * (g & 1));
            vw[kt][i][0] = y.x;
            vw[kt][i][VW > 1 ? 1 : 0] = y.y;
          } else {
            vw[kt][i][0] = *reinterpret_cast<const uint32_t*>(vb + value_offset<D>(t, g >> 2) + 4 * (g & 3));
          }
        }
      if (member >= 0 && t0 + kBlock > m_of[member].len) {
        // codes of events past the end are whatever an earlier history left there
        const int len = m_of[member].len;
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1) >= len)
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[kt][i][w] = 0;
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        // bytes of a pair of events side by side: n tiles 4w, 4w+1 and 4w+2, 4w+3
        uint32_t b[kBlock / 16][4][2];
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt) {
          const uint32_t l0 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x5140);
          const uint32_t l1 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x7362);
          const uint32_t h0 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x5140);
          const uint32_t h1 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x7362);
          b[kt][0][0] = e4m3x2_lo_to_f16x2(l0), b[kt][0][1] = e4m3x2_lo_to_f16x2(h0);
          b[kt][1][0] = e4m3x2_hi_to_f16x2(l0), b[kt][1][1] = e4m3x2_hi_to_f16x2(h0);
          b[kt][2][0] = e4m3x2_lo_to_f16x2(l1), b[kt][2][1] = e4m3x2_lo_to_f16x2(h1);
          b[kt][3][0] = e4m3x2_hi_to_f16x2(l1), b[kt][3][1] = e4m3x2_hi_to_f16x2(h1);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (!takes[mt]) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float acc[4];
#pragma unroll
            for (int kt = 0; kt < kBlock / 16; ++kt) mma_f16_from(acc, pa[mt][kt], b[kt][i][0], b[kt][i][1], kt > 0);
            float* out = o[mt][4 * w + i];
            if (kSplit) {
              out[0] = fmaf(vs, fmaf(acc[2], 1.f / 2048.f, acc[0]), out[0]);
              out[1] = fmaf(vs, fmaf(acc[3], 1.f / 2048.f, acc[1]), out[1]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) out[j] = fmaf(vs, acc[j], out[j]);
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the sets of warps
    __syncthreads();                              // every ring is done with: `joined` lies there
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r2 = 0; r2 < kR2; ++r2) {
        const float l = quad_sum(sum[mt][r2]);
        float* out = joined[set][(wr * MT + mt) * kTile + g + 8 * r2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          out[2 * c * (D / 8) + nt] = o[mt][nt][2 * r2];
          out[(2 * c + 1) * (D / 8) + nt] = o[mt][nt][2 * r2 + 1];
        }
        if (c == 0) {
          out[D] = top[mt][r2];
          out[D + 1] = l;
        }
      }
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int r = threadIdx.x;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kSets; ++w) m = fmaxf(m, joined[w][r][D]);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kSets; ++w) {
        const float f = exp2_approx(joined[w][r][D] - ref);
        l = fmaf(f, joined[w][r][D + 1], l);
        joined[w][r][D] = f;
      }
      joined[0][r][D + 1] = l;
      row_factor[r] = m;
    }
    __syncthreads();
    const bool split = chunk0 > 0 || chunk1 < s.chunks;
    constexpr int kPartial = kRows * kStride;
    float* mine = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (chunk0 > 0 ? 0 : 1)) * kPartial;
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
      const int r = e / D, d = e % D;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kSets; ++w) y = fmaf(joined[w][r][D], joined[w][r][d], y);
      if (split)
        mine[r * kStride + d] = y;
      else
        joined[0][r][d] = y;
    }
    if (split) {
      if (threadIdx.x < rows) {
        mine[threadIdx.x * kStride + D] = row_factor[threadIdx.x];
        mine[threadIdx.x * kStride + D + 1] = joined[0][threadIdx.x][D + 1];
      }
      // the CTAs that share this piece: first .. last, one part each. (A cut moves
      // out of short pieces only, so a split one's cuts are where they were.)
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
      auto part = [&](int i) { return p.partials + ((first + i) * 2 + (i > 0 ? 0 : 1)) * kPartial; };
      // maximum of each row over the parts, the parts' weights, then the weighted
      // sums, every thread with all its elements of a part under way
      for (int r = warp; r < rows; r += kWarps) {
        float m = -INFINITY;
        for (int i = lane; i < parts; i += kWarp) m = fmaxf(m, __ldcg(part(i) + r * kStride + D));
#pragma unroll
        for (int x = 16; x > 0; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (lane == 0) row_factor[r] = m;
      }
      constexpr int kPairs = kRows * D / 2 / kThreads;
      static_assert(kPairs * 2 * kThreads == kRows * D, "elements of a thread");
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
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
          const float* q = part(p0 + i);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const int of = 2 * (e * kThreads + threadIdx.x), r = of / D, d = of % D;
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
        const int of = 2 * (e * kThreads + threadIdx.x), r = of / D, d = of % D;
        joined[0][r][d] = acc[e].x;
        joined[0][r][d + 1] = acc[e].y;
      }
      if (threadIdx.x < rows) joined[0][threadIdx.x][D + 1] = l;
    }
    for (int r = threadIdx.x; r <= kRows; r += kThreads) odd[r] = 0;
    __syncthreads();

    // ---- outputs
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
      const int r = e / D, d = e % D;
      const int row = s.row0 + r, query = row / p.group;
      const float l = joined[0][r][D + 1];
      const float y = l == 0.f ? 0.f : joined[0][r][d] / l;
      const int64_t i = s.q0 + static_cast<int64_t>(query);
      const int hq = head * p.group + row - query * p.group;
      store_element<DT>(p.a.out, i * p.a.ld_out + hq * p.a.ld_out_head + d, y);
      if (d == 0 && p.a.lse)
        p.a.lse[i * p.a.n_heads + hq] = l == 0.f ? -INFINITY : row_factor[r] * kLn2 + logf(l * pow2f(-kLift));
      if (!finite(y) || l == 0.f) odd[r] = odd[kRows] = l == 0.f ? 2 : 1;   // 2: sees nothing, or has no weights
    }
    __syncthreads();
    if (odd[kRows]) {
      for (int r = 0; r < rows; ++r) {
        const int row = s.row0 + r, query = row / p.group, hq = head * p.group + row - query * p.group;
        const Visible v{see_end[r], see_gap0[r], see_gap1[r]};
        const int64_t i = s.q0 + static_cast<int64_t>(query);
        if (odd[r] == 1 || (odd[r] == 2 && sees_any(v)))
          careful_row<DT>(p.h, p.a, m_of[row_member[r]].slot, v, head, i * p.a.ld_q + hq * p.a.ld_q_head,
                          i * p.a.ld_out + hq * p.a.ld_out_head, i * p.a.n_heads + hq, &joined[0][0][0]);
      }
    }
    __syncthreads();                              // `joined` is read: the rings may be filled
  }
}

template <int D, int DT, int MT, int WR>
cudaError_t launch(Params& p, cudaStream_t stream) {
  using Sh = Shape<D, DT, MT, WR>;
  // set once on every device, by a bit each; the CTAs of an SM are the same on every GB300
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  int per_sm = 0;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prefix_attention_kernel<D, DT, MT, WR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, prefix_attention_kernel<D, DT, MT, WR>,
                                                      kThreads, Sh::kSmem);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, per_sm);
    resident.store(per_sm, std::memory_order_relaxed);
    done.fetch_or(bit, std::memory_order_acq_rel);
  } else {
    per_sm = resident.load(std::memory_order_relaxed);
  }
  // no more CTAs than counters, than partial results have space, and than pieces of
  // kLeastBlocks there can be
  const int64_t events = static_cast<int64_t>(p.h.max_pages) * p.h.page_tokens;
  const int64_t tiles = p.a.q_rows * p.group / Sh::kRows + p.n_groups;
  const int64_t blocks = (tiles * 2 + p.a.batch) * p.h.n_heads * (events / kBlock + 2);
  p.rows = Sh::kRows;
  p.split = Sh::kSets;
  p.grid = static_cast<int>(std::min<int64_t>(
      {std::max<int64_t>(blocks / kLeastBlocks, tiles * p.h.n_heads), static_cast<int64_t>(device_sm_count()) * per_sm,
       int64_t(kAttnMaxCtas), kAttnPartialFloats / (2 * Sh::kRows * Sh::kStride)}));
  e = launch_pdl(prefix_plan_kernel, dim3(p.n_groups), dim3(kPlanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_attention_kernel<D, DT, MT, WR>, dim3(p.grid), dim3(kThreads), Sh::kSmem, stream, p);
}

template <int D, int DT>
cudaError_t launch_rows(Params& p, cudaStream_t stream) {
  // by the rows of a group and kv head, on average
  constexpr int kTile = DT == DLRM_DTYPE_FP32 ? 8 : 16;
  const int64_t rows = (p.a.q_rows * p.group + p.n_groups - 1) / p.n_groups;
  if (rows <= kTile) return launch<D, DT, 1, 1>(p, stream);
  if (rows <= 2 * kTile) return launch<D, DT, 1, 2>(p, stream);
  return launch<D, DT, 1, 4>(p, stream);
}

template <int D>
cudaError_t launch_d(Params& p, cudaStream_t stream) {
  if (p.a.dtype == DLRM_DTYPE_FP32) return launch_rows<D, DLRM_DTYPE_FP32>(p, stream);
  if (p.a.dtype == DLRM_DTYPE_BF16) return launch_rows<D, DLRM_DTYPE_BF16>(p, stream);
  return launch_rows<D, DLRM_DTYPE_FP16>(p, stream);
}

}  // namespace

cudaError_t launch_history_prefix_attention(const dlrm_history_t& h, const dlrm_attention_t& a,
                                            const int32_t* groups, int n_groups, cudaStream_t stream) {
  const HistoryWork w = history_work(h);
  Params p;
  p.h = h;
  p.a = a;
  p.groups = groups;
  p.n_groups = n_groups;
  p.group = a.n_heads / h.n_heads;
  const int64_t four = 4 * dtype_bytes(a.dtype);
  p.vec_q = reinterpret_cast<uintptr_t>(a.q) % four == 0 && a.ld_q % 4 == 0 && a.ld_q_head % 4 == 0;
  p.head = work_part<int32_t>(h, w.prefix_head);
  p.members = work_part<Member>(h, w.members);
  p.found = work_part<Tile>(h, w.found_tiles);
  p.tiles = work_part<Tile>(h, w.tiles_of);
  p.cuts = work_part<int2>(h, w.cuts);
  p.counters = work_part<int32_t>(h, w.counters);
  p.partials = work_part<float>(h, w.partials);
  if (h.head_dim == 32) return launch_d<32>(p, stream);
  if (h.head_dim == 64) return launch_d<64>(p, stream);
  return launch_d<128>(p, stream);
}

}  // namespace dlrm
