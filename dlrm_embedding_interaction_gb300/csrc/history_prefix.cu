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
// keys and values, scales, splits of fp32, the join of parts) over a tile's list of
// blocks; a block of one request's own events is masked for the other rows.
#include "history_prefix.cuh"

namespace dlrm {
namespace prefix {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kHere = 256;                       // requests of a group that shared memory holds
constexpr int kTilesHere = 256;                  // tiles that shared memory holds

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
    const int s = lane < kPlanThreads / kWarp ? sums[lane] : 0;
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

// What bounds it: a chain of loads, each of which waits for the one before: groups, starts
// and slots, lengths, tables; then, in the last CTA, the tiles. What belongs to a group
// stays in shared memory in between, for up to kHere requests. 11 us for 64 groups, of which the
// last CTA takes 5.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ Params p) {
  __shared__ int sums[kWarp + 1];
  __shared__ int ref_s, len_s, gap_s, shared_s, last_s;
  __shared__ Member here[kHere];
  __shared__ Tile tiles_s[kTilesHere];
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, t = threadIdx.x, lane = t % kWarp, g = blockIdx.x;
  const int32_t* starts = p.a.q_starts;
  if (t == 0) {
    ref_s = INT32_MAX;
    len_s = INT32_MAX;
    gap_s = INT32_MAX;
  }
  pdl_wait();
  pdl_trigger();
  // everything that hangs by a group's place alone is loaded at once, from within the arrays
  // whatever the groups say
  const auto request = [&](int i) { return min(max(p.groups[i], 0), p.a.batch); };
  const int b0 = request(g), b1 = max(request(g + 1), b0), n_requests = b1 - b0;
  const int q0 = starts[b0], q1 = starts[b1], first_q = starts[request(0)], last_q = starts[request(p.n_groups)];
  const int64_t cap = static_cast<int64_t>(M) * G;
  const auto member_of = [&](int b) {            // of the call's
    Member m{};
    m.slot = p.a.slots[b];
    const int s0 = starts[b];
    m.queries = starts[b + 1] - s0;
    m.row0 = (s0 - q0) * p.group;
    m.rows = m.queries * p.group;
    if (m.slot >= 0 && m.slot < h.n_slots)
      m.len = static_cast<int>(min(static_cast<int64_t>(max(h.lengths[m.slot], 0)), cap));
    return m;
  };
  Member mine{};
  if (t < n_requests) mine = member_of(b0 + t);
  // starts or groups that decrease, leave their range or leave requests out: nothing is done
  // (no branch between two loads, which would wait for one another)
  const int q_rows = static_cast<int>(p.a.q_rows);
  int bad = (t == 0) & ((p.groups[0] != 0) | (p.groups[p.n_groups] != p.a.batch));
#pragma unroll 4
  for (int i = t; i <= p.n_groups; i += kPlanThreads) {
    const int x = p.groups[i], y = p.groups[min(i + 1, p.n_groups)];
    bad |= (x < 0) | (y < x);
  }
#pragma unroll 4
  for (int i = t; i <= p.a.batch; i += kPlanThreads) {
    const int x = starts[i], y = starts[min(i + 1, p.a.batch)];
    bad |= (x < 0) | (x > q_rows) | (y < x);
  }
  bad = __syncthreads_or(bad);
  // tiles of a group have places of their own, at least as many as it needs
  const auto place_of = [&](int start, int group) {
    return static_cast<int>(static_cast<int64_t>(start) * p.group >> (p.rows == 16 ? 4 : 3)) + group;
  };
  int first_place = 0, last_place = 0;
  if (!bad) {
    first_place = place_of(first_q, 0);
    last_place = place_of(last_q, p.n_groups);
    Member* members = n_requests <= kHere ? here : p.members + b0;   // of the group
    // ---- the events that every request with rows and events has
    const auto first_seen = [&](const Member& m) {   // of its first row
      return visible(p.a.causal ? m.len - m.queries : m.len - 1, m.len, p.a.window, p.a.sinks);
    };
    for (int b = t; b < n_requests; b += kPlanThreads) {
      const Member m = b == t ? mine : member_of(b0 + b);
      if (m.slot < 0 || m.slot >= h.n_slots) flag(h.err, DLRM_ERRBIT_INDEX_OOB);
      members[b] = m;
      if (m.rows > 0 && m.len > 0) {
        atomicMin(&ref_s, b);
        atomicMin(&len_s, m.len);
        atomicMin(&gap_s, first_seen(m).gap1);
      }
    }
    __syncthreads();
    const int ref = ref_s, pages = ref == INT32_MAX ? 0 : len_s / G;
    if (t == 0) shared_s = pages;
    __syncthreads();
    // ---- shared pages: the first entry that differs, 8 x 32 entries of a request at a time
    const int ref_slot = ref == INT32_MAX ? -1 : members[ref].slot;
    if (pages > 0) {
      const int32_t* mine = h.table + static_cast<int64_t>(ref_slot) * M;
      // (kAtOnce requests' entries are asked for before any is looked at)
      constexpr int kAtOnce = 4, kEach = 8, kWarps = kPlanThreads / kWarp;
      const unsigned pieces = (pages + kEach * kWarp - 1) / (kEach * kWarp);
      const unsigned work = n_requests * pieces;   // (as many as table entries at most)
      for (unsigned w0 = t / kWarp; w0 < work; w0 += kAtOnce * kWarps) {
        int32_t theirs[kAtOnce][kEach], ours[kAtOnce][kEach];
        int first[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const unsigned w = w0 + k * kWarps, b = min(w, work - 1) / pieces;
          const Member m = members[b];
          const int last = w < work && m.rows > 0 && m.len > 0 ? pages : 0;
          first[k] = static_cast<int>(w % pieces) * (kEach * kWarp) + lane;
          const int32_t* row = h.table + static_cast<int64_t>(last ? m.slot : ref_slot) * M;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int j = first[k] + i * kWarp;
            theirs[k][i] = ours[k][i] = 0;
            if (j < last) {
              theirs[k][i] = row[j];
              ours[k][i] = mine[j];
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          int differ = INT32_MAX;
#pragma unroll
          for (int i = kEach - 1; i >= 0; --i) differ = theirs[k][i] != ours[k][i] ? first[k] + i * kWarp : differ;
          differ = __reduce_min_sync(0xffffffffu, differ);
          if (lane == 0 && differ < pages) atomicMin(&shared_s, differ);
        }
      }
    }
    __syncthreads();
    const int shared = shared_s * G;             // events
    // ---- every request's blocks of its own, and how many lie before them
    int before = 0;
    for (int c0 = 0; c0 < n_requests; c0 += kPlanThreads) {
      const int b = c0 + t;
      int n = 0;
      Member m{};
      if (b < n_requests) {
        m = members[b];
        if (m.rows > 0 && m.len > 0) {
          const Visible v = first_seen(m);
          const int low = shared / kBlock;
          m.block0 = max(v.gap1 / kBlock, low);
          m.sinks = v.gap1 > shared ? max((min(v.gap0, m.len) + kBlock - 1) / kBlock - low, 0) : 0;
          if (low + m.sinks >= m.block0) {       // no gap: blocks from `shared` on
            m.sinks = 0;
            m.block0 = low;
          }
          n = blocks_of(m);
        }
      }
      int total;
      m.first = before + scan(n, sums, total);
      before += total;
      if (b < n_requests) {
        p.members[b0 + b] = m;
        members[b] = m;
      }
      __syncthreads();
    }
    // ---- tiles
    const int rows = (q1 - q0) * p.group, tiles = (rows + p.rows - 1) / p.rows;
    const int base = place_of(q0, g), next = place_of(q1, g + 1);
    const int gap1 = gap_s == INT32_MAX ? 0 : gap_s, gap0 = min(p.a.sinks, gap1);
    Tile x{};
    x.q0 = q0;
    x.slot = ref_slot;
    x.own0 = shared / kBlock;
    x.shared0 = min(gap1, shared) / kBlock;
    x.shared_sinks = min((min(gap0, shared) + kBlock - 1) / kBlock, x.shared0);
    if (x.shared_sinks == x.shared0) x.shared_sinks = x.shared0 = 0;
    x.shared_blocks = x.shared_sinks + x.own0 - x.shared0;
    const auto holds = [&](int row, int from) {  // the request of a row, `from` or a later one
      int lo = from, hi = n_requests;            // the last one that begins at or before it
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (members[mid].row0 <= row) lo = mid; else hi = mid;
      }
      return lo;
    };
    for (int i = t; base + i < next; i += kPlanThreads) {
      Tile y = x;
      if (i < tiles) {
        y.row0 = i * p.rows;
        y.rows = min(p.rows, rows - y.row0);
        const int m0 = holds(y.row0, 0), m1 = holds(y.row0 + y.rows - 1, m0);
        y.member0 = b0 + m0;
        y.member1 = b0 + m1;
        y.blocks = y.shared_blocks + members[m1].first + blocks_of(members[m1]) - members[m0].first;
      }
      p.found[base + i] = y;
    }
  }
  // ---- the last CTA: units, and the CTAs' parts
  __threadfence();
  __syncthreads();
  if (t == 0) {
    const unsigned n = atomicInc(reinterpret_cast<unsigned*>(p.arrived), gridDim.x - 1);
    last_s = n == gridDim.x - 1;
  }
  __syncthreads();
  if (!last_s) return;
  __threadfence();
  if (bad && t == 0) flag(h.err, DLRM_ERRBIT_OFFSETS);
  int work = 0, dense = 0;
  const int per = (last_place - first_place + kPlanThreads - 1) / kPlanThreads;
  const int mine0 = min(last_place, first_place + t * per), mine1 = min(last_place, mine0 + per);
  const auto copy_of = [](const Tile* tile) {
    Tile y;
    const int4* from = reinterpret_cast<const int4*>(tile);
    int4* to = reinterpret_cast<int4*>(&y);
#pragma unroll
    for (int w = 0; w < static_cast<int>(sizeof(Tile) / 16); ++w) to[w] = __ldcg(from + w);
    return y;
  };
  const auto tile_at = [&](int i) { return copy_of(&p.found[i]); };
  Tile only{};                                    // the thread's tile, if it is one
  for (int i = mine0; i < mine1; ++i) {
    only = tile_at(i);
    const int chunks = chunks_of(only);
    work += chunks > 0 ? (chunks + kCost) * h.n_heads : 0;
    dense += chunks > 0;
  }
  // the work of a CTA: of all, but kLeast chunks at least where pieces are longer on average
  int total, n_tiles;
  scan(work, sums, total);
  int place = scan(dense, sums, n_tiles);
  const int pieces = n_tiles * h.n_heads;
  const Cuts cuts(max((total + p.grid - 1) / p.grid, max(min(kLeast + kCost, pieces ? total / pieces : 1), 1)));
  work = 0;
  for (int i = mine0; i < mine1; ++i) {
    const int chunks = chunks_of(per == 1 ? only : tile_at(i));
    work += chunks > 0 ? cuts.work(chunks) * h.n_heads : 0;
  }
  int at = scan(work, sums, total);
  const int ctas = cuts.from(total);
  for (int i = mine0; i < mine1; ++i) {
    Tile y = per == 1 ? only : tile_at(i);
    const int chunks = chunks_of(y);
    if (chunks == 0) continue;
    y.first = at;
    p.tiles[place] = y;
    if (place < kTilesHere) tiles_s[place] = y;
    at += cuts.work(chunks) * h.n_heads;
    ++place;
  }
  __syncthreads();
  // a CTA begins with a piece, inside it, or with the next one
  for (int c = t; c <= p.grid; c += kPlanThreads) {
    Cut x{n_tiles, 0, 0, cuts.each, Tile{}};
    if (c < ctas) {
      const int w = c * cuts.each;
      int lo = 0, hi = n_tiles;                   // the last tile that begins at or before it
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if ((mid < kTilesHere ? tiles_s[mid].first : __ldcg(&p.tiles[mid].first)) <= w) lo = mid; else hi = mid;
      }
      x.place = lo;
      x.tile = lo < kTilesHere ? tiles_s[lo] : copy_of(&p.tiles[lo]);
      const int chunks = chunks_of(x.tile), length = cuts.work(chunks);
      x.piece = static_cast<unsigned>(w - x.tile.first) / static_cast<unsigned>(length);
      const int start = x.tile.first + x.piece * length, off = w - start;
      if (chunks > kWhole && off >= kNear && off < length - kNear)
        x.chunk = Cuts::chunk(off, length, chunks);
      else if (chunks > kWhole ? off >= kNear : off >= length / 2)
        ++x.piece;
    }
    p.cuts[c] = x;
  }
}

}  // namespace

cudaError_t launch_plan(const Params& p, cudaStream_t stream) {
  return launch_pdl(prefix_plan_kernel, dim3(p.n_groups), dim3(kPlanThreads), 0, stream, p);
}

}  // namespace prefix

cudaError_t launch_history_prefix_attention(const dlrm_history_t& h, const dlrm_attention_t& a,
                                            const int32_t* groups, int n_groups, cudaStream_t stream) {
  using namespace prefix;
  // Too little to share: history_attention's time over its least, by its pieces (a request's
  // rows of a kv head, 16 at a time, 0.007 us each) and the bytes that all requests together
  // can read (7.5 TB/s, most of them from L2), is not above the plan's time and that of the shared
  // pieces (a group's rows, a tile at a time, 0.0127 us each; how many events they share is not
  // known here). In us, apart against shared, one query a request: 1 user x 4 beams x 400 events
  // of 8 heads over 2 8.1 and 17, 17 x 12 x 430 fp16 18 and 29, 720 beams of five queries and 20
  // events 17 and 31; 36 x 3 x 1500 at head_dim 128 41 and 33, 64 x 16 x 1500 74 and 48.
  // The host knows what the tables have room for, not how long the histories are: in tables with
  // room for 8192 events 16 users x 8 x 1000 take 26 and would take 15 apart, 17 x 12 x 430 fp16 29
  // and 15, one user x 4 x 150 in room for 100,000 21 and 14.
  // bf16 calls of 64 rows a request and more and 4096 in all, which history_attention takes on
  // tcgen05 tiles with weights of 8 bits, are not read apart: here bf16 weights have 11. With 64
  // rows a request that costs little or nothing (apart against shared, head_dim 128: 64 users x 1
  // x 1024 49 and 54, 4 x 8 x 100,000 744 and 658; 64 x 4 x 64 at head_dim 64 19 and 42), with more
  // it does: 256 rows 61 and 148, 1265 and 2522, 23 and 128.
  constexpr double kPlan = 12.0, kPiece = 0.007, kShared = 0.0127, kBytes = 7.5e6;
  const int64_t cap = static_cast<int64_t>(h.max_pages) * h.page_tokens;
  const int64_t seen = a.window > 0 ? std::min<int64_t>(cap, int64_t(a.window) + a.sinks + 2 * kBlock) : cap;
  const int64_t rows = a.q_rows * (a.n_heads / h.n_heads);   // of a kv head
  const double apart = static_cast<double>(a.batch + rows / 16) * h.n_heads;
  const double tiles = static_cast<double>(n_groups + rows / (splits(a.dtype, rows, n_groups) ? 8 : 16)) * h.n_heads;
  if (apart * (kPiece + 2 * h.head_dim / kBytes * seen) <= kPlan + kShared * tiles && !history_tc_takes(h, a))
    return launch_history_attention(h, a, stream, groups, n_groups);
  const HistoryWork w = history_work(h);
  Params p;
  p.h = h;
  p.a = a;
  p.groups = groups;
  p.n_groups = n_groups;
  p.group = a.n_heads / h.n_heads;
  const int64_t four = 4 * dtype_bytes(a.dtype);
  p.vec_q = reinterpret_cast<uintptr_t>(a.q) % four == 0 && a.ld_q % 4 == 0 && a.ld_q_head % 4 == 0;
  p.vec_out = reinterpret_cast<uintptr_t>(a.out) % four == 0 && a.ld_out % 4 == 0 && a.ld_out_head % 4 == 0;
  p.arrived = work_part<int32_t>(h, w.prefix_head);
  p.members = work_part<Member>(h, w.members);
  p.found = work_part<Tile>(h, w.found_tiles);
  p.tiles = work_part<Tile>(h, w.tiles_of);
  p.cuts = work_part<Cut>(h, w.cuts);
  p.counters = work_part<int32_t>(h, w.counters);
  p.partials = work_part<float>(h, w.partials);
  if (h.head_dim == 32) return launch_32(p, stream);
  if (h.head_dim == 64) return launch_64(p, stream);
  return launch_128(p, stream);
}

}  // namespace dlrm
