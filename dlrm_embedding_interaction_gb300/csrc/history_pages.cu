// Pages of event histories: append (quantise), fork, copy, free, trim and
// compact. include/dlrm.h defines the pool and what each call does.
//
// Tables, reference counts and the free stack are read and changed on the
// device, so no call waits for the GPU and all can be captured in a graph.
// A call is a chain of small launches (programmatic dependent launches: each
// starts its set-up while the one before it ends):
//   append     plan (one CTA), write; of few requests every CTA plans for itself
//   fork       plan (one CTA), share and copy; likewise
//   copy       plan (one CTA), rows, copy
//   free/trim  one CTA for few pages; else release, count, push (a CTA a request)
//   reorder    plan (one CTA), take (references and copies), commit
//   compact    count, match, move, rename
// The plan gives every request its place in the free stack by a prefix sum
// over the requests, so page numbers do not depend on timing; freed pages are
// pushed in an order that is likewise a prefix sum over (request, page).
#include "history.cuh"

namespace dlrm {

namespace {

constexpr int kPlanThreads = 1024;

// Words of the scratch's head.
enum { kHeadItems = 0, kHeadTop = 1, kHeadLive = 2, kHeadMoves = 3, kHeadArrived = 4 };

// What the plan knows of one request. item0: its first work item.
struct Request {
  int32_t slot;      // destination, or -1: no effect
  int32_t source;
  int32_t length;    // events before the call (append), or of the source
  int32_t count;     // events to append
  int32_t base;      // pages taken from the stack by earlier requests
  int32_t need;      // pages this one takes
  int32_t item0;
  int32_t items;
};
static_assert(sizeof(Request) == 32, "scratch size of a request");

struct Pool {
  dlrm_history_t h;
  int32_t* head;
  int32_t* mark_slot;
  int32_t* mark_page;
  Request* request;
  int2* items;
  int32_t* stash;
  int32_t* remap;
  int32_t* holes;
  int32_t* movers;
  int32_t* tiles;
  int32_t* mark_keep;
  int32_t* dropped;
};

Pool make_pool(const dlrm_history_t& h) {
  const HistoryWork w = history_work(h);
  Pool p;
  p.h = h;
  p.head = work_part<int32_t>(h, w.head);
  p.mark_slot = work_part<int32_t>(h, w.mark_slot);
  p.mark_page = work_part<int32_t>(h, w.mark_page);
  p.request = work_part<Request>(h, w.request);
  p.items = work_part<int2>(h, w.items);
  p.stash = work_part<int32_t>(h, w.stash);
  p.remap = work_part<int32_t>(h, w.remap);
  p.holes = work_part<int32_t>(h, w.holes);
  p.movers = work_part<int32_t>(h, w.movers);
  p.tiles = work_part<int32_t>(h, w.tiles);
  p.mark_keep = work_part<int32_t>(h, w.mark_keep);
  p.dropped = work_part<int32_t>(h, w.dropped);
  return p;
}

__device__ __forceinline__ int warp_inclusive(int x) {
  const int lane = threadIdx.x % kWarp;
#pragma unroll
  for (int d = 1; d < kWarp; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Exclusive prefix sum over the block; total in every thread. sums: one int
// per warp and one more.
__device__ __forceinline__ int block_exclusive(int x, int* sums, int& total) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int warps = blockDim.x / kWarp;
  const int inc = warp_inclusive(x);
  __syncthreads();
  if (lane == kWarp - 1) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int s = lane < warps ? sums[lane] : 0;
    const int si = warp_inclusive(s);
    if (lane < warps) sums[lane] = si - s;
    if (lane == kWarp - 1) sums[kWarp] = si;
  }
  __syncthreads();
  total = sums[kWarp];
  return sums[warp] + inc - x;
}

// A page of the pool: not one trimmed away, nor what a broken table holds.
__device__ __forceinline__ bool is_page(const dlrm_history_t& h, int page) {
  return page >= 0 && page < h.n_pages;
}

enum PlanOp { kAppend, kFork, kCopy };

// What request b asks for, but for its place among the others; bad: the error
// bits of one that is refused. first: no earlier request writes its slot.
template <int OP>
__device__ __forceinline__ Request request_of(const Pool& p, int s, int d, bool first, const int32_t* starts,
                                              int b, int64_t rows, uint32_t& bad) {
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages;
  Request r{-1, -1, 0, 0, 0, 0, 0, 0};
  if (d < 0 || d >= h.n_slots || s < 0 || s >= h.n_slots) {
    bad = DLRM_ERRBIT_INDEX_OOB;
  } else if (!first) {
    bad = DLRM_ERRBIT_INVALID_ARG;
  } else {
    r.slot = d;
    r.source = s;
    const int64_t cap = static_cast<int64_t>(M) * G;
    r.length = static_cast<int>(min(static_cast<int64_t>(max(h.lengths[s], 0)), cap));
    if (OP == kAppend) {
      const int t0 = starts[b], t1 = starts[b + 1];
      if (t0 < 0 || t1 < t0 || t1 > rows) {
        bad = DLRM_ERRBIT_OFFSETS;
      } else if (r.length + static_cast<int64_t>(t1 - t0) > cap) {
        bad = DLRM_ERRBIT_INVALID_ARG;
      } else {
        r.count = t1 - t0;
        const int old = (r.length + G - 1) / G;
        r.need = static_cast<int>((r.length + static_cast<int64_t>(r.count) + G - 1) / G) - old;
        r.items = r.need + (r.count > 0 && r.length % G != 0 ? 1 : 0);
      }
    } else if (h.lengths[d] != 0) {
      bad = DLRM_ERRBIT_INVALID_ARG;
    } else if (OP == kFork) {
      r.need = r.length % G != 0 ? 1 : 0;
    }
  }
  return r;
}

// One CTA, a thread a request: gives every request its place in the free stack
// and in the list of work items by prefix sums. It reads tables and lengths
// but does not change them (the next launch does), so every request sees the
// pool as it was before the call. Of several requests that write one slot the
// first wins: phase 1 marks the slots.
template <int OP>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Pool p, const int32_t* src,
                                                            const int32_t* dst,
                                                            const int32_t* starts, int batch,
                                                            int64_t rows) {
  __shared__ int sums[kWarp + 1];
  __shared__ int done;
  __shared__ int count_s[OP == kCopy ? kPlanThreads : 1], source_s[OP == kCopy ? kPlanThreads : 1];
  const dlrm_history_t& h = p.h;
  const int lane = threadIdx.x % kWarp;
  const int G = h.page_tokens, M = h.max_pages;
  pdl_wait();
  pdl_trigger();
  const int nfree = min(max(*h.n_free, 0), h.n_pages);
  if (threadIdx.x == 0) done = 0;
  for (int b = threadIdx.x; b < batch; b += kPlanThreads) {
    const int d = dst[b];
    if (d >= 0 && d < h.n_slots) atomicMin(&p.mark_slot[d], b);
  }
  __syncthreads();

  int base = 0, items = 0;
  for (int b0 = 0; b0 < batch; b0 += kPlanThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    Request r{-1, -1, 0, 0, 0, 0, 0, 0};
    uint32_t bad = 0;
    bool marked = false;                          // the mark of its slot is this request's
    if (b < batch) {
      const int d = dst[b], s = OP == kAppend ? d : src[b];
      const bool in = d >= 0 && d < h.n_slots;
      marked = in && __ldcg(&p.mark_slot[d]) == b;
      const bool first = !in || marked;
      r = request_of<OP>(p, s, d, first, starts, b, rows, bad);
    }
    if (bad) {
      flag(h.err, bad);
      r.slot = -1;
      r.need = r.items = 0;
    }
    if (OP == kCopy) {
      // pages that a request copies (a trimmed history misses some), counted by
      // a warp a request
      count_s[threadIdx.x] = r.slot >= 0 ? (r.length + G - 1) / G : 0;
      source_s[threadIdx.x] = r.source;
      __syncthreads();
      for (int i = threadIdx.x / kWarp; i < min(kPlanThreads, batch - b0); i += kPlanThreads / kWarp) {
        int c = 0;
        for (int j = lane; j < count_s[i]; j += kWarp)
          c += is_page(h, h.table[static_cast<int64_t>(source_s[i]) * M + j]) ? 1 : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) count_s[i] = c;
      }
      __syncthreads();
      if (b < batch) r.need = r.items = count_s[threadIdx.x];
    }
    int total;
    r.base = base + block_exclusive(r.need, sums, total);
    // saturates: past nfree every later request that needs a page fails
    base = min(base + total, h.n_pages + 1);
    if (r.need > 0) {
      if (r.base + static_cast<int64_t>(r.need) > nfree) {
        flag(h.err, DLRM_ERRBIT_OOM);
        r.slot = -1;
        r.items = 0;
      } else {
        atomicMax(&done, r.base + r.need);
      }
    }
    if (OP != kFork) {
      r.item0 = items + block_exclusive(r.items, sums, total);
      items += total;
    }
    if (b < batch) {
      p.request[b] = r;
      // every reading of a mark lies before the barriers of the sum: the next call finds
      // none, whatever became of this request
      if (marked) p.mark_slot[dst[b]] = INT32_MAX;
    }
    if (OP == kAppend) {
      // work items (request, page of the history); long lists by the whole warp
      if (r.items <= 2) {
        for (int i = 0; i < r.items; ++i) p.items[r.item0 + i] = make_int2(b, r.length / G + i);
      }
      for (unsigned many = __ballot_sync(0xffffffffu, r.items > 2); many; many &= many - 1) {
        const int l = __ffs(many) - 1;
        const int n = __shfl_sync(0xffffffffu, r.items, l), at = __shfl_sync(0xffffffffu, r.item0, l);
        const int first = __shfl_sync(0xffffffffu, r.length / G, l);
        const int of = __shfl_sync(0xffffffffu, b, l);
        for (int i = lane; i < n; i += kWarp) p.items[at + i] = make_int2(of, first + i);
      }
    }
    __syncthreads();                              // `sums` before the next requests
  }
  if (threadIdx.x == 0) {
    p.head[kHeadItems] = items;
    p.head[kHeadTop] = nfree;
    *h.n_free = nfree - done;
  }
}

// The plan of a call of at most kSmallBatch requests, which every CTA of the next
// launch makes for itself instead: that launch is then the only one (one event for
// each of 32 users, forked, appended and freed: 19.1 us against 21.0). Lengths and the
// free stack's height change once every CTA has read them, in the CTA that is last to.
// (More requests: an earlier request for the same slot is found by comparison with
// each, and every CTA's plan takes longer than the launch.)
constexpr int kSmallBatch = 128;
struct SmallPlan {
  Request request[kSmallBatch];
  int4 slots[kSmallBatch / 4];
  int sums[kWarp + 1];
  int items, top, done;
};
// Returns the CTA's ticket, known to thread 0 alone and not before it asks for it:
// commit_small, at the kernel's end, takes it.
template <int OP>
__device__ __forceinline__ unsigned plan_small(const Pool& p, const int32_t* src, const int32_t* dst,
                                           const int32_t* starts, int batch, int64_t rows, SmallPlan& plan) {
  const dlrm_history_t& h = p.h;
  const int t = threadIdx.x;
  const bool report = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
  const int nfree = min(max(*h.n_free, 0), h.n_pages);
  const int d = t < batch ? dst[t] : -1, s = OP == kAppend || t >= batch ? d : src[t];
  if (t < kSmallBatch) reinterpret_cast<int*>(plan.slots)[t] = d;
  if (t == 0) plan.done = 0;
  __syncthreads();
  Request r{-1, -1, 0, 0, 0, 0, 0, 0};
  uint32_t bad = 0;
  if (t < batch) {
    bool first = true;
    for (int i = 0; i < t; i += 4) {
      const int4 x = plan.slots[i / 4];
      first &= x.x != d && (i + 1 >= t || x.y != d) && (i + 2 >= t || x.z != d) && (i + 3 >= t || x.w != d);
    }
    r = request_of<OP>(p, s, d, first, starts, t, rows, bad);
  }
  if (bad) {
    if (report) flag(h.err, bad);
    r.slot = -1;
    r.need = r.items = 0;
  }
  int total;
  r.base = block_exclusive(r.need, plan.sums, total);
  if (r.need > 0) {
    if (r.base + static_cast<int64_t>(r.need) > nfree) {
      if (report) flag(h.err, DLRM_ERRBIT_OOM);
      r.slot = -1;
      r.items = 0;
    } else {
      atomicMax(&plan.done, r.base + r.need);
    }
  }
  r.item0 = block_exclusive(r.items, plan.sums, total);
  if (t < kSmallBatch) plan.request[t] = r;
  if (t == 0) {
    plan.items = total;
    plan.top = nfree;
  }
  __syncthreads();                                // every thread has read what commit_small changes
  unsigned ticket = 0;
  if (t == 0) {
    __threadfence();
    ticket = atomicInc(reinterpret_cast<unsigned*>(&p.head[kHeadArrived]), gridDim.x * gridDim.y * gridDim.z - 1);
  }
  return ticket;
}
// By the first warp.
__device__ __forceinline__ void commit_small(const Pool& p, int batch, unsigned ticket, const SmallPlan& plan) {
  if (__shfl_sync(0xffffffffu, ticket, 0) != gridDim.x * gridDim.y * gridDim.z - 1) return;
  __threadfence();
  for (int i = threadIdx.x; i < batch; i += kWarp) {
    const Request& r = plan.request[i];
    if (r.slot >= 0) p.h.lengths[r.slot] = r.length + r.count;
  }
  if (threadIdx.x == 0) *p.h.n_free = plan.top - plan.done;
}

// Page number `rank` of request r.
__device__ __forceinline__ int granted(const Pool& p, const Request& r, int top, int rank) {
  return p.h.free_pages[top - 1 - (r.base + rank)];
}

// ------------------------------------------------------------------ copy

constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;                                    // 16-byte loads in flight a thread
constexpr int kCopyPiece = kCopyThreads * kCopyVec * 16;       // bytes

// Copies piece `piece` of the codes of one side of a page, and the scales with
// the first. Pages of H * G * D bytes, a multiple of 1 KB.
__device__ __forceinline__ void copy_piece(const dlrm_history_t& h, int side, int piece, int from,
                                           int to) {
  uint8_t* codes = side ? h.v_codes : h.k_codes;
  const int64_t bytes = static_cast<int64_t>(h.n_heads) * h.page_tokens * h.head_dim;
  const uint4* s = reinterpret_cast<const uint4*>(codes + from * bytes);
  uint4* d = reinterpret_cast<uint4*>(codes + to * bytes);
  const int n = static_cast<int>(bytes / 16);
  const int i0 = piece * (kCopyPiece / 16) + threadIdx.x;
  uint4 x[kCopyVec];
#pragma unroll
  for (int i = 0; i < kCopyVec; ++i)
    if (i0 + i * kCopyThreads < n) x[i] = s[i0 + i * kCopyThreads];
#pragma unroll
  for (int i = 0; i < kCopyVec; ++i)
    if (i0 + i * kCopyThreads < n) d[i0 + i * kCopyThreads] = x[i];
  if (piece == 0) {
    float* scales = side ? h.v_scales : h.k_scales;
    for (int i = threadIdx.x; i < h.n_heads; i += kCopyThreads)
      scales[static_cast<int64_t>(to) * h.n_heads + i] =
          scales[static_cast<int64_t>(from) * h.n_heads + i];
  }
}

__host__ __device__ __forceinline__ int pieces_of(const dlrm_history_t& h) {
  const int64_t bytes = static_cast<int64_t>(h.n_heads) * h.page_tokens * h.head_dim;
  return static_cast<int>((bytes + kCopyPiece - 1) / kCopyPiece);
}

// A fork's table row, by the CTAs (request, piece), pieces along y, and along z where a
// grid's y ends: full pages are shared, and piece by piece the last page that is not full
// is copied. Piece 0 writes the row.
__device__ __forceinline__ void fork_one(const Pool& p, const Request& r, int top, int pieces, bool lengths) {
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages;
  const int32_t* from = h.table + static_cast<int64_t>(r.source) * M;
  const int full = r.length / G;
  const int last = r.need > 0 ? from[full] : -1;
  const int page = r.need > 0 ? granted(p, r, top, 0) : -1;
  const int piece = blockIdx.z * gridDim.y + blockIdx.y;
  if (piece == 0) {
    int32_t* row = h.table + static_cast<int64_t>(r.slot) * M;
    for (int j = threadIdx.x; j < full; j += kCopyThreads) {
      const int old = from[j];
      row[j] = old;
      if (is_page(h, old)) atomicAdd(&h.refs[old], 1);
    }
    if (threadIdx.x == 0) {
      if (r.need > 0) {
        row[full] = page;
        h.refs[page] = 1;
      }
      if (lengths) h.lengths[r.slot] = r.length;
    }
  }
  // (a last page that is not full is never trimmed; a broken table's is not read)
  if (last >= 0 && last < h.n_pages && piece < 2 * pieces)
    copy_piece(h, piece / pieces, piece % pieces, last, page);
}

// dst: the call's requests where no plan came before.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(Pool p, int pieces, const int32_t* src,
                                                            const int32_t* dst) {
  __shared__ SmallPlan plan;
  pdl_wait();
  pdl_trigger();
  unsigned ticket = 0;
  if (dst) ticket = plan_small<kFork>(p, src, dst, nullptr, gridDim.x, 0, plan);
  const Request r = dst ? plan.request[blockIdx.x] : p.request[blockIdx.x];
  if (r.slot >= 0) fork_one(p, r, dst ? plan.top : p.head[kHeadTop], pieces, !dst);
  if (dst && threadIdx.x < kWarp) commit_small(p, gridDim.x, ticket, plan);
}

// A copy's table row, by one CTA a request: the list of pages to copy.
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(Pool p) {
  __shared__ int sums[kWarp + 1];
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages;
  const Request r = p.request[blockIdx.x];
  if (r.slot < 0) return;
  const int32_t* from = h.table + static_cast<int64_t>(r.source) * M;
  int32_t* row = h.table + static_cast<int64_t>(r.slot) * M;
  const int n = (r.length + G - 1) / G, top = p.head[kHeadTop];
  int taken = 0;
  for (int j0 = 0; j0 < n; j0 += kCopyThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    const int old = j < n ? from[j] : -1;
    const bool copied = is_page(h, old);
    int total;
    const int rank = taken + block_exclusive(copied ? 1 : 0, sums, total);
    if (copied) {
      const int page = granted(p, r, top, rank);
      row[j] = page;
      h.refs[page] = 1;
      p.items[r.item0 + rank] = make_int2(old, page);
    }
    taken += total;
  }
  if (threadIdx.x == 0) h.lengths[r.slot] = r.length;
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(Pool p, int pieces) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = static_cast<int64_t>(p.head[kHeadItems]) * 2 * pieces;
  for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
    const int2 item = p.items[w / (2 * pieces)];
    const int rest = static_cast<int>(w % (2 * pieces));
    copy_piece(p.h, rest / pieces, rest % pieces, item.x, item.y);
  }
}

// ------------------------------------------------------------------ append

constexpr int kWriteThreads = 256;   // at most: 128 where that holds a page's rows
constexpr int kHold = 8;             // chunks of eight elements that a thread holds
// CTAs of kWriteThreads that an SM holds, by the registers of the chunks
constexpr int write_ctas(int dtype) { return dtype == DLRM_DTYPE_FP32 ? 2 : 3; }

// Eight consecutive elements, as they are. VEC: at a 16-byte boundary.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(uint32_t* w, const void* x, int64_t at) {
  if (!VEC && DT == DLRM_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __ldg(static_cast<const uint32_t*>(x) + at + i);
  } else if (!VEC) {
    const uint16_t* p = static_cast<const uint16_t*>(x) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(__ldg(p + 2 * i)) | static_cast<uint32_t>(__ldg(p + 2 * i + 1)) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < (DT == DLRM_DTYPE_FP32 ? 2 : 1); ++i) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(
          static_cast<const char*>(x) + at * (DT == DLRM_DTYPE_FP32 ? 4 : 2)) + i);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
}

// Elements 2 i and 2 i + 1 of a chunk as fp32.
template <int DT>
__device__ __forceinline__ float2 pair_of(const uint32_t* w, int i) {
  if (DT == DLRM_DTYPE_FP32)
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  if (DT == DLRM_DTYPE_BF16)
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return f16x2_to_float2(w[i]);
}

// Quantises the new events of one page, head and side per iteration. The scale
// needs the largest magnitude before the first code, so the rows stay in
// registers in between: at most kHold chunks a thread, all under way at once.
// Magnitudes compare as unsigned integers, two 16-bit ones an instruction; only
// where the largest is no number does a second look leave out what is not
// finite. Where the page already holds events and its scale grows, their codes
// are re-rounded: exact but for codes that become subnormal, as scales are
// powers of two. What an item is takes a chain of four loads: the CTA's next
// items are looked up together, a thread each.
// What bounds it: HBM. 16 histories of 2000 to 4096 events, 8 heads of 128, bf16
// (310 MB moved): 52 us under the profiler, 87% of the copy rate; with the free before
// it 62 us (84 with the rows read twice, the second time from L1, and a plan of its own).
template <int DT, int D, bool VEC>
__global__ void __launch_bounds__(kWriteThreads, write_ctas(DT))
append_kernel(Pool p, const int32_t* slots, const int32_t* starts, int batch, int64_t rows,
              const void* k, int64_t ld_k, int64_t ld_k_head, const void* v, int64_t ld_v,
              int64_t ld_v_head) {
  __shared__ SmallPlan plan;
  __shared__ uint32_t top[2][kWriteThreads / kWarp];
  __shared__ int4 todo[kWriteThreads];            // page, first and last new event, row of event 0
  constexpr int kChunks = D / 8;                  // of a row
  constexpr int kWords = DT == DLRM_DTYPE_FP32 ? 8 : 4;
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, H = h.n_heads, T = blockDim.x, t = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const bool small = batch <= kSmallBatch;
  unsigned ticket = 0;
  if (small) ticket = plan_small<kAppend>(p, nullptr, slots, starts, batch, rows, plan);
  const int64_t n = static_cast<int64_t>(small ? plan.items : p.head[kHeadItems]) * H * 2;
  int left = 0;                                   // entries of `todo` from `at` on
  int at = 0, turn = 0;                           // `top` by turns: one barrier an item
  for (int64_t w = blockIdx.x; w < n; w += gridDim.x, ++at, --left) {
    if (left == 0) {
      left = T;
      at = 0;
      const int64_t w_of = w + static_cast<int64_t>(t) * gridDim.x;
      __syncthreads();                            // `todo` is read
      if (w_of < n) {
        const int which = static_cast<int>(w_of / (2 * H));
        int2 item;                                // request, page of the history
        Request r;
        if (small) {
          int b = 0;                              // the last one whose items begin at or before it
          for (int i = kSmallBatch / 2; i > 0; i /= 2)
            if (b + i < batch && plan.request[b + i].item0 <= which) b += i;
          r = plan.request[b];
          item = make_int2(b, r.length / G + which - r.item0);
        } else {
          item = p.items[which];
          r = p.request[item.x];
        }
        // the page there already, or one that the plan granted; one of the item's
        // workers writes it down, one of the last item's the new length
        int32_t* entry = h.table + static_cast<int64_t>(r.slot) * h.max_pages + item.y;
        const int had = (r.length + G - 1) / G;
        const bool fresh = item.y >= had;
        int page = fresh ? granted(p, r, small ? plan.top : p.head[kHeadTop], item.y - had) : *entry;
        if (page < 0 || page >= h.n_pages) {      // a broken table: a last page that is not full is never trimmed
          flag(h.err, DLRM_ERRBIT_INDEX_OOB);
          page = -1;
        }
        if (w_of == static_cast<int64_t>(which) * 2 * H) {
          if (fresh && page >= 0) {
            *entry = page;
            h.refs[page] = 1;
          }
          if (!small && which + 1 == r.item0 + r.items) h.lengths[r.slot] = r.length + r.count;
        }
        const int64_t first = static_cast<int64_t>(item.y) * G;   // the page's first event
        todo[t] = make_int4(page, static_cast<int>(max(r.length - first, int64_t(0))),
                            static_cast<int>(min(int64_t(r.length) + r.count - first, int64_t(G))),
                            static_cast<int>(starts[item.x] + first - r.length));
      }
      __syncthreads();
    }
    const int4 item = todo[at];
    const int page = item.x;
    if (page < 0) continue;
    // heads fastest, then sides: neighbouring CTAs read neighbouring rows
    const int rest = static_cast<int>(w % (2 * H));
    const int side = rest >= H ? 1 : 0, head = rest - side * H;
    const void* x = side ? v : k;
    const int64_t ld = side ? ld_v : ld_k;
    const int64_t x0 = item.w * ld + head * (side ? ld_v_head : ld_k_head);
    const int64_t place = static_cast<int64_t>(page) * H + head;
    uint8_t* codes = (side ? h.v_codes : h.k_codes) + place * G * D;
    float* scale = (side ? h.v_scales : h.k_scales) + place;

    const int kept = item.y;                      // events there already
    const float was = kept > 0 ? *scale : 1.f;
    const int e0 = kept * kChunks + t, e1 = item.z * kChunks;
    uint32_t f[kHold][kWords];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int e = e0 + i * T;
      if (e < e1) {
        load8<DT, VEC>(f[i], x, x0 + (e / kChunks) * ld + e % kChunks * 8);
      } else {
#pragma unroll
        for (int j = 0; j < kWords; ++j) f[i][j] = 0;
      }
    }
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < kHold; ++i)
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        big = DT == DLRM_DTYPE_FP32 ? max(big, f[i][j] & 0x7fffffffu) : __vmaxu2(big, f[i][j] & 0x7fff7fffu);
    if (DT != DLRM_DTYPE_FP32) {
      big = max(big >> 16, big & 0xffffu);
      big = DT == DLRM_DTYPE_BF16 ? big << 16 : __float_as_uint(f16x2_to_float2(big).x);
    }
    if (big >= 0x7f800000u) {
      big = 0;
#pragma unroll
      for (int i = 0; i < kHold; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x2 = pair_of<DT>(f[i], j);
          const uint32_t a = __float_as_uint(x2.x) & 0x7fffffffu, b = __float_as_uint(x2.y) & 0x7fffffffu;
          big = a < 0x7f800000u ? max(big, a) : big;
          big = b < 0x7f800000u ? max(big, b) : big;
        }
    }
    big = __reduce_max_sync(0xffffffffu, big);
    if (t % kWarp == 0) top[turn][t / kWarp] = big;
    __syncthreads();
    for (int i = 0; i < T / kWarp; ++i) big = max(big, top[turn][i]);
    turn ^= 1;
    int e_new = scale_exponent(big);
    if (kept > 0) {
      const int e_old = static_cast<int>(__float_as_uint(was) >> 23) - 127;
      e_new = max(e_new, min(max(e_old, -kScaleExpMax), kScaleExpMax));
      if (e_new > e_old) {
        const float g = pow2f(max(e_old - e_new, -126));
        uint32_t* c4 = reinterpret_cast<uint32_t*>(codes);
        for (int i = t; i < kept * D / 4; i += T) {
          const uint32_t c = c4[i];
          const float2 a = f16x2_to_float2(e4m3x2_lo_to_f16x2(c));
          const float2 b = f16x2_to_float2(e4m3x2_hi_to_f16x2(c));
          c4[i] = floats_to_e4m3x2(a.x * g, a.y * g) | (floats_to_e4m3x2(b.x * g, b.y * g) << 16);
        }
      }
    }
    if (t == 0) *scale = pow2f(e_new);
    const float inv = pow2f(-e_new);
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int e = e0 + i * T;
      if (e >= e1) break;
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x2 = pair_of<DT>(f[i], j);
        c[j] = floats_to_e4m3x2(x2.x * inv, x2.y * inv);
      }
      reinterpret_cast<uint2*>(codes)[e] = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
  }
  if (small && t < kWarp) commit_small(p, batch, ticket, plan);
}

// ------------------------------------------------------------------ free, trim

constexpr int kFreeThreads = 256;

// Takes the pages [first, last) of request b's slot out of its table; every
// page loses a reference and remembers the last (request, page) position that
// released it, which is the one that will push it.
__global__ void __launch_bounds__(kFreeThreads) release_kernel(Pool p, const int32_t* slots,
                                                               int window, int sinks) {
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, b = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int slot = slots[b];
  Request r{-1, -1, 0, 0, 0, 0, 0, 0};
  if (b == 0 && threadIdx.x == 0) p.head[kHeadTop] = min(max(*h.n_free, 0), h.n_pages);
  if (slot < 0 || slot >= h.n_slots) {
    if (threadIdx.x == 0) flag(h.err, DLRM_ERRBIT_INDEX_OOB);
  } else {
    bool again = false;                                         // listed before: nothing left
    for (int i = threadIdx.x; i < b; i += kFreeThreads) again |= slots[i] == slot;
    if (!__syncthreads_or(again)) {
      const int64_t len = max(h.lengths[slot], 0);
      r.slot = slot;
      r.count = static_cast<int>(min((len + G - 1) / G, static_cast<int64_t>(M)));
      if (window > 0) {
        r.base = static_cast<int>(min((static_cast<int64_t>(sinks) + G - 1) / G,
                                      static_cast<int64_t>(r.count)));
        r.count = static_cast<int>(max((len - window) / G, static_cast<int64_t>(r.base)));
        if (len < window) r.count = r.base;
      }
    }
  }
  if (threadIdx.x == 0) p.request[b] = r;
  if (r.slot < 0) return;
  int32_t* row = h.table + static_cast<int64_t>(slot) * M;
  for (int j = r.base + threadIdx.x; j < r.count; j += kFreeThreads) {
    int page = row[j];
    if (page < 0 || page >= h.n_pages) {
      page = -1;
    } else {
      atomicSub(&h.refs[page], 1);
      atomicMax(&p.mark_page[page], b * M + j);
    }
    row[j] = -1;
    p.stash[b * M + j] = page;
  }
}

__device__ __forceinline__ bool pushes(const Pool& p, const Request& r, int b, int j, int& page) {
  page = -1;
  if (r.slot < 0 || j >= r.count) return false;
  page = p.stash[b * p.h.max_pages + j];
  if (page < 0) return false;
  if (p.mark_page[page] != b * p.h.max_pages + j) {
    page = -1;
    return false;
  }
  return p.h.refs[page] <= 0;
}

__global__ void __launch_bounds__(kFreeThreads) count_freed_kernel(Pool p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  const Request r = p.request[b];
  int n = 0;
  for (int j0 = r.base; j0 < r.count; j0 += kFreeThreads) {
    int page;
    n += __syncthreads_count(pushes(p, r, b, j0 + static_cast<int>(threadIdx.x), page));
  }
  if (threadIdx.x == 0) p.request[b].items = n;
}

// Position q of the freed pages, counted from the last one down, goes to place
// top + q of the stack.
__global__ void __launch_bounds__(kFreeThreads) push_kernel(Pool p, int batch, int whole) {
  __shared__ int sums[kWarp + 1];
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int b = blockIdx.x;
  int before = 0, after = 0;
  for (int i = threadIdx.x; i < batch; i += kFreeThreads) {
    const int n = p.request[i].items;
    before += i <= b ? n : 0;
    after += i > b ? n : 0;
  }
  int upto, later;
  block_exclusive(before, sums, upto);
  block_exclusive(after, sums, later);
  const Request r = p.request[b];
  const int top = p.head[kHeadTop];
  int left = r.items;                                            // of this request, not pushed yet
  for (int j0 = r.base; j0 < r.count; j0 += kFreeThreads) {
    int page, n;
    const bool push = pushes(p, r, b, j0 + static_cast<int>(threadIdx.x), page);
    const int rank = block_exclusive(push ? 1 : 0, sums, n);
    if (push) {
      const int q = later + left - 1 - rank;
      if (top + q < h.n_pages) h.free_pages[top + q] = page;
      h.refs[page] = 0;
    }
    if (page >= 0) p.mark_page[page] = -1;
    left -= n;
  }
  if (threadIdx.x == 0) {
    if (whole && r.slot >= 0) h.lengths[r.slot] = 0;
    if (b == batch - 1) *h.n_free = min(top + upto, h.n_pages);
  }
}

// release, count and push in one CTA, with barriers for launches and a warp for each
// request. us of a fork and a free, this way against three launches: 32 slots of up
// to 32 pages 10.1 against 11.9, of up to 64 11.9 against 11.7; 16 of up to 64 10.9
// against 11.5. With several requests a warp: 48 slots of up to 16 pages 12.9 against
// 11.7, 256 of up to 3 31.7 against 13.8.
constexpr int kFreeSmallBatch = kWarp, kFreeSmallEntries = 2048;
static_assert(kFreeSmallBatch == kPlanThreads / kWarp, "a warp a request, a lane a request");

__global__ void __launch_bounds__(kPlanThreads) free_small_kernel(Pool p, const int32_t* slots,
                                                                  int batch, int window, int sinks) {
  __shared__ int freed_s[kFreeSmallBatch];
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages;
  const int lane = threadIdx.x % kWarp, b = threadIdx.x / kWarp;
  pdl_wait();
  pdl_trigger();
  const int top = min(max(*h.n_free, 0), h.n_pages);
  int first = 0, last = 0;                        // pages [first, last) of request b's table go
  if (b < batch) {
    const int slot = slots[b];
    const bool in = slot >= 0 && slot < h.n_slots;
    // listed before: nothing left
    const bool again = __any_sync(0xffffffffu, lane < b && slots[lane] == slot);
    if (in && !again) {
      const int64_t len = max(h.lengths[slot], 0);
      last = static_cast<int>(min((len + G - 1) / G, static_cast<int64_t>(M)));
      if (window > 0) {
        first = static_cast<int>(min((static_cast<int64_t>(sinks) + G - 1) / G,
                                     static_cast<int64_t>(last)));
        last = len < window ? first
                            : static_cast<int>(max((len - window) / G, static_cast<int64_t>(first)));
      }
    }
    if (!in && lane == 0) flag(h.err, DLRM_ERRBIT_INDEX_OOB);
    for (int j = first + lane; j < last; j += kWarp) {
      const int64_t at = static_cast<int64_t>(slot) * M + j;
      int page = h.table[at];
      if (page < 0 || page >= h.n_pages) {
        page = -1;
      } else {
        atomicSub(&h.refs[page], 1);
        atomicMax(&p.mark_page[page], b * M + j);
      }
      h.table[at] = -1;
      p.stash[b * M + j] = page;
    }
    __syncwarp();
    if (window == 0 && in && !again && lane == 0) h.lengths[slot] = 0;
  }
  __threadfence_block();
  __syncthreads();
  auto pushed = [&](int j, int& page) {
    page = j < last ? __ldcg(&p.stash[b * M + j]) : -1;
    if (page < 0) return false;
    if (__ldcg(&p.mark_page[page]) != b * M + j) {
      page = -1;
      return false;
    }
    return __ldcg(&h.refs[page]) <= 0;
  };
  int left = 0;
  for (int j0 = first; j0 < last; j0 += kWarp) {
    int page;
    left += __popc(__ballot_sync(0xffffffffu, pushed(j0 + lane, page)));
  }
  if (lane == 0) freed_s[b] = left;
  __syncthreads();
  const int freed = freed_s[lane];                // of request `lane`; none past the batch
  const int later = __reduce_add_sync(0xffffffffu, lane > b ? freed : 0);
  const int all = __reduce_add_sync(0xffffffffu, freed);
  for (int j0 = first; j0 < last; j0 += kWarp) {
    int page;
    const bool push = pushed(j0 + lane, page);
    const unsigned who = __ballot_sync(0xffffffffu, push);
    if (push) {
      const int q = later + left - 1 - __popc(who & ((1u << lane) - 1));
      if (top + q < h.n_pages) h.free_pages[top + q] = page;
      h.refs[page] = 0;
    }
    // only its own position's reader can still ask for this mark
    if (page >= 0) p.mark_page[page] = -1;
    left -= __popc(who);
  }
  if (threadIdx.x == 0) *h.n_free = min(top + all, h.n_pages);
}

// ------------------------------------------------------------------ reorder

// What the plan of a reordering knows of request b, in a Request: slot (-1: no effect),
// source (-1: the slot becomes empty), length of the source, count: events of the slot
// before the call, need: a page to copy the source's last one to, which is number
// `base` of the call's.
//
// A slot's table is read by every request that continues it and written by its own, and
// a page is free when all have counted, so three launches: the plan; references, copies
// and the new tables into scratch; then tables and lengths from there, and one CTA that
// pushes the pages that lost their last reference. Last pages that are not full have one
// holder: those of slots that nobody continues are known to the plan, and are the first
// that copies go to. What bounds it: three launches of dependent loads (835 requests 17 us,
// 135 that are five pages apart 12; their copies and tables would take 1).
// ONE: no more requests than threads, so that each stays in its thread's registers, and
// everything that does not wait for the other requests is loaded before they are asked.
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads) reorder_plan_kernel(Pool p, const int32_t* slots,
                                                                    const int32_t* parents, int batch) {
  __shared__ int sums[kWarp + 1];
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, t = threadIdx.x, T = blockDim.x;
  pdl_wait();
  pdl_trigger();
  const int nfree = min(max(*h.n_free, 0), h.n_pages);
  auto in = [&](int slot) { return slot >= 0 && slot < h.n_slots; };
  struct One {
    Request r;
    int own, part_own, part;                      // its slot; last pages, not full, of its slot and its source
    uint32_t bad;
  };
  auto look = [&](int b) {
    One x{{-1, -1, 0, 0, 0, 0, 0, 0}, -1, -1, -1, 0};
    if (b >= batch) return x;
    x.own = slots[b];
    const int from = parents[b];
    const int named = from >= 0 && from < batch ? slots[from] : -1;
    if (!in(x.own)) {
      x.bad = DLRM_ERRBIT_INDEX_OOB;
      return x;
    }
    const auto length_of = [&](int slot) {
      return static_cast<int>(min(static_cast<int64_t>(max(h.lengths[slot], 0)), static_cast<int64_t>(M) * G));
    };
    const auto part_of = [&](int slot, int length) {
      const int page = length % G != 0 ? h.table[static_cast<int64_t>(slot) * M + length / G] : -1;
      return is_page(h, page) ? page : -1;
    };
    x.r.slot = x.own;
    x.r.source = from == -1 ? -1 : named;
    if (from != -1 && !in(named)) {
      x.bad = DLRM_ERRBIT_INDEX_OOB;              // it keeps its history
      x.r.source = x.own;
    }
    x.r.count = length_of(x.own);
    if (x.r.source >= 0) x.r.length = length_of(x.r.source);
    x.part_own = part_of(x.own, x.r.count);
    if (x.r.source >= 0) x.part = part_of(x.r.source, x.r.length);
    return x;
  };
  One mine = look(t);
  for (int b = t; b < batch; b += T) {
    const int d = ONE ? mine.own : slots[b];
    if (in(d)) atomicMin(&p.mark_slot[d], b);
  }
  __syncthreads();
  // of the requests that continue a slot, its own or else the first one keeps its last page
  for (int b = t; b < batch; b += T) {
    if (!ONE) mine = look(b);
    if (mine.own == mine.r.slot && in(mine.own) && __ldcg(&p.mark_slot[mine.own]) != b) {
      mine.bad = DLRM_ERRBIT_INVALID_ARG;         // a slot that an earlier request has
      mine.r.slot = -1;
    }
    if (mine.bad) flag(h.err, mine.bad);
    if (mine.r.slot >= 0 && mine.r.source >= 0)
      atomicMin(&p.mark_keep[mine.r.source], mine.r.source == mine.r.slot ? -1 : b);
    if (!ONE) p.request[b] = mine.r;
  }
  __syncthreads();
  int copies = 0, given = 0;
  for (int b0 = 0; b0 < batch; b0 += T) {
    const int b = b0 + t;
    if (!ONE) {
      mine = look(b);
      if (b < batch) mine.r = p.request[b];
    }
    Request& r = mine.r;
    bool gives = false;
    if (r.slot >= 0) {
      gives = mine.part_own >= 0 && __ldcg(&p.mark_keep[r.slot]) == INT32_MAX;
      r.need = r.source >= 0 && mine.part >= 0 && __ldcg(&p.mark_keep[r.source]) != (r.source == r.slot ? -1 : b);
    }
    int total;                                    // of both counts, 16 bits each
    const int rank = block_exclusive(r.need | (gives ? 1 << 16 : 0), sums, total);
    static_assert(kPlanThreads < 1 << 15, "16 bits a count");
    r.base = copies + (rank & 0xffff);
    // (as many as pages at most, whatever a broken table says)
    if (gives && given + (rank >> 16) < h.n_pages) p.holes[given + (rank >> 16)] = mine.part_own;
    copies += total & 0xffff;
    given += total >> 16;
    if (!ONE && b < batch) p.request[b] = r;
    __syncthreads();                              // `sums` before the next requests
  }
  given = min(given, h.n_pages);
  const bool short_of = copies - given > nfree;   // then nothing at all is done
  for (int b = t; b < batch; b += T) {
    const int d = ONE ? mine.own : slots[b];
    if (in(d)) {
      p.mark_slot[d] = INT32_MAX;
      p.mark_keep[d] = INT32_MAX;
    }
    Request r = ONE ? mine.r : p.request[b];
    if (short_of) r.slot = -1;
    p.request[b] = r;
  }
  if (t == 0) {
    if (short_of) flag(h.err, DLRM_ERRBIT_OOM);
    p.head[kHeadItems] = given;
    p.head[kHeadTop] = nfree;
    p.head[kHeadMoves] = short_of ? 0 : max(copies - given, 0);   // taken from the stack
  }
}

// By the CTAs (request, piece): piece by piece the copy of a last page; piece 0 counts
// references, and writes down the new table row and, in order, the pages that the old one
// holds no more.
__global__ void __launch_bounds__(kCopyThreads) reorder_take_kernel(Pool p, int pieces) {
  __shared__ int sums[kWarp + 1];
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, b = blockIdx.x;
  const Request r = p.request[b];
  if (r.slot < 0 || r.source == r.slot) return;
  const int piece = blockIdx.z * gridDim.y + blockIdx.y;
  const int given = p.head[kHeadItems], top = p.head[kHeadTop];
  const int32_t* from = h.table + static_cast<int64_t>(max(r.source, 0)) * M;
  const int32_t* old_row = h.table + static_cast<int64_t>(r.slot) * M;
  const int n_new = r.source < 0 ? 0 : (r.length + G - 1) / G, n_old = (r.count + G - 1) / G;
  int page = -1;
  if (r.need) page = r.base < given ? p.holes[r.base] : h.free_pages[top - 1 - (r.base - given)];
  if (piece == 0) {
    int drops = 0;
    for (int j0 = 0; j0 < max(n_old, n_new); j0 += kCopyThreads) {
      const int j = j0 + static_cast<int>(threadIdx.x);
      const int was = j < n_old ? old_row[j] : -1;
      int now = j < n_new ? from[j] : -1;
      if (r.need && j == n_new - 1) now = page;
      if (j < n_new) p.stash[static_cast<int64_t>(b) * M + j] = now;
      const bool drop = was != now && is_page(h, was);
      int total;
      const int rank = drops + block_exclusive(drop ? 1 : 0, sums, total);
      drops += total;
      if (drop) {
        atomicSub(&h.refs[was], 1);
        atomicMax(&p.mark_page[was], b * M + rank);
        p.dropped[static_cast<int64_t>(b) * M + rank] = was;
      }
      if (was != now && is_page(h, now)) atomicAdd(&h.refs[now], 1);
    }
    if (threadIdx.x == 0) p.request[b].items = drops;
  }
  // (r.need: the source's last page is one of the pool's)
  if (r.need && is_page(h, page) && piece < 2 * pieces)
    copy_piece(h, piece / pieces, piece % pieces, from[n_new - 1], page);
}

constexpr int kCommitThreads = 1024;

// CTA 0 pushes freed pages, the last position of the last request first; the others
// write tables, a warp a request.
__global__ void __launch_bounds__(kCommitThreads) reorder_commit_kernel(Pool p, int batch) {
  __shared__ int sums[kWarp + 1];
  __shared__ int before[kCommitThreads];
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int G = h.page_tokens, M = h.max_pages, lane = threadIdx.x % kWarp;
  if (blockIdx.x > 0) {
    const int b = (blockIdx.x - 1) * (kCommitThreads / kWarp) + threadIdx.x / kWarp;
    if (b >= batch) return;
    const Request r = p.request[b];
    if (r.slot < 0 || r.source == r.slot) return;
    const int n_new = r.source < 0 ? 0 : (r.length + G - 1) / G, n_old = (r.count + G - 1) / G;
    int32_t* row = h.table + static_cast<int64_t>(r.slot) * M;
    for (int j = lane; j < max(n_old, n_new); j += kWarp)
      row[j] = j < n_new ? p.stash[static_cast<int64_t>(b) * M + j] : -1;
    if (lane == 0) h.lengths[r.slot] = r.length;
    return;
  }
  const int top = p.head[kHeadTop] - p.head[kHeadMoves];
  // Positions from the last one of the last request down, kCommitThreads at a time: whose they
  // are is found among the counts of as many requests. A page is its last position's to push, and that
  // one's mark to clear: no other position's reader takes it for its own, before or after.
  int pushed = 0;
  for (int e0 = 0; e0 < batch; e0 += kCommitThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    int all;
    const int first = block_exclusive(e < batch ? p.request[batch - 1 - e].items : 0, sums, all);
    __syncthreads();                              // (the one before is read)
    before[threadIdx.x] = first;
    __syncthreads();
    for (int f0 = 0; f0 < all; f0 += kCommitThreads) {
      const int f = f0 + static_cast<int>(threadIdx.x);
      int page = -1;
      bool push = false;
      if (f < all) {
        int k = 0;                                // the last request whose positions begin at or before it
#pragma unroll
        for (int d = kCommitThreads / 2; d > 0; d /= 2)
          if (before[k + d] <= f) k += d;
        const int b = batch - 1 - e0 - k;
        const int end = k + 1 < kCommitThreads ? before[k + 1] : all;
        const int64_t at = static_cast<int64_t>(b) * M + (end - 1 - f);
        page = p.dropped[at];
        if (__ldcg(&p.mark_page[page]) != at) page = -1;
        push = page >= 0 && __ldcg(&h.refs[page]) <= 0;
      }
      int n;
      const int q = top + pushed + block_exclusive(push ? 1 : 0, sums, n);
      if (push) {
        if (q < h.n_pages) h.free_pages[q] = page;
        h.refs[page] = 0;
      }
      if (page >= 0) p.mark_page[page] = -1;
      pushed += n;
    }
  }
  if (threadIdx.x == 0 && batch > 0) *h.n_free = min(top + pushed, h.n_pages);
}

// ------------------------------------------------------------------ compact

constexpr int kTile = 1024;   // pages a CTA looks at

__global__ void __launch_bounds__(kTile) count_live_kernel(Pool p) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * kTile + threadIdx.x;
  const int n = __syncthreads_count(i < p.h.n_pages && p.h.refs[i] > 0);
  if (threadIdx.x == 0) p.tiles[blockIdx.x] = n;
}

// Lists the free pages below n (n pages are live) and the live ones from n on,
// both in ascending order: equally many.
__global__ void __launch_bounds__(kTile) match_kernel(Pool p, int tiles) {
  __shared__ int sums[kWarp + 1];
  pdl_wait();
  pdl_trigger();
  const int P = p.h.n_pages;
  int mine = 0, all = 0;
  for (int t = threadIdx.x; t < tiles; t += kTile) {
    const int n = p.tiles[t];
    all += n;
    mine += t < static_cast<int>(blockIdx.x) ? n : 0;
  }
  int live, before;
  block_exclusive(all, sums, live);
  block_exclusive(mine, sums, before);
  // live pages below n: whole tiles, then the part of n's own tile
  int low = 0;
  for (int t = threadIdx.x; t < live / kTile; t += kTile) low += p.tiles[t];
  const int at = live / kTile * kTile + static_cast<int>(threadIdx.x);
  low += at < live && p.h.refs[at] > 0 ? 1 : 0;
  int kept;
  block_exclusive(low, sums, kept);
  const int i = blockIdx.x * kTile + threadIdx.x;
  const bool is_live = i < P && p.h.refs[i] > 0;
  int total;
  const int rank = before + block_exclusive(is_live ? 1 : 0, sums, total);
  if (i < live && !is_live) p.holes[i - rank] = i;
  if (i >= live && is_live) p.movers[rank - kept] = i;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.head[kHeadLive] = live;
    p.head[kHeadMoves] = live - kept;
  }
}

__global__ void __launch_bounds__(kCopyThreads) move_kernel(Pool p, int pieces) {
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int64_t n = static_cast<int64_t>(p.head[kHeadMoves]) * 2 * pieces;
  for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
    const int m = static_cast<int>(w / (2 * pieces));
    const int rest = static_cast<int>(w % (2 * pieces));
    const int from = p.movers[m], to = p.holes[m];
    copy_piece(h, rest / pieces, rest % pieces, from, to);
    if (rest == 0 && threadIdx.x == 0) {
      h.refs[to] = h.refs[from];
      h.refs[from] = 0;
      p.remap[from] = to;
    }
  }
}

__global__ void __launch_bounds__(256) rename_kernel(Pool p) {
  pdl_wait();
  pdl_trigger();
  const dlrm_history_t& h = p.h;
  const int live = p.head[kHeadLive];
  const int64_t entries = static_cast<int64_t>(h.n_slots) * h.max_pages;
  const int64_t first = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = first; i < entries; i += step) {
    const int page = h.table[i];
    if (page >= live && page < h.n_pages) h.table[i] = p.remap[page];
  }
  for (int64_t i = first; i < h.n_pages - live; i += step)
    h.free_pages[i] = h.n_pages - 1 - static_cast<int>(i);
  if (first == 0) *h.n_free = h.n_pages - live;
}

__global__ void __launch_bounds__(256) reset_kernel(Pool p, int32_t* counters, int n_counters,
                                                    int32_t* prefix_head) {
  const dlrm_history_t& h = p.h;
  const int64_t first = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t entries = static_cast<int64_t>(h.n_slots) * h.max_pages;
  for (int64_t i = first; i < entries; i += step) h.table[i] = -1;
  for (int64_t i = first; i < h.n_pages; i += step) {
    h.refs[i] = 0;
    h.free_pages[i] = h.n_pages - 1 - static_cast<int>(i);
    p.mark_page[i] = -1;
  }
  for (int64_t i = first; i < h.n_slots; i += step) {
    h.lengths[i] = 0;
    p.mark_slot[i] = INT32_MAX;
    p.mark_keep[i] = INT32_MAX;
  }
  for (int64_t i = first; i < n_counters; i += step) counters[i] = 0;
  if (first == 0) {
    *h.n_free = h.n_pages;
    *h.err = 0;
    p.head[kHeadArrived] = 0;
    *prefix_head = 0;
  }
}

unsigned grid_for(int64_t units, int per_sm) {
  return static_cast<unsigned>(std::max<int64_t>(
      1, std::min<int64_t>(units, static_cast<int64_t>(device_sm_count()) * per_sm)));
}

struct WriteArgs {
  const int32_t *slots, *starts;
  int batch;
  int64_t rows;
  const void *k, *v;
  int64_t ld_k, ld_k_head, ld_v, ld_v_head;
  bool vec;
};

template <int DT, int D>
cudaError_t launch_write_vec(const Pool& p, const WriteArgs& a, int64_t units, cudaStream_t stream) {
  // a page's rows of one head fit the registers of 128 or of 256 threads
  static_assert(kWriteThreads * kHold * 8 >= 128 * 128, "a page of 128 events of head_dim 128");
  const int threads = p.h.page_tokens * D <= 128 * kHold * 8 ? 128 : kWriteThreads;
  // all resident at once: a CTA begins by looking up its items, or by planning
  const unsigned grid = grid_for(units, write_ctas(DT) * (kWriteThreads / threads));
  return launch_pdl(a.vec ? append_kernel<DT, D, true> : append_kernel<DT, D, false>, dim3(grid),
                    dim3(threads), 0, stream, p, a.slots, a.starts, a.batch, a.rows, a.k,
                    a.ld_k, a.ld_k_head, a.v, a.ld_v, a.ld_v_head);
}

template <int DT>
cudaError_t launch_write(const Pool& p, const WriteArgs& a, int64_t units, cudaStream_t stream) {
  if (p.h.head_dim == 32) return launch_write_vec<DT, 32>(p, a, units, stream);
  if (p.h.head_dim == 64) return launch_write_vec<DT, 64>(p, a, units, stream);
  return launch_write_vec<DT, 128>(p, a, units, stream);
}

}  // namespace

cudaError_t launch_history_reset(const dlrm_history_t& h, cudaStream_t stream) {
  const int64_t most = std::max<int64_t>(static_cast<int64_t>(h.n_slots) * h.max_pages, h.n_pages);
  const HistoryWork w = history_work(h);
  reset_kernel<<<grid_for((most + 255) / 256, 8), 256, 0, stream>>>(
      make_pool(h), work_part<int32_t>(h, w.counters), kAttnMaxCtas, work_part<int32_t>(h, w.prefix_head));
  return cudaGetLastError();
}

cudaError_t launch_history_append(const dlrm_history_t& h, const int32_t* slots,
                                  const int32_t* starts, int batch, const void* k, int64_t ld_k,
                                  int64_t ld_k_head, const void* v, int64_t ld_v,
                                  int64_t ld_v_head, int64_t rows, int dtype,
                                  cudaStream_t stream) {
  const Pool p = make_pool(h);
  if (batch > kSmallBatch) {
    const cudaError_t e = launch_pdl(plan_kernel<kAppend>, dim3(1), dim3(kPlanThreads), 0, stream, p,
                                     static_cast<const int32_t*>(nullptr), slots, starts, batch, rows);
    if (e != cudaSuccess) return e;
  }
  // n new events touch at most n / G + 2 pages of a history
  const int64_t pages = std::min<int64_t>(rows, rows / h.page_tokens + 2 * int64_t(batch));
  const int64_t units = pages * h.n_heads * 2;
  const int64_t eb = dtype_bytes(dtype);
  auto vec = [&](const void* x, int64_t ld, int64_t ld_head) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld * eb % 16 == 0 && ld_head * eb % 16 == 0;
  };
  const WriteArgs a{slots, starts, batch, rows, k, v, ld_k, ld_k_head, ld_v, ld_v_head,
                    vec(k, ld_k, ld_k_head) && vec(v, ld_v, ld_v_head)};
  if (dtype == DLRM_DTYPE_FP32) return launch_write<DLRM_DTYPE_FP32>(p, a, units, stream);
  if (dtype == DLRM_DTYPE_BF16) return launch_write<DLRM_DTYPE_BF16>(p, a, units, stream);
  return launch_write<DLRM_DTYPE_FP16>(p, a, units, stream);
}

cudaError_t launch_history_fork(const dlrm_history_t& h, const int32_t* src, const int32_t* dst,
                                int batch, bool share, cudaStream_t stream) {
  const Pool p = make_pool(h);
  const int pieces = pieces_of(h);
  const int32_t* none = nullptr;
  // (a grid's y and z end at 65535)
  const unsigned z = (2 * pieces + 65534) / 65535;
  const dim3 grid(batch, (2 * pieces + z - 1) / z, z);
  if (share && batch <= kSmallBatch)
    return launch_pdl(fork_kernel, grid, dim3(kCopyThreads), 0, stream, p, pieces, src, dst);
  cudaError_t e = launch_pdl(share ? plan_kernel<kFork> : plan_kernel<kCopy>, dim3(1),
                             dim3(kPlanThreads), 0, stream, p, src, dst, none, batch, int64_t(0));
  if (e != cudaSuccess) return e;
  if (share)
    return launch_pdl(fork_kernel, grid, dim3(kCopyThreads), 0, stream, p, pieces,
                      none, none);
  e = launch_pdl(copy_rows_kernel, dim3(batch), dim3(kCopyThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  const int64_t pages = std::min<int64_t>(h.n_pages, int64_t(batch) * h.max_pages);
  return launch_pdl(copy_kernel, dim3(grid_for(pages * 2 * pieces, 8)), dim3(kCopyThreads), 0,
                    stream, p, pieces);
}

cudaError_t launch_history_free(const dlrm_history_t& h, const int32_t* slots, int batch,
                                int window, int sinks, cudaStream_t stream) {
  const Pool p = make_pool(h);
  if (batch <= kFreeSmallBatch && int64_t(batch) * h.max_pages <= kFreeSmallEntries)
    return launch_pdl(free_small_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, slots, batch,
                      window, sinks);
  cudaError_t e = launch_pdl(release_kernel, dim3(batch), dim3(kFreeThreads), 0, stream, p, slots,
                             window, sinks);
  if (e != cudaSuccess) return e;
  e = launch_pdl(count_freed_kernel, dim3(batch), dim3(kFreeThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(push_kernel, dim3(batch), dim3(kFreeThreads), 0, stream, p, batch,
                    window > 0 ? 0 : 1);
}

cudaError_t launch_history_reorder(const dlrm_history_t& h, const int32_t* slots, const int32_t* parents,
                                   int batch, cudaStream_t stream) {
  const Pool p = make_pool(h);
  const int threads = batch >= kPlanThreads ? kPlanThreads : (batch + kWarp - 1) / kWarp * kWarp;
  cudaError_t e = launch_pdl(batch <= kPlanThreads ? reorder_plan_kernel<true> : reorder_plan_kernel<false>, dim3(1),
                             dim3(threads), 0, stream, p, slots, parents, batch);
  if (e != cudaSuccess) return e;
  const int pieces = pieces_of(h);
  // (a grid's y and z end at 65535)
  const unsigned z = (2 * pieces + 65534) / 65535;
  e = launch_pdl(reorder_take_kernel, dim3(batch, (2 * pieces + z - 1) / z, z), dim3(kCopyThreads), 0, stream, p,
                 pieces);
  if (e != cudaSuccess) return e;
  constexpr int kPer = kCommitThreads / kWarp;
  return launch_pdl(reorder_commit_kernel, dim3(1 + (batch + kPer - 1) / kPer), dim3(kCommitThreads), 0, stream, p,
                    batch);
}

cudaError_t launch_history_compact(const dlrm_history_t& h, cudaStream_t stream) {
  const Pool p = make_pool(h);
  const int tiles = (h.n_pages + kTile - 1) / kTile;
  cudaError_t e = launch_pdl(count_live_kernel, dim3(tiles), dim3(kTile), 0, stream, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(match_kernel, dim3(tiles), dim3(kTile), 0, stream, p, tiles);
  if (e != cudaSuccess) return e;
  const int pieces = pieces_of(h);
  e = launch_pdl(move_kernel, dim3(grid_for(int64_t(h.n_pages) * pieces, 8)), dim3(kCopyThreads),
                 0, stream, p, pieces);
  if (e != cudaSuccess) return e;
  const int64_t entries = std::max<int64_t>(int64_t(h.n_slots) * h.max_pages, h.n_pages);
  return launch_pdl(rename_kernel, dim3(grid_for((entries + 255) / 256, 8)), dim3(256), 0, stream,
                    p);
}

}  // namespace dlrm
