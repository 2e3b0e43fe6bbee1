// The second launch of history_prefix_attention: its kernel and what its plan hands it
// (history_prefix.cu says how both work). One source file for each head_dim makes its
// instances.
#pragma once

#include <atomic>

#include "history_attention.cuh"

namespace dlrm {
namespace prefix {

constexpr int kWhole = 4;                        // chunks of a piece that is never split
constexpr int kLeast = 4;                        // chunks of a CTA at least, where pieces are longer
constexpr int kCost = 3;                         // chunks in whose time a piece is begun and ended
constexpr int kNear = 3;                         // a cut as near as this to a piece's end moves there
static_assert(kWhole >= 2 * kNear - kCost, "a piece that is split has an inside");
constexpr int kWeights = 32;                     // parts whose weights lie in shared memory at once

// What the plan knows of a request with rows, and of the tiles.
struct alignas(16) Member {
  int32_t slot, len, queries;
  int32_t row0, rows;                            // among the group's rows
  int32_t first;                                 // blocks of the group's earlier requests
  int32_t sinks, block0;                         // blocks of its own events: the sinks', then from block0 on
};
static_assert(sizeof(Member) == kPrefixMember, "scratch size of a member");
struct alignas(16) Tile {
  int32_t first, blocks;                         // work before it, as Cuts counts it; its blocks
  int32_t q0, row0, rows;                        // the group's first query row; rows among the group's
  int32_t member0, member1;                      // first and last request with rows in the tile
  int32_t slot;                                  // whose table gives the shared pages
  int32_t shared_sinks, shared0, shared_blocks;  // blocks of shared events: the sinks', then from shared0 on
  int32_t own0;                                  // first block that is not shared
};
static_assert(sizeof(Tile) == kPrefixTile, "scratch size of a tile");

struct alignas(16) Cut {                                     // where a CTA begins
  int32_t place, piece;                          // tile, and which of its pieces (kv heads)
  int32_t chunk;                                 // of the piece
  int32_t each;                                  // work of a CTA
  Tile tile;
};
static_assert(sizeof(Cut) == kPrefixCut, "scratch size of a cut");

// Chunks of a tile, a block a warp; one even where there is nothing to read, which writes zeros.
__device__ __forceinline__ int chunks_of(const Tile& t) {
  return t.rows > 0 ? max((t.blocks + kWarps - 1) / kWarps, 1) : 0;
}
// Cuts the pieces (a tile and kv head) of a call evenly over the CTAs. A piece counts as its
// chunks and kCost more, as it takes time to begin and to end, and, from four CTAs' work on, as a
// whole number of them, so that no CTA has parts of two such pieces. CTA c begins at c `each` of
// the whole, but where that lies within kNear of a piece's ends, or in a piece too short
// to be split, it begins with that piece or with the next.
struct Cuts {
  int each;
  __device__ __forceinline__ explicit Cuts(int each) : each(each) {}
  __device__ __forceinline__ int work(int chunks) const {
    const int n = chunks + kCost;
    return n >= 4 * each ? n / each * each : n;
  }
  // The first CTA that begins at or after `w`.
  __device__ __forceinline__ int from(int w) const { return static_cast<unsigned>(w + each - 1) / static_cast<unsigned>(each); }
  // CTAs [first, first + n) begin inside the piece of `chunks` chunks at `start`.
  __device__ __forceinline__ int inside(int start, int chunks, int& first) const {
    first = from(start + kNear);
    return chunks <= kWhole ? 0 : max(from(start + work(chunks) - kNear) - first, 0);
  }
  // The chunk at which one of them begins that lies `off` behind the start of a piece of
  // `length` in all: its share, and a chunk at least to either side. (In fp32, which keeps the
  // order; the CTAs lie kLeast chunks apart or more.)
  __device__ __forceinline__ static int chunk(int off, int length, int chunks) {
    const int n = static_cast<int>(static_cast<float>(off) / static_cast<float>(length) * static_cast<float>(chunks));
    return min(max(n, 1), chunks - 1);
  }
};

// Blocks of a request's own events.
__device__ __forceinline__ int blocks_of(const Member& m) {
  return m.rows > 0 && m.len > 0 ? m.sinks + max((m.len + kBlock - 1) / kBlock - m.block0, 0) : 0;
}

struct Params {
  dlrm_history_t h;
  dlrm_attention_t a;
  const int32_t* groups;
  int n_groups;
  int group;                                     // query heads of a kv head
  int rows;                                      // of a tile
  int grid;                                      // CTAs of the second launch
  int vec_q, vec_out;                            // four elements can be loaded, stored at once
  int32_t* arrived;                              // CTAs of the plan that are done
  Member* members;
  Tile* found;                                   // tiles, with gaps between the groups
  Tile* tiles;                                   // without
  Cut* cuts;                                     // of each CTA, and the end
  int32_t* counters;
  float* partials;
};

// Whether queries and weights are split (Shape) for so many rows of a kv head: fp32, and 16-bit
// rows that are no more than 8 of a group on average and leave half of an MMA's rows empty, whose
// place the rests take.
inline bool splits(int dtype, int64_t rows, int n_groups) {
  return dtype == DLRM_DTYPE_FP32 || rows <= int64_t(8) * n_groups;
}

cudaError_t launch_plan(const Params& p, cudaStream_t stream);
// By head_dim.
cudaError_t launch_32(Params& p, cudaStream_t stream);
cudaError_t launch_64(Params& p, cudaStream_t stream);
cudaError_t launch_128(Params& p, cudaStream_t stream);

template <int DT>
__device__ __forceinline__ void store_four(void* out, int64_t at, const float (&z)[4]) {
  if (DT == DLRM_DTYPE_FP32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(z[0], z[1], z[2], z[3]);
  else if (DT == DLRM_DTYPE_BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(pack_f16x2(z[0], z[1]), pack_f16x2(z[2], z[3]));
}

// Two fp32 at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// SPLIT: queries and weights as an f16 head and rest, in two MMA rows: fp32 rows, and
// 16-bit ones that are no more than 8, whose other MMA rows would be empty. Without it
// fp16 weights have their rest in a product of its own (an output has 11 bits too).
template <int D, bool SPLIT>
struct Shape {
  static constexpr int kRows = SPLIT ? 8 : 16;    // of a tile
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kBytes = 2 * kBlock * D;   // keys and values of a block
  static constexpr int kStride = D + 4;           // of a row's sums in shared memory
  static constexpr int kPartial = kRows * (D + 2);   // of a part in scratch: sums, maxima, sums of weights
  static constexpr int kRing = kWarps * kStages * kBytes;
  static constexpr int kJoin = (kWarps * kRows * (kStride + 2) + 2 * kWeights * kRows) * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

// Tiles of 16 rows (8 of fp32), a block a warp, whatever the rows of a group: two row tiles a
// warp, which halves the conversions, and warps that share a block, which reads it once for up
// to 64 rows, both took longer (64 users, 1500 events, 13 beams of 4 rows: 44 and 47 us
// against 43; 2 x 50,000 events at head_dim 128, 52 rows: 175 with shared blocks against 145,
// 1.4 times the time of the bytes). Each step of a warp is a chain of waits, so warps that go
// on by themselves are worth more than shorter work; tiles that follow one another find the
// events in L2. What bounds it: long histories, the codes' bytes (698 MB in 117 us, 6.0 TB/s);
// else a block's step of some 2000 cycles (conversions, two products, exponentials; issue slots
// 40% busy) and 11,000 cycles around each piece (64 users, 16 beams of bf16: 39 us).
template <int D, int DT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3)
prefix_attention_kernel(const __grid_constant__ Params p) {
  using Sh = Shape<D, SPLIT>;
  constexpr bool kRest = !SPLIT && DT == DLRM_DTYPE_FP16;
  constexpr int kRows = Sh::kRows, kStages = Sh::kStages, kStride = Sh::kStride, kPartial = Sh::kPartial;
  constexpr int KW = D / 16;                      // key words of a thread and event tile
  constexpr int VW = D / 32;                      // value words of a thread and event
  constexpr int NT = D / 8;                       // n tiles of the output
  constexpr int kR2 = SPLIT ? 1 : 2;              // rows of a thread
  extern __shared__ __align__(128) unsigned char smem[];
  // after the events: sums of each warp and row, then maxima, sums of weights; of parts, weights
  // and sums of weights
  float (*joined)[kRows][kStride] = reinterpret_cast<float (*)[kRows][kStride]>(smem);
  float (*tops)[kRows] = reinterpret_cast<float (*)[kRows]>(&joined[kWarps][0][0]);
  float (*totals)[kRows] = reinterpret_cast<float (*)[kRows]>(&tops[kWarps][0]);
  float (*weight)[kRows] = reinterpret_cast<float (*)[kRows]>(&totals[kWarps][0]);
  float (*weight_sum)[kRows] = reinterpret_cast<float (*)[kRows]>(&weight[kWeights][0]);
  __shared__ float row_top[kRows], row_total[kRows];
  __shared__ int odd[kRows + 1];
  __shared__ int see_end[kRows], see_gap0[kRows], see_gap1[kRows], row_member[kRows];
  __shared__ int64_t row_at[kRows];               // query row, of the call
  __shared__ int row_head[kRows];                 // head of the group
  // requests with rows in the tile: their rows [lo, hi) of it, first block
  __shared__ int n_members, n_arrived;
  __shared__ int clear_end, clear_gap;            // events that every row of the tile sees lie between
  __shared__ int m_lo[kRows], m_hi[kRows], m_first[kRows];
  __shared__ Member m_of[kRows];

  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int g = lane / 4, c = lane % 4;
  const int G = p.h.page_tokens, H = p.h.n_heads, shift = __ffs(G) - 1;   // G: a power of two
  const unsigned group = p.group;
  unsigned char* const ring = smem + warp * kStages * Sh::kBytes;
  // what this thread copies of a block: 16-byte chunks of keys and values, 32 apart
  constexpr int kSide = 2 * D;                    // chunks of a side
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t dst_k = ring_at + key_offset<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t dst_v = ring_at + kBlock * D + value_offset<D>(lane / (D / 16), lane % (D / 16));
  const uint8_t* const src_k = p.h.k_codes + lane * 16;
  const uint8_t* const src_v = p.h.v_codes + lane * 16;
  // those of a thread lie 8 events apart, or a multiple, for which the swizzles of keys and
  // values are alike, or 4, for which that of values changes in one bit
  constexpr uint32_t kFlip = D == 128 ? 64 : 0;
  pdl_wait();
  pdl_trigger();
  const Cut from = p.cuts[blockIdx.x], to = p.cuts[blockIdx.x + 1];
  const Cuts cuts(from.each);
  int place = from.place, head = from.piece, begin = from.chunk;
  Tile s = from.tile;
  bool fresh = true;                              // a tile whose requests are not known yet

  const auto ends = [&] {                         // nothing is left before `to`
    return place > to.place || (place == to.place && (head > to.piece || (head == to.piece && begin >= to.chunk)));
  };
  while (!ends()) {
    if (head == H) {
      ++place;
      head = begin = 0;
      fresh = true;
      if (ends()) break;
      s = p.tiles[place];
    }
    const int chunks = chunks_of(s);
    const int chunk0 = begin, chunk1 = place == to.place && head == to.piece ? to.chunk : chunks;
    const int piece = s.first + head * cuts.work(chunks);   // where it begins, as Cuts counts
    const int kv = head;
    const int rows = s.rows;
    begin = 0;
    ++head;

    // ---- the tile's requests; at the same time the queries and the first shared pages.
    // Everything below is a chain of loads, so what does not hang together starts together
    Member mine{};
    if (fresh && warp == 0 && s.member0 + lane <= s.member1) mine = p.members[s.member0 + lane];
    float x[2][KW][4];
#pragma unroll
    for (int r2 = 0; r2 < 2; ++r2) {
      const int r = SPLIT ? g : g + 8 * r2;
      const int row = s.row0 + min(r, rows - 1);
      const int query = group == 1 ? row : static_cast<unsigned>(row) / group;
      const int64_t q_at = (s.q0 + static_cast<int64_t>(query)) * p.a.ld_q +
                           (kv * p.group + row - query * p.group) * p.a.ld_q_head;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        if (r < rows && !(SPLIT && r2)) {
          load_four<DT>(x[r2][w], p.a.q, q_at + key_element<D>(c, w), p.vec_q);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[r2][w][e] = 0.f;
        }
      }
    }

    // ---- blocks of this warp: n0, n0 + kWarps, ..., shared ones first, then the requests' own;
    // lane l knows block l of the 32 at hand (info) and of the 32 after them (ahead)
    const int n0 = chunk0 * kWarps + warp, n1 = min(chunk1 * kWarps, s.blocks);
    const int count = n0 < n1 ? (n1 - n0 + kWarps - 1) / kWarps : 0;
    struct Info {
      int64_t codes;                              // first byte of the block's codes; -1: nothing to read
      int t0, member;                             // first event; whose own, or -1: shared
      float ks, vs;
    };
    auto open = [&](Info& x, int slot) {
      const int page = p.h.table[static_cast<int64_t>(slot) * p.h.max_pages + (x.t0 >> shift)];
      if (page < 0 || page >= p.h.n_pages) {
        flag(p.h.err, DLRM_ERRBIT_INDEX_OOB);     // trimmed, or a broken table: events that some row needs
      } else {
        const int64_t where = static_cast<int64_t>(page) * H + kv;
        x.codes = (where * G + (x.t0 & (G - 1))) * D;
        x.ks = p.h.k_scales[where];
        x.vs = p.h.v_scales[where];
      }
    };
    auto look_shared = [&](int i) {
      Info x{-1, 0, -1, 0.f, 0.f};
      const int n = n0 + i * kWarps;
      if (i < count && n < s.shared_blocks) {
        x.t0 = (n < s.shared_sinks ? n : n - s.shared_sinks + s.shared0) * kBlock;
        open(x, s.slot);
      }
      return x;
    };
    auto look_own = [&](int i, Info& x) {
      const int n = n0 + i * kWarps - s.shared_blocks;
      if (i < count && n >= 0) {
        int k = 0;                                // the last request whose blocks begin at or before it
        for (int d = n_members; d > 1;) {
          const int half = d / 2;
          if (m_first[k + half] <= n) k += half;
          d -= half;
        }
        const Member& m = m_of[k];
        const int j = n - m_first[k];
        x.member = k;
        x.t0 = (j < m.sinks ? s.own0 + j : j - m.sinks + m.block0) * kBlock;
        open(x, m.slot);
      }
    };
    Info info = look_shared(lane), ahead = look_shared(kWarp + lane);
    if (fresh) {
      __syncthreads();                            // the tile before is done with
      if (warp == 0) {
        int n = 0, first = 0;
        for (int b0 = s.member0; b0 <= s.member1; b0 += kWarp) {
          if (b0 > s.member0) {
            mine = Member{};
            if (b0 + lane <= s.member1) mine = p.members[b0 + lane];
          }
          const bool in = mine.rows > 0;
          const unsigned who = __ballot_sync(0xffffffffu, in);
          const int blocks = blocks_of(mine);
          int inc = blocks;
#pragma unroll
          for (int d = 1; d < kWarp; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
          }
          const int i = n + __popc(who & ((1u << lane) - 1));
          if (in && i < kRows) {                  // (each has a row of the tile)
            m_lo[i] = max(mine.row0 - s.row0, 0);
            m_hi[i] = min(mine.row0 + mine.rows - s.row0, s.rows);
            m_first[i] = first + inc - blocks;
            m_of[i] = mine;
          }
          n += __popc(who);
          first += __shfl_sync(0xffffffffu, inc, kWarp - 1);
        }
        if (lane == 0) {
          n_members = min(n, kRows);
          clear_end = INT32_MAX;
          clear_gap = 0;
        }
      }
      __syncthreads();
    }
    look_own(lane, info);
    look_own(kWarp + lane, ahead);
    int base = 0;                                 // blocks [base, base + 32) are in info
    auto fetch = [&](int i) {
      if (i < count) {
        const int64_t mine_codes = i - base < kWarp ? info.codes : ahead.codes;
        const int64_t codes = __shfl_sync(0xffffffffu, mine_codes, i % kWarp);
        if (codes >= 0) {
          const uint32_t at = (i % kStages) * Sh::kBytes;
#pragma unroll
          for (int y = 0; y < kSide / kWarp; ++y) copy16(dst_k + at + y * kWarp * 16, src_k + codes + y * kWarp * 16);
#pragma unroll
          for (int y = 0; y < kSide / kWarp; ++y)
            copy16((y % 2 ? dst_v ^ kFlip : dst_v) + at + y * kWarp * 16, src_v + codes + y * kWarp * 16);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ---- what each row sees (rows past the last stand for it)
    if (fresh) {
      if (threadIdx.x < kRows) {
        const int r = threadIdx.x, row = min(r, rows - 1), of = s.row0 + row;
        int i = 0;                                // the last request that begins at or before it
        for (int d = n_members; d > 1;) {
          const int half = d / 2;
          if (m_lo[i + half] <= row) i += half;
          d -= half;
        }
        const Member& m = m_of[i];
        const int query = static_cast<unsigned>(of - m.row0) / group;
        const Visible v = visible(p.a.causal ? m.len - m.queries + query : m.len - 1, m.len, p.a.window, p.a.sinks);
        see_end[r] = v.end;
        see_gap0[r] = v.gap0;
        see_gap1[r] = v.gap1;
        atomicMin(&clear_end, v.end);
        atomicMax(&clear_gap, v.gap1);
        row_member[r] = i;
        const int at = static_cast<unsigned>(of) / group;
        row_at[r] = s.q0 + static_cast<int64_t>(at);
        row_head[r] = of - at * p.group;
      }
      __syncthreads();
      fresh = false;
    }

    // ---- fragments of the queries, scaled to f16; a negative softmax scale is
    // theirs, so that the factors of the scores are positive
    uint32_t qa[KW][4];
    float qf[kR2];
#pragma unroll
    for (int r2 = 0; r2 < kR2; ++r2) {
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
    }
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float (&x0)[4] = x[0][w], (&x1)[4] = x[1][w];
      qa[w][0] = pack_f16x2(x0[0], x0[1]);
      qa[w][2] = pack_f16x2(x0[2], x0[3]);
      if (SPLIT) {
        const float2 h0 = f16x2_to_float2(qa[w][0]), h1 = f16x2_to_float2(qa[w][2]);
        qa[w][1] = pack_f16x2((x0[0] - h0.x) * 2048.f, (x0[1] - h0.y) * 2048.f);
        qa[w][3] = pack_f16x2((x0[2] - h1.x) * 2048.f, (x0[3] - h1.y) * 2048.f);
      } else {
        qa[w][1] = pack_f16x2(x1[0], x1[1]);
        qa[w][3] = pack_f16x2(x1[2], x1[3]);
      }
    }

    // ---- events
    float2 o[NT][kR2];
    float top[kR2], sum[kR2];
#pragma unroll
    for (int r2 = 0; r2 < kR2; ++r2) {
      top[r2] = -INFINITY;
      sum[r2] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[nt][r2] = make_float2(0.f, 0.f);
    }
    for (int it = 0; it < count; ++it) {
      if (it - base == kWarp) {
        base += kWarp;
        info = ahead;
        ahead = look_shared(base + kWarp + lane);
        look_own(base + kWarp + lane, ahead);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();                               // block `it` is there, and block it - 1 done with
      fetch(it + kStages - 1);
      const int at = it % kWarp;
      const bool there = __shfl_sync(0xffffffffu, info.codes >= 0, at);
      const int member = __shfl_sync(0xffffffffu, info.member, at);
      const float ks = __shfl_sync(0xffffffffu, info.ks, at);
      const float vs = __shfl_sync(0xffffffffu, info.vs, at);
      const int t0 = __shfl_sync(0xffffffffu, info.t0, at);
      if (!there) continue;
      // whether every row of the tile sees all of the block
      const bool clear = member < 0 && t0 + kBlock <= clear_end && t0 >= clear_gap;
      const unsigned char* kb = ring + (it % kStages) * Sh::kBytes;
      const unsigned char* vb = kb + kBlock * D;

      // S = Q K^T
      float sc[kBlock / 8][4];
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
        for (int w = 0; w < KW; ++w)
          mma_f16_from(sc[j], qa[w], e4m3x2_lo_to_f16x2(kw[w]), e4m3x2_hi_to_f16x2(kw[w]), w > 0);
      }
      if (SPLIT) {
#pragma unroll
        for (int j = 0; j < kBlock / 8; ++j) {
          sc[j][0] = fmaf(sc[j][2], 1.f / 2048.f, sc[j][0]);
          sc[j][1] = fmaf(sc[j][3], 1.f / 2048.f, sc[j][1]);
        }
      }
      if (!clear) {
        // rows of the tile that the block is for
        const int lo = member < 0 ? 0 : m_lo[member], hi = member < 0 ? kRows : m_hi[member];
#pragma unroll
        for (int r2 = 0; r2 < kR2; ++r2) {
          const int r = g + 8 * r2, row = min(r, rows - 1);
          // of the thread's events t0 + 2 c + 8 j (+ 1), those before `some`, but for a gap
          const int some = row >= lo && row < hi ? see_end[r] - t0 - 2 * c : 0;
#pragma unroll
          for (int j = 0; j < kBlock / 8; ++j) {
            if (8 * j >= some) sc[j][2 * r2] = -INFINITY;
            if (8 * j + 1 >= some) sc[j][2 * r2 + 1] = -INFINITY;
          }
          if (p.a.window > 0) {
            const int gap0 = see_gap0[r] - t0 - 2 * c, gap1 = see_gap1[r] - t0 - 2 * c;
#pragma unroll
            for (int j = 0; j < kBlock / 8; ++j) {
              if (8 * j >= gap0 && 8 * j < gap1) sc[j][2 * r2] = -INFINITY;
              if (8 * j + 1 >= gap0 && 8 * j + 1 < gap1) sc[j][2 * r2 + 1] = -INFINITY;
            }
          }
        }
      }
      // weights: exp2 of the scores times the factors, less the running maximum; a thread's
      // rows side by side
      float big[kR2], alpha[kR2], f[kR2], off[kR2];
#pragma unroll
      for (int r2 = 0; r2 < kR2; ++r2) {
        const float x0 = fmaxf(fmaxf(sc[0][2 * r2], sc[0][2 * r2 + 1]), fmaxf(sc[2][2 * r2], sc[2][2 * r2 + 1]));
        const float x1 = fmaxf(fmaxf(sc[1][2 * r2], sc[1][2 * r2 + 1]), fmaxf(sc[3][2 * r2], sc[3][2 * r2 + 1]));
        big[r2] = fmaxf(x0, x1);
      }
#pragma unroll
      for (int y = 1; y <= 2; y *= 2)
#pragma unroll
        for (int r2 = 0; r2 < kR2; ++r2) big[r2] = fmaxf(big[r2], __shfl_xor_sync(0xffffffffu, big[r2], y));
      bool grew = false;
#pragma unroll
      for (int r2 = 0; r2 < kR2; ++r2) {
        // (the factor is not zero, even for a softmax scale of zero: a masked score is -infinity)
        f[r2] = fmaxf(qf[r2] * ks, 1e-37f);
        const float m = fmaxf(top[r2], ceilf(big[r2] * f[r2]));
        const float ref = m == -INFINITY ? 0.f : m;
        off[r2] = kLift - ref;
        alpha[r2] = exp2_approx(top[r2] - ref);
        grew |= m > top[r2];
        top[r2] = m;
      }
#pragma unroll
      for (int r2 = 0; r2 < kR2; ++r2) {
        float2 add = make_float2(0.f, 0.f);
        const float2 f2 = make_float2(f[r2], f[r2]), off2 = make_float2(off[r2], off[r2]);
#pragma unroll
        for (int j = 0; j < kBlock / 8; ++j) {
          const float2 e = fma2(make_float2(sc[j][2 * r2], sc[j][2 * r2 + 1]), f2, off2);
          sc[j][2 * r2] = exp2_approx(e.x);
          sc[j][2 * r2 + 1] = exp2_approx(e.y);
          add = fma2(make_float2(sc[j][2 * r2], sc[j][2 * r2 + 1]), make_float2(1.f, 1.f), add);
        }
        sum[r2] = fmaf(sum[r2], alpha[r2], add.x + add.y);
      }
      // the output's correction, where the maximum of some row grew
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r2 = 0; r2 < kR2; ++r2) {
            o[nt][r2].x *= alpha[r2];
            o[nt][r2].y *= alpha[r2];
          }
      }
      uint32_t pa[kBlock / 16][4], pr[kBlock / 16][4];
#pragma unroll
      for (int kt = 0; kt < kBlock / 16; ++kt) {
        const float (&s0)[4] = sc[2 * kt], (&s1)[4] = sc[2 * kt + 1];
        uint32_t (&a)[4] = pa[kt];
        a[0] = pack_f16x2(s0[0], s0[1]);
        a[2] = pack_f16x2(s1[0], s1[1]);
        if (SPLIT) {
          const float2 h0 = f16x2_to_float2(a[0]), h1 = f16x2_to_float2(a[2]);
          a[1] = pack_f16x2((s0[0] - h0.x) * 2048.f, (s0[1] - h0.y) * 2048.f);
          a[3] = pack_f16x2((s1[0] - h1.x) * 2048.f, (s1[1] - h1.y) * 2048.f);
        } else {
          a[1] = pack_f16x2(s0[2], s0[3]);
          a[3] = pack_f16x2(s1[2], s1[3]);
        }
        if (kRest) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 h = f16x2_to_float2(a[i]);
            const float (&y)[4] = i < 2 ? s0 : s1;
            pr[kt][i] = pack_f16x2((y[2 * (i & 1)] - h.x) * 2048.f, (y[2 * (i & 1) + 1] - h.y) * 2048.f);
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
      const float2 vs2 = make_float2(vs, vs), less = make_float2(1.f / 2048.f, 1.f / 2048.f);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        float acc[4][4], rest[4][4];
#pragma unroll
        for (int kt = 0; kt < kBlock / 16; ++kt) {
          // bytes of a pair of events side by side: n tiles 4w, 4w+1 and 4w+2, 4w+3
          const uint32_t l0 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x5140);
          const uint32_t l1 = __byte_perm(vw[kt][0][w], vw[kt][1][w], 0x7362);
          const uint32_t h0 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x5140);
          const uint32_t h1 = __byte_perm(vw[kt][2][w], vw[kt][3][w], 0x7362);
          const uint32_t b[4][2] = {{e4m3x2_lo_to_f16x2(l0), e4m3x2_lo_to_f16x2(h0)},
                                    {e4m3x2_hi_to_f16x2(l0), e4m3x2_hi_to_f16x2(h0)},
                                    {e4m3x2_lo_to_f16x2(l1), e4m3x2_lo_to_f16x2(h1)},
                                    {e4m3x2_hi_to_f16x2(l1), e4m3x2_hi_to_f16x2(h1)}};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16_from(acc[i], pa[kt], b[i][0], b[i][1], kt > 0);
            if (kRest) mma_f16_from(rest[i], pr[kt], b[i][0], b[i][1], kt > 0);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2* out = o[4 * w + i];
          float2 y0 = make_float2(acc[i][0], acc[i][1]), y1 = make_float2(acc[i][2], acc[i][3]);
          if (SPLIT) {
            y0 = fma2(y1, less, y0);
          } else if (kRest) {
            y0 = fma2(make_float2(rest[i][0], rest[i][1]), less, y0);
            y1 = fma2(make_float2(rest[i][2], rest[i][3]), less, y1);
          }
          out[0] = fma2(vs2, y0, out[0]);
          if (!SPLIT) out[kR2 - 1] = fma2(vs2, y1, out[kR2 - 1]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps
    __syncthreads();                              // every ring is done with: `joined` lies there
#pragma unroll
    for (int r2 = 0; r2 < kR2; ++r2) {
      const int r = g + 8 * r2;
      const float l = quad_sum(sum[r2]);
      float* out = joined[warp][r];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        out[2 * c * (D / 8) + nt] = o[nt][r2].x;
        out[(2 * c + 1) * (D / 8) + nt] = o[nt][r2].y;
      }
      if (c == 0) {
        tops[warp][r] = top[r2];
        totals[warp][r] = l;
      }
    }
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int r = threadIdx.x;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, tops[w][r]);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_approx(tops[w][r] - ref);
        l = fmaf(f, totals[w][r], l);
        tops[w][r] = f;
      }
      row_top[r] = m;
      row_total[r] = l;
      odd[r] = 0;
      if (r == 0) odd[kRows] = 0;
    }
    __syncthreads();
    const bool split = chunk0 > 0 || chunk1 < chunks;
    float* mine_at = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (chunk0 > 0 ? 0 : 1)) * kPartial;
    auto sums_of = [&](int r, int d) {            // four sums of a row, over the warps
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = tops[w][r];
        const float4 z = *reinterpret_cast<const float4*>(&joined[w][r][d]);
        y.x = fmaf(f, z.x, y.x), y.y = fmaf(f, z.y, y.y), y.z = fmaf(f, z.z, y.z), y.w = fmaf(f, z.w, y.w);
      }
      return y;
    };
    // outputs, and which rows need a closer look
    auto finish = [&](int r, int d, const float4& y) {
      const float l = row_total[r];
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // (no weights: zeros)
      const float z[4] = {l == 0.f ? 0.f : y.x * inv, l == 0.f ? 0.f : y.y * inv, l == 0.f ? 0.f : y.z * inv,
                          l == 0.f ? 0.f : y.w * inv};
      const int hq = kv * p.group + row_head[r];
      const int64_t at = row_at[r] * p.a.ld_out + hq * p.a.ld_out_head + d;
      bool fine = l != 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) fine &= finite(z[e]);
      if (p.vec_out) {
        store_four<DT>(p.a.out, at, z);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_element<DT>(p.a.out, at + e, z[e]);
      }
      if (d == 0 && p.a.lse)
        p.a.lse[row_at[r] * p.a.n_heads + hq] = l == 0.f ? -INFINITY : row_top[r] * kLn2 + logf(l * pow2f(-kLift));
      if (!fine) odd[r] = odd[kRows] = l == 0.f ? 2 : 1;   // 2: sees nothing, or has no weights
    };
    constexpr int kQuads = (kRows * D / 4 + kThreads - 1) / kThreads;
    if (!split) {
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        const int of = 4 * (e * kThreads + threadIdx.x), r = of / D, d = of % D;
        if (r < rows) finish(r, d, sums_of(r, d));
      }
    } else {
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        const int of = 4 * (e * kThreads + threadIdx.x), r = of / D, d = of % D;
        if (r < rows) *reinterpret_cast<float4*>(mine_at + of) = sums_of(r, d);
      }
      if (threadIdx.x < rows) {
        mine_at[kRows * D + threadIdx.x] = row_top[threadIdx.x];
        mine_at[kRows * D + kRows + threadIdx.x] = row_total[threadIdx.x];
      }
      // the CTAs that share this piece, one part each: the one that begins it, and those
      // that begin inside
      int inner;
      const int parts = cuts.inside(piece, chunks, inner) + 1;
      const int64_t first = inner - 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int before = atomicAdd(&p.counters[first], 1);
        n_arrived = before;
        if (before == parts - 1) p.counters[first] = 0;
      }
      __syncthreads();
      if (n_arrived != parts - 1) continue;       // (`joined` was read before the barrier)
      __threadfence();
      auto part = [&](int i) { return p.partials + ((first + i) * 2 + (i > 0 ? 0 : 1)) * kPartial; };
      // maximum of each row over the parts, the parts' weights, then the weighted sums,
      // kWeights parts at a time
      float big = -INFINITY, l = 0.f;             // of row threadIdx.x
      auto load_tops = [&](int p0, int n) {
        for (int e = threadIdx.x; e < n * kRows; e += kThreads) {
          const int i = e / kRows, r = e % kRows;
          const float* q = part(p0 + i) + kRows * D;
          weight[i][r] = r < rows ? __ldcg(q + r) : -INFINITY;
          weight_sum[i][r] = r < rows ? __ldcg(q + kRows + r) : 0.f;
        }
        __syncthreads();
      };
      for (int p0 = 0; p0 < parts; p0 += kWeights) {
        const int n = min(kWeights, parts - p0);
        load_tops(p0, n);
        if (threadIdx.x < kRows)
          for (int i = 0; i < n; ++i) big = fmaxf(big, weight[i][threadIdx.x]);
        if (p0 + n < parts) __syncthreads();
      }
      if (threadIdx.x < kRows) row_top[threadIdx.x] = big;
      float4 acc[kQuads];
#pragma unroll
      for (int e = 0; e < kQuads; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p0 = 0; p0 < parts; p0 += kWeights) {
        const int n = min(kWeights, parts - p0);
        __syncthreads();
        if (parts > kWeights) load_tops(p0, n);   // (else they are there)
        if (threadIdx.x < kRows)
          for (int i = 0; i < n; ++i) {
            const float f = big == -INFINITY ? 0.f : exp2_approx(weight[i][threadIdx.x] - big);
            weight[i][threadIdx.x] = f;
            l = fmaf(f, weight_sum[i][threadIdx.x], l);
          }
        __syncthreads();
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const float* q = part(p0 + i);
#pragma unroll
          for (int e = 0; e < kQuads; ++e) {
            const int of = 4 * (e * kThreads + threadIdx.x), r = of / D;
            if (r >= rows) continue;
            const float4 y = __ldcg(reinterpret_cast<const float4*>(q + of));
            const float f = weight[i][r];
            acc[e].x = fmaf(f, y.x, acc[e].x), acc[e].y = fmaf(f, y.y, acc[e].y);
            acc[e].z = fmaf(f, y.z, acc[e].z), acc[e].w = fmaf(f, y.w, acc[e].w);
          }
        }
      }
      if (threadIdx.x < rows) row_total[threadIdx.x] = l;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        const int of = 4 * (e * kThreads + threadIdx.x), r = of / D, d = of % D;
        if (r < rows) finish(r, d, acc[e]);
      }
    }
    __syncthreads();
    if (odd[kRows]) {
      for (int r = 0; r < rows; ++r) {
        const int hq = kv * p.group + row_head[r];
        const Visible v{see_end[r], see_gap0[r], see_gap1[r]};
        if (odd[r] == 1 || (odd[r] == 2 && sees_any(v)))
          careful_row<DT>(p.h, p.a, m_of[row_member[r]].slot, v, kv, row_at[r] * p.a.ld_q + hq * p.a.ld_q_head,
                          row_at[r] * p.a.ld_out + hq * p.a.ld_out_head, row_at[r] * p.a.n_heads + hq,
                          &joined[0][0][0]);
      }
    }
    __syncthreads();                              // `joined` is read: the rings may be filled
  }
}

template <int D, int DT, bool SPLIT>
cudaError_t launch(Params& p, cudaStream_t stream) {
  using Sh = Shape<D, SPLIT>;
  // set once on every device, by a bit each; the CTAs of an SM are the same on every GB300
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  int per_sm = 0;
  if (!bit || !(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prefix_attention_kernel<D, DT, SPLIT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, prefix_attention_kernel<D, DT, SPLIT>,
                                                      kThreads, Sh::kSmem);
    if (e != cudaSuccess) return e;
    per_sm = std::max(1, per_sm);
    resident.store(per_sm, std::memory_order_relaxed);
    done.fetch_or(bit, std::memory_order_acq_rel);
  } else {
    per_sm = resident.load(std::memory_order_relaxed);
  }
  // no more CTAs than counters, than partial results have space, and than pieces of
  // kLeast chunks there can be
  const int64_t events = static_cast<int64_t>(p.h.max_pages) * p.h.page_tokens;
  const int64_t tiles = p.a.q_rows * p.group / Sh::kRows + p.n_groups;
  const int64_t blocks = (tiles * 2 + p.a.batch) * p.h.n_heads * (events / kBlock + 2);
  p.rows = Sh::kRows;
  p.grid = static_cast<int>(std::min<int64_t>(
      {std::max<int64_t>(blocks / (kLeast * kWarps), tiles * p.h.n_heads), static_cast<int64_t>(device_sm_count()) * per_sm,
       int64_t(kAttnMaxCtas), kAttnPartialFloats / (2 * Sh::kPartial)}));
  e = launch_plan(p, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_attention_kernel<D, DT, SPLIT>, dim3(p.grid), dim3(kThreads), Sh::kSmem, stream, p);
}

template <int D, int DT>
cudaError_t launch_rows(Params& p, cudaStream_t stream) {
  if constexpr (DT != DLRM_DTYPE_FP32) {
    if (!splits(DT, p.a.q_rows * p.group, p.n_groups)) return launch<D, DT, false>(p, stream);
  }
  return launch<D, DT, true>(p, stream);
}

template <int D>
cudaError_t launch_d(Params& p, cudaStream_t stream) {
  if (p.a.dtype == DLRM_DTYPE_FP32) return launch_rows<D, DLRM_DTYPE_FP32>(p, stream);
  if (p.a.dtype == DLRM_DTYPE_BF16) return launch_rows<D, DLRM_DTYPE_BF16>(p, stream);
  return launch_rows<D, DLRM_DTYPE_FP16>(p, stream);
}

}  // namespace prefix
}  // namespace dlrm
