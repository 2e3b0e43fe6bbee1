// Causal attention of ragged rows with a sliding window and sinks over plain
// keys and values (include/dlrm.h, window_attention).
//
// A CTA takes a tile of kWarps * 16 rows of one kv head of a request (rows
// are (query, head of the group) pairs), a warp 16 of them; every warp walks
// the blocks of 32 events that its own rows see, with a running maximum and
// sum, and keeps its output in registers. Fragments come straight from global
// memory (the four warps of a CTA read nearly the same events: L1 serves
// them), with the inner dimensions of the MMAs permuted so that loads are of 16
// bytes and the four threads of a row's queries and keys read 64 in a row (each a
// quarter of the row instead: 410 us against 358 at 2 x 4096 events, head_dim 128, whole
// rows at a time).
//   bf16, fp16: m16n8k16 in the input's own type; P is rounded to that type (fp16: 2^15
//     times as large, kLift).
//   fp32: m16n8k8 in tf32, three products per product (head * head, head * rest,
//     rest * head): 22 bits of each factor, the product of the rests left out. Outputs err
//     by 5.2e-7 of the values (norms; 32 users of up to 512 events, window 64), where fp32
//     products and sums err by 2.0e-7: a fourth product or a third part would cost more
//     than it gives a ranking.
// What bounds it: instructions (the splits of three products a product) and reads
// that wait for one another, as most warps walk few blocks. 32 users of up to 512
// events, 4 heads of 32, window 64, fp32: 20 us, four CTAs an SM (five by a register cap
// a fifth more). A block's keys and values loaded together take 28 us. 2 x 4096 events,
// window 512, fp32: 73 us at head_dim 32, 132 at 64, 305 at 128.
#include "window_attention.cuh"

namespace dlrm {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * kWarp;
constexpr int kBlock = 32;
constexpr int kTileRows = kWarps * 16;
// fp32: blocks after which the sums leave the MMA's accumulators. An MMA cuts its sum off
// where it should round, so a sum over 4096 events loses 2^-16 of itself, and one over
// 65,000 2^-11.5. The sums so far wait in shared memory (registers are short; a second set
// of sums in them took 30 us for 26 at head_dim 32) and are added with rounding: no
// accumulator sums more than 15 blocks. (The weights' sum goes with them: small ones are
// added up before they meet a large one.)
constexpr int kFlush = 8;
using Params = WindowParams;

// x as a tf32 head and rest, each rounded to nearest: 22 bits of x in all. (The
// MMA cuts its operands off, which would leave a bias.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& head, uint32_t& rest) {
  const float f = __uint_as_float(x);             // (x may be head)
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(head) : "f"(f));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(rest) : "f"(f - __uint_as_float(head)));
}

// N 32-bit words from a byte address on, 16 bytes at a time if aligned, a group of
// four each STEP bytes.
template <int N, bool HALF, int STEP = 16>
__device__ __forceinline__ void load_row_words(uint32_t* w, const uint8_t* p, bool vec) {
  if (vec && N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p + i * STEP));
      w[4 * i] = x.x;
      w[4 * i + 1] = x.y;
      w[4 * i + 2] = x.z;
      w[4 * i + 3] = x.w;
    }
  } else if (vec && N == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x;
    w[1] = x.y;
  } else if (!HALF) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p + i / 4 * STEP) + i % 4);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint16_t* two = reinterpret_cast<const uint16_t*>(p + i / 4 * STEP) + i % 4 * 2;
      const uint16_t lo = __ldg(two), hi = __ldg(two + 1);
      w[i] = lo | (static_cast<uint32_t>(hi) << 16);
    }
  }
}

// fp32: four CTAs an SM at head_dim 32 (27.4 us with 8 bytes of spills against 26.5: 32
// users, 4 heads, window 64); any number above, where the compiler would spill for a third
// CTA (4096 events, window 512, head_dim 64: 121 us against 84).
template <int D, int DT>
__global__ void __launch_bounds__(kThreads, DT != DLRM_DTYPE_FP32 ? 0 : D == 32 ? 4 : 1)
window_attention_kernel(const Params p) {
  constexpr bool kF32 = DT == DLRM_DTYPE_FP32;
  constexpr int kRaise = DT == DLRM_DTYPE_FP16 ? kLift : 0;   // log2 of the largest weight
  constexpr int EB = kF32 ? 4 : 2;
  constexpr int EW = 4 / EB;                      // elements of a word
  constexpr int KW = D / 4 / EW;                  // words of a thread and row: D/4 elements
  constexpr int VW = D / 8 / EW;
  constexpr int NT = D / 8;
  // Scores of a whole block from kGroup words of every row at a time, so that fp32
  // queries are split once a block (2 x 4096 events, window 512, 4 heads of 128: 305 us
  // against 364, of 64: 132 either way); at head_dim 32 from a whole row at a time, with
  // the queries' rests in registers (47.5 us against 48.5, one user). Unaligned bf16 rows:
  // 64 wide 82 us against 103, 128 wide 284 against 268, so whole rows there.
  constexpr bool kWholeRows = D == 32 || (D == 128 && !kF32);
  constexpr int kTogether = kWholeRows ? 1 : kBlock / 8, kGroup = kWholeRows ? KW : 4;
  __shared__ int64_t scan[40];
  // the thread's sums so far, of values and of weights, and the maxima that they are
  // relative to
  __shared__ float held[kF32 ? NT * 4 + 4 : 1][kThreads];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int g = lane / 4, c = lane % 4;
  const int heads = p.a.n_kv_heads;
  pdl_wait();
  pdl_trigger();
  int b;
  int64_t at, total;
  // CTA (tile, head) with the head fastest
  const int64_t unit = blockIdx.x / heads;
  const int head = blockIdx.x % heads;
  locate<kThreads>(p.a.batch, [&](int i) { return static_cast<int64_t>(window_span(p, i, kTileRows, false).tiles); },
                   unit, scan, b, at, total);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.a.batch; i += kThreads) window_span(p, i, kTileRows, true);
  if (unit >= total) return;
  const WindowSpan s = window_span(p, b, kTileRows, false);
  const int row0 = static_cast<int>(unit - at) * kTileRows + warp * 16;
  if (row0 >= s.rows) return;                     // no barrier follows
  const int last_row = min(row0 + 15, s.rows - 1);

  // queries: fragments of the 16 rows
  uint32_t qw[2][KW];
  Visible vis[2];
  float qf = p.a.scale * kLog2e;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = min(row0 + g + 8 * r, last_row);
    const int i = row / p.group;
    const uint8_t* q = static_cast<const uint8_t*>(p.a.q) +
                       ((s.q0 + static_cast<int64_t>(i)) * p.a.ld_q +
                        (head * p.group + row % p.group) * p.a.ld_q_head) * EB + c * 16;
    load_row_words<KW, !kF32, 64>(qw[r], q, p.vec);
    vis[r] = visible(s.len - s.rows / p.group + i, s.len, p.a.window, p.a.sinks);
  }
  constexpr bool kSplitQ = kF32 && D == 32;
  uint32_t q_rest[2][kSplitQ ? KW : 1];
  if (kSplitQ) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int w = 0; w < KW; ++w) split_tf32(qw[r][w], qw[r][w], q_rest[r][kSplitQ ? w : 0]);
  }
  // the events that any of the warp's rows sees
  const int i0 = row0 / p.group, i1 = last_row / p.group;
  const Visible v0 = visible(s.len - s.rows / p.group + i0, s.len, p.a.window, p.a.sinks);
  const Visible v1 = visible(s.len - s.rows / p.group + i1, s.len, p.a.window, p.a.sinks);

  float o[NT][4];
  float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[nt][i] = 0.f;

  const uint8_t* kp = static_cast<const uint8_t*>(p.a.k) +
                      (s.k0 * p.a.ld_k + head * p.a.ld_k_head) * EB + c * 16;
  const uint8_t* vp = static_cast<const uint8_t*>(p.a.v) +
                      (s.k0 * p.a.ld_v + head * p.a.ld_v_head + g * (D / 8)) * EB;
  const int64_t k_step = p.a.ld_k * EB, v_step = p.a.ld_v * EB;

  bool holds = false;
  // the sums, with those held: to be held, or (last) to stay
  auto gather = [&](bool last) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float f = holds ? exp2_approx(held[NT * 4 + r][threadIdx.x] - (top[r] == -INFINITY ? 0.f : top[r])) : 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 2 * r; i < 2 * r + 2; ++i) {
          float& there = held[nt * 4 + i][threadIdx.x];
          const float x = holds ? fmaf(there, f, o[nt][i]) : o[nt][i];
          if (last) {
            o[nt][i] = x;
          } else {
            there = x;
            o[nt][i] = 0.f;
          }
        }
      float& weights = held[NT * 4 + 2 + r][threadIdx.x];
      sum[r] = holds ? fmaf(weights, f, sum[r]) : sum[r];
      if (!last) {
        weights = sum[r];
        sum[r] = 0.f;
        held[NT * 4 + r][threadIdx.x] = top[r];
      }
    }
    holds = true;
  };
  for (int t0 = 0; t0 < v1.end; t0 += kBlock) {
    // past the sinks of every row and before the window of the first: skip to it
    if (t0 >= v1.gap0 && t0 + kBlock <= v0.gap1) {
      t0 = v0.gap1 / kBlock * kBlock - kBlock;
      continue;
    }
    float sc[kBlock / 8][4];
#pragma unroll
    for (int j0 = 0; j0 < kBlock / 8; j0 += kTogether) {
      const uint8_t* row[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[j0 + j][i] = 0.f;
        // an event past the end stands for the last one; its weight is zero
        row[j] = kp + min(t0 + 8 * (j0 + j) + g, s.len - 1) * k_step;
      }
#pragma unroll
      for (int w0 = 0; w0 < KW; w0 += kGroup) {
        uint32_t kw[kTogether][kGroup];
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          load_row_words<kGroup, !kF32, 64>(kw[j], row[j] + w0 * 16, p.vec);
#pragma unroll
        for (int w = w0; w < w0 + kGroup; w += 2) {
          if (!kF32) {
            const uint32_t a[4] = {qw[0][w], qw[1][w], qw[0][w + 1], qw[1][w + 1]};
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
              if (DT == DLRM_DTYPE_BF16)
                mma_bf16(sc[j0 + j], a, kw[j][w - w0], kw[j][w - w0 + 1]);
              else
                mma_f16(sc[j0 + j], a, kw[j][w - w0], kw[j][w - w0 + 1]);
            }
          } else {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hi[i] = qw[i & 1][w + (i >> 1)];
              if (kSplitQ)
                lo[i] = q_rest[i & 1][kSplitQ ? w + (i >> 1) : 0];
              else
                split_tf32(hi[i], hi[i], lo[i]);
            }
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
              uint32_t h0, h1, l0, l1;
              split_tf32(kw[j][w - w0], h0, l0);
              split_tf32(kw[j][w - w0 + 1], h1, l1);
              mma_tf32(sc[j0 + j], lo, h0, h1);
              mma_tf32(sc[j0 + j], hi, l0, l1);
              mma_tf32(sc[j0 + j], hi, h0, h1);
            }
          }
        }
      }
    }
    const bool whole = t0 + kBlock <= min(vis[0].end, vis[1].end) &&
                       (t0 >= vis[0].gap1 || t0 + kBlock <= vis[0].gap0) &&
                       (t0 >= vis[1].gap1 || t0 + kBlock <= vis[1].gap0);
    float big[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < kBlock / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[j][i] *= qf;
        if (!whole && !sees(vis[i >> 1], t0 + 8 * j + 2 * c + (i & 1))) sc[j][i] = -INFINITY;
        big[i >> 1] = fmaxf(big[i >> 1], sc[j][i]);
      }
    float alpha[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float most = quad_max(big[r]), m = fmaxf(top[r], kRaise ? ceilf(most) : most);
      const float none = m == -INFINITY ? 0.f : m, base = none - kRaise;
      alpha[r] = exp2_approx(top[r] - none);
      top[r] = m;
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        sc[j][2 * r] = exp2_approx(sc[j][2 * r] - base);
        sc[j][2 * r + 1] = exp2_approx(sc[j][2 * r + 1] - base);
        add += sc[j][2 * r] + sc[j][2 * r + 1];
      }
      sum[r] = fmaf(sum[r], alpha[r], add);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nt][i] *= alpha[i >> 1];
    if (!kF32) {
#pragma unroll
      for (int kt = 0; kt < kBlock / 16; ++kt) {
        uint32_t vw[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          load_row_words<VW, true>(vw[i], vp + min(t0 + 16 * kt + 2 * c + (i & 1) + 8 * (i >> 1), s.len - 1) * v_step, p.vec);
        uint32_t pa[4];
        if (DT == DLRM_DTYPE_BF16) {
          pa[0] = pack_bf16(sc[2 * kt][0], sc[2 * kt][1]);
          pa[1] = pack_bf16(sc[2 * kt][2], sc[2 * kt][3]);
          pa[2] = pack_bf16(sc[2 * kt + 1][0], sc[2 * kt + 1][1]);
          pa[3] = pack_bf16(sc[2 * kt + 1][2], sc[2 * kt + 1][3]);
        } else {
          pa[0] = pack_f16x2(sc[2 * kt][0], sc[2 * kt][1]);
          pa[1] = pack_f16x2(sc[2 * kt][2], sc[2 * kt][3]);
          pa[2] = pack_f16x2(sc[2 * kt + 1][0], sc[2 * kt + 1][1]);
          pa[3] = pack_f16x2(sc[2 * kt + 1][2], sc[2 * kt + 1][3]);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          // a pair of events side by side: n tiles 2w and 2w + 1
          const uint32_t l0 = __byte_perm(vw[0][w], vw[1][w], 0x5410);
          const uint32_t l1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
          const uint32_t h0 = __byte_perm(vw[2][w], vw[3][w], 0x5410);
          const uint32_t h1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
          if (DT == DLRM_DTYPE_BF16) {
            mma_bf16(o[2 * w], pa, l0, h0);
            mma_bf16(o[2 * w + 1], pa, l1, h1);
          } else {
            mma_f16(o[2 * w], pa, l0, h0);
            mma_f16(o[2 * w + 1], pa, l1, h1);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        uint32_t vw[2][VW], hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          load_row_words<VW, false>(vw[i], vp + min(t0 + 8 * j + 2 * c + i, s.len - 1) * v_step, p.vec);
        const float pr[4] = {sc[j][0], sc[j][2], sc[j][1], sc[j][3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          split_tf32(__float_as_uint(pr[i]), hi[i], lo[i]);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t h0, h1, l0, l1;
          split_tf32(vw[0][w], h0, l0);
          split_tf32(vw[1][w], h1, l1);
          mma_tf32(o[w], lo, h0, h1);
          mma_tf32(o[w], hi, l0, l1);
          mma_tf32(o[w], hi, h0, h1);
        }
      }
      if ((t0 & ((kFlush - 1) * kBlock)) == (kFlush - 1) * kBlock) gather(false);
    }
  }
  if (kF32 && holds) gather(true);

  uint32_t odd = 0;                               // rows to be done again, by bit
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float l = quad_sum(sum[r]);
    const int row = row0 + g + 8 * r;
    const bool in = row <= last_row;
    const int i = row / p.group, hq = head * p.group + row % p.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at_o = (s.q0 + static_cast<int64_t>(i)) * p.a.ld_out + hq * p.a.ld_out_head;
    bool bad = l == 0.f;                          // no events to see, or no weights: one look more
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = l == 0.f ? 0.f : o[nt][2 * r + e] * inv;
        bad |= !finite(x);
        if (in) store_element<DT>(p.a.out, at_o + (2 * c + e) * (D / 8) + nt, x);
      }
    }
    if (in && c == 0 && p.a.lse)
      p.a.lse[(s.q0 + static_cast<int64_t>(i)) * p.a.n_heads + hq] =
          l == 0.f ? -INFINITY : top[r] * kLn2 + logf(l * pow2f(-kRaise));
    const unsigned who = __ballot_sync(0xffffffffu, bad && in);
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if ((who >> (4 * x)) & 0xfu) odd |= 1u << (x + 8 * r);
  }
  __syncwarp();
  for (; odd; odd &= odd - 1) window_careful_row<D, DT>(p, s, head, row0 + __ffs(odd) - 1);
}

template <int D, int DT>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  const int64_t tiles = p.a.q_rows * p.group / kTileRows + p.a.batch;
  const int64_t grid = tiles * p.a.n_kv_heads;
  return launch_pdl(window_attention_kernel<D, DT>, dim3(static_cast<unsigned>(grid)),
                    dim3(kThreads), 0, stream, p);
}

template <int D>
cudaError_t launch_d(const Params& p, cudaStream_t stream) {
  if (p.a.dtype == DLRM_DTYPE_FP32) return launch<D, DLRM_DTYPE_FP32>(p, stream);
  if (p.a.dtype == DLRM_DTYPE_BF16) return launch<D, DLRM_DTYPE_BF16>(p, stream);
  return launch<D, DLRM_DTYPE_FP16>(p, stream);
}

}  // namespace

cudaError_t launch_window_attention(const dlrm_attention_t& a, cudaStream_t stream) {
  if (window_tc_takes(a)) return launch_window_attention_tc(a, stream);
  Params p;
  p.a = a;
  p.group = a.n_heads / a.n_kv_heads;
  const int64_t eb = dtype_bytes(a.dtype);
  auto vec = [&](const void* x, int64_t ld, int64_t ld_head) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld * eb % 16 == 0 && ld_head * eb % 16 == 0;
  };
  p.vec = vec(a.q, a.ld_q, a.ld_q_head) && vec(a.k, a.ld_k, a.ld_k_head) &&
          vec(a.v, a.ld_v, a.ld_v_head);
  if (a.head_dim == 32) return launch_d<32>(p, stream);
  if (a.head_dim == 64) return launch_d<64>(p, stream);
  return launch_d<128>(p, stream);
}

}  // namespace dlrm
