// pa_weights.cu -- attention weight that each cached position has drawn:
//   w[s][h][p] (+)= sum over the window's queries j that see p and the group's
//                   heads g of exp(scale q_jg . k_p - lse_jg)
// from the log-sum-exp that an attention call over the same queries returned,
// so one pass over K is enough (course README "Build an LLM Inference Engine
// From Scratch", curriculum row "Memory & KV Cache": what a cache keeps).
//
// A warp owns 32 or 64 consecutive positions (two or four blocks) of one KV head
// and all of their queries, so every weight has one writer and the sums have
// one order. S^T = K Q^T on mma.sync m16n8k16: rows are positions, columns eight
// query rows. K tiles arrive in a private ring of stages: bf16 by TMA with the
// 128-byte swizzle for ldmatrix, 8-bit by 1-D bulk copies. There a lane takes
// whole 16-byte pieces of its two rows of codes and of its query column, since
// the contraction does not care in which order it meets the head dimensions: a
// step's two k pairs are neighbouring pairs of a piece. The codes become f16
// (exact), and q enters times the power of two that puts its
// largest element in [2^14, 2^15) (exact: 8 significant bits; elements 2^-28
// below the largest lose bits that the fp32 sum does not hold either).
// Bound: the K stream. 8 contexts of 30,000..32,768 positions, one query: bf16
// 86 us, 6.1 TB/s (0.90 of the measured copy rate); FP8 50 us, 5.7 TB/s (0.83). A
// ragged step (256 sequences, log-uniform 1..4096): 51 us, 5.2 TB/s (0.77); about
// 8 us of a call are its launch, the plan and the first copies' latency.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_weights.cuh"

#include <type_traits>

namespace pa {
namespace {

// blocks of a tile: enough to spread a tile's fixed work (212 instructions a tile
// against some 100 a block), few enough for ten warps' two stages. Ragged bf16
// step: 52 us with two blocks, 62 us with four (six warps); 8 x 32k FP8: 57 us
// with four, 66 us with two.
template <int FMT>
constexpr int kSubOf = FMT == PA_KV_BF16 ? 2 : 4;
constexpr int kQRows = 8;                   // query rows that travel with a tile
// Windows with more query rows a KV head go to the tcgen05 kernel. 16 contexts of
// 1000..8192 positions, 16 / 24 rows: bf16 34 / 70 us here against 34 / 34 us
// there, FP8 27 / 89 us against 42 / 42 us (its codes have to be widened).
constexpr int kWgtTcRows = 16;

// Four one-byte codes as two exact f16 pairs. int8: the byte with its sign bit
// flipped is 128 + x, in the mantissa of a half it is 1024 + 128 + x.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == PA_KV_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
  }
}

template <int FMT>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (FMT == PA_KV_BF16) {
    mma_bf16_16816(d, a, b0, b1);
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

template <int FMT>
constexpr int kTileOf = FMT == PA_KV_BF16 ? kTileBytes : kInt8TileBytes;
// beside a stage of blocks: the tile's earlier weights, and for the first tile
// of a (sequence, KV head) up to kQRows query rows and their log-sum-exps
constexpr int kOffOld = 0;
constexpr int kOffQ = kOffOld + 4 * kBlock * 4;
constexpr int kOffLse = kOffQ + kQRows * kHeadDim * 2;
constexpr int kSide = kOffLse + kQRows * 4;
template <int FMT>
constexpr int kStagesOf = 2;
// warps of a CTA (one an SM), as many as two stages each leave room for; fewer
// when a large batch's plan needs the room
constexpr int kWgtWarps = 10;

// The B fragments of eight query rows (column = lane / 4), the lane's two
// columns' log-sum-exps in log2 units, as a leading part and the rest, and the
// factors that turn their products into log2 scores. A column that is no
// query, or whose query saw nothing, sees no position here.
struct QTile {
  uint32_t b[8][2];
  float l2[2], l2lo[2], scale[2];
  int last[2];  // last position that each of the lane's two columns sees
};

// staged: the rows and log-sum-exps in shared memory (col0 == 0), else null.
template <int FMT>
__device__ __forceinline__ void load_q(const WeightArgs& a, const unsigned char* staged,
                                       int64_t q0, int lq, int c, int h, int col0, int lane,
                                       QTile& t) {
  const int quad = lane & 3, rows = lq * a.G;
  const int col = col0 + (lane >> 2);
  const uint4* p = nullptr;
  if (col < rows)
    p = staged ? reinterpret_cast<const uint4*>(staged + col * (kHeadDim * 2))
               : reinterpret_cast<const uint4*>(
                     a.q + ((q0 + col / a.G) * a.Hq + (int64_t)h * a.G + col % a.G) * kHeadDim);
  float undo = 1.f;  // this lane's column: what its scaling has to be undone by
  if constexpr (FMT == PA_KV_BF16) {
    const uint32_t* pw = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      t.b[s][0] = p ? pw[8 * s + quad] : 0u;
      t.b[s][1] = p ? pw[8 * s + quad + 4] : 0u;
    }
  } else {
    uint4 x[4];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the two pieces of dims 16 (4 (j / 2) + quad) ..
      x[j] = p ? p[2 * (4 * (j >> 1) + quad) + (j & 1)] : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[u])), fabsf(bf_hi(w[u]))));
    }
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
    // 2^(14 - e) for m in [2^e, 2^(e+1)), within the normal range; a row of
    // zeros (or, all of it, below 2^-112) keeps factor 2^126
    const int e = min(max((int)((__float_as_uint(m) >> 23) & 255u) - 127, -112), 127);
    const float mul = __uint_as_float((uint32_t)(14 - e + 127) << 23);
    undo = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f[u]) : "f"(bf_hi(w[u]) * mul), "f"(bf_lo(w[u]) * mul));
      t.b[2 * j][0] = f[0];
      t.b[2 * j][1] = f[1];
      t.b[2 * j + 1][0] = f[2];
      t.b[2 * j + 1][1] = f[3];
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int cc = quad * 2 + e;
    t.scale[e] = a.scale_log2;
    if constexpr (FMT != PA_KV_BF16) t.scale[e] *= __shfl_sync(kFull, undo, cc * 4);
    t.l2[e] = 0.f;
    t.l2lo[e] = 0.f;
    t.last[e] = -1;
    if (col0 + cc < rows) {
      const int tok = (col0 + cc) / a.G;
      const float l =
          staged ? reinterpret_cast<const float*>(staged + kQRows * kHeadDim * 2)[cc]
                 : a.lse[(q0 + tok) * a.Hq + h * a.G + (col0 + cc) % a.G];
      if (l != neg_inf()) {  // a query that saw nothing draws nothing
        t.l2[e] = l * kLog2e;
        // what the product lost, and log2 e's own rounding
        t.l2lo[e] = fmaf(l, kLog2e, -t.l2[e]) + l * 1.925963033500e-8f;
        t.last[e] = c - lq + tok;
      }
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kWgtWarps * 32, 1)
    accumulate_weights_kernel(const __grid_constant__ CUtensorMap tmk, const WeightArgs a) {
  constexpr int kSub = kSubOf<FMT>, kTileKeys = kSub * kBlock;
  constexpr int kStages = kStagesOf<FMT>, kBytes = kTileOf<FMT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // the swizzle pattern needs 1024-byte alignment
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  unsigned char* ring = smem + warp * (kStages * kSub * kBytes);
  unsigned char* side = smem + warps * (kStages * kSub * kBytes) + warp * (kStages * kSide);
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + warps * kStages * (kSub * kBytes + kSide)) +
      warp * kStages;
  int* pm = reinterpret_cast<int*>(smem + warps * kStages * (kSub * kBytes + kSide + 8));
  if (lane == 0) {
    // a stage is full when its K bytes and every lane's weights have landed
    for (int i = 0; i < kStages; ++i) mbar_init(smem_addr(&bars[i]), 33);
    mbar_fence_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int S = a.S, Hkv = a.Hkv;
  PlanSmem P;
  P.pair_off = pm;
  P.seq_pair = P.pair_off + (S + 1);
  P.ctx = P.seq_pair + (S + 1);
  P.qstart = P.ctx + S;
  int* qlen = P.qstart + (S + 1);  // queries of each window (-1: refused)
  PlanInputs in;
  in.context_lens = a.context_lens;
  in.cu_seqlens_q = nullptr;
  in.S = S;
  in.Hkv = Hkv;
  in.max_ctx = (int)min((int64_t)a.max_blocks * kBlock, a.weights_len);
  in.qtile = 1;
  in.causal = 0;
  in.npairs_cap = S;
  in.num_q_rows = S;
  in.key_tile = kTileKeys;
  build_plan(in, P, nullptr);  // ends with a CTA barrier
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    int lq = 1;
    if (a.cu_seqlens_q) {
      const int q0 = a.cu_seqlens_q[s];
      lq = a.cu_seqlens_q[s + 1] - q0;
      P.qstart[s] = q0;
      if (q0 < 0 || lq < 0 || lq > P.ctx[s] || (int64_t)q0 + lq > a.num_q_tokens) {
        if (blockIdx.x == 0) flag_error(PA_DEVERR_QLEN_RANGE);
        lq = -1;
      }
    }
    qlen[s] = lq;
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int W = P.total;
  const int nw = min((int)gridDim.x * warps, W);
  const int w = warp * (int)gridDim.x + (int)blockIdx.x;  // ranges dealt out transposed
  if (w >= nw) return;
  const int R0 = range_start(w, W, nw), R1 = range_start(w + 1, W, nw);
  if (R0 >= R1) return;

  // ---- producer: block ids of eight tiles a window ahead, a bulk copy a block ----
  constexpr int kWin = 32 / kSub;
  TilePos pp = locate(P, S, Hkv, R0);
  int pidx = R0, wbase = R0;
  auto load_phys = [&](int base) -> int {  // lane: block lane % 4 of tile base + lane / 4
    const int idx = base + lane / kSub;
    if (idx >= R1) return 0;
    const TilePos t = locate_from(P, Hkv, pp, idx);
    const int b = t.b * kSub + lane % kSub;
    return b * kBlock < P.ctx[t.s] ? a.block_tables[(size_t)t.s * a.max_blocks + b] : 0;
  };
  const int my_tok = lane / a.G, my_head = lane - my_tok * a.G;  // of query row `lane`
  // of the producer's (sequence, KV head), renewed when it changes
  int p_left = 0, p_rows = 0, p_lq = 0;
  const float* p_w = nullptr;
  auto new_segment = [&]() {
    p_left = P.ctx[pp.s] - pp.b * kTileKeys;  // positions of the tile and beyond
    p_w = a.weights + ((int64_t)pp.s * Hkv + pp.h) * a.weights_len + pp.b * kTileKeys + lane;
    p_lq = qlen[pp.s];
    p_rows = p_lq * a.G;
    if (p_rows > kQRows) p_rows = 0;  // too many to travel with the tile
  };
  new_segment();
  bool p_first = true;  // the next tile brings the query rows
  int phys_cur = load_phys(wbase);
  int phys_next = load_phys(wbase + kWin);
  auto issue = [&](int stage) {
    int phys = __shfl_sync(kFull, phys_cur, (pidx - wbase) * kSub + (lane & (kSub - 1)));
    const uint32_t bar = smem_addr(&bars[stage]);
    if (a.accumulate) {
      const uint32_t dst = smem_addr(side + stage * kSide + kOffOld + lane * 4);
#pragma unroll
      for (int i = 0; i < kTileKeys / 32; ++i)
        if (lane + 32 * i < p_left)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + 128u * i),
                       "l"(p_w + 32 * i)
                       : "memory");
    }
    // the first tile of a (sequence, KV head) brings its few query rows
    uint32_t q_bytes = 0;
    if (p_first && p_rows > 0) {
      q_bytes = (uint32_t)p_rows * kHeadDim * 2;
      if (lane < p_rows)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         smem_addr(side + stage * kSide + kOffLse + lane * 4)),
                     "l"(a.lse + ((int64_t)P.qstart[pp.s] + my_tok) * a.Hq + pp.h * a.G + my_head)
                     : "memory");
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    const int nb = min(kSub, (p_left + kBlock - 1) / kBlock);
    if (lane == 0) {
      fence_proxy_async_smem();  // the stage's earlier reads come before the copies
      mbar_arrive_expect_tx(bar, (uint32_t)(nb * kBytes) + q_bytes);
    }
    __syncwarp();
    if (q_bytes && lane < p_lq)
      bulk_copy_g2s(smem_addr(side + stage * kSide + kOffQ + lane * a.G * kHeadDim * 2),
                    a.q + (((int64_t)P.qstart[pp.s] + lane) * a.Hq + (int64_t)pp.h * a.G) *
                              kHeadDim,
                    (uint32_t)a.G * kHeadDim * 2, bar);
    if (lane < nb) {
      if (phys < 0 || (int64_t)phys >= a.num_blocks) {
        flag_error(PA_DEVERR_BLOCK_RANGE);
        phys = 0;
      }
      const uint32_t d = smem_addr(ring + (stage * kSub + lane) * kBytes);
      if constexpr (FMT == PA_KV_BF16) {
        tma_load_block(d, &tmk, (int)(((int64_t)phys * Hkv + pp.h) * (kBlock / 8)), bar);
      } else {
        bulk_copy_g2s(d, a.k_cache + ((int64_t)phys * Hkv + pp.h) * kBytes, kBytes, bar);
      }
    }
    ++pidx;
    p_first = false;
    if (++pp.b < pp.nt) {
      p_left -= kTileKeys;
      p_w += kTileKeys;
    } else if (pidx < R1) {
      --pp.b;
      advance(P, S, Hkv, pp);
      new_segment();
      p_first = true;
    }
    if (pidx - wbase == kWin) {
      wbase += kWin;
      phys_cur = phys_next;
      phys_next = load_phys(wbase + kWin);
    }
  };
  for (int i = 0; i < kStages && pidx < R1; ++i) issue(i);

  // ---- consumer --------------------------------------------------------------------
  TilePos cp = locate(P, S, Hkv, R0);
  const int quad = lane & 3, r0 = lane >> 2;
  int q0 = 0, lq = 0, c = 0, cols = 0;
  bool write = false, begun = false;
  float* dst = nullptr;  // this lane's two rows of the tile
  QTile qt[2];
  int k = 0;
  for (int idx = R0; idx < R1; ++idx, ++k) {
    const int stage = k % kStages;
    if (!mbar_wait_bounded(smem_addr(&bars[stage]), (uint32_t)(k / kStages) & 1u)) {
      for (int j = k + 1; j < k + kStages && R0 + j < pidx; ++j)
        mbar_wait_bounded(smem_addr(&bars[j % kStages]), (uint32_t)(j / kStages) & 1u);
      return;
    }
    const unsigned char* st = side + stage * kSide;
    const unsigned char* kv = ring + stage * (kSub * kBytes);
    if (!begun) {
      begun = true;
      q0 = P.qstart[cp.s];
      lq = qlen[cp.s];
      c = P.ctx[cp.s];
      cols = lq * a.G;  // negative: refused
      write = quad < kSub && (lq > 0 || (lq == 0 && !a.accumulate));
      dst = a.weights + ((int64_t)cp.s * Hkv + cp.h) * a.weights_len + cp.b * kTileKeys +
            quad * kBlock + r0;
      if (cols > 0)
        load_q<FMT>(a, cols <= kQRows ? st + kOffQ : nullptr, q0, lq, c, cp.h, 0, lane, qt[0]);
      if (cols > 8) load_q<FMT>(a, nullptr, q0, lq, c, cp.h, 8, lane, qt[1]);
    }
    const int key0 = cp.b * kTileKeys;
    float sums[kSub][2];
#pragma unroll
    for (int u = 0; u < kSub; ++u) sums[u][0] = sums[u][1] = 0.f;
    // block u against the columns; blocks past the context give sums that
    // nothing writes, so the blocks need no branch between them
    auto block = [&](int u, auto few) {
      uint32_t f[8][4];
      [[maybe_unused]] float kscale[2] = {1.f, 1.f};
      if constexpr (FMT == PA_KV_BF16) {
        // ldmatrix leaves a step's fragment in four registers in a row (taking
        // whole 16-byte pieces instead costs 32 register moves a block); the
        // 128-byte swizzle keeps its rows in different banks
        const uint32_t blk = smem_addr(kv + u * kBytes);
        const int mi = lane >> 3, row = (mi & 1) * 8 + (lane & 7);
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int ch = 2 * s + (mi >> 1);
          ldsm_x4(blk + (row >> 3) * 2048 + (ch >> 3) * 1024 + (row & 7) * 128 +
                      (((ch & 7) ^ (row & 7)) << 4),
                  f[s][0], f[s][1], f[s][2], f[s][3]);
        }
      } else {
        const unsigned char* blk = kv + u * kBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = r0 + 8 * i;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 y =
                *reinterpret_cast<const uint4*>(blk + row * 128 + j * 64 + quad * 16);
            codes_to_f16<FMT>(y.x, f[4 * j][i], f[4 * j][2 + i]);
            codes_to_f16<FMT>(y.y, f[4 * j + 1][i], f[4 * j + 1][2 + i]);
            codes_to_f16<FMT>(y.z, f[4 * j + 2][i], f[4 * j + 2][2 + i]);
            codes_to_f16<FMT>(y.w, f[4 * j + 3][i], f[4 * j + 3][2 + i]);
          }
          kscale[i] = *reinterpret_cast<const float*>(blk + kBlock * kHeadDim + row * 4);
        }
      }
      const int pos = key0 + u * kBlock + r0;
      auto columns = [&](const QTile& t) {
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 8; s += 2) {
          mma_16816<FMT>(d0, f[s], t.b[s][0], t.b[s][1]);
          mma_16816<FMT>(d1, f[s + 1], t.b[s + 1][0], t.b[s + 1][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float sc = t.scale[e & 1];
          if constexpr (FMT != PA_KV_BF16) sc *= kscale[e >> 1];
          const float z = fmaf(d0[e] + d1[e], sc, -t.l2[e & 1]) - t.l2lo[e & 1];
          // (the exponential of a selected -inf: no branch around it)
          sums[u][e >> 1] += ex2(pos + 8 * (e >> 1) <= t.last[e & 1] ? z : neg_inf());
        }
      };
      columns(qt[0]);
      if constexpr (!few.value) {
        if (cols <= 16) {
          columns(qt[1]);
        } else {
          for (int col0 = 8; col0 < cols; col0 += 8) {
            load_q<FMT>(a, nullptr, q0, lq, c, cp.h, col0, lane, qt[1]);
            columns(qt[1]);
          }
        }
      }
    };
    if (cols > 8) {
#pragma unroll
      for (int u = 0; u < kSub; ++u)
        if (key0 + u * kBlock < c) block(u, std::false_type());
    } else if (cols > 0) {
#pragma unroll
      for (int u = 0; u < kSub; ++u) block(u, std::true_type());
    }
    // the four lanes of a row add their columns; lane quad u of the first kSub
    // writes block u's rows
    float mine[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = sums[u][i];
        x += __shfl_xor_sync(kFull, x, 1);
        x += __shfl_xor_sync(kFull, x, 2);
        if (quad == u) mine[i] = x;
      }
    }
    if (write) {
      const float* old = reinterpret_cast<const float*>(st + kOffOld) + quad * kBlock + r0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = key0 + quad * kBlock + r0 + 8 * i;
        // a window's own rows begin with this call
        if (a.accumulate && at < c - lq) mine[i] += old[8 * i];
        if (at < c) dst[8 * i] = mine[i];
      }
    }
    __syncwarp();
    if (pidx < R1) issue(stage);
    if (++cp.b < cp.nt) {
      dst += kTileKeys;
    } else if (idx + 1 < R1) {
      --cp.b;
      advance(P, S, Hkv, cp);
      begun = false;
    }
  }
}

// Shared memory of a CTA of `warps` warps; the plan has five words a sequence.
template <int FMT>
size_t weights_smem(int S, int warps) {
  return 1024 + (size_t)warps * kStagesOf<FMT> * (kSubOf<FMT> * kTileOf<FMT> + kSide + 8) +
         sizeof(int) * 5 * ((size_t)S + 1);
}

template <int FMT>
int launch_weights(const WeightArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  CUtensorMap tmk = {};
  if (FMT == PA_KV_BF16) {
    if (a.num_blocks * a.Hkv * kBlock > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if (!make_block_map(&tmk, a.k_cache, a.num_blocks * a.Hkv * kBlock)) return PA_ERR_CUDA;
  }
  int warps = kWgtWarps;
  while (warps > 0 && weights_smem<FMT>(a.S, warps) > (size_t)dev.max_smem_optin) --warps;
  if (warps == 0) return PA_ERR_UNSUPPORTED;
  const size_t smem = weights_smem<FMT>(a.S, warps);
  int per_sm = 0;
  if (!kernel_occupancy(reinterpret_cast<const void*>(accumulate_weights_kernel<FMT>), warps * 32,
                        smem, &per_sm) ||
      per_sm <= 0)
    return PA_ERR_CUDA;
  return launch_dependent(accumulate_weights_kernel<FMT>, dim3((unsigned)(dev.num_sms * per_sm)),
                          dim3(warps * 32), smem, st, tmk, a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

unsigned take_error_word_weights(cudaStream_t stream, int* rc) {
  unsigned v = 0, zero = 0;
  if (cudaStreamSynchronize(stream) != cudaSuccess ||
      cudaMemcpyFromSymbol(&v, g_pa_error_word, sizeof v) != cudaSuccess ||
      cudaMemcpyToSymbol(g_pa_error_word, &zero, sizeof zero) != cudaSuccess) {
    *rc = PA_ERR_CUDA;
    return 0;
  }
  return v;
}

}  // namespace pa

using namespace pa;

extern "C" int pa_accumulate_weights(const pa_bf16* q, const void* k_cache, int kv_format,
                                     const float* lse, const int32_t* block_tables,
                                     const int32_t* context_lens, const int32_t* cu_seqlens_q,
                                     int64_t num_q_tokens, int max_q_len, float scale,
                                     int accumulate, float* weights, int64_t weights_len,
                                     const pa_shape* shape, void* stream) {
  pa::NvtxRange nvtx_range("pa_accumulate_weights");
  int rc = check_shape_common(shape);
  if (rc != PA_OK) return rc;
  if (kv_format != PA_KV_BF16 && kv_format != PA_KV_INT8 && kv_format != PA_KV_FP8)
    return PA_ERR_ARG;
  if (num_q_tokens < 0 || num_q_tokens > 0x3fffffff || max_q_len < 0 || weights_len < 0)
    return PA_ERR_ARG;
  if (!cu_seqlens_q && num_q_tokens != shape->num_seqs) return PA_ERR_ARG;
  if (shape->num_seqs == 0) return PA_OK;
  if (!k_cache || !block_tables || !context_lens || !weights ||
      (num_q_tokens > 0 && (!q || !lse)))
    return PA_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(lse, 4) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(weights, 4))
    return PA_ERR_ARG;
  if (!(scale == scale)) return PA_ERR_ARG;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  WeightArgs a;
  a.q = q;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.lse = lse;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_seqlens_q = cu_seqlens_q;
  a.num_q_tokens = num_q_tokens;
  a.accumulate = accumulate ? 1 : 0;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.weights = weights;
  a.weights_len = weights_len;
  a.S = shape->num_seqs;
  a.Hq = shape->num_q_heads;
  a.Hkv = shape->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.max_blocks = shape->max_blocks_per_seq;
  a.num_blocks = shape->num_blocks;
  if (num_q_tokens > 0 && (int64_t)max_q_len * a.G > kWgtTcRows) {
    WeightsTcGeometry g;
    rc = weights_tc_geometry(shape, max_q_len, kv_format, &g);
    if (rc != PA_OK) return rc;
    if (g.enabled) return launch_weights_tc(g, a, kv_format, static_cast<cudaStream_t>(stream));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_format == PA_KV_BF16   ? launch_weights<PA_KV_BF16>(a, dev, st)
         : kv_format == PA_KV_INT8 ? launch_weights<PA_KV_INT8>(a, dev, st)
                                   : launch_weights<PA_KV_FP8>(a, dev, st);
}
