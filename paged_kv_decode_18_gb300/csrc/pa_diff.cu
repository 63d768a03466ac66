// pa_diff.cu -- differential attention over the paged pool: the difference of
// two softmax maps over values that they share, one query per sequence or short
// windows of them.
//
// Pages: course README "Build an LLM Inference Engine From Scratch", curriculum
// rows "Memory & KV Cache" (PagedAttention, GQA) and "Batching & Scheduling"
// (FlashAttention), and its claim that online softmax is exact and split-K
// variants agree: both maps are softmax maps, so both are cut and merged by it.
//
// KV heads 2p and 2p + 1 of a block lie side by side in the pool, so their two
// key tiles are one copy of 8 KB, and their value tiles another. K is read by
// one map, V by both: 2 FMA for each value of K and 4 for each of V per query
// row, which the CUDA cores could just do for one row of a map while HBM
// delivers; from two rows on (G >= 2) they could not, so both products run on
// the tensor cores (mma.sync m16n8k16) in tiles of 16 rows: rows 0-7 are (query
// token, head) rows of the first map, rows 8-15 the same of the second.
//   S: both maps' rows against either key tile; of a product with K[2p] rows 0-7
//      are kept, of one with K[2p + 1] rows 8-15. The other half is thrown away
//      (the tensor cores are a tenth busy), and a map never meets the other's
//      keys, whatever they hold.
//   O: P (16 rows x 16 keys) times V (16 keys x 256 dims), 128 accumulators a lane.
// The two results of a row end in the same lane, so difference, norm and scale
// cost no exchange but the sum of squares: a segment that one warp has worked
// through alone writes its bf16 output at once.
// Bound by HBM: 518 MB of 256 ragged contexts in 93.5 us, 514 MB of 8 x 30k .. 32k in 91.7,
// 5.5 and 5.6 TB/s, of which 5 us are launch, plan and first copy and 4 to 6 the merge;
// between them equal ranges end up to 15 us apart, some SMs getting a tenth more than
// others. Four short contexts, a CTA to a segment: 10.7 us, all latency.
// A warp is a worker with its own ring of 16 KB stages and an equal range of
// the batch's (sequence, query tile, pair, block) tiles; segments that ranges
// cut leave fp32 partials, which diff_fixup_kernel merges.
#include <cudaTypedefs.h>

#include "pa_diff.cuh"
#include "pa_diff_plan.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kDRows = 2 * kMapRows;
constexpr int kDStage = 4 * kTileBytes;     // K[2p] K[2p+1] V[2p] V[2p+1] = 16 KB
constexpr int kDWarps = 5;
constexpr int kDStages = 2;
// what a segment start weighs in the cut, in quarters of a tile
constexpr int kSegCost4 = 6;
constexpr int kDDesc = 8;
// a row of a part in shared memory: eight words apart, so that a warp's stores spread
constexpr int kPartStride = kDiffDim + 8;
static_assert(kDRows * kPartStride * 4 <= kDStages * kDStage, "a warp's parts in its ring");

struct DiffArgs {
  const uint16_t* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_seqlens_q;  // null: one query per sequence
  DiffOut o;
  float scale_log2;
  int S, Hq, Hkv, G, QT, max_blocks;
  int64_t num_blocks;
  int64_t num_q_tokens;
  int causal;
  int npairs_cap;
  int max_lq;       // longer windows belong to the tcgen05 kernel
  int max_q_len;    // no window is longer than this
  float* part_o;    // [NW*2][16][256]
  float* part_lse;  // [NW*2][16]
  int* desc;        // [NW][kDDesc]: of the segment that worker w's start cuts first, or
  int by_segment;   // of each of `segments`, where there are far fewer of those
  int segments;
};

// byte offset of a row's 16-byte chunk (0 .. 15) in a 16 x 128 tile that came in as
// (8-row group, 64-dim half) atoms of 1 KB with the 128-byte swizzle
__device__ __forceinline__ uint32_t atom_at(int row, int chunk) {
  return (uint32_t)((row >> 3) * 2048 + (chunk >> 3) * 1024 + (row & 7) * 128 +
                    (((chunk & 7) ^ (row & 7)) << 4));
}

// PieceCut without its array: the cost of tiles 0 .. x-1 is 4x + kSegCost4 * (segment
// starts below x), and worker w begins at the first tile whose cost reaches
// floor(w C / nw). A warp wants three starts and one owner only, in closed form behind
// one bisection; the array of all 608 took 2 us at the head of every call.
struct CostCut {
  const PlanSmem* P;
  int Hp, nw;
  bool narrow;  // 32-bit divisions do (a 64-bit one is 100 instructions)
  long long C;
  __device__ __forceinline__ CostCut(const PlanSmem& plan, int heads, int max_workers)
      : P(&plan), Hp(heads) {
    C = 4LL * plan.total + (long long)kSegCost4 * plan.npairs * heads;
    const long long n = C / (4 + kSegCost4);
    nw = (int)(n > max_workers ? max_workers : n);
    narrow = C * nw < (1LL << 32);
  }
  __device__ __forceinline__ long long base(int p) const {
    return 4LL * P->pair_off[p] + (long long)kSegCost4 * p * Hp;
  }
  __device__ __forceinline__ int start(int w) const {  // 0 <= w <= nw
    if (w <= 0) return 0;
    if (w >= nw) return P->total;
    const long long T = narrow ? (long long)((uint32_t)w * (uint32_t)C / (uint32_t)nw)
                               : ((long long)w * C) / nw;
    int lo = 0, hi = P->npairs - 1;  // the pair with base(lo) < T <= base(lo + 1)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base(mid) < T)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int o0 = P->pair_off[lo], nt = (P->pair_off[lo + 1] - o0) / Hp;
    const int D = (int)(T - base(lo));  // 1 .. Hp (4 nt + kSegCost4)
    const int seg = 4 * nt + kSegCost4, h = (D - 1) / seg, rem = D - h * seg;
    return o0 + h * nt + max(1, (rem - kSegCost4 + 3) / 4);
  }
  // the worker that holds the last tile of a segment of two tiles or more
  __device__ __forceinline__ int owner_of_last(const TilePos& t) const {
    const long long x = P->pair_off[t.p] + (long long)t.h * t.nt + t.nt - 1;
    const long long cost = 4 * x + (long long)kSegCost4 * (t.p * Hp + t.h + 1);
    return narrow ? (int)(((uint32_t)(cost + 1) * (uint32_t)nw - 1u) / (uint32_t)C)
                  : (int)(((cost + 1) * nw - 1) / C);
  }
};

// Two weights (not negative) as the pair of their upper halves and a pair of what those leave.
// Neither half of a weight of 2^-96 or more is 0, so that an infinite value times it is not a NaN.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t& high, uint32_t& low) {
  const uint32_t bx = __float_as_uint(x), by = __float_as_uint(y);
  high = __byte_perm(bx, by, 0x7632);
  const float lx = fmaxf(x - __uint_as_float(bx & 0xffff0000u), x * 0x1p-30f);
  const float ly = fmaxf(y - __uint_as_float(by & 0xffff0000u), y * 0x1p-30f);
  low = cvt_bf16x2(lx, ly);
}

struct MapSum {
  float m, sum;
  float acc[8];
};

// Adds (m, sum, acc) of another group.
__device__ __forceinline__ void join(MapSum& x, float mo, float so, const float (&ao)[8]) {
  if (mo == neg_inf()) return;
  const float mn = fmaxf(x.m, mo);
  const float mine = x.m == neg_inf() ? 0.f : ex2((x.m - mn) * kLog2e);
  const float other = ex2((mo - mn) * kLog2e);
  x.sum = x.sum * mine + so * other;
#pragma unroll
  for (int j = 0; j < 8; ++j) x.acc[j] = x.acc[j] * mine + ao[j] * other;
  x.m = mn;
  if (mo != mo) x.m = x.sum = mo;  // a NaN stays one
}

// Difference, norm and scale of a query row whose maps are merged: row r of a query
// tile, eight dims a lane.
__device__ __forceinline__ void finish_row(const MapSum (&x)[2], const DiffOut& out, int h, int r,
                                           int64_t qtok, int Hq, int G, int lane) {
  const int head = h * G + r % G;
  const float lam = out.lambdas[head];
  const float inv0 = x[0].sum != 0.f ? 1.f / x[0].sum : 0.f;
  const float inv1 = x[1].sum != 0.f ? 1.f / x[1].sum : 0.f;
  float y[8], squares = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = diff_value(x[0].acc[j], inv0, x[1].acc[j], inv1, lam);
    squares = fmaf(y[j], y[j], squares);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) squares += __shfl_xor_sync(kFull, squares, o);
  const float f = diff_factor(out, squares);
  if (out.weight) {
    const float4* wt = reinterpret_cast<const float4*>(out.weight + lane * 8);
    const float4 w0 = wt[0], w1 = wt[1];
    const float ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= f * ws[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= f;
  }
  *reinterpret_cast<uint4*>(out.out + (qtok * (Hq / 2) + head) * kDiffDim + lane * 8) =
      make_uint4(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]), cvt_bf16x2(y[4], y[5]),
                 cvt_bf16x2(y[6], y[7]));
  if (out.lse && lane == 0) {
    float* l = out.lse + qtok * Hq + (int64_t)(2 * h) * G + r % G;
    l[0] = x[0].sum != 0.f ? x[0].m + lg2(x[0].sum) * kLn2 : neg_inf();
    l[G] = x[1].sum != 0.f ? x[1].m + lg2(x[1].sum) * kLn2 : neg_inf();
  }
}

// kWhole: a CTA has a segment for itself, an equal part of its tiles a warp, and merges
// in shared memory: no second grid.
// kWeights: how the softmax weights enter the product with V (kTwin: of whole segments).
enum : int { kRounded, kSplit, kTwin };
template <bool kWhole, int kWeights>
__global__ void __launch_bounds__(kDWarps * 32, 1)
    paged_diff_kernel(const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const DiffArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char* wbuf = smem + warp * kDStages * kDStage;
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(smem + kDWarps * kDStages * kDStage) + warp * kDStages;
  const int S = a.S, Hq = a.Hq, G = a.G, QT = a.QT, Hp = a.Hkv >> 1;

  PlanSmem P;
  P.pair_off = reinterpret_cast<int*>(smem + kDWarps * kDStages * kDStage +
                                      kDWarps * kDStages * 8);
  P.seq_pair = P.pair_off + (a.npairs_cap + 1);
  P.ctx = P.seq_pair + (S + 1);
  P.qstart = P.ctx + S;
  // the norm's weights, in shared memory for the epilogue: from global memory its 32
  // loads a lane, few of them in flight beside 128 accumulators, cost a ragged batch of
  // short contexts a third of its time (a whole segment's rows are finished by finish_row)
  __shared__ float2 weights[kWhole ? 1 : kDiffDim / 2];
  __shared__ float part_lse[kWhole ? kDWarps : 1][kDRows];
  if (kWhole && lane < kDRows) part_lse[warp][lane] = neg_inf();  // a warp without tiles

  if (lane == 0) {
    for (int i = 0; i < kDStages; ++i) mbar_init(smem_addr(&bars[i]), 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  static_assert(kDWarps * 32 >= kDiffDim / 2, "a pair of weights a thread");
  float2 mine = make_float2(1.f, 1.f);
  if (!kWhole && a.o.weight && threadIdx.x < kDiffDim / 2)
    mine = reinterpret_cast<const float2*>(a.o.weight)[threadIdx.x];
  PlanInputs in;
  in.context_lens = a.context_lens;
  in.cu_seqlens_q = a.cu_seqlens_q;
  in.S = S;
  in.Hkv = Hp;
  in.max_ctx = a.max_blocks * kBlock;
  in.qtile = QT;
  in.causal = a.causal;
  in.npairs_cap = a.npairs_cap;
  in.num_q_rows = a.num_q_tokens;
  in.max_lq = a.max_lq;
  in.announced = a.max_q_len;
  in.skip_empty = a.cu_seqlens_q == nullptr;
  build_plan(in, P, nullptr);
  if (!kWhole) {
    if (threadIdx.x < kDiffDim / 2) weights[threadIdx.x] = mine;
    __syncthreads();
  }
  const int W = P.total;
  // two tiles a warp at least: cutting a short batch further costs more in the merge
  // than it saves
  const CostCut cut(P, Hp, min((int)gridDim.x * kDWarps, max(1, W / 2)));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // a sequence of the single-query form with an empty context has no tiles
  if (!a.cu_seqlens_q) {
    for (int s = blockIdx.x; s < S; s += gridDim.x) {
      if (P.ctx[s] != 0) continue;
      uint4* row = reinterpret_cast<uint4*>(a.o.out + (int64_t)s * (Hq / 2) * kDiffDim);
      for (int i = threadIdx.x; i < Hq / 2 * (kDiffDim / 8); i += blockDim.x)
        row[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.o.lse)
        for (int i = threadIdx.x; i < Hq; i += blockDim.x) a.o.lse[(int64_t)s * Hq + i] = neg_inf();
    }
  }

  if (a.by_segment && blockIdx.x == 0)  // (nor have those that the batch does not have)
    for (int i = P.npairs * Hp + (int)threadIdx.x; i < a.segments; i += blockDim.x)
      reinterpret_cast<int4*>(a.desc)[2 * i] = make_int4(-1, 0, 0, 0);

  const int w = warp * (int)gridDim.x + (int)blockIdx.x;
  int R0 = 0, R1 = 0, R0prev = 0;  // this worker's range, and where the one before begins
  if constexpr (kWhole) {
    const int p = (int)blockIdx.x / Hp, h = (int)blockIdx.x - p * Hp;
    if (p >= P.npairs) return;
    const int o0 = P.pair_off[p], nt = (P.pair_off[p + 1] - o0) / Hp;
    R0 = o0 + h * nt + nt * warp / kDWarps;
    R1 = o0 + h * nt + nt * (warp + 1) / kDWarps;
  } else if (w < cut.nw) {
    const int at = cut.start(w - 1 + (lane < 3 ? lane : 1));
    R0prev = __shfl_sync(kFull, at, 0);
    R0 = __shfl_sync(kFull, at, 1);
    R1 = __shfl_sync(kFull, at, 2);
  }
  TilePos cp;
  if (R0 < R1) cp = locate(P, S, Hp, R0);
  // the segment that this boundary cuts, if it is the first to do so
  auto describe = [&]() {
    int4 d0 = make_int4(-1, 0, 0, 0), d1 = d0;
    if (R0 < R1 && w > 0 && cp.b > 0) {
      const int A = R0 - cp.b;  // its first tile
      if (A >= R0prev) {
        d0 = make_int4(cp.s, cp.qt, cp.h, cut.owner_of_last(cp));
        d1 = make_int4(A == R0prev ? 0 : 1, P.qstart[cp.s], P.qstart[cp.s + 1] - P.qstart[cp.s], w);
      }
    }
    int4* d = reinterpret_cast<int4*>(a.desc);
    if (!a.by_segment) {
      d[2 * w] = d0;
      d[2 * w + 1] = d1;
      return;
    }
    if (R0 >= R1) return;
    if (d0.x >= 0) {
      d[2 * (cp.p * Hp + cp.h)] = d0;
      d[2 * (cp.p * Hp + cp.h) + 1] = d1;
    }
    // segments that lie in this range as a whole have no pieces
    TilePos t = cp;
    for (int at = R0 - cp.b;;) {
      if (at >= R0 && at + t.nt <= R1) d[2 * (t.p * Hp + t.h)] = make_int4(-1, 0, 0, 0);
      at += t.nt;
      if (at >= R1) break;
      t.b = t.nt - 1;
      advance(P, S, Hp, t);
    }
  };
  if (!kWhole && R0 >= R1) {
    if (lane == 0) describe();
    return;
  }

  // ---- producer --------------------------------------------------------------
  TilePos pp = cp;
  int pidx = R0, wbase = R0;
  // block id of flat tile idx; tiles of a window lie a few pairs past pp
  auto load_phys = [&](int idx) -> int {
    if (idx >= R1) return 0;
    const TilePos t = locate_from(P, Hp, pp, idx);
    return a.block_tables[(size_t)t.s * a.max_blocks + t.b];
  };
  int phys_cur = load_phys(wbase + lane);
  int phys_next = load_phys(wbase + 32 + lane);

  auto issue = [&](int stage) {
    int phys = __shfl_sync(kFull, phys_cur, pidx - wbase);
    if (lane == 0) {
      if (phys < 0 || (int64_t)phys >= a.num_blocks) {
        flag_error(PA_DEVERR_BLOCK_RANGE);
        phys = 0;
      }
      const uint32_t st = smem_addr(wbuf + stage * kDStage);
      const uint32_t bar = smem_addr(&bars[stage]);
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, kDStage);
      const int group = (int)(((int64_t)phys * a.Hkv + 2 * pp.h) * (kBlock / 8));
      tma_load_block(st, &tmk, group, bar);
      tma_load_block(st + 2 * kTileBytes, &tmv, group, bar);
    }
    ++pidx;
    if (pidx < R1) {
      advance(P, S, Hp, pp);
      if (pp.b == 0) {
        // a new segment: its query rows on their way to L2 before they are wanted
        const int row = lane >> 1;  // eight rows of either map, 128 bytes a lane
        const int n = P.qstart[pp.s + 1] - P.qstart[pp.s], rm = row & 7;
        const int tk = pp.qt * QT + rm / G;
        if (rm < QT * G && tk < n)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(
              a.q + (((int64_t)P.qstart[pp.s] + tk) * Hq + (int64_t)(2 * pp.h + (row >> 3)) * G +
                     rm % G) * kHeadDim + (lane & 1) * 64));
      }
    }
    if (pidx - wbase == 32) {
      wbase += 32;
      phys_cur = phys_next;
      phys_next = load_phys(wbase + 32 + lane);
    }
  };
  for (int i = 0; i < kDStages && pidx < R1; ++i) issue(i);
  if (!kWhole && lane == 0) describe();  // (while the first copies are on their way)

  // ---- consumer --------------------------------------------------------------
  // this lane's row of either map's tile, and the query row that it holds. A CTA's segment of
  // four rows or fewer holds them twice, for the weights' halves (four short contexts 10.7
  // us; a second product for the lower ones 11.7, rounded weights 10.4)
  const int rt = lane >> 2, quad = lane & 3;
  const int r = kWeights == kTwin ? rt & 3 : rt;
  const int mi = lane >> 3, rr = lane & 7;   // ldmatrix: matrix and row of this lane's address
  uint32_t qa[8][4];
  float o[32][4];
  float m_r[2], l_r[2];
  int lim = 0, lim_min = 0, lq = 0, ctx = 0, tok = 0;
  float lam = 0.f;
  bool valid = false;
  int piece_b0 = 0;
  bool piece_first = true;

  int stage = 0;
  uint32_t parity = 0;
  for (int idx = R0; idx < R1; ++idx) {
    unsigned char* st = wbuf + stage * kDStage;
    const uint32_t sK = smem_addr(st), sV = sK + 2 * kTileBytes;
    if (idx == R0 || cp.b == 0) {
      ctx = P.ctx[cp.s];
      lq = P.qstart[cp.s + 1] - P.qstart[cp.s];
      tok = cp.qt * QT + r / G;
      valid = r < QT * G && tok < lq;
      // row r of a map: token r / G, head r % G of the map's KV head. Padding rows
      // stay zero (never written out).
      const uint32_t* q0 = nullptr;
      if (valid)
        q0 = reinterpret_cast<const uint32_t*>(
            a.q + (((int64_t)P.qstart[cp.s] + tok) * Hq + (int64_t)(2 * cp.h) * G + r % G) *
                      kHeadDim);
      const uint32_t* q1 = q0 + (int64_t)G * (kHeadDim / 2);
      lam = valid ? a.o.lambdas[cp.h * G + r % G] : 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int c = kk * 8 + quad;  // 32-bit word of dims kk*16 + 2*quad
        qa[kk][0] = valid ? q0[c] : 0u;
        qa[kk][1] = valid ? q1[c] : 0u;
        qa[kk][2] = valid ? q0[c + 4] : 0u;
        qa[kk][3] = valid ? q1[c + 4] : 0u;
      }
#pragma unroll
      for (int n = 0; n < 32; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m_r[0] = m_r[1] = neg_inf();
      l_r[0] = l_r[1] = 0.f;
      lim = valid ? (a.causal ? ctx - lq + tok + 1 : ctx) : 0x7fffffff;
      lim_min = lim;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, off));
      piece_b0 = cp.b;
      piece_first = (idx == R0);
    }
    if (!mbar_wait_bounded(smem_addr(&bars[stage]), parity)) {
      // the copies in flight land before the warp leaves
      for (int j = idx + 1; j < pidx; ++j) {
        if (++stage == kDStages) {
          stage = 0;
          parity ^= 1u;
        }
        mbar_wait_bounded(smem_addr(&bars[stage]), parity);
      }
      if (!kWhole) return;
      break;  // (its results are of no use; the others wait for it below)
    }
    const int key0 = cp.b * kBlock;
    // keys past the context may hold anything: zero those V rows so that
    // P = 0 never meets a NaN in the product
    if (key0 + kBlock > ctx) {
      const int zr = ctx - key0;  // first row to clear
      for (int i = lane; i < (kBlock - zr) * 32; i += 32) {
        const int row = zr + (i >> 5), c = i & 31;
        *reinterpret_cast<uint4*>(st + 2 * kTileBytes + (c >> 4) * kTileBytes +
                                  atom_at(row, c & 15)) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
      asm volatile("" ::: "memory");  // the ldmatrix reads below stay after the stores
    }

    // ---- S = Q K^T: rows 0-7 from the first key tile, 8-15 from the second ----------
    float s[2][4];
    {
      float s0[2][4], s1[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s0[n][e] = s1[n][e] = 0.f;
      const int key = (mi >> 1) * 8 + rr;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t at = atom_at(key, 2 * kk + (mi & 1));
        uint32_t b0, b1, b2, b3;
        ldsm_x4(sK + at, b0, b1, b2, b3);
        mma_bf16_16816(s0[0], qa[kk], b0, b1);
        mma_bf16_16816(s0[1], qa[kk], b2, b3);
        ldsm_x4(sK + kTileBytes + at, b0, b1, b2, b3);
        mma_bf16_16816(s1[0], qa[kk], b0, b1);
        mma_bf16_16816(s1[1], qa[kk], b2, b3);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = s0[n][0];
        s[n][1] = s0[n][1];
        s[n][2] = s1[n][2];
        s[n][3] = s1[n][3];
      }
    }
    // ---- mask, online softmax of either map ------------------------------------------
    const bool need_mask = key0 + kBlock > lim_min;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = s[n][e] * a.scale_log2;
        if (need_mask && key0 + n * 8 + quad * 2 + (e & 1) >= lim) v = neg_inf();
        s[n][e] = v;
      }
    float alpha[2], mref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const float mn = fmaxf(m_r[i], mx);
      mref[i] = mn == neg_inf() ? 0.f : mn;
      alpha[i] = ex2(m_r[i] - mref[i]);
      m_r[i] = mn;
    }
    float rs[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = ex2(s[n][e] - mref[e >> 1]);
        s[n][e] = p;
        rs[e >> 1] += p;
      }
    l_r[0] = l_r[0] * alpha[0] + rs[0];
    l_r[1] = l_r[1] * alpha[1] + rs[1];
    if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < 32; ++n) {
        o[n][0] *= alpha[0];
        o[n][1] *= alpha[0];
        o[n][2] *= alpha[1];
        o[n][3] *= alpha[1];
      }
    }
    // a key that only some rows see may hold an infinity or a NaN, which the product
    // would spread to all of them (0 x NaN): such elements join the rows that see
    // them here and enter the product as zeros
    if (need_mask) {
      const int nk = min(kBlock, ctx - key0);
      for (int kk = max(0, lim_min - key0); kk < nk; ++kk) {
        uint4* at = reinterpret_cast<uint4*>(st + 2 * kTileBytes + (lane >> 4) * kTileBytes +
                                             atom_at(kk, lane & 15));
        const uint4 x = *at;
        const bool bad = bf2_nonfinite(x.x) || bf2_nonfinite(x.y) || bf2_nonfinite(x.z) ||
                         bf2_nonfinite(x.w);
        if (!__any_sync(kFull, bad)) continue;
        const bool sees = key0 + kk < lim;
#pragma unroll
        for (int n = 0; n < 32; ++n) {
          const uint32_t wv = *reinterpret_cast<const uint32_t*>(
              st + 2 * kTileBytes + (n >> 4) * kTileBytes + atom_at(kk, n & 15) + quad * 4);
          const uint32_t f = bf2_finite_part(wv);
          if (sees && ((wv ^ f) & 0x7f80u)) {
            o[n][0] += bf_lo(wv);
            o[n][2] += bf_lo(wv);
          }
          if (sees && ((wv ^ f) & 0x7f800000u)) {
            o[n][1] += bf_hi(wv);
            o[n][3] += bf_hi(wv);
          }
        }
        __syncwarp();
        if (bad)
          *at = make_uint4(bf2_finite_part(x.x), bf2_finite_part(x.y), bf2_finite_part(x.z),
                           bf2_finite_part(x.w));
        __syncwarp();
        asm volatile("" ::: "memory");
      }
    }
    // ---- O += P V --------------------------------------------------------------------
    // P enters the product in bf16, the type that V is stored in and the MMA takes
    // beside it. Of single queries a weight is two such numbers, its upper half and what
    // that leaves, off by 2^-15 of it together (1.5 us of the calls above); of windows, as
    // elsewhere, it is one, off by 2^-8 at most: their tiles are full, and a second product
    // takes 46.7 to 53.1 us for 64 windows of 16 rows over 512 keys. The sums of the weights,
    // and with them lse, are of the unrounded ones.
    uint32_t p4[4], p4_low[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = s[i >> 1][2 * (i & 1)], y = s[i >> 1][2 * (i & 1) + 1];
      if constexpr (kWeights == kRounded)
        p4[i] = cvt_bf16x2(x, y);
      else
        split_bf16x2(x, y, p4[i], p4_low[i]);
      if (kWeights == kTwin && rt != r) p4[i] = p4_low[i];
    }
    {
      const int key = (mi & 1) * 8 + rr;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_trans(sV + t * kTileBytes + atom_at(key, 2 * c + (mi >> 1)), b0, b1, b2, b3);
          mma_bf16_16816(o[t * 16 + 2 * c], p4, b0, b1);
          mma_bf16_16816(o[t * 16 + 2 * c + 1], p4, b2, b3);
          if constexpr (kWeights == kSplit) {
            mma_bf16_16816(o[t * 16 + 2 * c], p4_low, b0, b1);
            mma_bf16_16816(o[t * 16 + 2 * c + 1], p4_low, b2, b3);
          }
        }
    }
    __syncwarp();
    if (pidx < R1) issue(stage);
    if (++stage == kDStages) {
      stage = 0;
      parity ^= 1u;
    }

    if (idx == R1 - 1 || cp.b == cp.nt - 1) {
      float inv[2], lse[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l_r[i];
        x += __shfl_xor_sync(kFull, x, 1);
        x += __shfl_xor_sync(kFull, x, 2);
        // (a NaN score's NaN goes on into the row's results)
        inv[i] = x != 0.f ? 1.f / x : 0.f;
        lse[i] = x != 0.f ? (m_r[i] + lg2(x)) * kLn2 : neg_inf();
      }
      if constexpr (kWhole) {
        // the warp's ring is done with: its rows' parts go there
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* dst = reinterpret_cast<float*>(wbuf) + (i * kMapRows + rt) * kPartStride + quad * 2;
#pragma unroll
          for (int n = 0; n < 32; ++n)
            *reinterpret_cast<float2*>(dst + n * 8) =
                make_float2(o[n][2 * i] * inv[i], o[n][2 * i + 1] * inv[i]);
          if (quad == 0) part_lse[warp][i * kMapRows + rt] = lse[i];
        }
      } else if (piece_b0 == 0 && cp.b == cp.nt - 1) {
        const int head = cp.h * G + r % G;
        float squares = 0.f;
#pragma unroll
        for (int n = 0; n < 32; ++n) {
          o[n][0] = diff_value(o[n][0], inv[0], o[n][2], inv[1], lam);
          o[n][1] = diff_value(o[n][1], inv[0], o[n][3], inv[1], lam);
          squares = fmaf(o[n][0], o[n][0], fmaf(o[n][1], o[n][1], squares));
        }
        squares += __shfl_xor_sync(kFull, squares, 1);
        squares += __shfl_xor_sync(kFull, squares, 2);
        if (valid) {
          const float f = diff_factor(a.o, squares);
          const int64_t qtok = (int64_t)P.qstart[cp.s] + tok;
          uint16_t* dst = a.o.out + (qtok * (Hq / 2) + head) * kDiffDim + quad * 2;
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            const float2 x = weights[n * 4 + quad];
            *reinterpret_cast<uint32_t*>(dst + n * 8) =
                cvt_bf16x2(o[n][0] * (f * x.x), o[n][1] * (f * x.y));
          }
          if (a.o.lse && quad == 0) {
            float* l = a.o.lse + qtok * Hq + (int64_t)(2 * cp.h) * G + r % G;
            l[0] = lse[0];
            l[G] = lse[1];
          }
        }
      } else {
        const size_t slot = (size_t)w * 2 + (piece_first ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = i * kMapRows + r;
          float* dst = a.part_o + (slot * kDRows + row) * kDiffDim + quad * 2;
          if (valid) {
#pragma unroll
            for (int n = 0; n < 32; ++n)
              *reinterpret_cast<float2*>(dst + n * 8) =
                  make_float2(o[n][2 * i] * inv[i], o[n][2 * i + 1] * inv[i]);
          }
          if (quad == 0) a.part_lse[slot * kDRows + row] = lse[i];
        }
      }
    }
    if (idx + 1 < R1) advance(P, S, Hp, cp);
  }
  if constexpr (kWhole) {
    __syncthreads();
    const int p = (int)blockIdx.x / Hp, h = (int)blockIdx.x - p * Hp;
    const int s = upper_index(P.seq_pair, 0, S, p), qt = p - P.seq_pair[s];
    const int nrows = min(QT, P.qstart[s + 1] - P.qstart[s] - qt * QT) * G;
    for (int row = warp; row < nrows; row += kDWarps) {
      MapSum x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i].m = neg_inf();
        x[i].sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i].acc[j] = 0.f;
        for (int k = 0; k < kDWarps; ++k) {
          const float4* src = reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + k * kDStages * kDStage) +
              (i * kMapRows + row) * kPartStride + lane * 8);
          const float4 a0 = src[0], a1 = src[1];
          float ao[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
          if constexpr (kWeights == kTwin) {  // what the weights' lower halves gave
            const float4 b0 = src[kPartStride], b1 = src[kPartStride + 1];
            const float bo[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) ao[j] += bo[j];
          }
          join(x[i], part_lse[k][i * kMapRows + row], 1.f, ao);
        }
      }
      finish_row(x, a.o, h, row, (int64_t)P.qstart[s] + qt * QT + row / G, Hq, G, lane);
    }
  }
}

// Merge the pieces of (sequence, query tile, pair) segments cut by the workers'
// ranges, then difference, norm and scale. Grid (worker boundary, or segment where
// there are far fewer of those; chunk of chunk_rows rows); a CTA's warps are dealt out
// to its rows, several to a row where there are few, each taking every n-th round of
// four pieces with all their loads in flight. A lane holds eight of a row's 256 dims, of
// both maps. Partials are read through L2 (ld.global.cg): other SMs wrote them. Bound by
// launching and latency: 4 to 6 us of a call.
// Where segments have many pieces a CTA takes one row (8 x 32k contexts, 47 pieces of 4
// rows, 14 us with a CTA to a segment), and the grid has the segments: 32 x 4 CTAs come
// and go 3 us sooner than 760 x 4. Elsewhere four rows or fewer get four warps: 346
// live CTAs of eight (256 contexts of up to 4096) take a second round on the SMs, 2 us.
__global__ void __launch_bounds__(kDFixWarps * 32)
    diff_fixup_kernel(const int* desc, const float* part_o, const float* part_lse, const DiffOut out,
                      int chunk_rows, int Hq, int G, int QT) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4* d = reinterpret_cast<const int4*>(desc + (size_t)blockIdx.x * kDDesc);
  const int4 d0 = __ldcg(d), d1 = __ldcg(d + 1);
  if (d0.x < 0) return;
  const int qt = d0.y, h = d0.z, last = d0.w, slot_prev = d1.x, q0 = d1.y, lq = d1.z, w = d1.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int npieces = last - w + 2;                       // workers w-1 .. last
  const int row0 = (int)blockIdx.y * chunk_rows;
  const int nrows = min(chunk_rows, min(QT, lq - qt * QT) * G - row0);  // 1 .. chunk_rows of either map
  if (nrows <= 0) return;
  const DiffDeal deal = diff_deal((int)blockDim.x >> 5, nrows, warp);
  const int per_row = deal.per_row, rl = deal.row, group = deal.group;
  const int r = row0 + rl;
  const bool live = rl < nrows;
  MapSum x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i].m = neg_inf();
    x[i].sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[i].acc[j] = 0.f;
  }
  bool nan[2] = {false, false};  // a piece with a NaN score: the row's results are NaNs
  for (int i0 = 4 * group; live && i0 < npieces; i0 += 4 * per_row) {
    float li[2][4];
    float4 v[2][4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        li[i][u] = neg_inf();
        v[i][u][0] = v[i][u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + u < npieces) {
          const size_t sl = (size_t)(w - 1 + i0 + u) * 2 + (i0 + u == 0 ? slot_prev : 0);
          const size_t row = sl * kDRows + i * kMapRows + r;
          li[i][u] = __ldcg(part_lse + row);
          const float4* src = reinterpret_cast<const float4*>(part_o + row * kDiffDim + lane * 8);
          v[i][u][0] = __ldcg(src);
          v[i][u][1] = __ldcg(src + 1);
        }
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mn =
          fmaxf(fmaxf(x[i].m, fmaxf(li[i][0], li[i][1])), fmaxf(li[i][2], li[i][3]));
#pragma unroll
      for (int u = 0; u < 4; ++u) nan[i] = nan[i] || li[i][u] != li[i][u];
      if (mn == neg_inf()) continue;
      const float shrink = x[i].m == neg_inf() ? 0.f : ex2((x[i].m - mn) * kLog2e);
      x[i].sum *= shrink;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].acc[j] *= shrink;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float wt = li[i][u] == neg_inf() ? 0.f : ex2((li[i][u] - mn) * kLog2e);
        x[i].sum += wt;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[i].acc[4 * k + 0] = fmaf(wt, v[i][u][k].x, x[i].acc[4 * k + 0]);
          x[i].acc[4 * k + 1] = fmaf(wt, v[i][u][k].y, x[i].acc[4 * k + 1]);
          x[i].acc[4 * k + 2] = fmaf(wt, v[i][u][k].z, x[i].acc[4 * k + 2]);
          x[i].acc[4 * k + 3] = fmaf(wt, v[i][u][k].w, x[i].acc[4 * k + 3]);
        }
      }
      x[i].m = mn;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (nan[i]) x[i].m = x[i].sum = __int_as_float(0x7fc00000);
  __shared__ __align__(16) float left[kDFixWarps][2][kDiffDim];
  __shared__ float left_ms[kDFixWarps][2][2];
  if (per_row > 1) {
    if (live && group > 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4* dst = reinterpret_cast<float4*>(left[warp][i] + lane * 8);
        dst[0] = make_float4(x[i].acc[0], x[i].acc[1], x[i].acc[2], x[i].acc[3]);
        dst[1] = make_float4(x[i].acc[4], x[i].acc[5], x[i].acc[6], x[i].acc[7]);
        if (lane == 0) {
          left_ms[warp][i][0] = x[i].m;
          left_ms[warp][i][1] = x[i].sum;
        }
      }
    }
    __syncthreads();
    if (live && group == 0) {
      for (int g = 1; g < per_row; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float ao[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) ao[j] = left[warp + g][i][lane * 8 + j];
          join(x[i], left_ms[warp + g][i][0], left_ms[warp + g][i][1], ao);
        }
    }
  }
  if (!live || group > 0) return;
  finish_row(x, out, h, r, (int64_t)q0 + qt * QT + r / G, Hq, G, lane);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// make_block_map's view with boxes of two tiles: KV heads 2p and 2p + 1 of a block.
bool make_pair_map(CUtensorMap* map, const void* pool, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)(rows / 8)};
  cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * 2, 128, (cuuint64_t)kHeadDim * 2 * 8};
  cuuint32_t box[4] = {64, 8, 2, 2 * (cuuint32_t)kBlock / 8};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*DiffKernel)(const CUtensorMap, const CUtensorMap, const DiffArgs);

DiffKernel diff_kernel(bool whole, int weights) {
  if (whole)
    return weights == kTwin ? paged_diff_kernel<true, kTwin>
           : weights == kSplit ? paged_diff_kernel<true, kSplit>
                               : paged_diff_kernel<true, kRounded>;
  return weights == kRounded ? paged_diff_kernel<false, kRounded> : paged_diff_kernel<false, kSplit>;
}

struct DiffGeometry {
  int grid = 0, workers = 0, npairs_cap = 0;
  size_t smem = 0, ws_desc = 0, ws_lse = 0, ws_o = 0, ws_bytes = 0;
};

// what the kernels declare themselves (the norm's weights, or a CTA's log-sum-exps), rounded
// up by the ring's alignment
constexpr int kDeclared = 1024;

// longest: the longest window that comes here
int diff_geometry(const pa_shape* sh, int64_t num_q_tokens, int64_t longest, DiffGeometry* g) {
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  const int S = sh->num_seqs;
  const int G = sh->num_q_heads / sh->num_kv_heads, QT = kMapRows / G;
  const int64_t cap = diff_pairs(S, num_q_tokens, longest, QT);
  if (cap > (1 << 22)) return PA_ERR_UNSUPPORTED;
  g->npairs_cap = (int)(cap < S ? S : cap);
  if (!diff_tiles_fit(g->npairs_cap, sh->num_kv_heads / 2, sh->max_blocks_per_seq, kSegCost4))
    return PA_ERR_UNSUPPORTED;
  g->grid = dev.num_sms;
  g->workers = g->grid * kDWarps;
  const size_t plan = sizeof(int) * ((size_t)g->npairs_cap + 1 + 3 * (size_t)S + 2);
  g->smem = 1024 + (size_t)kDWarps * kDStages * kDStage + kDWarps * kDStages * 8 + plan;
  if (g->smem + kDeclared > (size_t)dev.max_smem_optin) return PA_ERR_UNSUPPORTED;
  for (int weights = kRounded; weights <= kTwin; ++weights)
    for (int whole = 0; whole < 2; ++whole)
      if (!raise_smem_limit(reinterpret_cast<const void*>(diff_kernel(whole, weights)),
                            kDeclared))
        return PA_ERR_CUDA;
  g->ws_desc = round_up(sizeof(int) * kDDesc * (size_t)g->workers, 256);
  g->ws_lse = round_up(sizeof(float) * 2 * kDRows * (size_t)g->workers, 256);
  g->ws_o = round_up(sizeof(float) * 2 * kDRows * kDiffDim * (size_t)g->workers, 256);
  g->ws_bytes = g->ws_desc + g->ws_lse + g->ws_o;
  return PA_OK;
}

constexpr int kMaxGroup = 128;

// The kernels of a call. A window whose rows of a KV head (query tokens x group) are
// fewer than this goes through warp tiles of eight rows, the others through tcgen05 tiles
// of 256; more than eight query heads to a KV head always do. Measured, warp tiles
// against tcgen05, two heads to a KV head: 32 x 4096 keys 16 rows 163 against 184 us, 24
// rows 214 against 185, 32 rows 263 against 182; 4 x 2048 keys 22 against 33, 29 against
// 33, 31 against 33, 48 rows 38 against 33; 64 x 512 keys 47 against 90, 62 against 91, 77
// against 90, 48 rows 100 against 92. One number for all lengths: at 24 rows it costs long
// contexts 14 % and spares short ones a third.
constexpr int kTcMinRows = 32;

// Whether every segment gets a CTA, which ends in one grid, in the place of a cut over all
// warps and a second grid. Without: 14.1 us for 16 segments of 24 blocks, 14.2 for 32
// blocks, 15.7 for 64, 23.0 and 33.0 for 128 segments of 32 and 64; with: 11.9, 14.3, 21.0,
// 18.1 and 27.3. The bound on the table keeps a batch whose contexts differ from waiting
// long for one of them. (The host knows the table's width, not the contexts: the same
// four short ones under a table of 2048 blocks are cut over all warps.)
bool whole_segments(int64_t segments, int max_blocks, int sms) {
  return segments <= sms && max_blocks <= (3 * segments >= 2 * sms ? 64 : 28);
}

struct DiffPlan {
  bool warp = false;  // some window may be short
  DiffGeometry g;
  DiffTcGeometry tc;
  size_t ws_bytes = 0;
};

int diff_plan(const pa_shape* sh, int64_t num_q_tokens, int max_q_len, DiffPlan* p) {
  const int G = sh->num_q_heads / sh->num_kv_heads;
  int min_lq = G > kMapRows ? 1 : (kTcMinRows + G - 1) / G;
  p->warp = G <= kMapRows;
  // as many rows as windows of max_q_len hold: every window has that length, as far as
  // the host can tell. One that is shorter after all (rows behind the last sequence) is
  // taken by the same kernel then
  if (max_q_len >= min_lq && num_q_tokens == (int64_t)sh->num_seqs * max_q_len) {
    min_lq = 1;
    p->warp = false;
  }
  int rc = diff_tc_geometry(sh, num_q_tokens, max_q_len, min_lq, &p->tc);
  if (rc != PA_OK) return rc;
  if (p->warp) {
    rc = diff_geometry(sh, num_q_tokens, diff_warp_longest(max_q_len, min_lq), &p->g);
    if (rc != PA_OK) return rc;
  }
  p->ws_bytes = (p->warp ? p->g.ws_bytes : 0) + p->tc.ws_bytes;
  return PA_OK;
}

int check_diff_args(const pa_shape* sh, int64_t num_q_tokens, int max_q_len) {
  const int rc = check_shape_common(sh);
  if (rc != PA_OK) return rc;
  if (sh->num_kv_heads % 2 != 0) return PA_ERR_UNSUPPORTED;
  if (sh->num_q_heads / sh->num_kv_heads > kMaxGroup) return PA_ERR_UNSUPPORTED;
  if (num_q_tokens < 0 || max_q_len < 0 || num_q_tokens > 0x3fffffff) return PA_ERR_ARG;
  if (sh->num_blocks * sh->num_kv_heads * kBlock > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace

unsigned take_error_word_diff(cudaStream_t stream, int* rc) {
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

extern "C" size_t pa_decode_diff_workspace_size(const pa_shape* shape, int64_t num_q_tokens,
                                                int max_q_len) {
  if (check_diff_args(shape, num_q_tokens, max_q_len) != PA_OK) return 0;
  if (shape->num_seqs == 0 || num_q_tokens == 0 || max_q_len == 0) return 0;
  DiffPlan p;
  return diff_plan(shape, num_q_tokens, max_q_len, &p) == PA_OK ? p.ws_bytes : 0;
}

extern "C" int pa_decode_diff(const pa_bf16* q, const pa_bf16* k_cache, const pa_bf16* v_cache,
                              const int32_t* block_tables, const int32_t* context_lens,
                              const int32_t* cu_seqlens_q, int64_t num_q_tokens, int max_q_len,
                              int causal, float scale, const float* lambdas,
                              const float* norm_weight, float norm_eps, float out_scale,
                              pa_bf16* out, float* lse, const pa_shape* shape, void* workspace,
                              size_t workspace_bytes, void* stream) {
  pa::NvtxRange nvtx_range("pa_decode_diff");
  int rc = check_diff_args(shape, num_q_tokens, max_q_len);
  if (rc != PA_OK) return rc;
  if (!cu_seqlens_q && (num_q_tokens != shape->num_seqs || max_q_len != 1)) return PA_ERR_ARG;
  if (!(scale == scale) || !(norm_eps >= 0.f) || !(out_scale == out_scale)) return PA_ERR_ARG;
  if (shape->num_seqs == 0 || num_q_tokens == 0) return PA_OK;
  if (max_q_len == 0) return PA_ERR_ARG;  // rows, but no window may hold one
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !lambdas || !out)
    return PA_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(lambdas, 4) || !aligned(norm_weight, 16) || !aligned(lse, 4))
    return PA_ERR_ARG;
  DiffPlan p;
  rc = diff_plan(shape, num_q_tokens, max_q_len, &p);
  if (rc != PA_OK) return rc;
  if (!workspace || workspace_bytes < p.ws_bytes || !aligned(workspace, 256))
    return PA_ERR_WORKSPACE;
  DiffOut o;
  o.out = out;
  o.lse = lse;
  o.lambdas = lambdas;
  o.weight = norm_weight;
  o.eps = norm_eps;
  o.gain = out_scale;
  causal = causal && cu_seqlens_q ? 1 : 0;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.tc.enabled) {
    rc = launch_diff_tc(p.tc, q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q,
                        num_q_tokens, max_q_len, causal, scale, o, shape, ws, st);
    if (rc != PA_OK) return rc;
  }
  if (!p.warp) return PA_OK;
  const DiffGeometry& g = p.g;
  const int64_t rows = shape->num_blocks * shape->num_kv_heads * kBlock;
  CUtensorMap tmk, tmv;
  if (!make_pair_map(&tmk, k_cache, rows) || !make_pair_map(&tmv, v_cache, rows))
    return PA_ERR_CUDA;
  DiffArgs a = {};
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_seqlens_q = cu_seqlens_q;
  a.o = o;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.S = shape->num_seqs;
  a.Hq = shape->num_q_heads;
  a.Hkv = shape->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.QT = kMapRows / a.G;
  a.max_blocks = shape->max_blocks_per_seq;
  a.num_blocks = shape->num_blocks;
  a.num_q_tokens = num_q_tokens;
  a.causal = causal;
  a.npairs_cap = g.npairs_cap;
  a.max_lq = p.tc.enabled ? p.tc.min_lq - 1 : 0x7fffffff;
  a.max_q_len = max_q_len;
  char* wws = ws + p.tc.ws_bytes;
  a.desc = reinterpret_cast<int*>(wws);
  a.part_lse = reinterpret_cast<float*>(wws + g.ws_desc);
  a.part_o = reinterpret_cast<float*>(wws + g.ws_desc + g.ws_lse);
  // more than eight pieces to a segment on average (if the batch fills its contexts)
  const int64_t segments = (int64_t)g.npairs_cap * (a.Hkv / 2);
  const bool whole = whole_segments(segments, a.max_blocks, g.grid);
  // single queries: four rows or fewer twice, where that is not the merge's to add
  const int weights = max_q_len > 1 ? kRounded : whole && a.G <= kMapRows / 2 ? kTwin : kSplit;
  const DiffKernel kern = diff_kernel(whole, weights);
  if (whole)
    return launch_dependent(kern, dim3((unsigned)segments), dim3(kDWarps * 32),
                            g.smem, st, tmk, tmv, a) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  const bool many = (int64_t)g.workers > 8 * segments;
  a.by_segment = many;
  a.segments = many ? (int)segments : 0;
  if (launch_dependent(kern, dim3(g.grid), dim3(kDWarps * 32), g.smem, st, tmk, tmv, a) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  const DiffMerge m = diff_merge(many, max_q_len, a.QT, a.G);
  // (a worker has two tiles at least: of a small call only the first ones work)
  const int64_t most = (int64_t)g.npairs_cap * (a.Hkv / 2) * a.max_blocks / 2;
  const int64_t boundaries = most < 1 ? 1 : most < g.workers ? most : g.workers;
  const dim3 grid((unsigned)(many ? segments : boundaries), (unsigned)m.chunks);
  if (launch_dependent(diff_fixup_kernel, grid, dim3(m.warps * 32), 0, st, (const int*)a.desc,
                       (const float*)a.part_o, (const float*)a.part_lse, a.o, m.chunk, a.Hq, a.G,
                       a.QT) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
