// pa_prefill_tc.cu -- chunked-prefill attention over the paged pool on the
// fifth-generation tensor cores (tcgen05 + tensor memory) of sm_103a.
//
// Pages: course README "Build an LLM Inference Engine From Scratch",
// curriculum row "Batching & Scheduling" (chunked prefill, FlashAttention) and
// the claims "chunked prefill produces a bit-identical KV cache" / "online
// softmax is exact"; "S20 - The Complete Engine", section "The conflicts"
// (prefill runs eagerly next to decode). A chunk of Lq queries at the end of a
// context of c tokens: query j sits at position c - Lq + j and (causal) sees
// keys 0 .. c - Lq + j, the earlier ones already in the cache.
//
// A prefill chunk gives each KV head (128/G) x G query rows that share every
// K/V tile: a real matrix product, so it runs on tcgen05 with accumulators in
// tensor memory. One CTA per SM, warp-specialised (12 warps):
//   warp 0    TMA producer for the query tiles (3-D tensor map over q; two
//             buffers, so the next piece's tile lands early) and for K, as
//             eight 16-key pool blocks per 128-key tile, one copy each, found
//             through the block table (ids fetched one tile ahead);
//   warp 10   TMA producer for V; K and V stages have their own full/empty
//             mbarriers, so a K stage refills as soon as its S is done;
//   warp 1    allocates 512 TMEM columns and, from one thread, issues
//             S = Q K^T into one of two S buffers (the next tile's S is computed
//             while softmax works on this one);
//   warp 11   issues, from one thread, O_h += P_h V_h for the two 64-key halves,
//             with P read from tensor memory (a thread that issued both spent
//             its time on the other product's waits); each finished group of
//             either is signalled by tcgen05.commit on an mbarrier;
//   warps 2-9 softmax, two threads per query row, one per 64-key half, each
//             with its own running max, sum and O accumulator: read the S
//             half from TMEM, mask, exp2, write P (bf16 pairs) back over the S
//             columns just read; rescale O in TMEM only when a row maximum
//             grows by more than 2^8 (exact either way); at the end of a piece
//             the halves exchange (max, sum) through shared memory and write
//             the normalised row during the next tile.
// Work is a cut of the batch's flat (query tile, KV head, key tile) list at
// CTA granularity in which a segment start weighs as much as one key tile
// (PieceCut); pieces of a segment cut between CTAs are merged by
// prefill_tc_fixup_kernel. Beside a verify grid of the same call the grid
// keeps only its share of the SMs (overlap_split). Optional fp32 row output
// with a row map serves the cascade's shared-prefix half.
#include <cudaTypedefs.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kRowsT = 128;                 // query rows per tile (MMA M)
constexpr int kKeysT = 128;                 // keys per tile (N of S, K of PV)
constexpr int kBlocksT = kKeysT / kBlock;   // pool blocks per key tile
constexpr int kHalfT = kRowsT * 128;        // one 64-column half of a 128-row bf16 operand
constexpr int kOpBytes = 2 * kHalfT;        // a 128 x 128 bf16 operand
constexpr int kOffQ = 0;                   // two query-tile buffers
constexpr int kOffKV = kOffQ + 2 * kOpBytes;  // stage s: K at kOffKV + s * 2 * kOpBytes, V after it
constexpr int kOffBar = kOffKV + 2 * 2 * kOpBytes;
constexpr int kNumBars = 20;
constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmemSlot + 4;
constexpr int kOffBadV = kOffAbort + 4;
static_assert(kOffBadV + 4 <= kOffBar + 256, "barrier area");
constexpr int kOffLx = kOffBar + 256;       // [2 pieces][2 halves][128 rows] x (m, l)
constexpr int kOffPlan = kOffLx + 2 * 2 * kRowsT * 8;
// a segment start weighs as much as one key tile in the cut between CTAs
// (measured: a CTA whose range starts many short segments spends about one
// tile's time more on each)
constexpr int kPieceCost4 = 4;
constexpr int kSoftmaxWarps = 8;            // warps 2-9, two per SM sub-partition
constexpr int kVWarp = 2 + kSoftmaxWarps;   // the V producer
constexpr int kPvWarp = kVWarp + 1;         // issues O += P V
constexpr int kThreadsT = 128 + kSoftmaxWarps * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;             // S/P buffers at columns 0 and 128; O halves at 256, 384
constexpr int kDescInts = 8;
constexpr float kRescaleLog2 = 8.f;         // lazy O rescale threshold (log2 units)

enum : int {
  B_QFULL = 0, B_QFULL1, B_QEMPTY, B_QEMPTY1,
  B_KFULL, B_KFULL1, B_KEMPTY, B_KEMPTY1,
  B_VFULL, B_VFULL1, B_VEMPTY, B_VEMPTY1,
  B_SFULL, B_SFULL1, B_SFREE, B_SFREE1,
  B_PFULL, B_ODONE, B_LX, B_LX1
};

struct TcArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_seqlens_q;
  uint16_t* out;
  float* lse;
  float scale_log2;
  int S, Hq, Hkv, G, QTb, max_blocks;
  int64_t num_blocks;
  int64_t num_q_tokens;
  int causal;
  int npairs_cap;
  int num_workers;
  // > 0: this grid runs beside the verify grid of the same call and keeps
  // overlap_split(...) of its split CTAs (one per SM); the others leave at once
  int split;
  int min_lq;
  float* part_o;    // [NW * 2][128 rows][128]
  float* part_lse;  // [NW * 2][128 rows]
  int* desc;        // [NW][kDescInts] the merge that each worker boundary owns
  RowsOut rows;     // fp32 row output instead of out / lse (rows.o set)
  const int32_t* row_map;  // rows mode: query token i -> output token row_map[i]
  // tree windows: mask rows, and V for the elements that the product leaves out
  const uint32_t* mask = nullptr;
  int mask_words = 0;
  const uint16_t* v_cache = nullptr;
  // 1: CTAs 2p and 2p + 1 take the same key ranges for neighbouring query tiles
  // (the plan's unit is two tiles), so the second's K and V come from L2
  int pair = 0;
};

// Output row (token * Hq + head) of query token qtok, head hd; -1 when the
// row map sends it outside the output (flagged, not written).
__device__ __forceinline__ int64_t out_row(const TcArgs& a, int64_t qtok, int hd) {
  if (!a.row_map) return qtok * a.Hq + hd;
  const int64_t t = a.row_map[qtok];
  if (t < 0 || t >= a.rows.tokens) {
    flag_error(PA_DEVERR_QLEN_RANGE);
    return -1;
  }
  return t * a.Hq + hd;
}

__device__ __forceinline__ void plan_inputs(const TcArgs& a, PlanInputs& in) {
  in.context_lens = a.context_lens;
  in.cu_seqlens_q = a.cu_seqlens_q;
  in.S = a.S;
  in.Hkv = a.Hkv;
  in.max_ctx = a.max_blocks * kBlock;
  in.qtile = a.QTb << a.pair;
  in.causal = a.causal;
  in.npairs_cap = a.npairs_cap;
  in.num_q_rows = a.num_q_tokens;
  in.key_tile = kKeysT;
  in.min_lq = a.min_lq;
  in.max_window = a.mask_words * 32;  // 0: not a tree
}

__device__ __forceinline__ void plan_view(unsigned char* base, const TcArgs& a, PlanSmem& P) {
  int* pm = reinterpret_cast<int*>(base);
  P.pair_off = pm;
  P.seq_pair = pm + (a.npairs_cap + 1);
  P.ctx = P.seq_pair + (a.S + 1);
  P.qstart = P.ctx + a.S;
}

// The worker starts of the piece-weighted cut, after the plan arrays.
__device__ __forceinline__ int* cut_view(unsigned char* base, const TcArgs& a) {
  return reinterpret_cast<int*>(base) + (a.npairs_cap + 1) + 3 * (a.S + 1);
}

// Two words for the SM split's reduction, after the cut (8-byte aligned).
__device__ __forceinline__ unsigned long long* split_view(unsigned char* base, const TcArgs& a) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(cut_view(base, a) + a.num_workers + 1);
  return reinterpret_cast<unsigned long long*>((p + 7) & ~uintptr_t(7));
}

// The CTAs this call's prefill grid works with (all of them unless it runs
// beside the verify grid).
__device__ __forceinline__ int prefill_workers(const TcArgs& a, unsigned char* plan_base) {
  if (a.split <= 0) return a.num_workers;
  const int K = overlap_split(a.cu_seqlens_q, a.context_lens, a.S, a.Hkv, a.G, a.causal,
                              a.min_lq, a.max_blocks * kBlock, a.split,
                              split_view(plan_base, a));
  return min(a.num_workers, K);
}

// TREE: the window's visibility comes from a.mask, and any group size is taken
// (rows past QTb x G of a tile are padding whose results nothing reads).
template <bool TREE>
__global__ void __launch_bounds__(kThreadsT, 1)
    paged_prefill_tc_kernel(const __grid_constant__ CUtensorMap tmq,
                            const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, const TcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmemSlot);
  // TREE: a window row of V held an infinity or a NaN (set once, kept)
  volatile int* bad_v = reinterpret_cast<volatile int*>(smem + kOffBadV);
  const int S = a.S, Hkv = a.Hkv, G = a.G, QTb = a.QTb;
  auto bar = [&](int i) { return smem_addr(&bars[i]); };

  PlanSmem P;
  plan_view(smem + kOffPlan, a, P);
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool all = i == B_PFULL || i == B_LX || i == B_LX1;
      mbar_init(bar(i), all ? (uint32_t)(kSoftmaxWarps * 32) : 1u);
    }
    *abort_flag = 0;
    *bad_v = 0;
    mbar_fence_init();
  }
  if (tid == 32) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  // launched as a programmatic dependent of the previous grid
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int max_workers = prefill_workers(a, smem + kOffPlan);
  const int w = blockIdx.x >> a.pair;
  const int odd = blockIdx.x & a.pair;  // which tile of a unit of two
  int* desc = a.desc + (size_t)w * kDescInts;
  // beside a verify grid: the CTAs past the split leave now, freeing their SMs
  if ((int)blockIdx.x >= max_workers) {
    if (tid == 0 && odd == 0) desc[0] = -1;
    return;
  }
  PlanInputs in;
  plan_inputs(a, in);
  build_plan(in, P, nullptr);  // ends with a CTA barrier
  const PieceCut cut = build_piece_cut(P, Hkv, max_workers >> a.pair, kPieceCost4,
                                       cut_view(smem + kOffPlan, a));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 32 * kPvWarp && odd == 0) {  // a warp whose own work begins last
    // what the merge grid needs of the plan (rebuilding it there, after this
    // grid has left its SMs, took most of that grid's time)
    const MergeJob j = merge_job_of(P, S, Hkv, w, cut.nw, cut);
    desc[0] = j.valid ? j.s : -1;
    if (j.valid) {
      desc[1] = j.qt;
      desc[2] = j.h;
      desc[3] = j.last;
      desc[4] = j.slot_prev;
      desc[5] = P.qstart[j.s];
      desc[6] = P.qstart[j.s + 1] - P.qstart[j.s];
    }
  }
  if (w >= cut.nw) return;  // the whole CTA is idle (uniform)
  const int R0 = cut.start(w), R1 = cut.start(w + 1);
  if (R0 >= R1) return;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](int b, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(b), parity)) return true;
    if (*abort_flag) return false;
    if (!mbar_wait_bounded(bar(b), parity)) {
      *abort_flag = 1;
      return false;
    }
    return true;
  };

  if (warp == 0 || warp == kVWarp) {
    // ------------------------------------------------------------------ producers
    // warp 0 loads the query tiles and K, warp kVWarp loads V: each stage's K
    // is refilled as soon as its S is done, without queueing behind the V of
    // the previous tile (which waits for that tile's PV)
    const bool is_k = warp == 0;
    TilePos t = locate(P, S, Hkv, R0);
    auto nblocks_of = [&](const TilePos& tp) {
      const int nb_seq = (P.ctx[tp.s] + kBlock - 1) / kBlock;
      return min(kBlocksT, nb_seq - tp.b * kBlocksT);
    };
    auto fetch_ids = [&](const TilePos& tp) -> int {
      return lane < nblocks_of(tp)
                 ? a.block_tables[(size_t)tp.s * a.max_blocks + tp.b * kBlocksT + lane]
                 : 0;
    };
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    const int b_full = is_k ? B_KFULL : B_VFULL, b_empty = is_k ? B_KEMPTY : B_VEMPTY;
    int ids = fetch_ids(t);
    int qn = 0;
    for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
      const bool first = (idx == R0) || (t.b == 0);
      if (is_k && first) {
        const int qs = qn & 1;
        if (qn >= 2 && !wait(B_QEMPTY + qs, (uint32_t)((qn >> 1) - 1) & 1u)) break;
        if (lane == 0) {
          // first query token of the tile (past the rows for the missing second
          // tile of a unit: zeros)
          const int z = P.qstart[t.s] + ((t.qt << a.pair) + odd) * QTb;
          const uint32_t qd = smem_addr(smem + kOffQ + qs * kOpBytes);
          mbar_arrive_expect_tx(bar(B_QFULL + qs),
                                TREE ? (uint32_t)(QTb * G) * 256u : (uint32_t)kOpBytes);
          tma_load_3d(qd, &tmq, 0, t.h * G, z, bar(B_QFULL + qs));
          tma_load_3d(qd + kHalfT, &tmq, 64, t.h * G, z, bar(B_QFULL + qs));
        }
        ++qn;
      }
      const int st = i & 1;
      const int nb = nblocks_of(t);
      int my_id = ids;
      if (idx + 1 < R1) {  // block ids of the next tile, one tile ahead
        TilePos tn = t;
        advance(P, S, Hkv, tn);
        ids = fetch_ids(tn);
      }
      if (lane < nb && (my_id < 0 || (int64_t)my_id >= a.num_blocks)) {
        if (is_k) flag_error(PA_DEVERR_BLOCK_RANGE);
        my_id = 0;
      }
      const int group = (int)(((int64_t)my_id * Hkv + t.h) * (kBlock / 8));
      // the stage is free once the S (K) or the PV (V) of tile i-2 is done
      if (i >= 2 && !wait(b_empty + st, (uint32_t)((i >> 1) - 1) & 1u)) break;
      if (lane == 0) mbar_arrive_expect_tx(bar(b_full + st), (uint32_t)nb * (uint32_t)kTileBytes);
      __syncwarp();
      const uint32_t d = smem_addr(smem + kOffKV + st * 2 * kOpBytes + (is_k ? 0 : kOpBytes) +
                                   lane * kTileBytes);
      if (lane < nb) tma_load_block(d, map, group, bar(b_full + st));
      __syncwarp();
      if (idx + 1 < R1) advance(P, S, Hkv, t);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer, S = Q K^T
    if (lane == 0) {
      const uint32_t idS = f16_idesc(kRowsT, kKeysT, 0);
      int qn = 0, qs = 0;  // query tiles seen; buffer of the current one
      // operand descriptors differ by their address alone (16-byte units)
      const uint64_t desc_q = sw128_desc(smem_addr(smem + kOffQ), 16, 1024);
      // K: 8-row groups every 2 KB, each the two 64-dim halves' 1 KB atoms
      const uint64_t desc_k = sw128_desc(smem_addr(smem + kOffKV), 16, 2048);
      auto issue_S = [&](int i, bool first) -> bool {
        if (first) {
          qs = qn & 1;
          if (!wait(B_QFULL + qs, (uint32_t)(qn >> 1) & 1u)) return false;
          ++qn;
        }
        const int st = i & 1;
        if (!wait(B_KFULL + st, (uint32_t)(i >> 1) & 1u)) return false;
        // the S/P buffer is free once the PV that read P of tile i-2 is done
        if (i >= 2 && !wait(B_SFREE + st, (uint32_t)((i >> 1) - 1) & 1u)) return false;
        tc_fence_after();
        const uint64_t dq = desc_q + (uint64_t)(qs * (kOpBytes >> 4));
        const uint64_t dk = desc_k + (uint64_t)(st * (2 * kOpBytes >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // head_dim 128 = 8 steps of 16
          tc_mma(tmem + (uint32_t)st * 128u, dq + (uint64_t)(((k >> 2) * kHalfT + (k & 3) * 32) >> 4),
                 dk + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), idS, k > 0);
        }
        tc_commit(bar(B_SFULL + st));
        tc_commit(bar(B_KEMPTY + st));
        return true;
      };
      TilePos t = locate(P, S, Hkv, R0);
      for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
        if (!issue_S(i, (idx == R0) || (t.b == 0))) break;
        if (idx + 1 >= R1 || t.b == t.nt - 1) tc_commit(bar(B_QEMPTY + qs));
        if (idx + 1 < R1) advance(P, S, Hkv, t);
      }
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ MMA issuer, O += P V
    if (lane == 0) {
      const uint32_t idPV = f16_idesc(kRowsT, 128, 1);
      // V: 8-row groups every 2 KB, each the two 64-dim halves' 1 KB atoms
      const uint64_t desc_v = sw128_desc(smem_addr(smem + kOffKV + kOpBytes), 1024, 2048);
      TilePos t = locate(P, S, Hkv, R0);
      for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
        const bool first = (idx == R0) || (t.b == 0);
        const int st = i & 1;
        if (!wait(B_VFULL + st, (uint32_t)(i >> 1) & 1u) || !wait(B_PFULL, (uint32_t)i & 1u)) break;
        tc_fence_after();
        const uint64_t dv = desc_v + (uint64_t)(st * (2 * kOpBytes >> 4));
        // O_hf += P[:, keys of half hf] V[keys of half hf, :]: one accumulator per
        // key half; P (bf16 pairs) sits in columns st*128 + hf*64 .. +31 of TMEM
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ts(tmem + kColO + (uint32_t)hf * 128u,
                      tmem + (uint32_t)st * 128u + (uint32_t)hf * 64u + (uint32_t)k * 8u,
                      dv + (uint64_t)((hf * 4 + k) * (4096 >> 4)), idPV,
                      (k > 0 || !first) ? 1u : 0u);
        tc_commit(bar(B_VEMPTY + st));
        tc_commit(bar(B_SFREE + st));
        tc_commit(bar(B_ODONE));
        if (idx + 1 < R1) advance(P, S, Hkv, t);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax
    // Thread (row r, half hf) owns keys hf*64 .. hf*64+63 of every tile of row r
    // with its own running maximum, sum and O accumulator; the two halves of a
    // row are merged once, at the end of a piece.
    const int q4 = warp & 3;
    const int hf = (warp - 2) >> 2;
    const int r = q4 * 32 + lane;  // this thread's query row (= TMEM lane)
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tO = tmem + lane_base + kColO;
    float* lx = reinterpret_cast<float*>(smem + kOffLx);
    const float sc = a.scale_log2;
    TilePos t = locate(P, S, Hkv, R0);
    float m_ref = neg_inf(), l = 0.f;
    int lim = 0, c = 0, lq = 0, tok = 0, piece_b0 = 0, np = 0;
    bool valid = false, piece_first = true;
    const uint32_t* mrow = nullptr;  // TREE: this row's mask words
    int pend_s = 0, pend_h = 0, pend_k0 = 0, pend_k1 = 0;
    // A finished piece's O stays in TMEM until the next tile's exponentials
    // are done (its last PV completes meanwhile); then it is written out.
    bool pend = false, pend_complete = false, pend_valid = false;
    int pend_np = 0;
    int64_t pend_orow = 0;
    size_t pend_slot = 0;
    float pend_m = 0.f, pend_l = 0.f;
    auto flush = [&]() -> bool {
      // merge the two key halves of the row: the partner's (m, l) from shared memory
      if (!wait(B_LX + (pend_np & 1), (uint32_t)(pend_np >> 1) & 1u)) return false;
      const float* other = lx + ((pend_np & 1) * 2 + (hf ^ 1)) * kRowsT * 2 + r * 2;
      const float m_o = other[0], l_o = other[1];
      const float M = fmaxf(pend_m, m_o);
      const float a_me = pend_m == neg_inf() ? 0.f : ex2(pend_m - M);
      const float a_o = m_o == neg_inf() ? 0.f : ex2(m_o - M);
      const float lt = pend_l * a_me + l_o * a_o;
      // (TREE: a NaN score's NaN goes on into the row's results)
      const bool any_weight = TREE ? lt != 0.f : lt > 0.f;
      const float inv = any_weight ? 1.f / lt : 0.f;
      const float c0 = (hf == 0 ? a_me : a_o) * inv, c1 = (hf == 0 ? a_o : a_me) * inv;
      const float lse_v = any_weight ? (M + lg2(lt)) * kLn2 : neg_inf();
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int d0 = hf * 64 + cc * 32;  // output dims d0 .. d0+31
        uint32_t u0[32], u1[32];
        tmem_ld32_async(tO + (uint32_t)d0, u0);
        tmem_ld32_async(tO + 128u + (uint32_t)d0, u1);
        tmem_wait_ld(u0);
        tmem_tie(u1);
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          o[j] = fmaf(__uint_as_float(u0[j]), c0, __uint_as_float(u1[j]) * c1);
        if constexpr (TREE) {
          // infinities and NaNs of window rows entered the product as zeros
          // (they must not reach queries that do not see their row): they join
          // the rows that see them here
          if (*bad_v && pend_valid) {
            const int lqp = P.qstart[pend_s + 1] - P.qstart[pend_s];
            const int p0 = P.ctx[pend_s] - lqp;
            const uint32_t* mr = a.mask + (pend_orow / a.Hq) * a.mask_words;
            const int i1 = min(lqp, pend_k1 - p0);  // the piece's window keys
            for (int i = max(0, pend_k0 - p0); i < i1; ++i) {
              if (!((mr[i >> 5] >> (i & 31)) & 1u)) continue;
              const int phys =
                  a.block_tables[(size_t)pend_s * a.max_blocks + (p0 + i) / kBlock];
              if (phys < 0 || (int64_t)phys >= a.num_blocks) continue;
              const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                  a.v_cache +
                  ((((int64_t)phys * Hkv + pend_h) * kBlock) + (p0 + i) % kBlock) * kHeadDim + d0);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t wv = vr[j], fin = bf2_finite_part(wv);
                if ((wv ^ fin) & 0x7f80u) o[2 * j] += bf_lo(wv);
                if ((wv ^ fin) & 0x7f800000u) o[2 * j + 1] += bf_hi(wv);
              }
            }
          }
        }
        if (pend_complete && a.rows.o) {
          if (pend_valid) {
            float4* dst = reinterpret_cast<float4*>(
                a.rows.o + (pend_orow * a.rows.stride + a.rows.slot) * kHeadDim + d0);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        } else if (pend_complete) {
          if (pend_valid) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + pend_orow * kHeadDim + d0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(cvt_bf16x2(o[8 * q + 0], o[8 * q + 1]),
                                  cvt_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                  cvt_bf16x2(o[8 * q + 4], o[8 * q + 5]),
                                  cvt_bf16x2(o[8 * q + 6], o[8 * q + 7]));
          }
        } else {
          float4* dst =
              reinterpret_cast<float4*>(a.part_o + (pend_slot * kRowsT + r) * kHeadDim + d0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (hf == 0) {
        if (pend_complete && a.rows.o) {
          if (pend_valid) a.rows.lse[pend_orow * a.rows.stride + a.rows.slot] = lse_v;
        } else if (pend_complete) {
          if (pend_valid && a.lse) a.lse[pend_orow] = lse_v;
        } else {
          a.part_lse[pend_slot * kRowsT + r] = lse_v;
        }
      }
      pend = false;
      return true;
    };
    int i = 0;
    for (int idx = R0; idx < R1; ++idx, ++i) {
      const bool first = (idx == R0) || (t.b == 0);
      const bool last = (idx == R1 - 1) || (t.b == t.nt - 1);
      if (first) {
        c = P.ctx[t.s];
        lq = P.qstart[t.s + 1] - P.qstart[t.s];
        tok = ((t.qt << a.pair) + odd) * QTb + r / G;
        valid = tok < lq;
        if constexpr (TREE) {
          valid = valid && r < QTb * G;
          mrow = a.mask + ((int64_t)P.qstart[t.s] + (valid ? tok : 0)) * a.mask_words;
        }
        lim = valid ? (a.causal ? c - lq + tok + 1 : c) : 0;
        m_ref = neg_inf();
        l = 0.f;
        piece_b0 = t.b;
        piece_first = (idx == R0);
      }
      const int sb = i & 1;
      if (!wait(B_SFULL + sb, (uint32_t)(i >> 1) & 1u)) break;
      tc_fence_after();
      uint32_t v0[32], v1[32];
      const uint32_t tS = tmem + lane_base + (uint32_t)sb * 128u + (uint32_t)hf * 64u;
      tmem_ld32_async(tS, v0);
      tmem_ld32_async(tS + 32u, v1);
      tmem_wait_ld(v0);
      tmem_tie(v1);

      // scores in log2 units
      float2 x[32];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = __fmul2_rn(make_float2(__uint_as_float(v0[2 * j]), __uint_as_float(v0[2 * j + 1])),
                          make_float2(sc, sc));
        x[16 + j] =
            __fmul2_rn(make_float2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1])),
                       make_float2(sc, sc));
      }
      const int kb = t.b * kKeysT + hf * 64;  // first key of this half
      if constexpr (TREE) {
        if (kb + 64 > c - lq) {  // the half reaches into the window
          const int i0 = kb - (c - lq);
          const uint32_t vis0 =
              valid ? tree_visible32(mrow, a.mask_words, i0, c - kb) : 0u;
          const uint32_t vis1 =
              valid ? tree_visible32(mrow, a.mask_words, i0 + 32, c - kb - 32) : 0u;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (!((vis0 >> (2 * j)) & 1u)) x[j].x = neg_inf();
            if (!((vis0 >> (2 * j + 1)) & 1u)) x[j].y = neg_inf();
            if (!((vis1 >> (2 * j)) & 1u)) x[16 + j].x = neg_inf();
            if (!((vis1 >> (2 * j + 1)) & 1u)) x[16 + j].y = neg_inf();
          }
        }
      } else if (kb + 64 > lim) {  // the causal diagonal or the end of the context
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (kb + 2 * j >= lim) x[j].x = neg_inf();
          if (kb + 2 * j + 1 >= lim) x[j].y = neg_inf();
        }
      }
      float mx;
      {
        float m8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float mu = fmaxf(x[u].x, x[u].y);
          float mv;
          asm("max.f32 %0, %1, %2, %3;" : "=f"(mv) : "f"(x[8 + u].x), "f"(x[8 + u].y), "f"(mu));
          asm("max.f32 %0, %1, %2, %3;" : "=f"(mu) : "f"(x[16 + u].x), "f"(x[16 + u].y), "f"(mv));
          asm("max.f32 %0, %1, %2, %3;" : "=f"(mv) : "f"(x[24 + u].x), "f"(x[24 + u].y), "f"(mu));
          m8[u] = mv;
        }
        float m3a, m3b;
        asm("max.f32 %0, %1, %2, %3;" : "=f"(m3a) : "f"(m8[0]), "f"(m8[1]), "f"(m8[2]));
        asm("max.f32 %0, %1, %2, %3;" : "=f"(m3b) : "f"(m8[3]), "f"(m8[4]), "f"(m8[5]));
        asm("max.f32 %0, %1, %2, %3;" : "=f"(mx) : "f"(m8[6]), "f"(m8[7]), "f"(m3a));
        mx = fmaxf(mx, m3b);
      }
      float alpha = 1.f;
      bool rescale = false;
      if (m_ref == neg_inf()) {
        m_ref = mx;  // nothing accumulated yet (O and l are zero)
      } else if (mx > m_ref + kRescaleLog2) {
        alpha = ex2(m_ref - mx);
        m_ref = mx;
        rescale = true;
      }
      const float ref = m_ref == neg_inf() ? 0.f : m_ref;
      const float2 nref = make_float2(-ref, -ref);
      float2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      // P enters the product in bf16, the type that V is stored in and that one
      // tcgen05.mma wants of both operands: a weight is off by at most 2^-8 of itself,
      // the output, itself bf16, by at most 2^-8 of sum p |v| (measured on trees of 64
      // nodes: 1.8e-3 at most against 1.6e-3 from the output's rounding alone). The
      // sum l, and with it lse, is of the unrounded ones.
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 d = __fadd2_rn(x[j], nref);
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        acc[j & 3] = __fadd2_rn(acc[j & 3], e);
        pk[j] = cvt_bf16x2(e.x, e.y);
      }
      const float2 s01 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l = fmaf(l, alpha, s01.x + s01.y);
      // the previous PV must be done before P is replaced, O is rescaled or the
      // previous piece's O is read
      if (i > 0 && !wait(B_ODONE, (uint32_t)(i - 1) & 1u)) break;
      tc_fence_after();
      if (pend && !flush()) break;
      // the tensor-memory accesses are warp-wide: the whole warp rescales when one
      // of its rows has to (the others by 1)
      if (__any_sync(kFull, rescale) && !first) {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t v[32];
          const uint32_t ta = tO + (uint32_t)hf * 128u + (uint32_t)cc * 32u;
          tmem_ld32(ta, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
          tmem_st32(ta, v);
        }
      }
      // P row r, keys of half hf, over the S columns this thread has read
      tmem_st32(tS, pk);
      tmem_wait_st();
      // keys past the context may hold anything (even NaN): zero their V rows
      // so that P = 0 never meets them (thread (r, hf) clears half hf of key row r)
      const int key0 = t.b * kKeysT;
      const int vsafe = TREE ? c - lq : c;  // rows before it enter the product as they are
      if (key0 + kKeysT > vsafe && key0 + r >= vsafe) {
        if (!wait(B_VFULL + sb, (uint32_t)(i >> 1) & 1u)) break;
        unsigned char* vrow = smem + kOffKV + sb * 2 * kOpBytes + kOpBytes + (r >> 3) * 2048 +
                              hf * 1024 + (r & 7) * 128;
        bool write = true;
        if constexpr (TREE) {
          if (key0 + r < c) {  // a window row: only its infinities and NaNs are left out
            bool bad = false;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              const uint4 x4 = *reinterpret_cast<const uint4*>(vrow + ch * 16);
              bad = bad || bf2_nonfinite(x4.x) || bf2_nonfinite(x4.y) || bf2_nonfinite(x4.z) ||
                    bf2_nonfinite(x4.w);
            }
            write = false;
            if (bad) {
              *bad_v = 1;
              for (int ch = 0; ch < 8; ++ch) {
                uint4 x4 = *reinterpret_cast<const uint4*>(vrow + ch * 16);
                x4.x = bf2_finite_part(x4.x);
                x4.y = bf2_finite_part(x4.y);
                x4.z = bf2_finite_part(x4.z);
                x4.w = bf2_finite_part(x4.w);
                *reinterpret_cast<uint4*>(vrow + ch * 16) = x4;
              }
              fence_proxy_async_smem();
            }
          }
        }
        if (write) {
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(vrow + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
      }
      tc_fence_before();
      mbar_arrive(bar(B_PFULL));

      if (last) {
        // hand (m, l) of this half to the partner thread; O is written out
        // during the next tile (or after the loop)
        float* mine = lx + ((np & 1) * 2 + hf) * kRowsT * 2 + r * 2;
        mine[0] = m_ref;
        mine[1] = l;
        mbar_arrive(bar(B_LX + (np & 1)));
        pend = true;
        pend_np = np++;
        pend_m = m_ref;
        pend_l = l;
        pend_complete = (piece_b0 == 0) && (t.b == t.nt - 1);
        pend_orow = valid ? out_row(a, (int64_t)P.qstart[t.s] + tok, t.h * G + r % G) : 0;
        pend_valid = valid && pend_orow >= 0;
        pend_s = t.s;
        pend_h = t.h;
        pend_k0 = piece_b0 * kKeysT;
        pend_k1 = (t.b + 1) * kKeysT;
        pend_slot = (size_t)blockIdx.x * 2 + (piece_first ? 0 : 1);
      }
      if (idx + 1 < R1) advance(P, S, Hkv, t);
    }
    if (pend && !*abort_flag && wait(B_ODONE, (uint32_t)(i - 1) & 1u)) {
      tc_fence_after();
      flush();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

// Merge the pieces of (sequence, query tile, KV head) segments cut between
// CTAs. Grid (CTA boundary, quarter of the tile's rows); eight lanes per
// query row, so each piece's row is one coalesced 512-byte read and a warp has
// four rows' loads in flight.
// GROUPS > 1: that many groups of the CTA's warps share its rows' pieces.
constexpr int kFixRowsPerCta = 32;
constexpr int kFixThreads = 256;
constexpr int kFixGroupsT = 4;

template <int GROUPS>
__global__ void __launch_bounds__(kFixThreads)
    prefill_tc_fixup_kernel(const TcArgs a) {
  // the next grid in the stream may start its own preparation now; it waits
  // for this grid before it reads anything this grid writes
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x >> a.pair, odd = blockIdx.x & a.pair;
  const int4* d = reinterpret_cast<const int4*>(a.desc + (size_t)w * kDescInts);
  const int4 d0 = __ldcg(d), d1 = __ldcg(d + 1);
  if (d0.x < 0) return;
  const int qt = d0.y, h = d0.z, last = d0.w, slot_prev = d1.x, q0 = d1.y, lq = d1.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int npieces = last - w + 2;  // workers w-1 .. last
  auto slot_of = [&](int i) -> size_t {
    return (size_t)(((w - 1 + i) << a.pair) + odd) * 2 + (i == 0 ? slot_prev : 0);
  };
  // a warp merges four rows at once: eight lanes per row, sixteen dims per lane
  constexpr int kRowWarps = kFixThreads / 32 / GROUPS;
  const int group = warp / kRowWarps, rl = (warp % kRowWarps) * 4 + (lane >> 3);
  const int r = blockIdx.y * (kFixRowsPerCta / GROUPS) + rl;
  const int dim0 = (lane & 7) * 16;
  const int tok = ((qt << a.pair) + odd) * a.QTb + r / a.G;
  const bool live = r < a.QTb * a.G && tok < lq;  // not a padding row
  if (GROUPS == 1 && !live) return;
  // online merge over the pieces, four at a time with all their loads in flight
  float m = neg_inf(), sum = 0.f;
  bool nan = false;  // a piece with a NaN score: the row's results are NaNs
  float acc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  for (int i0 = 4 * group; live && i0 < npieces; i0 += 4 * GROUPS) {
    float li[4];
    float4 x[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      li[u] = neg_inf();
      x[u][0] = x[u][1] = x[u][2] = x[u][3] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < npieces) {
        const size_t sl = slot_of(i0 + u);
        li[u] = a.part_lse[sl * kRowsT + r];
        const float4* src =
            reinterpret_cast<const float4*>(a.part_o + (sl * kRowsT + r) * kHeadDim + dim0);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[u][k] = src[k];
      }
    }
    const float mn = fmaxf(fmaxf(m, fmaxf(li[0], li[1])), fmaxf(li[2], li[3]));
#pragma unroll
    for (int u = 0; u < 4; ++u) nan = nan || li[u] != li[u];
    if (mn == neg_inf()) continue;
    const float shrink = m == neg_inf() ? 0.f : ex2((m - mn) * kLog2e);
    sum *= shrink;
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] *= shrink;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float wt = li[u] == neg_inf() ? 0.f : ex2((li[u] - mn) * kLog2e);
      sum += wt;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k + 0] = fmaf(wt, x[u][k].x, acc[4 * k + 0]);
        acc[4 * k + 1] = fmaf(wt, x[u][k].y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(wt, x[u][k].z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(wt, x[u][k].w, acc[4 * k + 3]);
      }
    }
    m = mn;
  }
  if (nan) m = sum = __int_as_float(0x7fc00000);
  if constexpr (GROUPS > 1) {
    __shared__ __align__(16) float left[GROUPS - 1][kFixRowsPerCta / GROUPS][kMergeRow];
    if (group > 0 && live) merge_store(left[group - 1][rl], dim0, m, sum, acc);
    __syncthreads();
    if (group > 0 || !live) return;
    for (int g = 0; g < GROUPS - 1; ++g) merge_take(left[g][rl], dim0, m, sum, acc);
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] *= inv;
  const float LSE = sum != 0.f ? m + lg2(sum) * kLn2 : neg_inf();
  const int64_t orow = out_row(a, (int64_t)q0 + tok, h * a.G + r % a.G);
  if (orow < 0) return;
  if (a.rows.o) {
    float4* dst = reinterpret_cast<float4*>(a.rows.o + (orow * a.rows.stride + a.rows.slot) * kHeadDim + dim0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      dst[k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
    if ((lane & 7) == 0) a.rows.lse[orow * a.rows.stride + a.rows.slot] = LSE;
    return;
  }
  uint4* dst = reinterpret_cast<uint4*>(a.out + orow * kHeadDim + dim0);
  dst[0] = make_uint4(cvt_bf16x2(acc[0], acc[1]), cvt_bf16x2(acc[2], acc[3]),
                      cvt_bf16x2(acc[4], acc[5]), cvt_bf16x2(acc[6], acc[7]));
  dst[1] = make_uint4(cvt_bf16x2(acc[8], acc[9]), cvt_bf16x2(acc[10], acc[11]),
                      cvt_bf16x2(acc[12], acc[13]), cvt_bf16x2(acc[14], acc[15]));
  if ((lane & 7) == 0 && a.lse) a.lse[orow] = LSE;
}

// plan arrays, then the worker starts of the cut, then the split's two words
size_t plan_bytes(int S, int npairs_cap, int workers) {
  return sizeof(int) * ((size_t)npairs_cap + 1 + 3 * ((size_t)S + 1) + (size_t)workers + 1) + 24;
}

}  // namespace

// 3-D view of q as [Tq][Hq][128] bf16, boxes of (128/G) tokens x G heads x 64 dims,
// 128-byte swizzle: one box lands as 128 rows (token-major, head-minor) of 128 B.
bool make_q_map(CUtensorMap* map, const void* q, int64_t num_q_tokens, int Hq, int G, int QTb) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hq, (cuuint64_t)num_q_tokens};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)Hq * kHeadDim * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)QTb};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int tc_geometry(const pa_shape* sh, int64_t num_q_tokens, int max_q_len,
                       PrefillTcGeometry* g, int min_q_len, int max_ctas, bool tree) {
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  const int G = sh->num_q_heads / sh->num_kv_heads;
  if (G > kRowsT || (kRowsT % G != 0 && !tree) || max_q_len < min_q_len || max_q_len < 1) {
    g->enabled = false;
    g->ws_bytes = 0;
    return PA_OK;
  }
  const int QTb = kRowsT / G, S = sh->num_seqs;
  const int64_t cap1 = (int64_t)S * ((max_q_len + QTb - 1) / QTb);
  const int64_t cap2 = (num_q_tokens + QTb - 1) / QTb + S;
  const int64_t cap = cap1 < cap2 ? cap1 : cap2;
  if (cap > (1 << 20)) return PA_ERR_UNSUPPORTED;
  g->enabled = true;
  g->npairs_cap = (int)(cap < 1 ? 1 : cap);
  g->QTb = QTb;
  // one CTA per SM (shared memory and TMEM limit it to one)
  g->grid = max_ctas > 0 && max_ctas < dev.num_sms ? max_ctas : dev.num_sms;
  g->workers = g->grid;
  g->smem = 1024 + kOffPlan + round_up(plan_bytes(S, g->npairs_cap, g->workers), 16);
  if (g->smem > (size_t)dev.max_smem_optin) return PA_ERR_UNSUPPORTED;
  if (!raise_smem_limit(tree ? reinterpret_cast<const void*>(paged_prefill_tc_kernel<true>)
                             : reinterpret_cast<const void*>(paged_prefill_tc_kernel<false>)))
    return PA_ERR_CUDA;
  g->ws_lse = round_up(sizeof(float) * 2 * kRowsT * (size_t)g->workers, 256);
  g->ws_o = round_up(sizeof(float) * 2 * kRowsT * kHeadDim * (size_t)g->workers, 256);
  g->ws_bytes = g->ws_lse + g->ws_o + round_up(sizeof(int) * kDescInts * (size_t)g->workers, 256);
  return PA_OK;
}

int prefill_tc_geometry(const pa_shape* sh, int64_t num_q_tokens, int max_q_len,
                        PrefillTcGeometry* g, int min_q_len, int max_ctas) {
  return tc_geometry(sh, num_q_tokens, max_q_len, g, min_q_len, max_ctas, false);
}

int tree_tc_geometry(const pa_shape* sh, int64_t num_q_tokens, int max_q_len,
                     PrefillTcGeometry* g) {
  return tc_geometry(sh, num_q_tokens, max_q_len, g, 1, 0, true);
}

static int launch_tc(const PrefillTcGeometry& g, const pa_bf16* q, const pa_bf16* k_cache,
                     const pa_bf16* v_cache, TcArgs a, int64_t num_q_tokens, float scale,
                     const pa_shape* sh, void* workspace, cudaStream_t st, int parts) {
  const int G = sh->num_q_heads / sh->num_kv_heads;
  CUtensorMap tmq, tmk, tmv;
  const int64_t pool_rows = sh->num_blocks * sh->num_kv_heads * kBlock;
  if (!make_q_map(&tmq, q, num_q_tokens, sh->num_q_heads, G, g.QTb) ||
      !make_block_map(&tmk, k_cache, pool_rows) || !make_block_map(&tmv, v_cache, pool_rows))
    return PA_ERR_CUDA;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.S = sh->num_seqs;
  a.Hq = sh->num_q_heads;
  a.Hkv = sh->num_kv_heads;
  a.G = G;
  a.QTb = g.QTb;
  a.max_blocks = sh->max_blocks_per_seq;
  a.num_blocks = sh->num_blocks;
  a.num_q_tokens = num_q_tokens;
  a.npairs_cap = g.npairs_cap;
  a.num_workers = g.workers;
  char* ws = static_cast<char*>(workspace);
  a.part_lse = reinterpret_cast<float*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + g.ws_lse);
  a.desc = reinterpret_cast<int*>(ws + g.ws_lse + g.ws_o);
  if (parts & 1) {
    const cudaError_t e =
        a.mask ? launch_dependent(paged_prefill_tc_kernel<true>, dim3(g.grid), dim3(kThreadsT),
                                  g.smem, st, tmq, tmk, tmv, a)
               : launch_dependent(paged_prefill_tc_kernel<false>, dim3(g.grid), dim3(kThreadsT),
                                  g.smem, st, tmq, tmk, tmv, a);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  if (parts & 2) {
    // trees over few contexts: more than eight pieces to a segment on average
    const bool many = a.mask && (int64_t)g.workers > 8 * (int64_t)a.S * a.Hkv;
    const dim3 grid(g.workers, kRowsT / kFixRowsPerCta * (many ? kFixGroupsT : 1));
    if (launch_dependent(many ? prefill_tc_fixup_kernel<kFixGroupsT> : prefill_tc_fixup_kernel<1>,
                         grid, dim3(kFixThreads), 0, st, a) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  return PA_OK;
}

int launch_prefill_tc(const PrefillTcGeometry& g, const pa_bf16* q, const pa_bf16* k_cache,
                      const pa_bf16* v_cache, const int32_t* block_tables,
                      const int32_t* context_lens, const int32_t* cu_seqlens_q,
                      int64_t num_q_tokens, int causal, float scale, pa_bf16* out, float* lse,
                      const pa_shape* sh, void* workspace, cudaStream_t st, int min_q_len,
                      const RowsOut* rows, const int32_t* row_map, int parts, int split) {
  TcArgs a;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_seqlens_q = cu_seqlens_q;
  a.out = out;
  a.lse = lse;
  a.causal = causal ? 1 : 0;
  a.split = split > 0 ? g.grid : 0;
  a.min_lq = min_q_len;
  if (rows) a.rows = *rows;
  a.row_map = row_map;
  return launch_tc(g, q, k_cache, v_cache, a, num_q_tokens, scale, sh, workspace, st, parts);
}

int launch_tree_tc(const PrefillTcGeometry& g, const pa_bf16* q, const pa_bf16* k_cache,
                   const pa_bf16* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* cu_seqlens_q,
                   const uint32_t* tree_mask, int mask_words, int64_t num_q_tokens, float scale,
                   pa_bf16* out, float* lse, const pa_shape* sh, void* workspace,
                   cudaStream_t st) {
  TcArgs a;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_seqlens_q = cu_seqlens_q;
  a.out = out;
  a.lse = lse;
  a.causal = 0;
  a.split = 0;
  a.min_lq = 1;
  a.row_map = nullptr;
  a.mask = tree_mask;
  a.mask_words = mask_words;
  a.v_cache = v_cache;
  // windows of more than one tile on average: the second tile of a unit is seldom
  // missing (and costs nothing of the bandwidth that bounds the call where it is)
  a.pair = num_q_tokens * (sh->num_q_heads / sh->num_kv_heads) > (int64_t)kRowsT * 17 / 16 * sh->num_seqs;
  return launch_tc(g, q, k_cache, v_cache, a, num_q_tokens, scale, sh, workspace, st, 3);
}

unsigned take_error_word_prefill(cudaStream_t stream, int* rc) {
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
