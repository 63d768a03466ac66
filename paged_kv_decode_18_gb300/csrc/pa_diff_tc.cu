// pa_diff_tc.cu -- differential attention for longer windows (and for many query
// heads to a KV head) on the fifth-generation tensor cores, in tiles that a pair
// of SMs works on together (tcgen05, cta_group::2).
//
// Per key tile of 128 keys, each map needs S = Q K^T (128 dims) and O += P V with V
// twice as wide (256 dims): 6.3 M products per 128 query rows, 0.8 us of one SM's
// tensor core, against 96 KB of K and V. An SM takes its tiles in at 44 to 60
// GB/s (measured on the prefill kernel, whatever else was changed), so a tile of
// one SM would wait 2 us for its loads. A pair of SMs shares them: M = 256 query
// rows, 128 in each SM, and of every operand B each SM holds one half,
//   S: keys 0-63 of the tile in one SM, 64-127 in the other;
//   O: the value dims of KV head 2p in one SM, of 2p + 1 in the other,
// 48 KB per SM and tile, three stages of them beside two query tiles. One thread
// of the leading CTA issues each product for both.
//
// The flat work list is (query tile of 256 rows, pair of KV heads, map, key tile):
// the two maps of a pair follow one another, so a segment -- (query tile, pair) --
// is both. A worker (a cluster of two CTAs) has an equal range of it (PieceCut).
// Where a worker has a whole segment, the first map's normalised rows wait in its
// own scratch (read back by the threads that wrote them, from L2) and
// difference, norm and scale happen when the second map is done; segments that
// ranges cut leave both maps' partials for diff_tc_fixup_kernel.
//
// Roles in each CTA (12 warps): warp 0 loads query tiles and K, warp 10 V; in the
// leading CTA warp 1 issues S and warp 11 O; warps 2-9 are the softmax, two
// threads to a query row, one per 64-key half. O has the whole 256 columns that
// S/P leave of tensor memory, one accumulator for both halves, so the halves
// agree on the row's reference: they exchange their maxima every tile. The
// reference moves only when a maximum grows by more than 2^32 (exact either way).
#include <cudaTypedefs.h>

#include "pa_diff.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kRowsT = 128;                   // query rows of one CTA
constexpr int kKeysT = 128;                   // keys per tile
constexpr int kBlocksT = kKeysT / kBlock;
constexpr int kHalfT = kRowsT * 128;          // one 64-dim half of a 128-row bf16 operand
constexpr int kQBytes = 2 * kHalfT;           // a query tile: 32 KB
constexpr int kKBytes = kBlocksT / 2 * kTileBytes;  // this CTA's half of the keys: 16 KB
constexpr int kVBytes = kBlocksT * kTileBytes;      // this CTA's value head: 32 KB
constexpr int kStageT = kKBytes + kVBytes;
constexpr int kMaxStagesT = 3;
constexpr int kSoftmaxWarps = 8;              // warps 2-9
constexpr int kVWarp = 2 + kSoftmaxWarps;
constexpr int kPvWarp = kVWarp + 1;
constexpr int kThreadsT = 128 + kSoftmaxWarps * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;               // S/P buffers at columns 0 and 128, O at 256 .. 511
constexpr int kSegCost4 = 6;                  // a segment start in quarters of a key tile
constexpr int kTDesc = 8;
// The reference of a row's exponentials moves only when its maximum has grown by more
// than this power of two: weights up to 2^32 are as exact in bf16 and fp32 as those below
// 1, and leave 95 powers of two for V and the sums. (At 2^8, with one key in a hundred
// eight times as long as the others, nearly every warp rescaled its 256 columns of O in
// every tile, at 700 clocks each.)
constexpr float kRescaleLog2 = 32.f;

enum : int {
  B_QFULL = 0,                        // [2], leader: both CTAs' query rows
  B_QEMPTY = 2,                       // [2], both
  B_KFULL = 4,                        // [3], leader: both CTAs' keys
  B_KEMPTY = 7,                       // [3], both
  B_VFULL = 10,                       // [3], each CTA its own values
  B_VEMPTY = 13,                      // [3], both
  B_SFULL = 16,                       // [2], both
  B_SFREE = 18,                       // [2], both: the product that read this buffer's P is done
  // [2], leader: all softmax warps of both. Two, since a warp may be through with the
  // next tile's exponentials before another has arrived for this one
  B_PFULL = 20,
  B_XCH = 22,                         // [4]: the two warps of 32 rows, every exchange a phase
  kNumBarsT = 26
};

// shared memory past the operands
constexpr int kOffBars = 0;
constexpr int kOffSlot = kNumBarsT * 8;
constexpr int kOffAbort = kOffSlot + 4;
constexpr int kOffBad = kOffAbort + 4;
constexpr int kOffXch = 256;                       // [2][2 halves][128] floats
constexpr int kOffPlanT = kOffXch + 2 * 2 * kRowsT * 4;
static_assert(kOffBad + 4 <= kOffXch, "barrier area");

struct DiffTcArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_seqlens_q;
  const uint16_t* v_cache;
  DiffOut o;
  float scale_log2;
  int S, Hq, Hkv, G, QTb, max_blocks;
  int64_t num_blocks;
  int64_t num_q_tokens;
  int causal;
  int npairs_cap;
  int num_workers;
  int min_lq;
  int nstage;
  float* part_o;    // [workers * 2 pieces][2 maps][256 rows][256]
  float* part_lse;  // [workers * 2 pieces][2 maps][256 rows]
  int* desc;        // [workers][kTDesc]
};

// ---------------------------------------------------------------------------
// pair-of-CTAs wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// this CTA's shared address, in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}
// Arrives on a barrier of either CTA. What it tells of is in tensor memory (ordered by
// the tcgen05 fences); a thread that has written shared memory for the peer's products
// to read makes a fence of the cluster's scope first. (An arrive that releases at that
// scope costs every softmax warp 600 clocks a tile.)
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
// tiled copies whose completion counts on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_block(uint32_t dst, const CUtensorMap* map, int group,
                                               uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate));
}
// the barrier at this address of both CTAs
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__global__ void __launch_bounds__(kThreadsT, 1)
    paged_diff_tc_kernel(const __grid_constant__ CUtensorMap tmq,
                         const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv, const DiffTcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank();
  const int nstage = a.nstage;
  unsigned char* stages = smem + 2 * kQBytes;  // stage s: K at s * kStageT, V after it
  unsigned char* rest = stages + nstage * kStageT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rest + kOffBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rest + kOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(rest + kOffAbort);
  // a window row of V held an infinity or a NaN (set once in both CTAs, kept)
  volatile int* bad_v = reinterpret_cast<volatile int*>(rest + kOffBad);
  float* xch = reinterpret_cast<float*>(rest + kOffXch);
  const int S = a.S, Hkv = a.Hkv, Hp = a.Hkv >> 1, G = a.G, QTb = a.QTb;
  auto bar = [&](int i) { return smem_addr(&bars[i]); };

  PlanSmem P;
  P.pair_off = reinterpret_cast<int*>(rest + kOffPlanT);
  P.seq_pair = P.pair_off + (a.npairs_cap + 1);
  P.ctx = P.seq_pair + (S + 1);
  P.qstart = P.ctx + S;
  int* cut_at = P.qstart + (S + 1);

  if (tid == 0) {
    for (int i = 0; i < kNumBarsT; ++i)
      mbar_init(bar(i), i >= B_XCH ? 2 : i == B_PFULL || i == B_PFULL + 1 ? 2 * kSoftmaxWarps : 1);
    *abort_flag = 0;
    *bad_v = 0;
    mbar_fence_init();
  }
  if (tid == 32) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  PlanInputs in;
  in.context_lens = a.context_lens;
  in.cu_seqlens_q = a.cu_seqlens_q;
  in.S = S;
  in.Hkv = Hkv;
  in.max_ctx = a.max_blocks * kBlock;
  in.qtile = 2 * QTb;
  in.causal = a.causal;
  in.npairs_cap = a.npairs_cap;
  in.num_q_rows = a.num_q_tokens;
  in.key_tile = kKeysT;
  in.min_lq = a.min_lq;
  in.skip_empty = a.cu_seqlens_q == nullptr;
  build_plan(in, P, nullptr);
  // segments are pairs of KV heads: n tiles of the first map, then n of the second
  const PieceCut cut = build_piece_cut(P, Hp, a.num_workers, kSegCost4, cut_at);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // a sequence of the single-query form with an empty context has no tiles
  if (!a.cu_seqlens_q) {
    for (int s = blockIdx.x; s < S; s += gridDim.x) {
      if (P.ctx[s] != 0) continue;
      uint4* row = reinterpret_cast<uint4*>(a.o.out + (int64_t)s * (a.Hq / 2) * kDiffDim);
      for (int i = tid; i < a.Hq / 2 * (kDiffDim / 8); i += blockDim.x)
        row[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.o.lse)
        for (int i = tid; i < a.Hq; i += blockDim.x) a.o.lse[(int64_t)s * a.Hq + i] = neg_inf();
    }
  }

  const int w = blockIdx.x >> 1;  // the worker: a cluster
  const bool work = P.total > 0 && w < cut.nw;
  if (tid == 32 * kPvWarp && rank == 0) {
    int* d = a.desc + (size_t)w * kTDesc;
    MergeJob j;
    j.valid = false;
    if (work) j = merge_job_of(P, S, Hp, w, cut.nw, cut);
    d[0] = j.valid ? j.s : -1;
    if (j.valid) {
      d[1] = j.qt;
      d[2] = j.h;
      d[3] = j.last;
      d[4] = j.slot_prev;
      d[5] = P.qstart[j.s];
      d[6] = P.qstart[j.s + 1] - P.qstart[j.s];
    }
  }
  if (!work) return;  // both CTAs of the cluster
  const int R0 = cut.start(w), R1 = cut.start(w + 1);
  if (R0 >= R1) return;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // the peer's barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](int b, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(b), parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!*abort_flag) {
      if (mbar_try_wait(bar(b), parity)) return true;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        flag_error(PA_DEVERR_PIPE_TIMEOUT);
        *abort_flag = 1;
      }
    }
    return false;
  };
  // the same for a whole warp: its lanes go on or leave together
  auto wait_all = [&](int b, uint32_t parity) -> bool {
    return __all_sync(kFull, wait(b, parity));
  };
  // map and key tile of a segment's tile b
  auto map_of = [](const TilePos& t) { return 2 * t.b >= t.nt ? 1 : 0; };
  auto key_tile_of = [&](const TilePos& t) { return t.b - map_of(t) * (t.nt >> 1); };
  // whether a tile begins a map of a piece
  auto begins = [&](const TilePos& t, int idx) { return idx == R0 || key_tile_of(t) == 0; };

  if (warp == 0 || warp == kVWarp) {
    // ------------------------------------------------------------------ producers
    const bool is_k = warp == 0;
    TilePos t = locate(P, S, Hp, R0);
    auto nblocks_of = [&](const TilePos& tp) {
      const int nb_seq = (P.ctx[tp.s] + kBlock - 1) / kBlock;
      return min(kBlocksT, nb_seq - key_tile_of(tp) * kBlocksT);
    };
    auto fetch_ids = [&](const TilePos& tp) -> int {
      return lane < nblocks_of(tp)
                 ? a.block_tables[(size_t)tp.s * a.max_blocks + key_tile_of(tp) * kBlocksT + lane]
                 : 0;
    };
    const uint32_t lead_q = in_cta(bar(B_QFULL), 0), lead_k = in_cta(bar(B_KFULL), 0);
    int ids = fetch_ids(t);
    int qn = 0, st = 0, i = 0;
    uint32_t use = 0;  // how often the ring has come round
    bool fine = true;
    for (int idx = R0; idx < R1; ++idx, ++i) {
      const int map = map_of(t);
      if (is_k && begins(t, idx)) {
        const int qs = qn & 1;
        if (qn >= 2 && !wait_all(B_QEMPTY + qs, (uint32_t)((qn >> 1) - 1) & 1u)) {
          fine = false;
          break;
        }
        if (lane == 0) {
          // this CTA's query rows (past the window's: zeros, or a neighbour's rows that
          // nothing reads the results of)
          const int z = P.qstart[t.s] + (t.qt * 2 + rank) * QTb;
          const uint32_t qd = smem_addr(smem + qs * kQBytes);
          const int y = (2 * t.h + map) * G;
          if (rank == 0)
            mbar_arrive_expect_tx(bar(B_QFULL + qs), 2u * (uint32_t)(QTb * G) * 256u);
          tma_pair_3d(qd, &tmq, 0, y, z, lead_q + qs * 8);
          tma_pair_3d(qd + kHalfT, &tmq, 64, y, z, lead_q + qs * 8);
        }
        ++qn;
      }
      const int nb = nblocks_of(t);
      int my_id = ids;
      const int h0 = 2 * t.h;
      if (idx + 1 < R1) {  // block ids of the next tile, one tile ahead
        advance(P, S, Hp, t);
        ids = fetch_ids(t);
      }
      if (lane < nb && (my_id < 0 || (int64_t)my_id >= a.num_blocks)) {
        if (is_k && rank == 0) flag_error(PA_DEVERR_BLOCK_RANGE);
        my_id = 0;
      }
      // the stage is free once the product that read it is done
      if (use > 0 && !wait_all((is_k ? B_KEMPTY : B_VEMPTY) + st, (use - 1) & 1u)) {
        fine = false;
        break;
      }
      unsigned char* base = stages + st * kStageT;
      if (is_k) {
        if (lane == 0 && rank == 0)
          mbar_arrive_expect_tx(bar(B_KFULL + st), (uint32_t)nb * (uint32_t)kTileBytes);
        __syncwarp();
        const int half = lane - rank * (kBlocksT / 2);  // this CTA's four blocks
        if (half >= 0 && half < kBlocksT / 2 && lane < nb)
          tma_pair_block(smem_addr(base + half * kTileBytes), &tmk,
                         (int)(((int64_t)my_id * Hkv + h0 + map) * (kBlock / 8)), lead_k + st * 8);
      } else {
        if (lane == 0) mbar_arrive_expect_tx(bar(B_VFULL + st), (uint32_t)nb * (uint32_t)kTileBytes);
        __syncwarp();
        if (lane < nb)
          tma_load_block(smem_addr(base + kKBytes + lane * kTileBytes), &tmv,
                         (int)(((int64_t)my_id * Hkv + h0 + rank) * (kBlock / 8)), bar(B_VFULL + st));
      }
      __syncwarp();
      if (++st == nstage) {
        st = 0;
        ++use;
      }
    }
    if (!fine && (rank == 0 || !is_k)) {
      // copies in flight land (within the limit) before the CTA leaves; the leading
      // CTA's barriers count the peer's K and Q as well
      for (int k = i < nstage ? i : nstage; k > 0; --k) {
        if (--st < 0) {
          st = nstage - 1;
          --use;
        }
        mbar_wait_bounded(bar((is_k ? B_KFULL : B_VFULL) + st), use & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    if (lane == 0 && rank == 0) {
      const uint32_t idS = f16_idesc(2 * kRowsT, kKeysT, 0);
      const uint64_t desc_q = sw128_desc(smem_addr(smem), 16, 1024);
      const uint64_t desc_k = sw128_desc(smem_addr(stages), 16, 2048);
      TilePos t = locate(P, S, Hp, R0);
      int qn = 0, qs = 0, st = 0;
      uint32_t use = 0;
      for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
        if (begins(t, idx)) {
          qs = qn & 1;
          if (!wait(B_QFULL + qs, (uint32_t)(qn >> 1) & 1u)) break;
          ++qn;
        }
        const int sb = i & 1;
        if (!wait(B_KFULL + st, use & 1u)) break;
        // the S/P buffer is free once the product that read P of tile i-2 is done
        if (i >= 2 && !wait(B_SFREE + sb, (uint32_t)((i >> 1) - 1) & 1u)) break;
        tc_fence_after();
        const uint64_t dq = desc_q + (uint64_t)(qs * (kQBytes >> 4));
        const uint64_t dk = desc_k + (uint64_t)(st * (kStageT >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          pair_mma(tmem + (uint32_t)sb * 128u,
                   dq + (uint64_t)(((k >> 2) * kHalfT + (k & 3) * 32) >> 4),
                   dk + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), idS, k > 0);
        pair_commit(bar(B_SFULL + sb));
        pair_commit(bar(B_KEMPTY + st));
        if (++st == nstage) {
          st = 0;
          ++use;
        }
        if (idx + 1 < R1) advance(P, S, Hp, t);
        if (idx + 1 >= R1 || key_tile_of(t) == 0) pair_commit(bar(B_QEMPTY + qs));
      }
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ O += P V
    if (lane == 0 && rank == 0) {
      const uint32_t idPV = f16_idesc(2 * kRowsT, kDiffDim, 1);
      const uint64_t desc_v = sw128_desc(smem_addr(stages + kKBytes), 1024, 2048);
      TilePos t = locate(P, S, Hp, R0);
      int st = 0;
      for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
        const bool first = begins(t, idx);
        const uint32_t sb = (uint32_t)(i & 1);
        // (a softmax warp of either CTA has seen its values land before it arrives)
        if (!wait(B_PFULL + (int)sb, (uint32_t)(i >> 1) & 1u)) break;
        tc_fence_after();
        const uint64_t dv = desc_v + (uint64_t)(st * (kStageT >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          pair_mma_ts(tmem + kColO, tmem + sb * 128u + (uint32_t)((k >> 2) * 64 + (k & 3) * 8),
                      dv + (uint64_t)(k * (kTileBytes >> 4)), idPV, (k > 0 || !first) ? 1u : 0u);
        pair_commit(bar(B_VEMPTY + st));
        pair_commit(bar(B_SFREE + (int)sb));
        if (++st == nstage) st = 0;
        if (idx + 1 < R1) advance(P, S, Hp, t);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax
    const int q4 = warp & 3;
    const int hf = (warp - 2) >> 2;
    const int r = q4 * 32 + lane;  // this thread's query row (= TMEM lane)
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tO = tmem + lane_base + kColO + (uint32_t)hf * 128u;  // its 128 output dims
    const uint32_t lead_p = in_cta(bar(B_PFULL), 0);
    const float sc = a.scale_log2;
    uint32_t xphase = 0;
    // Gives `mine` to the thread of the row's other half and takes its value.
    auto exchange = [&](float mine, float& other) -> bool {
      float* x = xch + (xphase & 1u) * (2 * kRowsT);
      x[hf * kRowsT + r] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_XCH + q4));
      if (!wait_all(B_XCH + q4, xphase & 1u)) return false;
      ++xphase;
      other = x[(hf ^ 1) * kRowsT + r];
      return true;
    };
    TilePos t = locate(P, S, Hp, R0);
    float m_ref = neg_inf(), l = 0.f;
    int lim = 0, c = 0, lq = 0, tok = 0, piece_b0 = 0, st = 0;
    uint32_t use = 0;
    bool valid = false, piece_first = true;
    // A finished map's O stays in tensor memory until the next tile's exponentials are
    // done (its last product completes meanwhile); then it is written out.
    struct Pending {
      bool on, valid, whole, last_of_piece;
      int s, h, map, b0, b1, n;  // the piece's tiles b0 .. b1 of a segment of 2n
      int64_t qtok;
      int k0, k1, vis;           // its keys, and the row's limit
      size_t slot;
      float m, l;
    } pend;
    pend.on = false;
    auto flush = [&]() -> bool {
      float l_o = 0.f;
      if (!exchange(pend.l, l_o)) return false;
      const float lt = hf == 0 ? pend.l + l_o : l_o + pend.l;
      // (a NaN score's NaN goes on into the row's results)
      const float inv = lt != 0.f ? 1.f / lt : 0.f;
      const float lse_v = lt != 0.f ? (pend.m + lg2(lt)) * kLn2 : neg_inf();
      const int head = pend.h * G + r % G;
      const bool merge = pend.whole && pend.map == 1;  // both maps are here: the row's output
      const float lam = merge && pend.valid ? a.o.lambdas[head] : 0.f;
      const int row = rank * kRowsT + r;
      float* part = a.part_o + ((pend.slot * 2 + pend.map) * (2 * kRowsT) + row) * kDiffDim + hf * 128;
      const float* first_map = a.part_o + ((pend.slot * 2) * (2 * kRowsT) + row) * kDiffDim + hf * 128;
      float squares = 0.f;
      // twice over a row's dims where it is normed: sum of squares, then the output
      const int passes = merge && a.o.weight ? 2 : 1;
      float factor = a.o.gain;
      for (int pass = 0; pass < passes; ++pass) {
        const bool out = merge && pass == passes - 1;
        if (pass == 1) {
          float sq_o = 0.f;
          if (!exchange(squares, sq_o)) return false;
          factor = diff_factor(a.o, hf == 0 ? squares + sq_o : sq_o + squares);
        }
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t u[32];
          __syncwarp();
          tmem_ld32(tO + (uint32_t)cc * 32u, u);
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(u[j]);
          if (*bad_v && pend.valid) {
            // infinities and NaNs of window rows entered the product as zeros (they must
            // not reach queries that do not see their row): they join the rows that see
            // them here
            const int lqp = P.qstart[pend.s + 1] - P.qstart[pend.s];
            const int p0 = P.ctx[pend.s] - lqp;
            const int k1 = min(pend.vis, pend.k1);
            for (int k = max(p0 + 1, pend.k0); k < k1; ++k) {
              const int phys = a.block_tables[(size_t)pend.s * a.max_blocks + k / kBlock];
              if (phys < 0 || (int64_t)phys >= a.num_blocks) continue;
              const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                  a.v_cache + ((((int64_t)phys * Hkv + 2 * pend.h + hf) * kBlock) + k % kBlock) *
                                  kHeadDim + cc * 32);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t wv = vr[j], fin = bf2_finite_part(wv);
                if ((wv ^ fin) & 0x7f80u) y[2 * j] += bf_lo(wv);
                if ((wv ^ fin) & 0x7f800000u) y[2 * j + 1] += bf_hi(wv);
              }
            }
          }
          if (!merge) {
            if (pend.valid) {
              float4* dst = reinterpret_cast<float4*>(part + cc * 32);
#pragma unroll
              for (int q = 0; q < 8; ++q)
                dst[q] = make_float4(__fmul_rn(y[4 * q], inv), __fmul_rn(y[4 * q + 1], inv),
                                     __fmul_rn(y[4 * q + 2], inv), __fmul_rn(y[4 * q + 3], inv));
            }
            continue;
          }
          if (!pend.valid) continue;
          const float4* src = reinterpret_cast<const float4*>(first_map + cc * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = src[q];
            y[4 * q] = diff_value(x.x, 1.f, y[4 * q], inv, lam);
            y[4 * q + 1] = diff_value(x.y, 1.f, y[4 * q + 1], inv, lam);
            y[4 * q + 2] = diff_value(x.z, 1.f, y[4 * q + 2], inv, lam);
            y[4 * q + 3] = diff_value(x.w, 1.f, y[4 * q + 3], inv, lam);
          }
          if (!out) {
#pragma unroll
            for (int j = 0; j < 32; ++j) squares = fmaf(y[j], y[j], squares);
            continue;
          }
          if (a.o.weight) {
            const float4* wt = reinterpret_cast<const float4*>(a.o.weight + hf * 128 + cc * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 x = wt[q];
              y[4 * q] *= factor * x.x;
              y[4 * q + 1] *= factor * x.y;
              y[4 * q + 2] *= factor * x.z;
              y[4 * q + 3] *= factor * x.w;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] *= factor;
          }
          uint4* dst = reinterpret_cast<uint4*>(
              a.o.out + (pend.qtok * (a.Hq / 2) + head) * kDiffDim + hf * 128 + cc * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(cvt_bf16x2(y[8 * q + 0], y[8 * q + 1]),
                                cvt_bf16x2(y[8 * q + 2], y[8 * q + 3]),
                                cvt_bf16x2(y[8 * q + 4], y[8 * q + 5]),
                                cvt_bf16x2(y[8 * q + 6], y[8 * q + 7]));
        }
      }
      if (hf == 0 && pend.valid) {
        if (pend.whole) {
          if (a.o.lse)
            a.o.lse[pend.qtok * a.Hq + (int64_t)(2 * pend.h + pend.map) * G + r % G] = lse_v;
        } else {
          float* pl = a.part_lse + (pend.slot * 2) * (2 * kRowsT) + row;
          pl[pend.map * (2 * kRowsT)] = lse_v;
          // a map that the piece has no tile of weighs nothing in the merge
          if (pend.map == 0 && pend.last_of_piece) pl[2 * kRowsT] = neg_inf();
          if (pend.map == 1 && pend.b0 >= pend.n) pl[0] = neg_inf();
        }
      }
      pend.on = false;
      return true;
    };
    int i = 0;
    for (int idx = R0; idx < R1; ++idx, ++i) {
      const int n = t.nt >> 1, map = map_of(t), kt = t.b - map * n;
      const bool first = idx == R0 || kt == 0;
      const bool piece_last = idx == R1 - 1 || t.b == t.nt - 1;
      const bool last = piece_last || kt == n - 1;
      if (idx == R0 || t.b == 0) {
        c = P.ctx[t.s];
        lq = P.qstart[t.s + 1] - P.qstart[t.s];
        tok = (t.qt * 2 + rank) * QTb + r / G;
        valid = tok < lq && r < QTb * G;
        lim = valid ? (a.causal ? c - lq + tok + 1 : c) : 0;
        piece_b0 = t.b;
        piece_first = idx == R0;
      }
      if (first) {
        m_ref = neg_inf();
        l = 0.f;
      }
      const int sb = i & 1;
      if (!wait_all(B_SFULL + sb, (uint32_t)(i >> 1) & 1u)) break;
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
      const int key0 = kt * kKeysT, kb = key0 + hf * 64;  // first key of the tile, of this half
      if (kb + 64 > lim) {  // the causal diagonal or the end of the context
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (kb + 2 * j >= lim) x[j].x = neg_inf();
          if (kb + 2 * j + 1 >= lim) x[j].y = neg_inf();
        }
      }
      float mx = fmaxf(x[0].x, x[0].y);
      {
        float m4[4] = {mx, neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int j = 1; j < 32; ++j)
          asm("max.f32 %0, %1, %2, %3;"
              : "=f"(m4[j & 3])
              : "f"(x[j].x), "f"(x[j].y), "f"(m4[j & 3]));
        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      float mo;
      if (!exchange(mx, mo)) break;
      mx = fmaxf(mx, mo);  // the same in both halves of the row
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
      // tcgen05.mma wants of both operands: a weight is off by at most 2^-8 of itself.
      // The sum l, and with it lse, is of the unrounded ones.
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
      // the previous product must be done before O is rescaled or the previous map's O is
      // read. Its P buffer says so: the product before it on that buffer is done, or this
      // tile's S would not be there, so its phase is not mistaken for an earlier one. (The
      // tensor-memory accesses are warp-wide: the whole warp rescales when one of its
      // rows has to, the others by 1.)
      const bool scale_o = __any_sync(kFull, rescale) && !first;
      if (scale_o || pend.on) {
        if (!wait_all(B_SFREE + (sb ^ 1), (uint32_t)((i - 1) >> 1) & 1u)) break;
        tc_fence_after();
      }
      if (pend.on && !flush()) break;
      if (scale_o) {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t v[32];
          tmem_ld32(tO + (uint32_t)cc * 32u, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
          tmem_st32(tO + (uint32_t)cc * 32u, v);
        }
      }
      // P row r, keys of half hf, over the S columns this thread has read
      __syncwarp();
      tmem_st32(tS, pk);
      tmem_wait_st();
      // keys past the context may hold anything (even NaN): zero their V rows so that P
      // = 0 never meets them; of the window's rows, which only some queries see, the
      // infinities and NaNs (thread (r, hf) has half hf of key row r of this CTA's head)
      // (Only one warp of a CTA sees to it that V is there before the product begins; a
      // wait costs 130 clocks even when it is over.)
      const int vsafe = a.causal ? c - lq + 1 : c;  // rows before it enter as they are
      if ((warp == 2 || key0 + kKeysT > vsafe) && !wait_all(B_VFULL + st, use & 1u)) break;
      if (key0 + kKeysT > vsafe && key0 + r >= vsafe) {
        unsigned char* vrow = stages + st * kStageT + kKBytes + (r >> 3) * 2048 + hf * 1024 +
                              (r & 7) * 128;
        if (key0 + r >= c) {
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(vrow + ch * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          fence_cluster();
        } else {
          bool bad = false;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(vrow + ch * 16);
            bad = bad || bf2_nonfinite(x4.x) || bf2_nonfinite(x4.y) || bf2_nonfinite(x4.z) ||
                  bf2_nonfinite(x4.w);
          }
          if (bad) {
            for (int ch = 0; ch < 8; ++ch) {
              uint4 x4 = *reinterpret_cast<const uint4*>(vrow + ch * 16);
              x4.x = bf2_finite_part(x4.x);
              x4.y = bf2_finite_part(x4.y);
              x4.z = bf2_finite_part(x4.z);
              x4.w = bf2_finite_part(x4.w);
              *reinterpret_cast<uint4*>(vrow + ch * 16) = x4;
            }
            fence_proxy_async_smem();
            // both CTAs write dims of both heads out
            const uint32_t flag = smem_addr(rest + kOffBad);
            for (uint32_t to = 0; to < 2; ++to)
              asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(
                               in_cta(flag, to)),
                           "r"(1u)
                           : "memory");
            fence_cluster();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_in_cluster(lead_p + sb * 8);
      if (++st == nstage) {
        st = 0;
        ++use;
      }

      if (last) {
        pend.on = true;
        pend.valid = valid;
        pend.whole = piece_b0 == 0 && (map == 0 ? cut.start(w + 1) - idx > n : t.b == t.nt - 1);
        pend.last_of_piece = piece_last;
        pend.s = t.s;
        pend.h = t.h;
        pend.map = map;
        pend.b0 = piece_b0;
        pend.b1 = t.b;
        pend.n = n;
        pend.qtok = (int64_t)P.qstart[t.s] + tok;
        pend.k0 = (map == 0 || piece_b0 < n ? (map == 0 ? piece_b0 : 0) : piece_b0 - n) * kKeysT;
        pend.k1 = key0 + kKeysT;
        pend.vis = lim;
        pend.slot = (size_t)w * 2 + (piece_first ? 0 : 1);
        pend.m = m_ref;
        pend.l = l;
      }
      if (idx + 1 < R1) advance(P, S, Hp, t);
    }
    if (pend.on && wait_all(B_SFREE + ((i - 1) & 1), (uint32_t)((i - 1) >> 1) & 1u)) {
      tc_fence_after();
      flush();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_meet();  // nothing of the pair reaches into a CTA that has left
  tc_fence_after();
  __syncwarp();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

// Merge the pieces of the (query tile, pair) segments that the ranges cut, both
// maps, then difference, norm and scale. Grid (worker boundary, chunk of rows): a
// warp takes a row at a time, eight of its 256 dims a lane.
constexpr int kTFixWarps = 8;
constexpr int kTFixChunks = 16;  // 256 rows: 16 of them a CTA

__global__ void __launch_bounds__(kTFixWarps * 32)
    diff_tc_fixup_kernel(const DiffTcArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x;
  const int* d = a.desc + (size_t)w * kTDesc;
  if (__ldcg(d) < 0) return;
  const int qt = __ldcg(d + 1), h = __ldcg(d + 2), last = __ldcg(d + 3), slot_prev = __ldcg(d + 4),
            q0 = __ldcg(d + 5), lq = __ldcg(d + 6);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int npieces = last - w + 2;  // workers w-1 .. last
  constexpr int kRowsPerCta = 2 * kRowsT / kTFixChunks;
  for (int row = blockIdx.y * kRowsPerCta + warp; row < (int)(blockIdx.y + 1) * kRowsPerCta;
       row += kTFixWarps) {
    const int r = row & (kRowsT - 1);
    const int tok = (qt * 2 + row / kRowsT) * a.QTb + r / a.G;
    if (r >= a.QTb * a.G || tok >= lq) continue;
    float y[8], lse[2];
    float a0[8];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      float m = neg_inf(), sum = 0.f, acc[8];
      bool nan = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      for (int i0 = 0; i0 < npieces; i0 += 4) {
        float li[4];
        float4 v[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          li[u] = neg_inf();
          v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + u < npieces) {
            const size_t sl = (size_t)(w - 1 + i0 + u) * 2 + (i0 + u == 0 ? slot_prev : 0);
            const size_t at = (sl * 2 + map) * (2 * kRowsT) + row;
            li[u] = __ldcg(a.part_lse + at);
            const float4* src = reinterpret_cast<const float4*>(a.part_o + at * kDiffDim + lane * 8);
            if (li[u] != neg_inf()) {
              v[u][0] = __ldcg(src);
              v[u][1] = __ldcg(src + 1);
            }
          }
        }
        const float mn = fmaxf(fmaxf(m, fmaxf(li[0], li[1])), fmaxf(li[2], li[3]));
#pragma unroll
        for (int u = 0; u < 4; ++u) nan = nan || li[u] != li[u];
        if (mn == neg_inf()) continue;
        const float shrink = m == neg_inf() ? 0.f : ex2((m - mn) * kLog2e);
        sum *= shrink;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] *= shrink;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wt = li[u] == neg_inf() ? 0.f : ex2((li[u] - mn) * kLog2e);
          sum += wt;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            acc[4 * k + 0] = fmaf(wt, v[u][k].x, acc[4 * k + 0]);
            acc[4 * k + 1] = fmaf(wt, v[u][k].y, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(wt, v[u][k].z, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(wt, v[u][k].w, acc[4 * k + 3]);
          }
        }
        m = mn;
      }
      if (nan) m = sum = __int_as_float(0x7fc00000);
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      lse[map] = sum != 0.f ? m + lg2(sum) * kLn2 : neg_inf();
      const float lam = a.o.lambdas[h * a.G + r % a.G];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (map == 0)
          a0[j] = __fmul_rn(acc[j], inv);
        else
          y[j] = diff_value(a0[j], 1.f, acc[j], inv, lam);
      }
    }
    float squares = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) squares = fmaf(y[j], y[j], squares);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) squares += __shfl_xor_sync(kFull, squares, o);
    const float f = diff_factor(a.o, squares);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= a.o.weight ? f * a.o.weight[lane * 8 + j] : f;
    const int head = h * a.G + r % a.G;
    const int64_t qtok = (int64_t)q0 + tok;
    *reinterpret_cast<uint4*>(a.o.out + (qtok * (a.Hq / 2) + head) * kDiffDim + lane * 8) =
        make_uint4(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]), cvt_bf16x2(y[4], y[5]),
                   cvt_bf16x2(y[6], y[7]));
    if (a.o.lse && lane == 0) {
      float* l = a.o.lse + qtok * a.Hq + (int64_t)(2 * h) * a.G + r % a.G;
      l[0] = lse[0];
      l[a.G] = lse[1];
    }
  }
}

}  // namespace

int diff_tc_geometry(const pa_shape* sh, int64_t num_q_tokens, int max_q_len, int min_q_len,
                     DiffTcGeometry* g) {
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  const int G = sh->num_q_heads / sh->num_kv_heads;
  g->enabled = max_q_len >= min_q_len;
  g->ws_bytes = 0;
  if (!g->enabled) return PA_OK;
  const int S = sh->num_seqs, unit = 2 * (kRowsT / G);
  const int64_t cap1 = (int64_t)S * (((int64_t)max_q_len + unit - 1) / unit);
  const int64_t cap2 = (num_q_tokens + unit - 1) / unit + S;
  const int64_t cap = cap1 < cap2 ? cap1 : cap2;
  if (cap > (1 << 20)) return PA_ERR_UNSUPPORTED;
  g->npairs_cap = (int)(cap < 1 ? 1 : cap);
  g->min_lq = min_q_len;
  g->workers = dev.num_sms / 2;
  const size_t plan =
      sizeof(int) * ((size_t)g->npairs_cap + 1 + 3 * ((size_t)S + 1) + (size_t)g->workers + 1);
  for (g->nstage = kMaxStagesT; g->nstage >= 2; --g->nstage) {
    g->smem = 1024 + 2 * kQBytes + (size_t)g->nstage * kStageT + kOffPlanT + round_up(plan, 16);
    if (g->smem <= (size_t)dev.max_smem_optin) break;
  }
  if (g->nstage < 2) return PA_ERR_UNSUPPORTED;
  // as many clusters as are resident at once
  int clusters = 0;
  if (!cluster_occupancy(reinterpret_cast<const void*>(paged_diff_tc_kernel), kThreadsT, g->smem, 2,
                         &clusters) ||
      clusters <= 0)
    return PA_ERR_CUDA;
  if (clusters < g->workers) g->workers = clusters;
  g->ws_lse = round_up(sizeof(float) * 8 * kRowsT * (size_t)g->workers, 256);
  g->ws_o = round_up(sizeof(float) * 8 * kRowsT * kDiffDim * (size_t)g->workers, 256);
  g->ws_bytes = g->ws_lse + g->ws_o + round_up(sizeof(int) * kTDesc * (size_t)g->workers, 256);
  return PA_OK;
}

int launch_diff_tc(const DiffTcGeometry& g, const pa_bf16* q, const pa_bf16* k_cache,
                   const pa_bf16* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* cu_seqlens_q, int64_t num_q_tokens,
                   int causal, float scale, const DiffOut& out, const pa_shape* sh, void* workspace,
                   cudaStream_t st) {
  const int G = sh->num_q_heads / sh->num_kv_heads, QTb = kRowsT / G;
  CUtensorMap tmq, tmk, tmv;
  const int64_t pool_rows = sh->num_blocks * sh->num_kv_heads * kBlock;
  if (!make_q_map(&tmq, q, num_q_tokens, sh->num_q_heads, G, QTb) ||
      !make_block_map(&tmk, k_cache, pool_rows) || !make_block_map(&tmv, v_cache, pool_rows))
    return PA_ERR_CUDA;
  DiffTcArgs a = {};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_seqlens_q = cu_seqlens_q;
  a.v_cache = v_cache;
  a.o = out;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.S = sh->num_seqs;
  a.Hq = sh->num_q_heads;
  a.Hkv = sh->num_kv_heads;
  a.G = G;
  a.QTb = QTb;
  a.max_blocks = sh->max_blocks_per_seq;
  a.num_blocks = sh->num_blocks;
  a.num_q_tokens = num_q_tokens;
  a.causal = causal;
  a.npairs_cap = g.npairs_cap;
  a.num_workers = g.workers;
  a.min_lq = g.min_lq;
  a.nstage = g.nstage;
  char* ws = static_cast<char*>(workspace);
  a.part_lse = reinterpret_cast<float*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + g.ws_lse);
  a.desc = reinterpret_cast<int*>(ws + g.ws_lse + g.ws_o);
  if (launch_dependent_cluster(paged_diff_tc_kernel, dim3(2 * g.workers), dim3(kThreadsT), g.smem, 2,
                               st, tmq, tmk, tmv, a) != cudaSuccess)
    return PA_ERR_CUDA;
  if (launch_dependent(diff_tc_fixup_kernel, dim3(g.workers, kTFixChunks), dim3(kTFixWarps * 32), 0,
                       st, a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

unsigned take_error_word_diff_tc(cudaStream_t stream, int* rc) {
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
