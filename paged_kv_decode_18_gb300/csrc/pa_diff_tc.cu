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
// Roles in each CTA (20 warps): warp 0 loads query tiles and K, warp 18 V; in the
// leading CTA warp 1 issues S and warp 19 O; warps 2-17 are the softmax, four
// threads to a query row, 32 keys each. Tensor memory holds O (256 columns), one S and
// two P: a tile's scores go to registers at once, so the next S is computed beside
// the exponentials of this one and the product of the last. (S and P in one buffer,
// two of those: the next S but one waited for the product, 2400 clocks a tile.) O is
// one accumulator for all keys, so a row's threads agree on its reference. It moves
// only when a maximum grows by more than 2^32 (exact either way): the four warps of 32
// rows vote whether one does, by a hardware barrier, and exchange maxima through
// shared memory only then. (Exchanging them every tile, with an mbarrier: 365 clocks, 7
// us of the call below.)
//
// Four chunks of 512 queries over 2816 to 7424 keys, 16 heads over 8: 104 us and the
// merge's 15, 119 in all, of which the products' own operations are 64. A tile takes 1.1
// us: its products and their hand-offs by themselves (no exponentials) 1.0 to 1.2, the
// softmax by itself (no products) as much, and leaving the loads out changes neither. A
// map's end (its diagonal tiles, O read out with nothing beside it) costs 3 to 4 us.
#include <cudaTypedefs.h>

#include "pa_diff.cuh"
#include "pa_diff_plan.h"
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
constexpr int kParts = 4;                     // softmax threads to a query row
constexpr int kPartKeys = kKeysT / kParts;    // keys of a tile that each has
constexpr int kPartDims = kDiffDim / kParts;  // output dims
constexpr int kSoftmaxWarps = 4 * kParts;     // warps 2-17
constexpr int kVWarp = 2 + kSoftmaxWarps;
constexpr int kPvWarp = kVWarp + 1;
constexpr int kThreadsT = 128 + kSoftmaxWarps * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 128;               // S at columns 0 .. 127, two P buffers of 64,
constexpr uint32_t kColO = 256;               // O at 256 .. 511
// a map's start in quarters of a key tile: what its diagonal tiles and its write-out take
// on top of the others (four chunks over 2816 .. 7424 keys: 12: 128 us, 16: 125.3, 20:
// 124.3, 24: 124.5, 28: 127.4; 24 charged where both maps' segment starts: 127.4)
constexpr int kMapCost4 = 20;
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
  B_VFULL = 10,                       // [3], leader: both CTAs' values
  B_VEMPTY = 13,                      // [3], both
  B_SFULL = 16,                       // both
  B_SEMPTY = 17,                      // leader: all softmax warps of both hold their scores
  B_PFREE = 18,                       // [2], both: the product that read this P is done
  // [2], leader: all softmax warps of both. Two, since a warp may be through with the
  // next tile's exponentials before another has arrived for this one
  B_PFULL = 20,
  B_VSEEN = 22,                       // both: the values of a tile that has to be cleaned are there
  B_XCH = 23,                         // [4]: the four warps of 32 rows, every exchange a phase
  kNumBarsT = 27
};

// shared memory past the operands
constexpr int kOffBars = 0;
constexpr int kOffSlot = kNumBarsT * 8;
constexpr int kOffAbort = kOffSlot + 4;
constexpr int kOffBad = kOffAbort + 4;
constexpr int kOffXch = 256;                       // [2][kParts][128] floats
constexpr int kOffPend = kOffXch + 2 * kParts * kRowsT * 4;  // [softmax warps] Pending
constexpr int kOffPlanT = kOffPend + kSoftmaxWarps * 32;
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
  int max_q_len;
  int nstage;
  // [workers * 2 pieces][2 maps][64 groups of 4 dims][256 rows][4]: neighbouring
  // threads hold neighbouring rows
  float* part_o;
  float* part_lse;  // [workers * 2 pieces][2 maps][256 rows]
  int* desc;        // [workers][kTDesc]
};

__device__ __forceinline__ float4* part_rows(const DiffTcArgs& a, int slot, int map) {
  return reinterpret_cast<float4*>(a.part_o) +
         ((size_t)slot * 2 + map) * (kDiffDim / 4) * (2 * kRowsT);
}

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
// The same for what the peer is to read by ordinary loads, and the wait for it.
__device__ __forceinline__ void release_in_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ bool try_acquire_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
// mbar_try_wait that may sleep for up to 20 us: a warp that spins takes issue slots from
// the softmax warps of its sub-partition
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// Whether `yes` holds in one of the four warps of 32 rows. Every warp votes once a tile;
// one that leaves early makes up for the votes that the others wait for.
__device__ __forceinline__ bool vote(int rows, bool yes) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)yes), "r"(1 + rows), "n"(kParts * 32)
      : "memory");
  return any != 0;
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
      mbar_init(bar(i), i >= B_XCH ? kParts
                        : i == B_PFULL || i == B_PFULL + 1 ? 2 * kSoftmaxWarps
                        : i == B_SEMPTY                  ? 2 * 4
                                                         : 1);
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
  in.announced = a.max_q_len;
  in.skip_empty = a.cu_seqlens_q == nullptr;
  build_plan(in, P, nullptr);
  // segments are pairs of KV heads, n tiles of the first map, then n of the second; the
  // cut charges every map by itself, as if each KV head had a segment of n
  const PieceCut cut = build_piece_cut(P, Hkv, a.num_workers, kMapCost4, cut_at);
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
    MergeJob j;
    j.valid = false;
    if (work) j = merge_job_of(P, S, Hp, w, cut.nw, cut);
    int4 d0 = make_int4(-1, 0, 0, 0), d1 = d0;
    if (j.valid) {
      d0 = make_int4(j.s, j.qt, j.h, j.last);
      d1 = make_int4(j.slot_prev, P.qstart[j.s], P.qstart[j.s + 1] - P.qstart[j.s], 0);
    }
    int4* d = reinterpret_cast<int4*>(a.desc + (size_t)w * kTDesc);
    d[0] = d0;
    d[1] = d1;
  }
  if (!work) return;  // both CTAs of the cluster
  const int R0 = cut.start(w), R1 = cut.start(w + 1);
  if (R0 >= R1) return;

  // map and key tile of a segment's tile b
  auto map_of = [](const TilePos& t) { return 2 * t.b >= t.nt ? 1 : 0; };
  auto key_tile_of = [&](const TilePos& t) { return t.b - map_of(t) * (t.nt >> 1); };
  auto nblocks_of = [&](const TilePos& tp) {
    const int nb_seq = (P.ctx[tp.s] + kBlock - 1) / kBlock;
    return min(kBlocksT, nb_seq - key_tile_of(tp) * kBlocksT);
  };
  auto fetch_ids = [&](const TilePos& tp) -> int {
    return lane < nblocks_of(tp)
               ? a.block_tables[(size_t)tp.s * a.max_blocks + key_tile_of(tp) * kBlocksT + lane]
               : 0;
  };
  // the producers' first tile, its block ids on their way while the pair meets (2 us of
  // the call of the head comment)
  TilePos t0;
  int ids0 = 0;
  if (warp == 0 || warp == kVWarp) {
    t0 = locate(P, S, Hp, R0);
    ids0 = fetch_ids(t0);
  }
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
    if (try_wait_long(bar(b), parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!*abort_flag) {
      if (try_wait_long(bar(b), parity)) return true;
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
  // keys before it are seen by every query of the tile
  auto safe_keys = [&](const TilePos& t) {
    const int c = P.ctx[t.s];
    return a.causal ? c - (P.qstart[t.s + 1] - P.qstart[t.s]) + t.qt * 2 * QTb + 1 : c;
  };
  // whether a tile begins a map of a piece
  auto begins = [&](const TilePos& t, int idx) { return idx == R0 || key_tile_of(t) == 0; };

  if (warp == 0 || warp == kVWarp) {
    // ------------------------------------------------------------------ producers
    const bool is_k = warp == 0;
    TilePos t = t0;
    const uint32_t lead_q = in_cta(bar(B_QFULL), 0), lead_k = in_cta(bar(B_KFULL), 0),
                   lead_v = in_cta(bar(B_VFULL), 0);
    int ids = ids0;
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
        if (lane == 0 && rank == 0)
          mbar_arrive_expect_tx(bar(B_VFULL + st), 2u * (uint32_t)nb * (uint32_t)kTileBytes);
        __syncwarp();
        if (lane < nb)
          tma_pair_block(smem_addr(base + kKBytes + lane * kTileBytes), &tmv,
                         (int)(((int64_t)my_id * Hkv + h0 + rank) * (kBlock / 8)), lead_v + st * 8);
      }
      __syncwarp();
      if (++st == nstage) {
        st = 0;
        ++use;
      }
    }
    if (!fine && rank == 0) {
      // copies in flight land (within the limit) before the CTA leaves; the leading
      // CTA's barriers count the peer's as well
      for (int k = qn < 2 ? 0 : qn - 2; is_k && k < qn; ++k)
        mbar_wait_bounded(bar(B_QFULL + (k & 1)), (uint32_t)(k >> 1) & 1u);
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
        if (!wait(B_KFULL + st, use & 1u)) break;
        // the softmax holds the scores of the last tile in registers
        if (i >= 1 && !wait(B_SEMPTY, (uint32_t)(i - 1) & 1u)) break;
        // and the P buffer that it will fill next is free: S says so to every warp
        if (i >= 2 && !wait(B_PFREE + (i & 1), (uint32_t)((i >> 1) - 1) & 1u)) break;
        tc_fence_after();
        const uint64_t dq = desc_q + (uint64_t)(qs * (kQBytes >> 4));
        const uint64_t dk = desc_k + (uint64_t)(st * (kStageT >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          pair_mma(tmem, dq + (uint64_t)(((k >> 2) * kHalfT + (k & 3) * 32) >> 4),
                   dk + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), idS, k > 0);
        pair_commit(bar(B_SFULL));
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
      uint32_t use = 0;
      for (int idx = R0, i = 0; idx < R1; ++idx, ++i) {
        const bool first = begins(t, idx);
        const uint32_t sb = (uint32_t)(i & 1);
        if (!wait(B_VFULL + st, use & 1u)) break;
        // the softmax warps clean these values before they arrive
        if ((key_tile_of(t) + 1) * kKeysT > safe_keys(t))
          for (uint32_t to = 0; to < 2; ++to) release_in_cluster(in_cta(bar(B_VSEEN), to));
        if (!wait(B_PFULL + (int)sb, (uint32_t)(i >> 1) & 1u)) break;
        tc_fence_after();
        const uint64_t dv = desc_v + (uint64_t)(st * (kStageT >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          pair_mma_ts(tmem + kColO, tmem + kColP + sb * 64u + (uint32_t)k * 8u, dv + (uint64_t)(k * (kTileBytes >> 4)), idPV, (k > 0 || !first) ? 1u : 0u);
        pair_commit(bar(B_VEMPTY + st));
        pair_commit(bar(B_PFREE + (int)sb));
        if (++st == nstage) {
          st = 0;
          ++use;
        }
        if (idx + 1 < R1) advance(P, S, Hp, t);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax
    const int q4 = warp & 3;
    const int part = (warp - 2) >> 2;  // which keys of a tile and which output dims
    const int r = q4 * 32 + lane;  // this thread's query row (= TMEM lane)
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tO = tmem + lane_base + kColO + (uint32_t)(part * kPartDims);  // its output dims
    // arrives on a barrier of the leading CTA
    auto arrive = [&](int b) {
      if (rank == 0)
        mbar_arrive(bar(b));
      else
        arrive_in_cluster(in_cta(bar(b), 0));
    };
    const float sc = a.scale_log2;
    uint32_t xphase = 0, cleaned = 0;  // exchanges; tiles whose values were cleaned
    int st = 0, votes = 0;
    // Gives `mine` to the other threads of the row; all take the four values.
    auto exchange = [&](float mine, float (&all)[kParts]) -> bool {
      float* x = xch + (xphase & 1u) * (kParts * kRowsT) + r;
      x[part * kRowsT] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_XCH + q4));
      if (!wait_all(B_XCH + q4, xphase & 1u)) return false;
      ++xphase;
#pragma unroll
      for (int k = 0; k < kParts; ++k) all[k] = x[k * kRowsT];
      return true;
    };
    TilePos t = locate(P, S, Hp, R0);
    float m_ref = neg_inf(), l = 0.f;
    int lim = 0, c = 0, vsafe = 0, piece_b0 = 0;
    bool piece_first = true;
    // A finished map's O stays in tensor memory until the next tile's exponentials are
    // done (its last product completes meanwhile); then it is written out.
    // What it takes is the same for a warp's rows and kept in shared memory: registers
    // that do not spill are what this loop is short of (beside 218 KB of shared memory a
    // spilled word comes back from L2).
    struct Pending {
      int flags, s, h, k1;   // 1: whole, 2: last tile of the piece; where its keys end
      int map, b0, n, slot;  // b0: the piece's first tile, of a segment of 2n
    };
    static_assert(sizeof(Pending) == 32, "kOffPend");
    Pending* pending = reinterpret_cast<Pending*>(rest + kOffPend) + (warp - 2);
    bool pend_on = false;
    int pend_tok = -1;  // the row's token (-1: padding)
    float pend_m = 0.f, pend_l = 0.f;
    auto flush = [&]() -> bool {
      const Pending pend = *pending;
      const bool pend_valid = pend_tok >= 0;
      float ls[kParts];
      if (!exchange(pend_l, ls)) return false;
      float lt = ls[0];
#pragma unroll
      for (int k = 1; k < kParts; ++k) lt += ls[k];
      // (a NaN score's NaN goes on into the row's results)
      const float inv = lt != 0.f ? 1.f / lt : 0.f;
      const float lse_v = lt != 0.f ? (pend_m + lg2(lt)) * kLn2 : neg_inf();
      const int head = pend.h * G + r % G;
      const bool merge = (pend.flags & 1) && pend.map == 1;  // both maps are here: the row's output
      const int64_t qtok = (int64_t)P.qstart[pend.s] + pend_tok;
      const float lam = merge && pend_valid ? a.o.lambdas[head] : 0.f;
      const int row = rank * kRowsT + r;
      float4* mine = part_rows(a, pend.slot, pend.map) + part * (kPartDims / 4) * (2 * kRowsT) + row;
      const float4* first_map =
          part_rows(a, pend.slot, 0) + part * (kPartDims / 4) * (2 * kRowsT) + row;
      float4 x[4];  // the first map's values
      float squares = 0.f;
#pragma unroll 1
      for (int cc = 0; cc < kPartDims / 16; ++cc) {
        float z[16];
        if (merge && pend_valid) {
#pragma unroll
          for (int q = 0; q < 4; ++q) x[q] = first_map[(cc * 4 + q) * (2 * kRowsT)];
        }
        __syncwarp();
        tmem_ld16(tO + (uint32_t)cc * 16u, z);
        if (*bad_v && pend_valid) {
          // infinities and NaNs of rows that not all of the tile's queries see entered the
          // product as zeros (they must not reach the others): they join the rows that
          // see them here
          const int lqp = P.qstart[pend.s + 1] - P.qstart[pend.s];
          const int p0 = P.ctx[pend.s] - lqp;
          const int k0 =
              pend.b0 < pend.n && pend.map == 1 ? 0 : (pend.b0 - pend.map * pend.n) * kKeysT;
          const int k1 = min(p0 + pend_tok + 1, pend.k1);  // (a causal window)
          const int seen = p0 + pend_tok / (2 * QTb) * (2 * QTb) + 1;  // by all of the tile
          for (int k = max(seen, k0); k < k1; ++k) {
            const int phys = a.block_tables[(size_t)pend.s * a.max_blocks + k / kBlock];
            if (phys < 0 || (int64_t)phys >= a.num_blocks) continue;
            const int dim = part * kPartDims + cc * 16;
            const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                a.v_cache + ((((int64_t)phys * Hkv + 2 * pend.h + dim / kHeadDim) * kBlock) +
                             k % kBlock) * kHeadDim + dim % kHeadDim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t wv = vr[j], fin = bf2_finite_part(wv);
              if ((wv ^ fin) & 0x7f80u) z[2 * j] += bf_lo(wv);
              if ((wv ^ fin) & 0x7f800000u) z[2 * j + 1] += bf_hi(wv);
            }
          }
        }
        if (!merge) {
          if (pend_valid) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mine[(cc * 4 + q) * (2 * kRowsT)] = make_float4(__fmul_rn(z[4 * q], inv), __fmul_rn(z[4 * q + 1], inv),
                                   __fmul_rn(z[4 * q + 2], inv), __fmul_rn(z[4 * q + 3], inv));
          }
          continue;
        }
        uint32_t d[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = x[q];
          const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = diff_value(fs[e], 1.f, z[4 * q + e], inv, lam);
            squares = fmaf(v, v, squares);
            d[4 * q + e] = __float_as_uint(v);
          }
        }
        // the difference waits in tensor memory for its norm
        __syncwarp();
        tmem_st16(tO + (uint32_t)cc * 16u, d);
      }
      if (merge) {
        tmem_wait_st();
        float factor = a.o.gain;
        if (a.o.weight) {
          float sq[kParts];
          if (!exchange(squares, sq)) return false;
          float sum = sq[0];
#pragma unroll
          for (int k = 1; k < kParts; ++k) sum += sq[k];
          factor = diff_factor(a.o, sum);
        }
#pragma unroll 1
        for (int cc = 0; cc < kPartDims / 16; ++cc) {
          float v[16];
          __syncwarp();
          tmem_ld16(tO + (uint32_t)cc * 16u, v);
          if (!pend_valid) continue;
          const float4* wt = reinterpret_cast<const float4*>(a.o.weight + part * kPartDims + cc * 16);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 w0 = a.o.weight ? wt[q] : make_float4(1.f, 1.f, 1.f, 1.f);
            v[4 * q] *= factor * w0.x;
            v[4 * q + 1] *= factor * w0.y;
            v[4 * q + 2] *= factor * w0.z;
            v[4 * q + 3] *= factor * w0.w;
          }
          uint4* dst = reinterpret_cast<uint4*>(
              a.o.out + (qtok * (a.Hq / 2) + head) * kDiffDim + part * kPartDims + cc * 16);
          dst[0] = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                              cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
          dst[1] = make_uint4(cvt_bf16x2(v[8], v[9]), cvt_bf16x2(v[10], v[11]),
                              cvt_bf16x2(v[12], v[13]), cvt_bf16x2(v[14], v[15]));
        }
      }
      if (part == 0 && pend_valid) {
        if (pend.flags & 1) {
          if (a.o.lse)
            a.o.lse[qtok * a.Hq + (int64_t)(2 * pend.h + pend.map) * G + r % G] = lse_v;
        } else {
          float* pl = a.part_lse + (size_t)pend.slot * 2 * (2 * kRowsT) + row;
          pl[pend.map * (2 * kRowsT)] = lse_v;
          // a map that the piece has no tile of weighs nothing in the merge
          if (pend.map == 0 && (pend.flags & 2)) pl[2 * kRowsT] = neg_inf();
          if (pend.map == 1 && pend.b0 >= pend.n) pl[0] = neg_inf();
        }
      }
      pend_on = false;
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
        const int lq = P.qstart[t.s + 1] - P.qstart[t.s];
        const int tok = (t.qt * 2 + rank) * QTb + r / G;
        // keys that the row sees (padding: none; a query sees one at least)
        lim = tok < lq && r < QTb * G ? (a.causal ? c - lq + tok + 1 : c) : 0;
        vsafe = safe_keys(t);
        piece_b0 = t.b;
        piece_first = idx == R0;
      }
      if (first) {
        m_ref = neg_inf();
        l = 0.f;
      }
      const uint32_t sb = (uint32_t)(i & 1);
      if (!wait_all(B_SFULL, sb)) break;
      tc_fence_after();
      float2 x[kPartKeys / 2];
      {
        uint32_t v[kPartKeys / 32][32];
#pragma unroll
        for (int g = 0; g < kPartKeys / 32; ++g)
          tmem_ld32_async(tmem + lane_base + (uint32_t)(part * kPartKeys + g * 32), v[g]);
        tmem_wait_ld(v[0]);
#pragma unroll
        for (int g = 0; g < kPartKeys / 32; ++g) {
          if (g > 0) tmem_tie(v[g]);
          // scores in log2 units
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[g * 16 + j] =
                __fmul2_rn(make_float2(__uint_as_float(v[g][2 * j]), __uint_as_float(v[g][2 * j + 1])),
                           make_float2(sc, sc));
        }
      }
      // the scores are in registers: the next tile's may come
      tc_fence_before();
      const int key0 = kt * kKeysT, kb = key0 + part * kPartKeys;  // first key of the tile, of this part
      if (kb + kPartKeys > lim) {  // the causal diagonal or the end of the context
#pragma unroll
        for (int j = 0; j < kPartKeys / 2; ++j) {
          if (kb + 2 * j >= lim) x[j].x = neg_inf();
          if (kb + 2 * j + 1 >= lim) x[j].y = neg_inf();
        }
      }
      float mx;
      {
        float m4[4] = {fmaxf(x[0].x, x[0].y), fmaxf(x[1].x, x[1].y), fmaxf(x[2].x, x[2].y),
                       fmaxf(x[3].x, x[3].y)};
#pragma unroll
        for (int j = 4; j < kPartKeys / 2; ++j)
          asm("max.f32 %0, %1, %2, %3;"
              : "=f"(m4[j & 3])
              : "f"(x[j].x), "f"(x[j].y), "f"(m4[j & 3]));
        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      // m_ref moves only where a maximum is 2^kRescaleLog2 above it, in one of the row's
      // parts: mostly nowhere, and then no maxima have to be exchanged.
      const bool moves = vote(q4, mx > m_ref + kRescaleLog2);
      ++votes;
      if (part == 0) {  // (the other parts' scores are in registers, too)
        tc_fence_after();
        tc_fence_before();
        if (lane == 0) arrive(B_SEMPTY);
      }
      float alpha = 1.f;
      bool rescale = false;
      if (moves) {
        float ms[kParts];
        if (!exchange(mx, ms)) break;
#pragma unroll
        for (int k = 0; k < kParts; ++k) mx = fmaxf(mx, ms[k]);  // the same in all parts of the row
        if (mx > m_ref + kRescaleLog2) {
          // (with m_ref = -inf nothing has accumulated yet: O and l are zero)
          rescale = m_ref != neg_inf();
          if (rescale) alpha = ex2(m_ref - mx);
          m_ref = mx;
        }
      }
      const bool scale_o = __any_sync(kFull, rescale) && !first;
      const float ref = m_ref == neg_inf() ? 0.f : m_ref;
      const float2 nref = make_float2(-ref, -ref);
      float2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      // P enters the product in bf16, the type that V is stored in and that one
      // tcgen05.mma wants of both operands: a weight is off by at most 2^-8 of itself.
      // The sum l, and with it lse, is of the unrounded ones.
      uint32_t pk[kPartKeys / 32][16];
#pragma unroll
      for (int j = 0; j < kPartKeys / 2; ++j) {
        const float2 d = __fadd2_rn(x[j], nref);
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        acc[j & 3] = __fadd2_rn(acc[j & 3], e);
        pk[j >> 4][j & 15] = cvt_bf16x2(e.x, e.y);
      }
      const float2 s01 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l = fmaf(l, alpha, s01.x + s01.y);
      // P row r, keys of this part
      __syncwarp();
#pragma unroll
      for (int g = 0; g < kPartKeys / 32; ++g)
        tmem_st16(tmem + lane_base + kColP + sb * 64u + (uint32_t)(part * (kPartKeys / 2) + g * 16),
                  pk[g]);
      // the previous product must be done before O is rescaled or the previous map's O is
      // read. Its P buffer says so: the product before it on that buffer is done, or this
      // tile's S would not be there, so its phase is not mistaken for an earlier one. (The
      // tensor-memory accesses are warp-wide: the whole warp rescales when one of its
      // rows has to, the others by 1.)
      if (scale_o || pend_on) {
        if (!wait_all(B_PFREE + (int)(sb ^ 1u), (uint32_t)((i - 1) >> 1) & 1u)) break;
        tc_fence_after();
      }
      if (pend_on && !flush()) break;
      if (scale_o) {
        __syncwarp();
#pragma unroll 1
        for (int cc = 0; cc < kPartDims / 16; ++cc) {
          float y[16];
          uint32_t u[16];
          tmem_ld16(tO + (uint32_t)cc * 16u, y);
#pragma unroll
          for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(y[j] * alpha);
          tmem_st16(tO + (uint32_t)cc * 16u, u);
        }
      }
      tmem_wait_st();
      // keys past the context may hold anything (even NaN): zero their V rows so that P
      // = 0 never meets them; of the rows that only some of the tile's queries see, the
      // infinities and NaNs. (Other tiles' values are the issuing thread's to wait for: a wait
      // costs 130 clocks even when it is over, and the divisions for its stage as much again;
      // one warp that made it for its CTA held up its rows by 400 clocks a tile.)
      if (key0 + kKeysT > vsafe) {
        bool there = try_acquire_cluster(bar(B_VSEEN), cleaned & 1u);
        if (!there)
          there = wait(B_VSEEN, cleaned & 1u) && try_acquire_cluster(bar(B_VSEEN), cleaned & 1u);
        if (!__all_sync(kFull, there)) break;
        ++cleaned;
        // chunks of 16 bytes in the order in which they lie: (16 keys, 8 of them, 64 dims, key)
        constexpr int kChunks = kVBytes / (kSoftmaxWarps * 32 * 16);
        unsigned char* vt = stages + st * kStageT + kKBytes;
        uint4 x4[kChunks];
        uint32_t unfit = 0;  // chunks to be put right
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          x4[k] = *reinterpret_cast<uint4*>(vt + (k * kSoftmaxWarps * 32 + tid - 64) * 16);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int at = (k * kSoftmaxWarps * 32 + tid - 64) * 16;
          const int key = key0 + (at >> 12) * 16 + ((at >> 11) & 1) * 8 + ((at >> 7) & 7);
          // (all exponent bits set: one more in their lowest place carries to the sign's)
          const uint32_t e = 0x7f807f80u, one = 0x00800080u;
          const bool odd = ((((x4[k].x & e) + one) | ((x4[k].y & e) + one) |
                             ((x4[k].z & e) + one) | ((x4[k].w & e) + one)) & 0x80008000u) != 0;
          if (key >= c || (key >= vsafe && odd)) unfit |= 1u << k;
          if (key >= c) x4[k] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (unfit) {
          const uint32_t flag = smem_addr(rest + kOffBad);
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            if (!((unfit >> k) & 1u)) continue;
            const int at = (k * kSoftmaxWarps * 32 + tid - 64) * 16;
            const uint4 y = make_uint4(bf2_finite_part(x4[k].x), bf2_finite_part(x4[k].y),
                                       bf2_finite_part(x4[k].z), bf2_finite_part(x4[k].w));
            // both CTAs write dims of both heads out
            if ((x4[k].x ^ y.x) | (x4[k].y ^ y.y) | (x4[k].z ^ y.z) | (x4[k].w ^ y.w))
              for (uint32_t to = 0; to < 2; ++to)
                asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(
                                 in_cta(flag, to)),
                             "r"(1u)
                             : "memory");
            *reinterpret_cast<uint4*>(vt + at) = y;
          }
          fence_proxy_async_smem();
          fence_cluster();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(B_PFULL + (int)sb);
      if (++st == nstage) st = 0;

      if (last) {
        pend_on = true;
        pend_tok = lim > 0 ? (t.qt * 2 + rank) * QTb + r / G : -1;
        pend_m = m_ref;
        pend_l = l;
        __syncwarp();
        if (lane == 0) {
          Pending p;
          p.flags = (piece_b0 == 0 && (map == 0 ? R1 - idx > n : t.b == t.nt - 1) ? 1 : 0) |
                    (piece_last ? 2 : 0);
          p.k1 = key0 + kKeysT;
          p.s = t.s;
          p.h = t.h;
          p.map = map;
          p.b0 = piece_b0;
          p.n = n;
          p.slot = w * 2 + (piece_first ? 0 : 1);
          *pending = p;
        }
        __syncwarp();
      }
      if (idx + 1 < R1) advance(P, S, Hp, t);
    }
    for (; votes < R1 - R0; ++votes) vote(q4, false);
    if (pend_on && wait_all(B_PFREE + ((i - 1) & 1), (uint32_t)((i - 1) >> 1) & 1u)) {
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
// maps, then difference, norm and scale. Grid (worker boundary, chunk of 8 rows): a
// thread has 16 dims of a row, eight neighbours the same dims of the chunk (128 bytes of
// partials), whose sums of squares meet in shared memory. 18 us after the call of the
// head comment with chunks of 32 rows in CTAs of 16 warps, since a quarter of them came
// in a second round on the SMs; 16 us of 16 rows, 15 of 8, for 52 MB out of L2. Four
// pieces at a time: two are as fast there (two or three pieces to a segment) and 2 us
// slower where 19 meet.
constexpr int kTFixWarps = 4;
constexpr int kTFixRows = 8;
constexpr int kTFixChunks = 2 * kRowsT / kTFixRows;
constexpr int kTFixDims = 16;  // of a thread
constexpr int kTFixParts = kDiffDim / kTFixDims;
static_assert(kTFixWarps * 32 == kTFixRows * kTFixParts, "a thread has 16 dims of a row");

__global__ void __launch_bounds__(kTFixWarps * 32, 8)
    diff_tc_fixup_kernel(const DiffTcArgs a) {
  __shared__ float squares_of[kTFixParts][kTFixRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x;
  const int4* d = reinterpret_cast<const int4*>(a.desc + (size_t)w * kTDesc);
  const int4 d0 = __ldcg(d), d1 = __ldcg(d + 1);
  if (d0.x < 0) return;
  const int qt = d0.y, h = d0.z, last = d0.w, slot_prev = d1.x, q0 = d1.y, lq = d1.z;
  const int at = threadIdx.x % kTFixRows, part = threadIdx.x / kTFixRows;
  const int npieces = last - w + 2;  // workers w-1 .. last
  const int row = blockIdx.y * kTFixRows + at, r = row & (kRowsT - 1);
  const int tok = (qt * 2 + row / kRowsT) * a.QTb + r / a.G;
  const bool live = r < a.QTb * a.G && tok < lq;
  if (!__syncthreads_or(live)) return;
  auto slot_of = [&](int i) { return (w - 1 + i) * 2 + (i == 0 ? slot_prev : 0); };
  const int head = h * a.G + r % a.G;
  float y[kTFixDims], lse[2] = {neg_inf(), neg_inf()};
  float squares = 0.f;
  if (live) {
    float m[2] = {neg_inf(), neg_inf()}, sum[2] = {0.f, 0.f}, acc[2][kTFixDims];
    bool nan[2] = {false, false};  // a piece with a NaN score: the row's results are NaNs
#pragma unroll
    for (int j = 0; j < kTFixDims; ++j) acc[0][j] = acc[1][j] = 0.f;
    const float lam = a.o.lambdas[head];
    for (int i0 = 0; i0 < npieces; i0 += 4) {  // online, four pieces' sums in flight
      float li[2][4], wt[2][4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int map = 0; map < 2; ++map)
          li[map][u] = i0 + u < npieces
                           ? __ldcg(a.part_lse + ((size_t)slot_of(i0 + u) * 2 + map) * (2 * kRowsT) + row)
                           : neg_inf();
#pragma unroll
      for (int map = 0; map < 2; ++map) {
        float mn = m[map];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          nan[map] = nan[map] || li[map][u] != li[map][u];
          mn = fmaxf(mn, li[map][u]);
        }
        const float shrink = m[map] == neg_inf() ? 0.f : ex2((m[map] - mn) * kLog2e);
        sum[map] *= shrink;
#pragma unroll
        for (int j = 0; j < kTFixDims; ++j) acc[map][j] *= shrink;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          wt[map][u] = li[map][u] == neg_inf() ? 0.f : ex2((li[map][u] - mn) * kLog2e);
          sum[map] += wt[map][u];
        }
        m[map] = mn;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int map = 0; map < 2; ++map) {
          if (li[map][u] == neg_inf()) continue;  // nothing was written there
          const float4* src =
              part_rows(a, slot_of(i0 + u), map) + part * (kTFixDims / 4) * (2 * kRowsT) + row;
          float4 v[kTFixDims / 4];
#pragma unroll
          for (int q = 0; q < kTFixDims / 4; ++q) v[q] = __ldcg(src + q * (2 * kRowsT));
#pragma unroll
          for (int q = 0; q < kTFixDims / 4; ++q) {
            acc[map][4 * q + 0] = fmaf(wt[map][u], v[q].x, acc[map][4 * q + 0]);
            acc[map][4 * q + 1] = fmaf(wt[map][u], v[q].y, acc[map][4 * q + 1]);
            acc[map][4 * q + 2] = fmaf(wt[map][u], v[q].z, acc[map][4 * q + 2]);
            acc[map][4 * q + 3] = fmaf(wt[map][u], v[q].w, acc[map][4 * q + 3]);
          }
        }
    }
    float inv[2];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      if (nan[map]) m[map] = sum[map] = __int_as_float(0x7fc00000);
      inv[map] = sum[map] != 0.f ? 1.f / sum[map] : 0.f;
      lse[map] = sum[map] != 0.f ? m[map] + lg2(sum[map]) * kLn2 : neg_inf();
    }
#pragma unroll
    for (int j = 0; j < kTFixDims; ++j) {
      y[j] = diff_value(acc[0][j], inv[0], acc[1][j], inv[1], lam);
      squares = fmaf(y[j], y[j], squares);
    }
  }
  squares_of[part][at] = squares;
  float weight[kTFixDims];
#pragma unroll
  for (int q = 0; q < kTFixDims / 4; ++q) {
    const float4 x = a.o.weight
                         ? reinterpret_cast<const float4*>(a.o.weight + part * kTFixDims)[q]
                         : make_float4(1.f, 1.f, 1.f, 1.f);
    weight[4 * q] = x.x;
    weight[4 * q + 1] = x.y;
    weight[4 * q + 2] = x.z;
    weight[4 * q + 3] = x.w;
  }
  __syncthreads();
  if (!live) return;
  squares = 0.f;
#pragma unroll
  for (int k = 0; k < kTFixParts; ++k) squares += squares_of[k][at];
  const float f = diff_factor(a.o, squares);
  const int64_t qtok = (int64_t)q0 + tok;
  uint4* dst = reinterpret_cast<uint4*>(a.o.out + (qtok * (a.Hq / 2) + head) * kDiffDim +
                                        part * kTFixDims);
#pragma unroll
  for (int q = 0; q < kTFixDims / 8; ++q) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 8 * q + 2 * e;
      u[e] = cvt_bf16x2(y[j] * (f * weight[j]), y[j + 1] * (f * weight[j + 1]));
    }
    dst[q] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (a.o.lse && part == 0) {
    float* l = a.o.lse + qtok * a.Hq + (int64_t)(2 * h) * a.G + r % a.G;
    l[0] = lse[0];
    l[a.G] = lse[1];
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
  const int64_t cap = diff_pairs(S, num_q_tokens, max_q_len, unit);
  if (cap > (1 << 20)) return PA_ERR_UNSUPPORTED;
  g->npairs_cap = (int)(cap < 1 ? 1 : cap);
  // (a KV head is a segment of its own in the cut)
  if (!diff_tiles_fit(g->npairs_cap, sh->num_kv_heads,
                      ((int64_t)sh->max_blocks_per_seq + kBlocksT - 1) / kBlocksT, kMapCost4))
    return PA_ERR_UNSUPPORTED;
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
                   int max_q_len, int causal, float scale, const DiffOut& out, const pa_shape* sh,
                   void* workspace, cudaStream_t st) {
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
  a.max_q_len = max_q_len;
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
