// pa_weights_tc.cu -- pa_accumulate_weights for windows of many queries on the
// fifth-generation tensor cores (tcgen05 + tensor memory) of sm_103a.
//
//   w[s][h][p] (+)= sum_j sum_g exp(scale q_jg . k_p - lse_jg)
//
// S^T = K Q^T with the keys as the rows of the product: a thread of the
// epilogue owns one key (one tensor-memory lane) and sums its exponentials over
// the query columns in its own registers. A work item is (sequence, KV head, 128
// keys) with all of the window's query tiles, so a weight has one writer and its
// sum one order. One CTA per SM, warp-specialised:
//   warp 0     K producer: eight 16-key pool blocks a tile through the block
//              table (4-D TMA, 8-bit codes 3-D, with the 128-byte swizzle);
//   warp 10    query tiles of 128 rows ((128/G) tokens x G heads, 3-D TMA) and
//              their columns' log-sum-exps and causal limits;
//   warps 1,11 tensor memory and, from one thread each, the products: 128 keys x
//              up to 128 columns into the next accumulator; they take the items
//              (windows of several query tiles: the tiles) in turn: one thread
//              alone spends 2,000 cycles an item on waits, issue and commits,
//              more than anything else of it takes;
//   warps 2-9  the epilogue: two groups of four warps that take the items in
//              turn, so that one's exponentials hide the other's waits (two
//              threads a key with half the columns each, who met at every
//              item's end, took 45 us where this took 38), or in windows of
//              several query tiles half the columns each (SPLIT below);
//   warps 12-15 (8-bit pools) turn the raw codes into bf16 (exact) in tensor
//              memory, where the products take them from; the row scales
//              multiply the scores in the epilogue.
// Bound: windows of up to 128 rows by the K stream and the call's start: 16
// contexts of 1000..8192 positions with 64 queries of two heads (157 MB) take
// 36.2 us in bf16, 34.4 us with all of the epilogue's column work left out; FP8
// codes (81 MB) 42.6 us, 4 us less without their conversion. Longer windows by the
// epilogue and the waits between its tiles: 1024 rows take 187 us, 0.75 us a tile
// (135 us without the column work, 132 without the queries' loads as well and 109
// with one product in eight). No unit is near its limit meanwhile: tensor pipe 35 %,
// exponentials 35 %, issue 46 % of one a clock and SM quarter; windows of 128 FP8
// rows 20, 20 and 49 %. A tile is a chain of waits.
#include <cudaTypedefs.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_tcgen05.cuh"
#include "pa_weights.cuh"
#include "pa_weights_plan.h"

namespace pa {
namespace {

constexpr int kKeys = kWeightKeys;            // keys per item (MMA M)
constexpr int kCols = 128;                    // query rows per tile (MMA N, at most)
constexpr int kBlocksK = kKeys / kBlock;
constexpr int kHalfB = 128 * 128;             // 64 dims of a 128-row bf16 operand
constexpr int kOperand = 2 * kHalfB;
constexpr int kCodes = kKeys * kHeadDim;      // the raw codes of an item
constexpr int kRawTile = kCodes + 1024;       // and its row scales
constexpr int kScaleSlots = 8;                // items whose row scales are kept (see below)
constexpr int kPartSlots = 8;                 // items whose second half may wait (see below)
constexpr int kEpiWarps = 8;
constexpr int kQWarp = 2 + kEpiWarps;
constexpr int kMma2Warp = kQWarp + 1;
constexpr int kConvWarps = 4;

constexpr int kNumBarsMax = 48;

// SPLIT: windows of several query tiles may come. A tile then passes a chain of
// query load, product and epilogue with nothing to hide behind but the next
// tiles. So there are more query tiles in shared memory and fewer of K, the two
// issuing threads take tiles in turn, and both groups of the epilogue take half
// the columns of every tile (16 x 1000..8192, bf16, windows of 1024 rows: 189 us
// where the other form takes 224; windows of 128 rows: 41 us where that takes 36).
// Halves of columns, not every other tile: with two accumulators, all that
// the 8-bit pools leave room for, that took 206 us instead of 194, in bf16 180.
template <int FMT, bool SPLIT>
struct Lay {
  static constexpr bool q8 = FMT != PA_KV_BF16;
  static constexpr int kQBufs = SPLIT ? 4 : 2;       // query tiles in shared memory
  // bf16 K tiles: in shared memory, or widened into tensor memory (64 columns each)
  static constexpr int kStages = SPLIT && !q8 ? 2 : 4;
  static constexpr int kRawStages = SPLIT ? 4 : 6;   // of raw 8-bit tiles
  static constexpr int kDBufs = q8 ? 2 : 4;  // accumulators in tensor memory
  // A waiter knows a phase by its parity: it may neither look two phases late nor
  // while the phase before the one it wants is still running. Whoever waits for
  // every use of a slot has a part in emptying it (query tiles: the thread that
  // leaves a tile to the other arrives too). An issuing thread waits for its own
  // accumulators, without SPLIT also for its own items' K only and an epilogue group
  // for its own accumulators. Either meets a slot at every use or never: since the
  // two take items or tiles in turn, the rings have to be even. (Should a window of several tiles come to the form without SPLIT and
  // shift the turns, the wait for its query tile, the second after one that all
  // have done with, keeps them together.)
  static_assert(kDBufs % 2 == 0 && (SPLIT || (kStages % 2 == 0 && kQBufs == 2)),
                "a slot has one thread or group");
  static constexpr int kATmem = kDBufs * kCols;
  static_assert(kATmem + (q8 ? kStages * kHeadDim / 2 : 0) <= 512, "tensor memory");
  static constexpr int q = 0;                 // query tiles
  static constexpr int k = q + kQBufs * kOperand;  // K as it arrives
  static constexpr int bars = k + (q8 ? kRawStages * kRawTile : kStages * kOperand);
  static constexpr int misc = bars + kNumBarsMax * 8;  // tmem slot, abort flag
  static constexpr int l2 = misc + 16;              // a query tile's 128 -log-sum-exps, log2 units
  static constexpr int last = l2 + kQBufs * kCols * 4;   // last key seen; -1: no query
  static constexpr int clean = last + kQBufs * kCols * 4;  // all 128 columns are queries
  static constexpr int scale = clean + 16;          // [kScaleSlots][128] row scales
  static constexpr int part = scale + (q8 ? kScaleSlots * kKeys * 4 : 0);
  static constexpr int plan = part + kPartSlots * kKeys * 4;
  static constexpr int threads = 32 * (kMma2Warp + 1 + (q8 ? kConvWarps : 0));
};

enum : int {
  B_KFULL = 0, B_KEMPTY = 4, B_QFULL = 8, B_QEMPTY = 12, B_DFULL = 16, B_DEMPTY = 20,
  B_RFULL = 24, B_REMPTY = 30, B_PART = 36, kNumBars = 44
};

static_assert(kNumBars <= kNumBarsMax, "barrier area");

struct TcWeightArgs {
  WeightArgs w;
  int QTb;
};

// Per sequence, in shared memory: items and cost before it, lengths.
struct WPlan {
  int* cost;   // [S + 1] (query tiles + 1) summed over the items of earlier sequences
  int* item;   // [S + 1]
  int* ctx;    // [S]
  int* q0;     // [S]
  int* lq;     // [S]
};

struct Item {
  int s, h, i, nt;
};

__device__ __forceinline__ Item item_at(const WPlan& P, int S, int Hkv, int x) {
  Item t;
  t.s = upper_index(P.item, 0, S, x);
  t.nt = (P.item[t.s + 1] - P.item[t.s]) / Hkv;
  const int local = x - P.item[t.s];
  t.h = local / t.nt;
  t.i = local - t.h * t.nt;
  return t;
}
__device__ __forceinline__ void next_item(const WPlan& P, int Hkv, Item& t) {
  if (++t.i < t.nt) return;
  t.i = 0;
  if (++t.h < Hkv) return;
  t.h = 0;
  do {
    ++t.s;
  } while (P.item[t.s + 1] == P.item[t.s]);
  t.nt = (P.item[t.s + 1] - P.item[t.s]) / Hkv;
}
// Key tiles from both ends in turn: under the causal mask of a long window an
// early tile meets many query tiles and a late one few, so neighbours even out.
__device__ __forceinline__ int key_tile(const Item& t) {
  return (t.i & 1) ? t.nt - 1 - (t.i >> 1) : t.i >> 1;
}

template <int FMT, bool SPLIT>
__global__ void __launch_bounds__((Lay<FMT, SPLIT>::threads), 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk, const TcWeightArgs arg) {
  using L = Lay<FMT, SPLIT>;
  const WeightArgs& a = arg.w;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t rawp = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + (((rawp + 1023u) & ~1023u) - rawp);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc + 4);
  float* col_l2 = reinterpret_cast<float*>(smem + L::l2);
  int* col_last = reinterpret_cast<int*>(smem + L::last);
  volatile int* col_clean = reinterpret_cast<volatile int*>(smem + L::clean);
  const int S = a.S, Hkv = a.Hkv, G = a.G, QTb = arg.QTb;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(B_KFULL + i), L::q8 ? kConvWarps * 32u : 1u);
      mbar_init(bar(B_KEMPTY + i), SPLIT ? 2u : 1u);  // the issuing threads' commits
      mbar_init(bar(B_DFULL + i), 2u);  // the issuing thread and its commit
      mbar_init(bar(B_DEMPTY + i), kEpiWarps * (SPLIT ? 32u : 16u));  // who reads it
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(bar(B_RFULL + i), 1u);
      mbar_init(bar(B_REMPTY + i), kConvWarps * 32u);
    }
    for (int i = 0; i < kPartSlots; ++i) mbar_init(bar(B_PART + i), kEpiWarps * 16u);
    for (int i = 0; i < L::kQBufs; ++i) {
      mbar_init(bar(B_QFULL + i), 33u);  // warp 10's lanes and the expected bytes
      // the epilogue, and whoever of the issuing threads may still have to look for it
      mbar_init(bar(B_QEMPTY + i), (SPLIT ? 1u : 2u) + kEpiWarps * 32u);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (tid == 32) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- plan ---------------------------------------------------------------------
  WPlan P;
  P.cost = reinterpret_cast<int*>(smem + L::plan);
  P.item = P.cost + (S + 1);
  P.ctx = P.item + (S + 1);
  P.q0 = P.ctx + S;
  P.lq = P.q0 + S;
  const int max_ctx = (int)min((int64_t)a.max_blocks * kBlock, a.weights_len);
  for (int s = tid; s < S; s += blockDim.x) {
    int c = a.context_lens[s];
    if (c < 0 || c > max_ctx) {
      flag_error(PA_DEVERR_CONTEXT_RANGE);
      c = c < 0 ? 0 : max_ctx;
    }
    const int q0 = a.cu_seqlens_q ? a.cu_seqlens_q[s] : s;
    const int lq = a.cu_seqlens_q ? a.cu_seqlens_q[s + 1] - q0 : (c > 0 ? 1 : 0);
    const bool bad = q0 < 0 || lq < 0 || lq > c || (int64_t)q0 + lq > a.num_q_tokens;
    if (bad) flag_error(PA_DEVERR_QLEN_RANGE);
    // no query: nothing to add, zeros to write
    const int nt = bad || (lq == 0 && a.accumulate) ? 0 : (c + kKeys - 1) / kKeys;
    P.ctx[s] = c;
    P.q0[s] = q0;
    P.lq[s] = bad ? 0 : lq;
    P.item[s] = Hkv * nt;
    P.cost[s] = window_cost(nt, c, lq, QTb, Hkv, S);
  }
  __syncthreads();
  if (warp == 0) {
    const int n = warp0_exclusive_scan(P.item, S);
    if (lane == 0) P.item[S] = n;
    const int n2 = warp0_exclusive_scan(P.cost, S);
    if (lane == 0) P.cost[S] = n2;
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int total = P.item[S], cost_total = P.cost[S];
  // CTA w begins at the item in which its share of the cost begins
  auto begin_of = [&](int w) -> int {
    if (w >= (int)gridDim.x) return total;
    const int T = (int)((long long)w * cost_total / gridDim.x);
    const int s = upper_index(P.cost, 0, S, T);
    const int items = P.item[s + 1] - P.item[s], cost = P.cost[s + 1] - P.cost[s];
    if (cost <= 0) return total;
    return P.item[s] + (int)((long long)(T - P.cost[s]) * items / cost);
  };
  if (total == 0) return;
  const int I0 = begin_of((int)blockIdx.x), I1 = begin_of((int)blockIdx.x + 1);
  if (I0 >= I1) return;  // the whole CTA

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512u)
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
  // Query tiles of the window: one stays for all key tiles of a head, several
  // are loaded for each key tile again.
  auto tiles_of = [&](const Item& t) { return (P.lq[t.s] + QTb - 1) / QTb; };
  auto fresh_q = [&](const Item& t, int nq, int x) { return nq > 1 || t.i == 0 || x == I0; };

  if (warp == 0) {
    // -------------------------------------------------------------- K producer
    Item t = item_at(P, S, Hkv, I0);
    auto blocks_of = [&](const Item& it, int kt) {
      return min(kBlocksK, (P.ctx[it.s] + kBlock - 1) / kBlock - kt * kBlocksK);
    };
    auto fetch = [&](const Item& it) -> int {
      const int kt = key_tile(it);
      return lane < blocks_of(it, kt)
                 ? a.block_tables[(size_t)it.s * a.max_blocks + kt * kBlocksK + lane]
                 : 0;
    };
    int ids = fetch(t), n = 0;  // n: items with queries so far
    for (int x = I0; x < I1; ++x) {
      const Item cur = t;
      const int nb = blocks_of(cur, key_tile(cur));
      int id = ids;
      if (x + 1 < I1) {
        next_item(P, Hkv, t);
        ids = fetch(t);
      }
      if (P.lq[cur.s] == 0) continue;
      if (lane < nb && (id < 0 || (int64_t)id >= a.num_blocks)) {
        flag_error(PA_DEVERR_BLOCK_RANGE);
        id = 0;
      }
      constexpr int kRing = L::q8 ? L::kRawStages : L::kStages;
      const int st = n % kRing;
      const uint32_t full = bar((L::q8 ? B_RFULL : B_KFULL) + st);
      if (n >= kRing &&
          !wait((L::q8 ? B_REMPTY : B_KEMPTY) + st, (uint32_t)((n / kRing) - 1) & 1u))
        break;
      if (lane == 0)
        mbar_arrive_expect_tx(full, (uint32_t)nb * (uint32_t)(L::q8 ? kInt8TileBytes : kTileBytes));
      __syncwarp();
      if (lane < nb) {
        if constexpr (L::q8) {
          // the codes with the 128-byte swizzle, the row scales behind the tile's codes
          const int64_t tile = (int64_t)id * Hkv + cur.h;
          unsigned char* raw = smem + L::k + st * kRawTile;
          tma_load_3d(smem_addr(raw + lane * kBlock * kHeadDim), &tmk, 0, 0, (int)tile, full);
          bulk_copy_g2s(smem_addr(raw + kCodes + lane * kBlock * 4),
                        a.k_cache + tile * kInt8TileBytes + kBlock * kHeadDim, kBlock * 4, full);
        } else {
          const int group = (int)(((int64_t)id * Hkv + cur.h) * (kBlock / 8));
          tma_load_block(smem_addr(smem + L::k + st * kOperand + lane * kTileBytes), &tmk, group,
                         full);
        }
      }
      __syncwarp();
      ++n;
    }
  } else if (warp == kQWarp) {
    // -------------------------------------------------------------- query tiles
    // The log-sum-exps of the next tile are on their way while this one waits for
    // its buffer (windows of 1024 rows: 288 -> 232 us).
    int tok_of[kCols / 32], off[kCols / 32];
#pragma unroll
    for (int i = 0; i < kCols / 32; ++i) {
      const int col = i * 32 + lane;
      tok_of[i] = col < QTb * G ? col / G : 1 << 30;
      off[i] = col / G * a.Hq + col % G;
    }
    Item t = item_at(P, S, Hkv, I0);
    int x = I0, c = 0, lq = 0, q0 = 0, nq = 0, qt = 0;
    auto settle = [&] {  // on the first item from x on with a tile to load
      while (x < I1) {
        c = P.ctx[t.s], lq = P.lq[t.s], q0 = P.q0[t.s], nq = tiles_of(t);
        if (nq > 0 && fresh_q(t, nq, x)) {
          qt = nq > 1 ? first_tile(key_tile(t), c, lq, QTb) : 0;
          return;
        }
        if (++x < I1) next_item(P, Hkv, t);
      }
    };
    float l[kCols / 32];
    auto fetch = [&] {
      if (x >= I1) return;
      const float* row = a.lse + ((int64_t)q0 + qt * QTb) * a.Hq + t.h * G;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i)
        l[i] = tok_of[i] < lq - qt * QTb ? row[off[i]] : neg_inf();
    };
    settle();
    fetch();
    for (int qn = 0; x < I1; ++qn) {
      const int b = qn % L::kQBufs;
      if (qn >= L::kQBufs &&
          !__all_sync(kFull, wait(B_QEMPTY + b, (uint32_t)(qn / L::kQBufs - 1) & 1u)))
        break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(B_QFULL + b), (uint32_t)(QTb * G) * 256u);
        const uint32_t d = smem_addr(smem + L::q + b * kOperand);
        tma_load_3d(d, &tmq, 0, t.h * G, q0 + qt * QTb, bar(B_QFULL + b));
        tma_load_3d(d + kHalfB, &tmq, 64, t.h * G, q0 + qt * QTb, bar(B_QFULL + b));
      }
      bool all = true;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int col = i * 32 + lane;
        const bool draws = l[i] != neg_inf();  // a query that saw nothing draws nothing
        // rounded once, to half a step of lse log2 e: exp is off by 2^-24 |lse| of
        // itself, about what the fp32 score is off by; its low part, which the warp
        // kernel carries, would take a second addition a column here (64 queries over
        // 1000..8192 keys: 5.2e-7 off the 64-bit sums, a plain fp32 form 2.8e-7)
        col_l2[b * kCols + col] = draws ? -(l[i] * kLog2e) : 0.f;
        col_last[b * kCols + col] = draws ? c - lq + qt * QTb + tok_of[i] : -1;
        all = all && draws;
      }
      all = __all_sync(kFull, all);
      if (lane == 0) col_clean[b] = all;
      __syncwarp();
      mbar_arrive(bar(B_QFULL + b));
      if (++qt >= nq) {
        if (++x < I1) next_item(P, Hkv, t);
        settle();
      }
      fetch();
    }
  } else if (warp == 1 || warp == kMma2Warp) {
    // -------------------------------------------------------------- products
    if (lane == 0) {
      const int me = warp == 1 ? 0 : 1;
      // one thread issues for the whole CTA: what does not change within a
      // sequence or at all is kept out of its loop (built anew for each item it
      // cost 1,700 cycles, more than the item's exponentials)
      const uint64_t desc_q = sw128_desc(smem_addr(smem + L::q), 16, 1024);
      // K: 8-row groups every 2 KB, each the two halves' 1 KB atoms
      const uint64_t desc_k = sw128_desc(smem_addr(smem + L::k), 16, 2048);
      Item t = item_at(P, S, Hkv, I0);
      int n = 0, qn = 0, dn = 0, c = 0, lq = 0, nq = 0;
      uint32_t idesc_last = 0;  // of the window's last tile
      bool ok = true, begun = false;
      for (int x = I0; ok && x < I1; ++x) {
        if (!begun || t.i == 0) {
          begun = true;
          c = P.ctx[t.s];
          lq = P.lq[t.s];
          nq = tiles_of(t);
          const int cols = min(kCols, (lq - (nq - 1) * QTb) * G);
          idesc_last = f16_idesc(kKeys, (cols + 15) & ~15, 0);
        }
        if (lq > 0) {
          const int st = n % L::kStages;
          // SPLIT: the two take tiles in turn, else items
          const bool item_mine = (n & 1) == me;
          if ((SPLIT || item_mine) && !wait(B_KFULL + st, (uint32_t)(n / L::kStages) & 1u)) break;
          const bool fresh = fresh_q(t, nq, x);
          const bool last_use = nq > 1 || t.i == t.nt - 1 || x + 1 == I1;
          const uint64_t dk = desc_k + (uint64_t)(st * (kOperand >> 4));
          for (int qt = nq > 1 ? first_tile(key_tile(t), c, lq, QTb) : 0; qt < nq; ++qt, ++dn) {
            if (fresh) {
              if (!wait(B_QFULL + qn % L::kQBufs, (uint32_t)(qn / L::kQBufs) & 1u)) {
                ok = false;
                break;
              }
              ++qn;
            }
            const int qb = (qn - 1) % L::kQBufs, db = dn % L::kDBufs;
            if (SPLIT ? (dn & 1) != me : !item_mine) {
              // The other's; this one's products with the query tile come first. The
              // epilogue answers for the thread that issues the tile's last product,
              // nobody for the one that does not: unless its having passed QFULL
              // counts, the buffer can be filled again before it has looked, two
              // phases that it cannot tell from none.
              if (last_use) {
                if (SPLIT)
                  mbar_arrive(bar(B_QEMPTY + qb));
                else
                  tc_commit(bar(B_QEMPTY + qb));
              }
              continue;
            }
            if (dn >= L::kDBufs && !wait(B_DEMPTY + db, (uint32_t)((dn / L::kDBufs) - 1) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t idesc =
                qt == nq - 1 ? idesc_last : f16_idesc(kKeys, (QTb * G + 15) & ~15, 0);
            const uint64_t dq = desc_q + (uint64_t)(qb * (kOperand >> 4));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint64_t dqk = dq + (uint64_t)(((k >> 2) * kHalfB + (k & 3) * 32) >> 4);
              if constexpr (L::q8)
                tc_mma_ts(tmem + (uint32_t)db * kCols,
                          tmem + L::kATmem + st * (kHeadDim / 2) + k * 8, dqk, idesc, k > 0);
              else
                tc_mma(tmem + (uint32_t)db * kCols,
                       dk + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), dqk, idesc, k > 0);
            }
            tc_commit(bar(B_DFULL + db));
            mbar_arrive(bar(B_DFULL + db));
            // the query tile is done with after its last product (SPLIT: when both
            // groups of the epilogue, who wait for every product, have arrived, and
            // the thread without that product has passed by)
            if (!SPLIT && last_use) tc_commit(bar(B_QEMPTY + qb));
          }
          if (SPLIT || item_mine) tc_commit(bar(B_KEMPTY + st));
          ++n;
        }
        if (x + 1 < I1) next_item(P, Hkv, t);
      }
    }
    __syncwarp();
  } else if (warp < kQWarp) {  // warps 2 .. 9
    // -------------------------------------------------------------- epilogue
    const int q4 = warp & 3, group = (warp - 2) >> 2;
    const int r = q4 * 32 + lane;  // this thread's key (tensor-memory lane)
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const float* kscale = reinterpret_cast<const float*>(smem + L::scale);
    Item t = item_at(P, S, Hkv, I0);
    float* part = reinterpret_cast<float*>(smem + L::part);
    int n = 0, qn = 0, dn = 0, pn = 0;
    int c = 0, lq = 0, nq = 0;
    float* row = nullptr;  // weights of the item's sequence and head
    bool ok = true, begun = false;
    for (int x = I0; ok && x < I1; ++x) {
      if (!begun || t.i == 0) {
        begun = true;
        c = P.ctx[t.s];
        lq = P.lq[t.s];
        nq = tiles_of(t);
        row = a.weights + ((int64_t)t.s * Hkv + t.h) * a.weights_len;
      }
      const int kt = key_tile(t), key = kt * kKeys + r;
      // the group that the item falls to (SPLIT: that writes it)
      const int mine = !SPLIT && lq > 0 ? n & 1 : 0;
      float old = 0.f;
      if (mine == group && a.accumulate && key < c - lq) old = row[key];
      float2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      if (lq > 0) {
        const bool fresh = fresh_q(t, nq, x);
        const bool last_use = nq > 1 || t.i == t.nt - 1 || x + 1 == I1;
        for (int qt = nq > 1 ? first_tile(kt, c, lq, QTb) : 0; qt < nq; ++qt, ++dn) {
          // both groups wait for a new query tile and release it, so that neither
          // runs a tile ahead
          if (fresh) {
            if (!__all_sync(kFull, wait(B_QFULL + qn % L::kQBufs, (uint32_t)(qn / L::kQBufs) & 1u))) {
              ok = false;
              break;
            }
            ++qn;
          }
          const int qb = (qn - 1) % L::kQBufs, db = dn % L::kDBufs;
          if (SPLIT || mine == group) {
            const int cols = min(kCols, min(QTb, lq - qt * QTb) * G);
            if (!__all_sync(kFull, wait(B_DFULL + db, (uint32_t)(dn / L::kDBufs) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            float sc = a.scale_log2;
            if constexpr (L::q8) sc *= kscale[(n % kScaleSlots) * kKeys + r];
            const float2 sc2 = make_float2(sc, sc);
            const uint32_t ta = tmem + lane_base + (uint32_t)db * kCols;
            // every key of the tile is seen by every column, and all are queries
            const bool clean = col_clean[qb] && kt * kKeys + kKeys <= c - lq + qt * QTb + 1;
            auto columns = [&](const uint32_t (&v)[32], int c0) {
              const float* l2 = col_l2 + qb * kCols + c0;
              if (clean) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float4 l = *reinterpret_cast<const float4*>(l2 + 4 * j);
                  const float2 z0 = __ffma2_rn(
                      make_float2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), sc2,
                      make_float2(l.x, l.y));
                  const float2 z1 = __ffma2_rn(
                      make_float2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])),
                      sc2, make_float2(l.z, l.w));
                  acc[(2 * j) & 3] =
                      __fadd2_rn(acc[(2 * j) & 3], make_float2(ex2(z0.x), ex2(z0.y)));
                  acc[(2 * j + 1) & 3] =
                      __fadd2_rn(acc[(2 * j + 1) & 3], make_float2(ex2(z1.x), ex2(z1.y)));
                }
              } else {
                const int* last = col_last + qb * kCols + c0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 l = *reinterpret_cast<const float2*>(l2 + 2 * j);
                  const int2 e = *reinterpret_cast<const int2*>(last + 2 * j);
                  const float z0 = fmaf(__uint_as_float(v[2 * j]), sc, l.x);
                  const float z1 = fmaf(__uint_as_float(v[2 * j + 1]), sc, l.y);
                  acc[j & 3] = __fadd2_rn(acc[j & 3], make_float2(ex2(key <= e.x ? z0 : neg_inf()),
                                                                  ex2(key <= e.y ? z1 : neg_inf())));
                }
              }
            };
            // 32 columns at a time; the other group's exponentials fill the wait for
            // them. (With the next 32 on their way during these, an epilogue warp
            // keeps its scheduler to itself: 37.9 us instead of 35.5 in bf16, 51
            // instead of 43.5 in FP8, where the codes' conversion waits for it.)
            const int c_lo = SPLIT ? group * (kCols / 2) : 0;
            const int c_hi = SPLIT ? min(cols, c_lo + kCols / 2) : cols;
            uint32_t v0[32];
#pragma unroll 1
            for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
              tmem_ld32(ta + (uint32_t)c0, v0);
              columns(v0, c0);
            }
            tc_fence_before();
            mbar_arrive(bar(B_DEMPTY + db));
          }
          if (last_use) mbar_arrive(bar(B_QEMPTY + qb));
        }
        if (!ok) break;
        ++n;
      }
      const float2 s2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      float sum = s2.x + s2.y;
      if (SPLIT && lq > 0) {
        // The second group's half goes through one of eight slots. It is at most
        // kDBufs items ahead: a tile is written anew only after both have read it.
        float* slot = part + (pn % kPartSlots) * kKeys + r;
        if (group == 1) {
          *slot = sum;
          mbar_arrive(bar(B_PART + pn % kPartSlots));
        } else {
          if (!__all_sync(kFull, wait(B_PART + pn % kPartSlots,
                                      (uint32_t)(pn / kPartSlots) & 1u)))
            break;
          sum += *slot;
        }
        ++pn;
      }
      if (mine == group && key < c) row[key] = old + sum;
      if (x + 1 < I1) next_item(P, Hkv, t);
    }
  } else if constexpr (L::q8) {
    // -------------------------------------------------------------- codes to bf16
    // thread = key row = tensor-memory lane: 128 codes of the swizzled raw tile to
    // the 64 columns of a K operand, which the products read from tensor memory
    // (a swizzled bf16 tile in shared memory and the fence that it needs: 64 us
    // instead of 61 for FP8 windows of 128 rows). The next item's codes are loaded
    // while this one's stores end (61 -> 51 us).
    // Row scales go to slot n mod 8: by the time slot n is written again, item
    // n + 8's, the accumulator of item n has been read (K stages and accumulators
    // between them hold fewer items).
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    float* kscale = reinterpret_cast<float*>(smem + L::scale);
    int m = 0;  // items with queries
    {
      Item t = item_at(P, S, Hkv, I0);
      for (int x = I0; x < I1; ++x) {
        m += P.lq[t.s] > 0;
        if (x + 1 < I1) next_item(P, Hkv, t);
      }
    }
    uint4 x16[8];  // 16 codes each; rows behind the context hold anything
    float scale = 0.f;
    auto load = [&](int n) {
      const int rs = n % L::kRawStages;
      const unsigned char* raw = smem + L::k + rs * kRawTile;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x16[i] = *reinterpret_cast<const uint4*>(raw + r * kHeadDim + ((i ^ (r & 7)) << 4));
      scale = *reinterpret_cast<const float*>(raw + kCodes + r * 4);
      mbar_arrive(bar(B_REMPTY + rs));
    };
    bool loaded = false;
    for (int n = 0; n < m; ++n) {
      const int st = n % L::kStages;
      if (!loaded) {
        if (!__all_sync(kFull, wait(B_RFULL + n % L::kRawStages, (uint32_t)(n / L::kRawStages) & 1u)))
          break;
        load(n);
      }
      if (n >= L::kStages &&
          !__all_sync(kFull, wait(B_KEMPTY + st, (uint32_t)((n / L::kStages) - 1) & 1u)))
        break;
      tc_fence_after();
      kscale[(n % kScaleSlots) * kKeys + r] = scale;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = x16[half * 4 + i];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            codes_to_bf16<FMT>(w[u], o[8 * i + 2 * u], o[8 * i + 2 * u + 1]);
        }
        tmem_st32(tmem + lane_base + L::kATmem + st * (kHeadDim / 2) + half * 32, o);
      }
      // the next item's codes, if they are there, come while the stores end
      loaded = n + 1 < m && __all_sync(kFull, mbar_test(bar(B_RFULL + (n + 1) % L::kRawStages),
                                                            (uint32_t)((n + 1) / L::kRawStages) & 1u));
      if (loaded) load(n + 1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(B_KFULL + st));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
}

template <int FMT>
size_t smem_bytes(int S, bool split) {
  return 1024 + (size_t)(split ? Lay<FMT, true>::plan : Lay<FMT, false>::plan) +
         sizeof(int) * (5 * (size_t)S + 2);
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, TcWeightArgs);

template <bool SPLIT>
Kernel kernel_for(int fmt) {
  return fmt == PA_KV_BF16   ? weights_tc_kernel<PA_KV_BF16, SPLIT>
         : fmt == PA_KV_INT8 ? weights_tc_kernel<PA_KV_INT8, SPLIT>
                             : weights_tc_kernel<PA_KV_FP8, SPLIT>;
}
Kernel kernel_of(int fmt, bool split) { return split ? kernel_for<true>(fmt) : kernel_for<false>(fmt); }

}  // namespace

int weights_tc_geometry(const pa_shape* sh, int max_q_len, int kv_format, WeightsTcGeometry* g) {
  g->enabled = false;
  const int G = sh->num_q_heads / sh->num_kv_heads;
  if (G > kCols || max_q_len < 1) return PA_OK;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  g->QTb = kCols / G < max_q_len ? kCols / G : max_q_len;
  g->split = max_q_len > g->QTb;
  g->smem = kv_format == PA_KV_BF16 ? smem_bytes<PA_KV_BF16>(sh->num_seqs, g->split)
                                    : smem_bytes<PA_KV_INT8>(sh->num_seqs, g->split);
  if (g->smem > (size_t)dev.max_smem_optin) return PA_OK;
  // costs are summed in 32 bits, and K's rows are 32-bit coordinates
  const int64_t tiles = (int64_t)sh->max_blocks_per_seq / kBlocksK + 1;
  const int64_t steps = (int64_t)(max_q_len + g->QTb - 1) / g->QTb + 1;
  if (steps > (int64_t(1) << 30) / sh->num_seqs / sh->num_kv_heads / tiles) return PA_OK;
  if (sh->num_blocks * sh->num_kv_heads * (kv_format == PA_KV_BF16 ? kBlock : 1) > 0x7fffffff)
    return PA_OK;
  if (!raise_smem_limit(reinterpret_cast<const void*>(kernel_of(kv_format, g->split))))
    return PA_ERR_CUDA;
  g->grid = dev.num_sms;
  g->enabled = true;
  return PA_OK;
}

int launch_weights_tc(const WeightsTcGeometry& g, const WeightArgs& a, int kv_format,
                      cudaStream_t st) {
  CUtensorMap tmq, tmk;
  if (!make_q_map(&tmq, a.q, a.num_q_tokens, a.Hq, a.G, g.QTb)) return PA_ERR_CUDA;
  if (kv_format == PA_KV_BF16 ? !make_block_map(&tmk, a.k_cache, a.num_blocks * a.Hkv * kBlock)
                              : !make_code_map(&tmk, a.k_cache, a.num_blocks * a.Hkv))
    return PA_ERR_CUDA;
  TcWeightArgs t;
  t.w = a;
  t.QTb = g.QTb;
  const int threads = kv_format == PA_KV_BF16 ? Lay<PA_KV_BF16, false>::threads : Lay<PA_KV_INT8, false>::threads;
  const cudaError_t e = launch_dependent(kernel_of(kv_format, g.split), dim3(g.grid), dim3(threads),
                                         g.smem, st, tmq, tmk, t);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

unsigned take_error_word_weights_tc(cudaStream_t stream, int* rc) {
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
