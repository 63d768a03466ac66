// pa_evict.cu -- eviction from the paged cache by accumulated attention weight
// (course README "Build an LLM Inference Engine From Scratch", curriculum row
// "Memory & KV Cache"): per (sequence, KV head) the first `sinks` and the last
// `recent` positions stay, and of those between the ones that have drawn the
// most weight; what stays is moved together in order, in place.
//
// A cluster of CTAs serves one (sequence, KV head), each a slice of the
// positions, read once into shared memory. Selection is a radix select: four
// passes over the weights' 32-bit keys, each a 256-bin histogram of the next
// byte among the keys that match the bits found so far, summed over the
// cluster through distributed shared memory; they give the key of the last
// position that stays and how many of its equals do (the lowest positions
// first). The first eight bits are a sign and an exponent, which most weights
// share: that histogram has a column a lane, so that no two lanes of a warp add
// to one word. (Longer digits make fewer passes, but 4096 bins read from every
// CTA of the cluster cost more than a pass: 102 us against 54 us at 8 x 32k.)
// An ordered scan then lists the positions.
// Moving: the i-th row that stays comes from a position kept[i] >= i, and kept
// increases. So the rows go in waves of as many as the cluster's shared memory
// holds twice over: all CTAs read their rows of a wave, the cluster meets, all
// write. A wave's writes fall before every later wave's sources, so the next
// wave's reads begin before the cluster has met.
// Bound: HBM for large moves, the chain of passes and meetings for small ones.
// Calls one after another, each on caches and weights of its own that no call has
// touched since they left L2: 8 contexts of 30,000..32,768 positions, 8 KV heads,
// int8, cut to 4096: 51 us, weights of 8 MB read and 4080 rows a head moved, 149 MB
// or 2.9 TB/s; 32 of 1030..1153, bf16, to 1024: 46 us for 785 rows a head, 210 MB or
// 4.5 TB/s. (A call on a cache that is still in L2 is faster: 25 us for the second.)
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kMaxCluster = 8;
// Shared memory: the first pass's histogram, two of a CTA's sums, the slice's
// weights; later a wave's rows. Two CTAs an SM.
constexpr int kBins = 256;
constexpr int kOffB = kBins * 32 * 4;
constexpr int kOffSlice = kOffB + 2 * kBins * 4;
constexpr int kArea = 112 * 1024;
constexpr int kSliceMax = (kArea - kOffSlice) / 4;  // a longer slice is read again each time
constexpr int kEvictSmem = kArea + (3 * kEvictWarps + 4) * 4;
template <bool Q8>
constexpr int kRowBytes = Q8 ? 2 * kHeadDim : 4 * kHeadDim;  // a row's K and V (8-bit: the codes)
// rows of a wave a warp (two waves' rows are in shared memory): data, and 16
// bytes for the weight and the 8-bit scales
template <bool Q8>
constexpr int kWarpRows = kArea / 2 / (kRowBytes<Q8> + 16) / kEvictWarps / (Q8 ? 2 : 1) * (Q8 ? 2 : 1);

struct EvictArgs {
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* weights;
  int64_t weights_len;  // row length of weights
  const int32_t* budgets;
  int max_budget, sinks, recent;
  int32_t* kept;
  int32_t* new_lens;
  int max_blocks, Hkv;
  int64_t num_blocks;
};

// Order-preserving integer of a weight: larger weight, larger key; -0 counts as
// 0 and a NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster meet; what they wrote (shared and global memory)
// is seen by all afterwards.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at this CTA's shared address `p`, in CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_load(const int* p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool Q8>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const EvictArgs a) {
  extern __shared__ __align__(128) unsigned char area[];
  int* warp_tot = reinterpret_cast<int*>(area + kArea);  // [kEvictWarps]
  int* run_tot = warp_tot + kEvictWarps;   // [2][kEvictWarps] keys above the last one, equal to it
  int* found = run_tot + 2 * kEvictWarps;  // digit, how many are still needed inside it
  int* counts = found + 2;                 // run_tot summed over this CTA
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
  const int h = (int)blockIdx.x / ctas, s = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gtid = rank * kEvictThreads + tid, gthreads = ctas * kEvictThreads;
  const int c = a.context_lens[s];
  const int budget = a.budgets[s];
  int32_t* kept = a.kept + ((int64_t)s * a.Hkv + h) * a.max_budget;
  const int max_ctx = (int)min((int64_t)a.max_blocks * kBlock, a.weights_len);
  const bool bad_ctx = c < 0 || c > max_ctx;
  const bool bad_budget = budget > a.max_budget || budget < a.sinks + a.recent;
  if (bad_ctx || bad_budget) {  // the sequence stays as it is
    if (gtid == 0 && h == 0) {
      flag_error(bad_ctx ? PA_DEVERR_CONTEXT_RANGE : PA_DEVERR_BUDGET_RANGE);
      a.new_lens[s] = c;
    }
    for (int i = gtid; i < a.max_budget; i += gthreads) kept[i] = -1;
    return;
  }
  const int n = min(c, budget);
  if (gtid == 0 && h == 0) a.new_lens[s] = n;
  if (c <= budget) {
    for (int i = gtid; i < a.max_budget; i += gthreads) kept[i] = i < c ? i : -1;
    return;
  }
  float* w = a.weights + ((int64_t)s * a.Hkv + h) * a.weights_len;
  // ---- this CTA's slice of the positions to choose among --------------------------
  const int lo = a.sinks, hi = c - a.recent;
  const int per = (hi - lo + ctas - 1) / ctas;
  const int p0 = min(hi, lo + rank * per), p1 = min(hi, p0 + per), len = p1 - p0;
  const bool held = per <= kSliceMax;
  uint32_t* slice = reinterpret_cast<uint32_t*>(area + kOffSlice);  // keys
  if (held) {
    for (int i = tid; i < len; i += 8 * kEvictThreads) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * kEvictThreads < len) x[u] = w[p0 + i + u * kEvictThreads];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * kEvictThreads < len) slice[i + u * kEvictThreads] = weight_key(x[u]);
    }
  }
  auto key_of = [&](int i) { return held ? slice[i] : weight_key(w[p0 + i]); };
  // every key of [i, end) in steps of `step`, several reads on their way at once
  auto each_key = [&](int i, int end, int step, auto&& use) {
    for (; i + 3 * step < end; i += 4 * step) {
      const uint32_t k0 = key_of(i), k1 = key_of(i + step), k2 = key_of(i + 2 * step),
                     k3 = key_of(i + 3 * step);
      use(k0);
      use(k1);
      use(k2);
      use(k3);
    }
    for (; i < end; i += step) use(key_of(i));
  };
  // ---- the key of the last one that stays -----------------------------------------
  int need = budget - a.sinks - a.recent;  // how many of the middle stay, < hi - lo
  const bool some = need > 0;
  uint32_t prefix = 0u;
  if (some) {
    // clearing and adding up the columns pays from some thousand weights on
    const bool columns = per > 2048;
    for (int i = (columns ? 0 : kOffB / 16) + tid; i < kOffSlice / 16; i += kEvictThreads)
      reinterpret_cast<int4*>(area)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int pass = 0, shift = 24; pass < 4; ++pass, shift -= 8) {
      int* hs = reinterpret_cast<int*>(area + kOffB) + (pass & 1) * kBins;
      if (pass == 0 && columns) {
        int* ha = reinterpret_cast<int*>(area);
        each_key(tid, len, kEvictThreads,
                 [&](uint32_t key) { atomicAdd(&ha[(key >> 24) * 32 + lane], 1); });
        __syncthreads();
        // two threads a bin, sixteen columns each, beginning at their own so that
        // a warp's reads fall into different banks
        int sum = 0;
        const int* col = ha + (tid >> 1) * 32 + (tid & 1) * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += col[(i + (lane >> 1)) & 15];
        sum += __shfl_xor_sync(kFull, sum, 1);
        if (!(tid & 1)) hs[tid >> 1] = sum;
      } else {
        if (pass >= 2) {  // read by the cluster two passes ago: all have met since
          if (tid < kBins) hs[tid] = 0;
          __syncthreads();
        }
        const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
        each_key(tid, len, kEvictThreads, [&](uint32_t key) {
          if ((key & above) == prefix) atomicAdd(&hs[(key >> shift) & 255u], 1);
        });
      }
      cluster_meet();
      // thread t owns bin 255 - t
      int sum = 0;
      if (tid < kBins)
        for (int r = 0; r < ctas; ++r) sum += cluster_load(&hs[kBins - 1 - tid], (uint32_t)r);
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_tot[warp] = x;
      __syncthreads();
      // keys in higher bins
      const int run = x - sum + __reduce_add_sync(kFull, lane < warp ? warp_tot[lane] : 0);
      if (run < need && run + sum >= need) {
        found[0] = kBins - 1 - tid;
        found[1] = need - run;
      }
      __syncthreads();
      prefix |= (uint32_t)found[0] << shift;
      need = found[1];
    }
  }
  // ---- the positions that stay, in order ------------------------------------------
  // need: how many keys equal to prefix stay. A warp scans a run of the slice.
  const int wlen = (len + kEvictWarps - 1) / kEvictWarps;
  const int i0 = min(len, warp * wlen), i1 = min(len, i0 + wlen);
  int gt = 0, eq = 0;  // of this warp's run
  if (some) {
    each_key(i0 + lane, i1, 32, [&](uint32_t key) {
      gt += key > prefix;
      eq += key == prefix;
    });
    gt = __reduce_add_sync(kFull, gt);
    eq = __reduce_add_sync(kFull, eq);
  }
  int before_gt = 0, before_eq = 0;
  {
    if (lane == 0) {
      run_tot[warp] = gt;
      run_tot[kEvictWarps + warp] = eq;
    }
    __syncthreads();
    const int g = lane < kEvictWarps ? run_tot[lane] : 0;
    const int e = lane < kEvictWarps ? run_tot[kEvictWarps + lane] : 0;
    before_gt = __reduce_add_sync(kFull, lane < warp ? g : 0);
    before_eq = __reduce_add_sync(kFull, lane < warp ? e : 0);
    const int tg = __reduce_add_sync(kFull, g), te = __reduce_add_sync(kFull, e);
    if (tid == 0) {
      counts[0] = tg;
      counts[1] = te;
    }
  }
  cluster_meet();
  for (int r = 0; r < rank; ++r) {
    before_gt += cluster_load(&counts[0], (uint32_t)r);
    before_eq += cluster_load(&counts[1], (uint32_t)r);
  }
  if (some) {
    for (int i = i0; i < i1; i += 32) {
      const bool in = i + lane < i1;
      const uint32_t key = in ? key_of(i + lane) : 0u;
      const unsigned bg = __ballot_sync(kFull, in && key > prefix);
      const unsigned be = __ballot_sync(kFull, in && key == prefix);
      const unsigned below = (1u << lane) - 1u;
      const int ig = before_gt + __popc(bg & below), ie = before_eq + __popc(be & below);
      if (((bg >> lane) & 1u) || (((be >> lane) & 1u) && ie < need))
        kept[lo + ig + min(ie, need)] = p0 + i + lane;
      before_gt += __popc(bg);
      before_eq += __popc(be);
    }
  }
  for (int i = gtid; i < lo; i += gthreads) kept[i] = i;
  for (int i = gtid; i < a.recent; i += gthreads) kept[n - a.recent + i] = hi + i;
  for (int i = n + gtid; i < a.max_budget; i += gthreads) kept[i] = -1;
  cluster_meet();  // the list is complete, and nobody reads the weights by slices any more
  // ---- weights and rows, wave by wave ---------------------------------------------
  constexpr int kMine = kWarpRows<Q8>, kRow = kRowBytes<Q8>, kRows = kMine * kEvictWarps;
  static_assert(kMine <= 32, "a lane a row");
  // this warp's rows in each half of the area
  unsigned char* data = area + (size_t)warp * kMine * kRow;
  unsigned char* aux = area + (size_t)kRows * kRow + ((size_t)warp * kMine + lane) * 16;
  constexpr int kHalfArea = kRows * (kRow + 16);
  static_assert(2 * kHalfArea <= kArea, "two waves");
  PoolView pool;
  pool.k = a.k_cache;
  pool.v = a.v_cache;
  pool.table = a.block_tables + (int64_t)s * a.max_blocks;
  pool.num_blocks = a.num_blocks;
  pool.Hkv = a.Hkv;
  pool.h = h;
  // 16-byte chunks of a row: bf16 one row of 16 + 16 (K, V), 8-bit two rows of 8 + 8
  constexpr int kAtOnce = Q8 ? 2 : 1, kHalfChunks = Q8 ? 8 : 16;
  const int sub = Q8 ? lane >> 4 : 0, chunk = lane & (2 * kHalfChunks - 1);
  uint8_t* mybase = (chunk < kHalfChunks ? a.k_cache : a.v_cache) + (chunk & (kHalfChunks - 1)) * 16;
  auto row_at = [&](const RowPlace& p) -> int64_t {  // byte offset of a row's data in K and V
    return Q8 ? p.tile * kInt8TileBytes + p.off * kHeadDim
              : (p.tile * kBlock + p.off) * (kHeadDim * 2);
  };
  // lane j looks up row j of the warp's: where it comes from and goes to (-1: stays)
  struct Move {
    int64_t from, to;
    int64_t scale_from, scale_to;  // 8-bit: byte offsets of the scales
    int src;
  };
  auto look_up = [&](int base) -> Move {
    Move m{-1, -1, 0, 0, 0};
    const int i = base + rank * kRows + warp * kMine + lane;
    if (lane < kMine && i < n) {
      m.src = kept[i];
      RowPlace from, to;
      if (m.src != i) {
        const bool ok1 = pool.place(m.src, &from), ok2 = pool.place(i, &to);
        if (ok1 && ok2) {
          m.from = row_at(from);
          m.to = row_at(to);
          if (Q8) {
            m.scale_from = from.tile * kInt8TileBytes + kBlock * kHeadDim + from.off * 4;
            m.scale_to = to.tile * kInt8TileBytes + kBlock * kHeadDim + to.off * 4;
          }
        } else {
          flag_error(PA_DEVERR_BLOCK_RANGE);
        }
      }
    }
    return m;
  };
  auto read_rows = [&](const Move& m, int half) {
    const uint32_t x = smem_addr(aux + half * kHalfArea);
    if (m.from >= 0) {
      copy4_async(x + 8, w + m.src);
      if (Q8) {
        copy4_async(x, a.k_cache + m.scale_from);
        copy4_async(x + 4, a.v_cache + m.scale_from);
      }
    }
    const uint32_t d = smem_addr(data + half * kHalfArea) + lane * 16;
#pragma unroll
    for (int j = 0; j < kMine; j += kAtOnce) {
      const int64_t f = __shfl_sync(kFull, m.from, j + sub);
      if (f >= 0) copy16_async(d + j * kRow, mybase + f);
    }
  };
  const int step = ctas * kRows;
  Move mv = look_up(0);
  read_rows(mv, 0);
  Move next = look_up(step);
  for (int base = 0, half = 0; base < n; base += step, half ^= 1) {
    // this wave's rows are here; while the others' land too, the next wave's set
    // out (their sources lie behind everything that this wave writes). Relaxed: the
    // meeting keeps reads before others' writes, and these reads have ended; an
    // arrival that also waits for this CTA's last writes costs 2 to 5 % of a call.
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    read_rows(next, half ^ 1);
    const Move after = look_up(base + 2 * step);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < kMine; j += kAtOnce) {
      const int64_t to = __shfl_sync(kFull, mv.to, j + sub);
      if (to >= 0)
        *reinterpret_cast<uint4*>(mybase + to) =
            *reinterpret_cast<const uint4*>(data + half * kHalfArea + j * kRow + lane * 16);
    }
    if (mv.from >= 0) {
      const float* x = reinterpret_cast<const float*>(aux + half * kHalfArea);
      w[base + rank * kRows + warp * kMine + lane] = x[2];
      if (Q8) {
        *reinterpret_cast<float*>(a.k_cache + mv.scale_to) = x[0];
        *reinterpret_cast<float*>(a.v_cache + mv.scale_to) = x[1];
      }
    }
    __syncwarp();  // this half is read before the copies of the wave after next
    mv = next;
    next = after;
  }
}

}  // namespace

unsigned take_error_word_evict(cudaStream_t stream, int* rc) {
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

extern "C" int pa_evict(void* k_cache, void* v_cache, int kv_format, const int32_t* block_tables,
                        const int32_t* context_lens, float* weights, int64_t weights_len,
                        const int32_t* budgets, int max_budget, int num_sinks, int num_recent,
                        int32_t* kept, int32_t* new_lens, const pa_shape* shape, void* stream) {
  pa::NvtxRange nvtx_range("pa_evict");
  int rc = check_shape_common(shape);
  if (rc != PA_OK) return rc;
  if (kv_format != PA_KV_BF16 && kv_format != PA_KV_INT8 && kv_format != PA_KV_FP8)
    return PA_ERR_ARG;
  if (weights_len < 0 || max_budget < 0 || max_budget > (1 << 30) || num_sinks < 0 ||
      num_recent < 0 || (int64_t)num_sinks + num_recent > max_budget)
    return PA_ERR_ARG;
  if (shape->num_seqs > 65535) return PA_ERR_UNSUPPORTED;  // grid rows
  if (shape->num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !weights || !budgets ||
      (!kept && max_budget > 0) || !new_lens)
    return PA_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(weights, 4) || !aligned(budgets, 4) ||
      !aligned(kept, 4) || !aligned(new_lens, 4))
    return PA_ERR_ARG;
  // every (sequence, KV head) reads context_lens and budgets while one writes new_lens
  auto overlaps = [&](const int32_t* x) {
    return x < new_lens + shape->num_seqs && new_lens < x + shape->num_seqs;
  };
  if (overlaps(context_lens) || overlaps(budgets)) return PA_ERR_ARG;
  EvictArgs a;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.weights = weights;
  a.weights_len = weights_len;
  a.budgets = budgets;
  a.max_budget = max_budget;
  a.sinks = num_sinks;
  a.recent = num_recent;
  a.kept = kept;
  a.new_lens = new_lens;
  a.max_blocks = shape->max_blocks_per_seq;
  a.Hkv = shape->num_kv_heads;
  a.num_blocks = shape->num_blocks;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  const bool q8 = kv_format != PA_KV_BF16;
  auto kernel = q8 ? evict_kernel<true> : evict_kernel<false>;
  if (!raise_smem_limit(reinterpret_cast<const void*>(kernel))) return PA_ERR_CUDA;
  // clusters as large as leave every (sequence, KV head) resident at two CTAs an
  // SM (twice as large, in two rounds: 41 us against 28.6 us at 8 x 32k in L2), but
  // no larger than a slice of 1024 positions calls for in the longest context that
  // the table has room for -- the host knows no other bound. With a table of 32768
  // positions the 32 contexts of 1030..1153 take the same 46 us.
  const int64_t heads = (int64_t)shape->num_seqs * a.Hkv;
  const int64_t most = (int64_t)a.max_blocks * kBlock / 1024;
  int cluster = 1;
  while (cluster < kMaxCluster && heads * cluster * 2 <= 2 * dev.num_sms && cluster * 2 <= most)
    cluster *= 2;
  if (launch_dependent_cluster(kernel, dim3((unsigned)(a.Hkv * cluster), (unsigned)shape->num_seqs),
                               dim3(kEvictThreads), kEvictSmem, cluster,
                               static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
