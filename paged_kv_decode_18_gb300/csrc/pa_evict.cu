// pa_evict.cu -- eviction from the paged cache by accumulated attention weight
// (course README "Build an LLM Inference Engine From Scratch", curriculum row
// "Memory & KV Cache"): per (sequence, KV head) the first `sinks` and the last
// `recent` positions stay, and of those between the ones that have drawn the
// most weight; what stays is moved together in order, in place.
//
// Selection is a radix select: four passes over the weights' 32-bit keys, each
// a 256-bin histogram of one byte among the keys that match the bytes found so
// far, give the key of the last position that stays and how many of its equals
// do (the lowest positions first). One ordered scan then lists the positions.
// Moving: the i-th row that stays comes from a position kept[i] >= i, and kept
// increases, so groups of rows that are read before any of them is written,
// group after group, never read a row that is already overwritten.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kMoveRows = 4;  // rows a warp holds between reading and writing

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

template <bool Q8>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_tot[kEvictWarps];
  __shared__ int found[2];  // digit, how many are still needed inside it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int h = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = a.context_lens[s];
  const int budget = a.budgets[s];
  int32_t* kept = a.kept + ((int64_t)s * a.Hkv + h) * a.max_budget;
  const int max_ctx = (int)min((int64_t)a.max_blocks * kBlock, a.weights_len);
  const bool bad_ctx = c < 0 || c > max_ctx;
  const bool bad_budget = budget > a.max_budget || budget < a.sinks + a.recent;
  if (bad_ctx || bad_budget) {  // the sequence stays as it is
    if (tid == 0 && h == 0) {
      flag_error(bad_ctx ? PA_DEVERR_CONTEXT_RANGE : PA_DEVERR_BUDGET_RANGE);
      a.new_lens[s] = c;
    }
    for (int i = tid; i < a.max_budget; i += kEvictThreads) kept[i] = -1;
    return;
  }
  const int n = min(c, budget);
  if (tid == 0 && h == 0) a.new_lens[s] = n;
  if (c <= budget) {
    for (int i = tid; i < a.max_budget; i += kEvictThreads) kept[i] = i < c ? i : -1;
    return;
  }
  float* w = a.weights + ((int64_t)s * a.Hkv + h) * a.weights_len;
  const int lo = a.sinks, hi = c - a.recent;  // positions to choose among
  int need = budget - a.sinks - a.recent;     // how many of them stay, < hi - lo
  // ---- the key of the last one that stays --------------------------------------
  uint32_t prefix = 0u;
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int p = lo + tid; p < hi; p += kEvictThreads) {
      const uint32_t key = weight_key(w[p]);
      if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l owns bins 255 - 8l .. 248 - 8l: running counts from the top
      int cnt[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cnt[i] = hist[255 - lane * 8 - i];
        sum += cnt[i];
      }
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      int run = x - sum;  // keys in higher bins
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (run < need && run + cnt[i] >= need) {
          found[0] = 255 - lane * 8 - i;
          found[1] = need - run;
        }
        run += cnt[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    need = found[1];
  }
  // ---- the positions that stay, in order ---------------------------------------
  // need: how many keys equal to prefix stay (0: nothing of the middle does)
  const bool some = budget > a.sinks + a.recent;
  int run_gt = 0, run_eq = 0;
  for (int p0 = 0; p0 < c; p0 += kEvictThreads) {
    const int p = p0 + tid;
    int gt = 0, eq = 0;
    if (p < c) {
      if (p < lo || p >= hi) {
        gt = 1;
      } else if (some) {
        const uint32_t key = weight_key(w[p]);
        gt = key > prefix;
        eq = key == prefix;
      }
    }
    const unsigned bg = __ballot_sync(kFull, gt), be = __ballot_sync(kFull, eq);
    if (lane == 0) warp_tot[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kEvictWarps; ++i) {
      const int t = warp_tot[i];
      if (i < warp) before += t;
      total += t;
    }
    __syncthreads();
    const unsigned below = (1u << lane) - 1u;
    const int ig = run_gt + (before & 0xffff) + __popc(bg & below);
    const int ie = run_eq + (before >> 16) + __popc(be & below);
    if (gt || (eq && ie < need)) kept[ig + min(ie, need)] = p;
    run_gt += total & 0xffff;
    run_eq += total >> 16;
  }
  for (int i = n + tid; i < a.max_budget; i += kEvictThreads) kept[i] = -1;
  __syncthreads();
  // ---- weights, then rows ---------------------------------------------------------
  for (int i0 = 0; i0 < n; i0 += 4 * kEvictThreads) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kEvictThreads + tid;
      if (i < n) x[u] = w[kept[i]];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kEvictThreads + tid;
      if (i < n) w[i] = x[u];
    }
  }
  PoolView pool;
  pool.k = a.k_cache;
  pool.v = a.v_cache;
  pool.table = a.block_tables + (int64_t)s * a.max_blocks;
  pool.num_blocks = a.num_blocks;
  pool.Hkv = a.Hkv;
  pool.h = h;
  for (int i0 = 0; i0 < n; i0 += kMoveRows * kEvictWarps) {
    uint4 x[kMoveRows];
    uint8_t* to[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      to[u] = nullptr;
      const int i = i0 + u * kEvictWarps + warp;
      if (i >= n) continue;
      const int src = kept[i];
      if (src == i) continue;
      RowPlace from, dst;
      const bool ok1 = pool.place(src, &from), ok2 = pool.place(i, &dst);
      if (!ok1 || !ok2) {
        if (lane == 0) flag_error(PA_DEVERR_BLOCK_RANGE);
        continue;
      }
      x[u] = load_chunk<Q8>(row_chunk<Q8>(pool, from, lane), lane);
      to[u] = row_chunk<Q8>(pool, dst, lane);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (to[u]) store_chunk<Q8>(to[u], lane, x[u]);
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
  auto kernel = kv_format == PA_KV_BF16 ? evict_kernel<false> : evict_kernel<true>;
  if (launch_dependent(kernel, dim3((unsigned)a.Hkv, (unsigned)shape->num_seqs),
                       dim3(kEvictThreads), 0, static_cast<cudaStream_t>(stream),
                       a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
