// pa_tree.cu -- the two ends of verifying a tree of drafted tokens
// (speculative decoding, "S20 - The Complete Engine", section "Core idea": step
// 3 PROPOSE, step 5 verify): the ancestor bits that the attention over the
// drafted window needs, and the commit that turns the accepted path's cached
// rows into the next tokens of the context.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// pa_tree_mask. Row j of a window: bit j and the bits of j's ancestors, found by
// following the parents (each smaller than its child, so a walk ends). A
// thread makes one 32-bit word of one row. The parents are staged in shared
// memory, so a step of a walk costs a shared-memory read: the call is bound by
// its launch and the longest chain, not by bytes (4 windows of 8 nodes 2.6 us,
// 256 of 20..64 nodes 3.1 us a call among others).
// ---------------------------------------------------------------------------
constexpr int kMaskThreads = 128;
constexpr int kMaskStage = 8192;  // parents staged in shared memory (32 KB); longer windows read global

__global__ void __launch_bounds__(kMaskThreads)
    tree_mask_kernel(const int32_t* parents, const int32_t* cu, int64_t num_q_tokens,
                     int max_q_len, int words, uint32_t* __restrict__ mask,
                     int32_t* __restrict__ depths) {
  extern __shared__ int32_t sp[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x;
  const int q0 = cu[s], lq = cu[s + 1] - q0;
  if (q0 < 0 || lq < 0 || lq > max_q_len || (int64_t)q0 + lq > num_q_tokens) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(PA_DEVERR_QLEN_RANGE);
    return;
  }
  const bool staged = lq <= kMaskStage;
  bool bad = false;
  if (staged) {
    for (int j = threadIdx.x; j < lq; j += blockDim.x) {
      const int p = parents[(int64_t)q0 + j];
      bad = bad || p < -1 || p >= j;
      sp[j] = p < -1 || p >= j ? -1 : p;  // a bad parent makes its node a root
    }
    __syncthreads();
  }
  auto parent = [&](int j) -> int {
    if (staged) return sp[j];
    const int p = parents[(int64_t)q0 + j];
    if (p < -1 || p >= j) {
      bad = true;
      return -1;
    }
    return p;
  };
  const int64_t items = (int64_t)lq * words;
  for (int64_t it = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; it < items;
       it += (int64_t)gridDim.y * blockDim.x) {
    const int j = (int)(it / words), w = (int)(it - (int64_t)j * words);
    uint32_t bits = 0u;
    int depth = -1;
    // the ancestors below this word's first bit matter for the depth alone
    for (int a = j; a >= 0 && (a >= w * 32 || w == 0); a = parent(a)) {
      if ((a >> 5) == w) bits |= 1u << (a & 31);
      ++depth;
    }
    mask[((int64_t)q0 + j) * words + w] = bits;
    if (w == 0 && depths) depths[(int64_t)q0 + j] = depth;
  }
  if (bad) flag_error(PA_DEVERR_TREE_RANGE);
}

// ---------------------------------------------------------------------------
// pa_commit_path. One CTA per sequence, one warp per KV head at a time. A path
// of increasing window indices has path[i] >= i, so a warp that reads a group
// of rows before it writes any of them, group after group, never reads a row
// that it has already written. The call is a chain of dependent reads -- the
// lengths and the path, the block table, the rows -- so lane i looks up row i
// of 32 at once. 4 windows 3.2 us, 256 windows of an int8 pool (5.4 MB) 5.2 us.
// ---------------------------------------------------------------------------
constexpr int kCommitWarps = 8;
constexpr int kCommitGroup = 8;  // rows a warp holds between reading and writing

template <bool Q8>
__global__ void __launch_bounds__(kCommitWarps * 32)
    commit_path_kernel(uint8_t* k_cache, uint8_t* v_cache,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* cu, const int32_t* path, const int32_t* path_lens,
                       int max_path_len,
                       int32_t* new_lens, int max_blocks, int64_t num_blocks, int Hkv) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* row = path + (int64_t)s * max_path_len;
  // path entries base + lane - 1 and base + lane (-1 before the first)
  auto entry = [&](int base, int& before) -> int {
    const int i = base + lane;
    const int x = i < max_path_len ? row[i] : 0;
    before = __shfl_up_sync(kFull, x, 1);
    if (lane == 0) before = base > 0 ? row[base - 1] : -1;
    return x;
  };
  int before;
  const int x0 = entry(0, before);  // read beside the lengths, whether used or not
  const int c = context_lens[s], n = path_lens[s];
  const int lq = cu[s + 1] - cu[s];
  const bool bad_ctx = c < 0 || c > max_blocks * kBlock;
  const bool bad_len = lq < 0 || lq > c;
  bool bad_path = n < 0 || n > max_path_len || n > lq;
  if (!bad_ctx && !bad_len && !bad_path) {
    // increasing from -1 and below lq; every warp checks the whole path
    bad_path = lane < n && (x0 <= before || x0 >= lq);
    for (int base = 32; base < n; base += 32) {
      const int x = entry(base, before);
      bad_path = bad_path || (base + lane < n && (x <= before || x >= lq));
    }
    bad_path = __any_sync(kFull, bad_path);
  }
  const int p0 = c - lq;
  if (bad_ctx || bad_len || bad_path) {  // the sequence stays as it is
    if (threadIdx.x == 0)
      flag_error(bad_ctx ? PA_DEVERR_CONTEXT_RANGE
                         : (bad_len ? PA_DEVERR_QLEN_RANGE : PA_DEVERR_TREE_RANGE));
  } else {
    PoolView pool;
    pool.k = k_cache;
    pool.v = v_cache;
    pool.table = block_tables + (int64_t)s * max_blocks;
    pool.num_blocks = num_blocks;
    pool.Hkv = Hkv;
    for (int base = 0; base < n; base += 32) {
      const int src = base == 0 ? x0 : entry(base, before);
      const int i = base + lane;
      // tiles of head 0 and rows of where lane's row comes from and goes to
      bool moves = i < n && src != i;
      RowPlace from{0, 0}, to{0, 0};
      pool.h = 0;
      if (moves) {
        const bool ok1 = pool.place(p0 + src, &from), ok2 = pool.place(p0 + i, &to);
        if (!ok1 || !ok2) {
          if (warp == 0) flag_error(PA_DEVERR_BLOCK_RANGE);
          moves = false;
        }
      }
      const unsigned moving = __ballot_sync(kFull, moves);
      for (int h = warp; h < Hkv; h += kCommitWarps) {
        unsigned m = moving;
        while (m) {
          uint4 x[kCommitGroup];
          uint8_t* dst[kCommitGroup];
#pragma unroll
          for (int u = 0; u < kCommitGroup; ++u) {
            dst[u] = nullptr;
            if (!m) continue;
            const int j = __ffs(m) - 1;
            m &= m - 1;
            RowPlace f, d;
            f.tile = __shfl_sync(kFull, from.tile, j) + h;
            f.off = __shfl_sync(kFull, from.off, j);
            d.tile = __shfl_sync(kFull, to.tile, j) + h;
            d.off = __shfl_sync(kFull, to.off, j);
            x[u] = load_chunk<Q8>(row_chunk<Q8>(pool, f, lane), lane);
            dst[u] = row_chunk<Q8>(pool, d, lane);
          }
          __syncwarp();
#pragma unroll
          for (int u = 0; u < kCommitGroup; ++u)
            if (dst[u]) store_chunk<Q8>(dst[u], lane, x[u]);
        }
      }
    }
  }
  // new_lens may be context_lens: every warp has read it
  __syncthreads();
  if (threadIdx.x == 0) new_lens[s] = bad_ctx || bad_len || bad_path ? c : p0 + n;
}

}  // namespace

unsigned take_error_word_tree(cudaStream_t stream, int* rc) {
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

extern "C" int pa_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, int num_seqs,
                            int64_t num_q_tokens, int max_q_len, uint32_t* tree_mask,
                            int mask_words, int32_t* depths, void* stream) {
  pa::NvtxRange nvtx_range("pa_tree_mask");
  if (num_seqs < 0 || num_q_tokens < 0 || num_q_tokens > 0x3fffffff || max_q_len < 0 ||
      mask_words < 0 || mask_words > (1 << 20) || max_q_len > (int64_t)mask_words * 32)
    return PA_ERR_ARG;
  if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
  if (max_q_len == 0) return PA_ERR_ARG;  // rows, but no window may hold one
  if (!parents || !cu_seqlens_q || !tree_mask) return PA_ERR_ARG;
  if (!aligned(parents, 4) || !aligned(cu_seqlens_q, 4) || !aligned(tree_mask, 4) ||
      (depths && !aligned(depths, 4)))
    return PA_ERR_ARG;
  const int stage = max_q_len < kMaskStage ? max_q_len : kMaskStage;
  const int64_t items = (int64_t)max_q_len * mask_words;
  const int64_t ctas = (items + 8 * kMaskThreads - 1) / (8 * kMaskThreads);
  const unsigned gy = (unsigned)(ctas < 1 ? 1 : (ctas > 1024 ? 1024 : ctas));
  if (launch_dependent(tree_mask_kernel, dim3((unsigned)num_seqs, gy), dim3(kMaskThreads),
                       sizeof(int32_t) * (size_t)stage, static_cast<cudaStream_t>(stream),
                       parents, cu_seqlens_q, num_q_tokens, max_q_len, mask_words, tree_mask,
                       depths) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

extern "C" int pa_commit_path(void* k_cache, void* v_cache, int kv_format,
                              const int32_t* block_tables, const int32_t* context_lens,
                              const int32_t* cu_seqlens_q, const int32_t* path,
                              const int32_t* path_lens, int max_path_len, int32_t* new_lens,
                              const pa_shape* shape, void* stream) {
  pa::NvtxRange nvtx_range("pa_commit_path");
  int rc = check_shape_common(shape);
  if (rc != PA_OK) return rc;
  if (kv_format != PA_KV_BF16 && kv_format != PA_KV_INT8 && kv_format != PA_KV_FP8)
    return PA_ERR_ARG;
  if (max_path_len < 0) return PA_ERR_ARG;
  if (shape->num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !cu_seqlens_q || !path_lens ||
      !new_lens || (max_path_len > 0 && !path))
    return PA_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4) || !aligned(new_lens, 4))
    return PA_ERR_ARG;
  // a sequence's new length may replace its old one, not another's
  if (new_lens != context_lens && context_lens < new_lens + shape->num_seqs &&
      new_lens < context_lens + shape->num_seqs)
    return PA_ERR_ARG;
  auto kernel = kv_format == PA_KV_BF16 ? commit_path_kernel<false> : commit_path_kernel<true>;
  if (launch_dependent(kernel, dim3((unsigned)shape->num_seqs), dim3(kCommitWarps * 32), 0,
                       static_cast<cudaStream_t>(stream), static_cast<uint8_t*>(k_cache),
                       static_cast<uint8_t*>(v_cache), block_tables, context_lens, cu_seqlens_q,
                       path, path_lens, max_path_len, new_lens, shape->max_blocks_per_seq,
                       shape->num_blocks, shape->num_kv_heads) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
