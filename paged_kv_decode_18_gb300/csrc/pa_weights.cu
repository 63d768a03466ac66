// pa_weights.cu -- attention weight that each cached position has drawn:
//   w[s][h][p] (+)= sum over the window's queries j that see p and the group's
//                   heads g of exp(scale q_jg . k_p - lse_jg)
// from the log-sum-exp that an attention call over the same queries returned,
// so one pass over K is enough (course README "Build an LLM Inference Engine
// From Scratch", curriculum row "Memory & KV Cache": what a cache keeps).
//
// A warp owns 16 consecutive positions (one block) of one KV head and all of
// their queries, so every weight has one writer and the sums have one order.
// S^T = K Q^T on mma.sync m16n8k16: rows are positions, columns eight query
// rows. The contraction does not care in which order it meets the head
// dimensions, so a lane takes 16-byte pieces of its two K rows and of its
// query column straight from global memory as fragments (no shared memory):
// the fragment's two k pairs of a step are neighbouring pairs of the piece.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_weights.cuh"

namespace pa {
namespace {

constexpr int kWgtWarps = 8;
constexpr int kWgtTcRows = 16;  // windows with more query rows a KV head go to the tcgen05 kernel

// One warp's K tile as loaded: two rows per lane. bf16: four 16-byte pieces a
// row (dims (4i + quad) * 8 ..); 8-bit: two (dims (4i + quad) * 16 ..) and the
// rows' scales.
template <int FMT>
struct KTile {
  static constexpr int kPieces = FMT == PA_KV_BF16 ? 4 : 2;
  uint4 x[2][kPieces];
  float scale[2];
};

template <int FMT>
__device__ __forceinline__ void load_k(const WeightArgs& a, int64_t tile, int lane,
                                       KTile<FMT>& t) {
  const int r0 = lane >> 2, quad = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + 8 * i;
    if constexpr (FMT == PA_KV_BF16) {
      const uint8_t* p = a.k_cache + (tile * kBlock + row) * (kHeadDim * 2) + quad * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) t.x[i][j] = __ldg(reinterpret_cast<const uint4*>(p + j * 64));
    } else {
      const uint8_t* p = a.k_cache + tile * kInt8TileBytes;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        t.x[i][j] =
            __ldg(reinterpret_cast<const uint4*>(p + row * kHeadDim + j * 64 + quad * 16));
      t.scale[i] = __ldg(reinterpret_cast<const float*>(p + kBlock * kHeadDim) + row);
    }
  }
}

// The A fragments of the tile: step t's k pairs are pairs 2t and 2t + 1 of the
// lane's values in order.
template <int FMT>
__device__ __forceinline__ void fragments(const KTile<FMT>& t, uint32_t (&f)[8][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < KTile<FMT>::kPieces; ++j) {
      const uint32_t w[4] = {t.x[i][j].x, t.x[i][j].y, t.x[i][j].z, t.x[i][j].w};
      if constexpr (FMT == PA_KV_BF16) {
        f[2 * j][i] = w[0];
        f[2 * j][2 + i] = w[1];
        f[2 * j + 1][i] = w[2];
        f[2 * j + 1][2 + i] = w[3];
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          f[4 * j + u][i] = codes_to_bf16x2<FMT>(w[u] & 0xffffu);
          f[4 * j + u][2 + i] = codes_to_bf16x2<FMT>(w[u] >> 16);
        }
      }
    }
  }
}

// The B fragments of eight query rows (column = lane / 4) and the columns'
// log-sum-exps in log2 units, as a leading part and the rest; a column that is
// no query, or whose query saw nothing, sees no position here.
struct QTile {
  uint32_t b[8][2];
  float l2[2], l2lo[2];
  int last[2];  // last position that each of the lane's two columns sees
};

template <int FMT>
__device__ __forceinline__ void load_q(const WeightArgs& a, int64_t q0, int lq, int c, int h,
                                       int col0, int lane, QTile& t) {
  const int quad = lane & 3, rows = lq * a.G;
  {
    const int col = col0 + (lane >> 2);
    const uint4* p = nullptr;
    if (col < rows)
      p = reinterpret_cast<const uint4*>(
          a.q + ((q0 + col / a.G) * a.Hq + (int64_t)h * a.G + col % a.G) * kHeadDim);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // bf16: 16-byte piece 4j + quad; 8-bit: the two pieces of 16 dims
      const int piece = FMT == PA_KV_BF16 ? 4 * j + quad : 2 * (4 * (j >> 1) + quad) + (j & 1);
      const uint4 x = p ? __ldg(p + piece) : make_uint4(0u, 0u, 0u, 0u);
      t.b[2 * j][0] = x.x;
      t.b[2 * j][1] = x.y;
      t.b[2 * j + 1][0] = x.z;
      t.b[2 * j + 1][1] = x.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int col = col0 + quad * 2 + e;
    t.l2[e] = 0.f;
    t.l2lo[e] = 0.f;
    t.last[e] = -1;
    if (col < rows) {
      const float l = __ldg(a.lse + (q0 + col / a.G) * a.Hq + h * a.G + col % a.G);
      if (l != neg_inf()) {  // a query that saw nothing draws nothing
        t.l2[e] = l * kLog2e;
        // what the product lost, and log2 e's own rounding
        t.l2lo[e] = fmaf(l, kLog2e, -t.l2[e]) + l * 1.925963033500e-8f;
        t.last[e] = c - lq + col / a.G;
      }
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kWgtWarps * 32, 2)
    accumulate_weights_kernel(const WeightArgs a) {
  extern __shared__ __align__(16) int pm[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = a.S, Hkv = a.Hkv;
  PlanSmem P;
  P.pair_off = pm;
  P.seq_pair = P.pair_off + (S + 1);
  P.ctx = P.seq_pair + (S + 1);
  P.qstart = P.ctx + S;
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
  build_plan(in, P, nullptr);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int W = P.total;
  const int nw = min((int)gridDim.x * kWgtWarps, W);
  const int w = warp * (int)gridDim.x + (int)blockIdx.x;  // ranges dealt out transposed
  if (w >= nw) return;
  const int R0 = range_start(w, W, nw), R1 = range_start(w + 1, W, nw);
  if (R0 >= R1) return;

  TilePos pp = locate(P, S, Hkv, R0);
  auto load_phys = [&](int idx) -> int {
    if (idx >= R1) return 0;
    const TilePos t = locate_from(P, Hkv, pp, idx);
    return a.block_tables[(size_t)t.s * a.max_blocks + t.b];
  };
  int wbase = R0;
  int phys_cur = load_phys(wbase + lane);
  int phys_next = load_phys(wbase + 32 + lane);
  auto fetch = [&](int idx, const TilePos& t, KTile<FMT>& k) {
    int phys = __shfl_sync(kFull, phys_cur, idx - wbase);
    if (phys < 0 || (int64_t)phys >= a.num_blocks) {
      if (lane == 0) flag_error(PA_DEVERR_BLOCK_RANGE);
      phys = 0;
    }
    load_k<FMT>(a, (int64_t)phys * Hkv + t.h, lane, k);
  };

  TilePos cp = pp;
  KTile<FMT> cur, nxt;
  fetch(R0, pp, cur);
  int q0 = 0, lq = 0;
  bool ok = false;
  QTile qt;
  const int quad = lane & 3, r0 = lane >> 2;
  for (int idx = R0; idx < R1; ++idx) {
    // the next tile's rows land while this one is computed
    if (idx + 1 < R1) {
      advance(P, S, Hkv, pp);
      if (idx + 1 - wbase == 32) {
        wbase += 32;
        phys_cur = phys_next;
        phys_next = load_phys(wbase + 32 + lane);
      }
      fetch(idx + 1, pp, nxt);
    }
    const int c = P.ctx[cp.s];
    if (idx == R0 || cp.b == 0) {
      q0 = cp.s;
      lq = 1;
      if (a.cu_seqlens_q) {
        q0 = a.cu_seqlens_q[cp.s];
        lq = a.cu_seqlens_q[cp.s + 1] - q0;
      }
      ok = q0 >= 0 && lq >= 0 && lq <= c && (int64_t)q0 + lq <= a.num_q_tokens;
      if (!ok && lane == 0) flag_error(PA_DEVERR_QLEN_RANGE);
      if (ok) load_q<FMT>(a, q0, lq, c, cp.h, 0, lane, qt);
    }
    if (ok) {
      const int pos[2] = {cp.b * kBlock + r0, cp.b * kBlock + r0 + 8};
      float* dst = a.weights + ((int64_t)cp.s * Hkv + cp.h) * a.weights_len;
      float old[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (a.accumulate && quad == 0 && pos[i] < c - lq) old[i] = dst[pos[i]];
      uint32_t f[8][4];
      fragments<FMT>(cur, f);
      float sum[2] = {0.f, 0.f};
      for (int col0 = 0; col0 < lq * a.G; col0 += 8) {
        if (lq * a.G > 8) load_q<FMT>(a, q0, lq, c, cp.h, col0, lane, qt);
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
          mma_bf16_16816(d0, f[t], qt.b[t][0], qt.b[t][1]);
          mma_bf16_16816(d1, f[t + 1], qt.b[t + 1][0], qt.b[t + 1][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float sc = a.scale_log2;
          if constexpr (FMT != PA_KV_BF16) sc *= cur.scale[e >> 1];
          const float z = fmaf(d0[e] + d1[e], sc, -qt.l2[e & 1]) - qt.l2lo[e & 1];
          if (pos[e >> 1] <= qt.last[e & 1]) sum[e >> 1] += ex2(z);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(kFull, sum[i], 1);
        sum[i] += __shfl_xor_sync(kFull, sum[i], 2);
        if (quad == 0 && pos[i] < c) dst[pos[i]] = old[i] + sum[i];
      }
    }
    cur = nxt;
    if (idx + 1 < R1) cp = pp;
  }
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
  const size_t smem = sizeof(int) * 4 * ((size_t)shape->num_seqs + 1);
  if (smem > (size_t)dev.max_smem_optin) return PA_ERR_UNSUPPORTED;
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
  auto kernel = kv_format == PA_KV_BF16   ? accumulate_weights_kernel<PA_KV_BF16>
                : kv_format == PA_KV_INT8 ? accumulate_weights_kernel<PA_KV_INT8>
                                          : accumulate_weights_kernel<PA_KV_FP8>;
  int per_sm = 0;
  if (!kernel_occupancy(reinterpret_cast<const void*>(kernel), kWgtWarps * 32, smem, &per_sm) ||
      per_sm <= 0)
    return PA_ERR_CUDA;
  if (launch_dependent(kernel, dim3((unsigned)(dev.num_sms * per_sm)), dim3(kWgtWarps * 32), smem,
                       static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
