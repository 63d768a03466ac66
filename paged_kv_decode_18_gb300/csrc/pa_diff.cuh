// pa_diff.cuh -- differential attention: what its kernels share. A pair of KV
// heads (2p, 2p + 1) holds two key maps and one value of 256 dims; a
// differential head combines the two maps' results,
//   d = a_0 - lambda a_1,   out = out_scale d [w / sqrt(mean d^2 + eps)].
#pragma once

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

constexpr int kDiffDim = 2 * kHeadDim;  // values of a pair, and of an output row

struct DiffOut {
  uint16_t* out;        // [tokens][Hq / 2][256]
  float* lse;           // [tokens][Hq], or null
  const float* lambdas; // [Hq / 2]
  const float* weight;  // [256], or null: no norm
  float eps, gain;
};

// One value of the difference. Both maps' values are rounded before they meet, so
// that equal ones cancel (a norm without an eps would blow up what is left).
__device__ __forceinline__ float diff_value(float o0, float inv0, float o1, float inv1, float lam) {
  return fmaf(-lam, __fmul_rn(o1, inv1), __fmul_rn(o0, inv0));
}

// The factor on a row's difference whose squares sum to `squares`.
__device__ __forceinline__ float diff_factor(const DiffOut& o, float squares) {
  if (!o.weight) return o.gain;
  const float mean = squares * (1.f / kDiffDim) + o.eps;
  // a row of zeros without an eps: 0, not 0 x infinity
  return mean > 0.f || mean != mean ? o.gain * rsqrtf(mean) : 0.f;
}

// ---------------------------------------------------------------------------
// tcgen05 path (pa_diff_tc.cu): windows of min_q_len tokens and more
// ---------------------------------------------------------------------------
struct DiffTcGeometry {
  bool enabled = false;
  int workers = 0, npairs_cap = 0, nstage = 0, min_lq = 0;
  size_t smem = 0, ws_lse = 0, ws_o = 0, ws_bytes = 0;
};

int diff_tc_geometry(const pa_shape* sh, int64_t num_q_tokens, int max_q_len, int min_q_len,
                     DiffTcGeometry* g);
int launch_diff_tc(const DiffTcGeometry& g, const pa_bf16* q, const pa_bf16* k_cache,
                   const pa_bf16* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* cu_seqlens_q, int64_t num_q_tokens,
                   int max_q_len, int causal, float scale, const DiffOut& out, const pa_shape* sh,
                   void* workspace, cudaStream_t st);

}  // namespace pa
