// pa_weights.cuh -- what the two kernels of pa_accumulate_weights share.
#pragma once

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {

struct WeightArgs {
  const uint16_t* q;
  const uint8_t* k_cache;
  const float* lse;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_seqlens_q;  // null: one query per sequence
  int64_t num_q_tokens;
  int accumulate;
  float scale_log2;
  float* weights;
  int64_t weights_len;
  int S, Hq, Hkv, G, max_blocks;
  int64_t num_blocks;
};

// Four one-byte codes as two exact bf16 pairs.
// int8: 128 + the low seven bits, less 128 or (sign bit set) 256; both are
// bf16 bit patterns 0x43xx, and the difference, at most 8 bits, is exact.
__device__ __forceinline__ uint32_t int8x2_to_bf16x2(uint32_t spread) {  // bytes c0, 0, c1, 0
  const uint32_t hi = (spread & 0x007f007fu) | 0x43004300u;
  const uint32_t lo = (spread & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(hi), "r"(lo));
  return r;
}
// E4M3: a code's exponent and mantissa bits are those of a bf16 value 2^-120
// times as large (biases 7 and 127; subnormals included), so a shift and an
// exact product give it. (The hardware's conversions go through f16 and fp32
// at 16 a clock and made the tcgen05 kernel's tile 1.6 us instead of 0.5.)
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t t) {  // bytes 0, c0, 0, c1
  const uint32_t x = (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7b807b80u));  // 2^120
  return r;
}
template <int FMT>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == PA_KV_INT8) {
    lo = int8x2_to_bf16x2(__byte_perm(w, 0u, 0x4140));
    hi = int8x2_to_bf16x2(__byte_perm(w, 0u, 0x4342));
  } else {
    lo = e4m3x2_to_bf16x2(__byte_perm(w, 0u, 0x1404));
    hi = e4m3x2_to_bf16x2(__byte_perm(w, 0u, 0x3424));
  }
}

// The tcgen05 kernel for windows (pa_weights_tc.cu). False in `enabled`: the
// batch does not fit it (group or plan size).
struct WeightsTcGeometry {
  bool enabled = false;
  bool split = false;  // a window may have several query tiles
  int grid = 0, QTb = 0;
  size_t smem = 0;
};
int weights_tc_geometry(const pa_shape* sh, int max_q_len, int kv_format, WeightsTcGeometry* g);
int launch_weights_tc(const WeightsTcGeometry& g, const WeightArgs& a, int kv_format,
                      cudaStream_t st);

}  // namespace pa
