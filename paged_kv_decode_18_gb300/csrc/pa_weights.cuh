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

// Two one-byte codes (low 16 bits of c) as an exact bf16 pair.
// int8: 128 + the low seven bits, less 128 or (sign bit set) 256; both are
// bf16 bit patterns 0x43xx, and the difference, at most 8 bits, is exact.
__device__ __forceinline__ uint32_t int8x2_to_bf16x2(uint32_t c) {
  const uint32_t spread = __byte_perm(c, 0u, 0x4140);  // bytes c0, 0, c1, 0
  const uint32_t hi = (spread & 0x007f007fu) | 0x43004300u;
  const uint32_t lo = (spread & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(hi), "r"(lo));
  return r;
}
// E4M3: the hardware's exact f16 pair, then fp32, whose upper halves are the
// bf16 values (4 significant bits, exponents -9 .. 8: exact).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float lo, hi;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t c) {
  return FMT == PA_KV_INT8 ? int8x2_to_bf16x2(c) : e4m3x2_to_bf16x2(c);
}

// The tcgen05 kernel for windows (pa_weights_tc.cu). False in `enabled`: the
// batch does not fit it (group or plan size).
struct WeightsTcGeometry {
  bool enabled = false;
  int grid = 0, QTb = 0;
  size_t smem = 0;
};
int weights_tc_geometry(const pa_shape* sh, int max_q_len, int kv_format, WeightsTcGeometry* g);
int launch_weights_tc(const WeightsTcGeometry& g, const WeightArgs& a, int kv_format,
                      cudaStream_t st);

}  // namespace pa
