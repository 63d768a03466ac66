// pa_rows.cuh -- moving whole cached rows (one position's K and V of one KV
// head) inside the paged pool, shared by the accepted-path commit and the
// eviction.
#pragma once

#include "pa_device.cuh"

namespace pa {

// Where a position's row of one KV head lies: its (block, KV head) tile and
// the row inside the tile.
struct RowPlace {
  int64_t tile;
  int off;
};

struct PoolView {
  uint8_t* k;
  uint8_t* v;
  const int32_t* table;  // this sequence's block table
  int64_t num_blocks;
  int Hkv, h;
  // False: the position's block id lies outside the pool.
  __device__ __forceinline__ bool place(int pos, RowPlace* p) const {
    const int phys = table[pos / kBlock];
    p->tile = (int64_t)phys * Hkv + h;
    p->off = pos % kBlock;
    return phys >= 0 && (int64_t)phys < num_blocks;
  }
};

// One lane's share of a row. bf16: lanes 0-15 hold the 16-byte chunks of the K
// row, lanes 16-31 those of the V row. 8-bit: lanes 0-7 and 8-15 the chunks of
// the codes, lanes 16 and 17 the two scales.
template <bool Q8>
__device__ __forceinline__ uint8_t* row_chunk(const PoolView& p, const RowPlace& at, int lane) {
  if constexpr (!Q8) {
    uint8_t* base = lane < 16 ? p.k : p.v;
    return base + ((at.tile * kBlock + at.off) * kHeadDim) * 2 + (lane & 15) * 16;
  } else {
    if (lane >= 16) {
      uint8_t* base = lane == 16 ? p.k : p.v;
      return base + at.tile * kInt8TileBytes + kBlock * kHeadDim + at.off * 4;
    }
    uint8_t* base = lane < 8 ? p.k : p.v;
    return base + at.tile * kInt8TileBytes + at.off * kHeadDim + (lane & 7) * 16;
  }
}

template <bool Q8>
__device__ __forceinline__ uint4 load_chunk(const uint8_t* p, int lane) {
  if (Q8 && lane >= 16) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 18) x.x = *reinterpret_cast<const uint32_t*>(p);
    return x;
  }
  return *reinterpret_cast<const uint4*>(p);
}

template <bool Q8>
__device__ __forceinline__ void store_chunk(uint8_t* p, int lane, const uint4& x) {
  if (Q8 && lane >= 16) {
    if (lane < 18) *reinterpret_cast<uint32_t*>(p) = x.x;
    return;
  }
  *reinterpret_cast<uint4*>(p) = x;
}

}  // namespace pa
