// pa_rotate.cu -- rotary positions: of rows (pa_rotate), of a step's queries
// and keys on their way into the paged cache (pa_rotate_and_cache), and of keys
// that the cache already holds (pa_rotate_cached).
//
// Pages: course README "Build an LLM Inference Engine From Scratch", curriculum
// row of the model layer (RoPE) and "Memory & KV Cache" (quantization);
// Work-log, "KV Cache > The Idea" (the new K and V are appended to the cache).
//
// Pair i of a row, (a, b), becomes (a cos - b sin, b cos + a sin) for the angle
// position * theta_i. theta_i comes as a fraction of a turn in steps of 2^-64
// (pa_rotation), so position * theta_i modulo one turn is one 64-bit integer
// product: exact for any position, where an fp32 product would be off by
// 2^-24 of an angle of many turns. Its upper 23 bits go to the fast sine and cosine,
// which are off by 2^-19.7 then, far below the 2^-9 of the bf16 result.
//
// Everything here is bound by HBM, or by the launch where there are few rows:
// 16 FMA and 8 sines and cosines per 64 bytes moved. Eight lanes hold a row, 16
// values each in two 16-byte chunks that hold both sides of its pairs, so that
// a pair never leaves its lane: chunks c and c + rot_dim / 16 (half layout), c
// and c + 8 (interleaved, where a chunk holds whole pairs). Half layouts whose
// rot_dim is no multiple of 16 have pairs across lanes: they exchange their
// values through shared memory.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_quant.cuh"
#include "pa_tcgen05.cuh"

#include <math.h>

namespace pa {
namespace {

constexpr int kHalf = 0;  // pairs (i, i + r/2), r a multiple of 16
constexpr int kSide = 1;  // pairs (2i, 2i + 1)
constexpr int kAny = 2;   // pairs (i, i + r/2), any even r

constexpr int kFmtBf16 = 0, kFmtInt8 = 1, kFmtFp8 = 2;
static_assert(kFmtBf16 == PA_KV_BF16 && kFmtInt8 == PA_KV_INT8 && kFmtFp8 == PA_KV_FP8, "formats");

constexpr int kRotWarps = 8;

// What a lane knows of the rows it turns: its place c among the row's eight
// lanes, its two chunks, and which of its eight words (two values each) are
// rotated.
template <int MODE>
struct Lane {
  int c, a, b;
  uint32_t words;  // bit w: word w of the lane (0-3: chunk a, 4-7: chunk b) is rotated
  __device__ __forceinline__ Lane(int lane, int r) {
    c = lane & 7;
    a = c;
    b = c + 8;
    words = 0xffu;
    if constexpr (MODE == kHalf) {
      const int hr = r >> 4;
      if (c < hr) {
        b = c + hr;
      } else {
        a = 2 * c;
        b = 2 * c + 1;
        words = 0u;
      }
    } else {
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (dim(2 * w) >= r) words &= ~(1u << w);
    }
  }
  // dimension of the lane's value e (0-7: chunk a, 8-15: chunk b)
  __device__ __forceinline__ int dim(int e) const { return (e < 8 ? a : b) * 8 + (e & 7); }
};

// The rotation's turns in shared memory, a word of padding after every eight: a warp's
// lanes want eight of them at a time, which the constant bank gives one by one (32 x 1024
// cached keys behind an eviction 29.0 us, with sines made anew in every row; 26.2 so).
constexpr int kTurns = 64 + 8;
__device__ __forceinline__ int turn_at(int pair) { return pair + (pair >> 3); }
__device__ __forceinline__ void load_turns(unsigned long long* turns, const pa_rotation& rot) {
  if (threadIdx.x < 64) turns[turn_at(threadIdx.x)] = rot.turns[threadIdx.x];
  __syncthreads();
}

// Cosines and sines for a lane's values at one position. kHalf: of the pairs
// (value j, value 8 + j); kSide: of the pairs (value 2j, value 2j + 1); kAny: of
// each value on its own, the sine with the sign that its side takes.
template <int MODE>
struct Spin {
  static constexpr int N = MODE == kAny ? 16 : 8;
  float c[N], s[N];
  __device__ __forceinline__ void set(const unsigned long long* turns, int r,
                                      const Lane<MODE>& me, int pos, float magnitude, float sign) {
    // (volatile: read where they are wanted, or a loop around this would hold them all)
    const volatile unsigned long long* mine =
        turns + (MODE == kHalf ? turn_at(me.c * 8) : MODE == kSide ? turn_at(me.c * 4) : 0);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      int at;
      float sg = sign;
      if constexpr (MODE == kHalf) {
        at = j;  // pair c * 8 + j
      } else if constexpr (MODE == kSide) {
        at = j < 4 ? j : turn_at(32) + j - 4;  // pairs c * 4 + j, 32 + c * 4 + j - 4
      } else {
        const int d = me.dim(j), h = r >> 1;
        at = turn_at(d < h ? d : (d < 2 * h ? d - h : 0));
        if (d < h) sg = -sign;
      }
      const unsigned long long phase = mine[at] * (unsigned long long)(long long)pos;
      // the phase's upper 23 bits as the fraction of a number in [1, 2), half a turn on, so
      // that 1.5 stands for 0: an integer conversion would take a third turn on the unit
      // that sine and cosine share
      const uint32_t hi = ((uint32_t)(phase >> 32) + 0x80000100u) >> 9;
      float sn, cs;
      __sincosf((__uint_as_float(0x3f800000u | hi) - 1.5f) * 6.28318530717959f, &sn, &cs);
      c[j] = cs * magnitude;
      s[j] = sn * (magnitude * sg);
    }
  }
};

// Turns a lane's values. kAny: rows holds this warp's four rows of shared
// memory; the whole warp calls it.
// (a word more every 32, and rows 134 apart: a warp's accesses, eight words apart in four
// rows, then fall into 32 banks; 4-way conflicts made these layouts twice as slow)
constexpr int kRowPad = kHeadDim + 6;
__device__ __forceinline__ int skewed(int d) { return d + (d >> 5); }

template <int MODE>
__device__ __forceinline__ void turn(float (&f)[16], const Spin<MODE>& sp, const Lane<MODE>& me,
                                     int r, float* rows, int sub) {
  if constexpr (MODE == kHalf) {
    if (me.words) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = f[j], y = f[8 + j];
        f[j] = x * sp.c[j] - y * sp.s[j];
        f[8 + j] = y * sp.c[j] + x * sp.s[j];
      }
    }
  } else if constexpr (MODE == kSide) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!((me.words >> j) & 1u)) continue;
      const float x = f[2 * j], y = f[2 * j + 1];
      f[2 * j] = x * sp.c[j] - y * sp.s[j];
      f[2 * j + 1] = y * sp.c[j] + x * sp.s[j];
    }
  } else {
    float* row = rows + sub * kRowPad;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) row[skewed(me.dim(e))] = f[e];
    __syncwarp();
    const int h = r >> 1;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = me.dim(e);
      if (d < r) f[e] = f[e] * sp.c[e] + row[skewed(d < h ? d + h : d - h)] * sp.s[e];
    }
  }
}

__device__ __forceinline__ void unpack16(const uint4& xa, const uint4& xb, float (&f)[16]) {
  const uint32_t w[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf_lo(w[i]);
    f[2 * i + 1] = bf_hi(w[i]);
  }
}

// The words of `rotated` from f, the others as they were.
__device__ __forceinline__ void repack16(const float (&f)[16], uint32_t rotated, uint4& xa,
                                         uint4& xb) {
  uint32_t w[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((rotated >> i) & 1u) w[i] = cvt_bf16x2(f[2 * i], f[2 * i + 1]);
  xa = make_uint4(w[0], w[1], w[2], w[3]);
  xb = make_uint4(w[4], w[5], w[6], w[7]);
}

// Largest magnitude of a row whose eight lanes hold 16 values each.
__device__ __forceinline__ float row_amax(const float (&f)[16]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  return m;
}

__device__ __forceinline__ void store_row(uint2 ca, uint2 cb, float scale, int a, int b, int c,
                                          uint8_t* tile, int off) {
  uint8_t* row = tile + off * kHeadDim;
  *reinterpret_cast<uint2*>(row + a * 8) = ca;
  *reinterpret_cast<uint2*>(row + b * 8) = cb;
  if (c == 0) *(reinterpret_cast<float*>(tile + kBlock * kHeadDim) + off) = scale;
}

// Quantises a row held by eight lanes into the tile's row `off`. The whole warp
// calls it; write: this lane's row goes to memory.
template <bool FP8>
__device__ __forceinline__ void store_codes(const float (&f)[16], int a, int b, int c,
                                            uint8_t* tile, int off, bool write) {
  const float amax = row_amax(f);
  if (!write) return;
  uint2 ca = make_uint2(0u, 0u), cb = ca;
  if (amax > 0.f) {
    const float inv = code_factor<FP8>(amax);
    ca = codes_of8<FP8>(f, inv);
    cb = codes_of8<FP8>(f + 8, inv);
  }
  store_row(ca, cb, amax > 0.f ? __fdiv_rn(amax, code_range<FP8>()) : 0.f, a, b, c, tile, off);
}

// The same for a row that the tile held with `scale` and whose codes' own values were
// turned: a turn is linear, so the scale passes by it. One that is infinite or NaN (keys
// that had overflowed) stays one, and so does an FP8 code that is a NaN.
template <bool FP8>
__device__ __forceinline__ void store_turned(const float (&f)[16], float scale, int a, int b,
                                             int c, uint8_t* tile, int off, bool write) {
  const float amax = row_amax(f);
  if (!write) return;
  const float inv = amax > 0.f ? __fdiv_rn(code_range<FP8>(), amax) : 1.f;
  store_row(codes_of8<FP8>(f, inv), codes_of8<FP8>(f + 8, inv),
            __fmul_rn(scale, __fdiv_rn(amax, code_range<FP8>())), a, b, c, tile, off);
}

// ---------------------------------------------------------------------------
// rows, and a step's rows into the cache
// ---------------------------------------------------------------------------

struct View {
  uint16_t* p = nullptr;
  int64_t ts = 0, hs = 0;
};

struct RowsArgs {
  View q, k, v, qo;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* kc;
  uint8_t* vc;
  int64_t num_slots;
  int Hq, Hkv;      // rows of a token: Hq queries, Hkv keys, Hkv values
  int warps_per_token;
  int num_warps;
  float sign;       // -1: the transposed map
  pa_rotation rot;
};

// A warp turns 16 rows of one token, four at a time, all loads first, with one set of
// sines and cosines. Measured: 16,200 x 16 rows 22.5 us, 5.9 TB/s; 12,000 tokens of 16 + 8
// + 8 rows into the cache 32.1 us, 6.2 TB/s. (Eight rows a warp: 23.5 and 37.8; twelve: 26.9
// and 34.9; twenty: 23.1 and 37.8. At a decode step's 256 tokens all take the 4 us of a
// launch.) 8,100 such tokens: bf16 22.8 us, FP8 24.5, int8 25.8, of which their bytes are
// 19.6, 17.2 and 17.2: the quantiser's instructions, 1.9 a clock in all (12 bytes of
// registers spill). A token of few rows leaves its warp's others empty: 65,536 tokens of
// one, two or four heads take 37 to 39 us, their bytes 5, 10 and 20.
// kAny's sines and cosines of 16 values (each side of a pair makes its own) want 128
// registers: 46.6 us for 16,200 x 16 rows of r = 72 with two CTAs to an SM, 49.3 with three,
// where the other layouts take 23.
constexpr int kIter = 4;

template <int MODE, int FMT>
__global__ void __launch_bounds__(kRotWarps * 32, MODE == kAny ? 2 : 3)
    rotate_rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float exchange[MODE == kAny ? kRotWarps * 4 * kRowPad : 1];
  __shared__ unsigned long long turns[kTurns];
  load_turns(turns, a.rot);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = (int)blockIdx.x * kRotWarps + warp;
  const Lane<MODE> me(lane, a.rot.rot_dim);
  const int sub = lane >> 3;
  float* rows = exchange + (MODE == kAny ? warp * 4 * kRowPad : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (w >= a.num_warps) return;
  const int t = w / a.warps_per_token;
  const int r0 = (w - t * a.warps_per_token) * 4 * kIter;
  const int total = a.Hq + 2 * a.Hkv;
  uint4 xa[kIter], xb[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int r = r0 + i * 4 + sub;
    xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < total) {
      const uint16_t* src;
      if (r < a.Hq)
        src = a.q.p + t * a.q.ts + r * a.q.hs;
      else if (r < a.Hq + a.Hkv)
        src = a.k.p + t * a.k.ts + (r - a.Hq) * a.k.hs;
      else
        src = a.v.p + t * a.v.ts + (r - a.Hq - a.Hkv) * a.v.hs;
      xa[i] = *reinterpret_cast<const uint4*>(src + me.a * 8);
      xb[i] = *reinterpret_cast<const uint4*>(src + me.b * 8);
    }
  }
  int64_t slot = -1;
  if (a.Hkv > 0 && r0 + 4 * kIter > a.Hq) {
    slot = a.slots[t];
    if (slot >= a.num_slots) {
      // one row of the token tells
      if (r0 <= a.Hq && lane == 0) flag_error(PA_DEVERR_SLOT_RANGE);
      slot = -1;
    }
  }
  Spin<MODE> sp;
  if (r0 < a.Hq + a.Hkv) sp.set(turns, a.rot.rot_dim, me, a.positions[t], a.rot.magnitude, a.sign);
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (r0 + i * 4 >= total) break;  // the same for the whole warp
    const int r = r0 + i * 4 + sub;
    const bool turned = r < a.Hq + a.Hkv;
    const bool query = r < a.Hq;
    float f[16];
    unpack16(xa[i], xb[i], f);
    if constexpr (MODE == kAny) {
      if (r0 + i * 4 < a.Hq + a.Hkv) {
        float g[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = f[e];
        turn<MODE>(g, sp, me, a.rot.rot_dim, rows, sub);
        if (turned) {
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = g[e];
        }
      }
    } else {
      if (turned) turn<MODE>(f, sp, me, a.rot.rot_dim, rows, sub);
    }
    if (FMT == kFmtBf16 || query) {
      if (turned) repack16(f, me.words, xa[i], xb[i]);
      uint16_t* dst = nullptr;
      if (query) {
        dst = a.qo.p + t * a.qo.ts + r * a.qo.hs;
      } else if (FMT == kFmtBf16 && r < total && slot >= 0) {
        const int64_t blk = slot / kBlock, off = slot % kBlock;
        const int h = turned ? r - a.Hq : r - a.Hq - a.Hkv;
        dst = reinterpret_cast<uint16_t*>(turned ? a.kc : a.vc) +
              ((blk * a.Hkv + h) * kBlock + off) * kHeadDim;
      }
      if (dst) {
        *reinterpret_cast<uint4*>(dst + me.a * 8) = xa[i];
        *reinterpret_cast<uint4*>(dst + me.b * 8) = xb[i];
      }
    }
    if constexpr (FMT != kFmtBf16) {
      if (r0 + i * 4 + 3 >= a.Hq) {  // some row of the four goes to the cache
        const bool write = !query && r < total && slot >= 0;
        const int64_t blk = write ? slot / kBlock : 0;
        const int h = turned ? r - a.Hq : r - a.Hq - a.Hkv;
        uint8_t* tile = (turned ? a.kc : a.vc) + (write ? (blk * a.Hkv + h) * kInt8TileBytes : 0);
        store_codes<FMT == kFmtFp8>(f, me.a, me.b, me.c, tile, write ? (int)(slot % kBlock) : 0,
                                    write);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// keys that the cache holds
// ---------------------------------------------------------------------------

struct CachedArgs {
  uint8_t* kc;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* shifts;
  const int32_t* kept;
  int first, kept_len;
  int S, Hkv, max_blocks;
  int64_t num_blocks;
  pa_rotation rot;
};

// One warp turns a (block, KV head) tile of 16 keys, four at a time, the loads of
// eight ahead; the batch's tiles are cut into equal ranges, one per warp (tiles of a
// sequence and head in order, so that a warp's positions follow one another).
// Sines and cosines are made anew only where a row's turn differs from the last.
// Measured: 8 x 24,000..28,700 keys of 8 heads by a shift 143 us (6.0 TB/s); 32 x 1024
// behind an eviction 26 us, of which some 7 us is the chain launch, lengths, block
// ids and turns, first rows. (Loads of the next eight keys held ahead of the present
// ones: 33 us, for the registers that it takes.) 16 x 4096 keys of 8 heads by a shift: bf16
// 47 us, FP8 35.4, int8 41.6, behind an eviction 47.6, 43 and 51; the 8-bit ones, 20 us
// by their bytes, issue 2.4 and 2.5 instructions a clock with a third of the warp slots
// filled. kAny: bf16 70 us (68 bytes spilled), FP8 54, int8 59 with two CTAs to an SM; three,
// at 80 registers and 900 bytes of spill loads a thread, 70 and 76.
template <int MODE, int FMT>
__global__ void __launch_bounds__(kRotWarps * 32, MODE == kAny ? 2 : 3)
    rotate_cached_kernel(const __grid_constant__ CachedArgs a) {
  extern __shared__ __align__(16) int area[];  // turns, kAny: the exchange, the plan
  unsigned long long* turns = reinterpret_cast<unsigned long long*>(area);
  float* exchange = reinterpret_cast<float*>(turns + kTurns);
  int* plan = area + 2 * kTurns + (MODE == kAny ? kRotWarps * 4 * kRowPad : 0);
  load_turns(turns, a.rot);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<MODE> me(lane, a.rot.rot_dim);
  const int sub = lane >> 3;
  float* rows = exchange + (MODE == kAny ? warp * 4 * kRowPad : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  PlanSmem P;
  P.pair_off = plan;
  P.seq_pair = P.pair_off + a.S + 1;
  P.ctx = P.seq_pair + a.S + 1;
  P.qstart = P.ctx + a.S;
  PlanInputs in;
  in.context_lens = a.context_lens;
  in.cu_seqlens_q = nullptr;
  in.S = a.S;
  in.Hkv = a.Hkv;
  in.max_ctx = a.max_blocks * kBlock;
  in.qtile = 1;
  in.causal = 0;
  in.npairs_cap = a.S;
  in.num_q_rows = a.S;
  build_plan(in, P, nullptr);
  const int W = P.total, nw = min((int)gridDim.x * kRotWarps, W);
  const int w = warp * (int)gridDim.x + (int)blockIdx.x;
  if (w >= nw) return;
  const int R0 = range_start(w, W, nw), R1 = range_start(w + 1, W, nw);
  TilePos t = locate(P, a.S, a.Hkv, R0);
  Spin<MODE> sp;
  int spun = 0;  // the turn that sp holds (0: none yet)
  // a tile's block, and the turns of this lane's rows in it
  auto fetch = [&](int& phys, int (&by)[4]) {
    phys = a.block_tables[(int64_t)t.s * a.max_blocks + t.b];
    const int c = P.ctx[t.s];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = t.b * kBlock + i * 4 + sub;
      by[i] = 0;
      if (pos < c) {
        if (a.kept) {
          if (pos < a.kept_len) {
            const int old = a.kept[((int64_t)t.s * a.Hkv + t.h) * a.kept_len + pos];
            if (old >= 0) by[i] = pos - old;
          }
        } else if (pos >= a.first) {
          by[i] = a.shifts[t.s];
        }
      }
    }
  };
  // (a tile ahead with bf16 keys; 8-bit ones have no registers left for it: 36 us against
  // 33.5 for 16 x 4096 FP8 keys of 8 heads, bf16 46.4 against 47.7)
  constexpr bool kAhead = FMT == kFmtBf16;
  int phys_next = 0, by_next[4] = {0, 0, 0, 0};
  if (kAhead) fetch(phys_next, by_next);
  for (int idx = R0; idx < R1; ++idx) {
    if (!kAhead) fetch(phys_next, by_next);
    const int phys = phys_next, h = t.h;
    int by[4];
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      by[i] = by_next[i];
      any = any || by[i] != 0;
    }
    if (idx + 1 < R1) {
      advance(P, a.S, a.Hkv, t);
      if (kAhead) fetch(phys_next, by_next);
    }
    const bool inside = phys >= 0 && (int64_t)phys < a.num_blocks;
    if (!inside && lane == 0) flag_error(PA_DEVERR_BLOCK_RANGE);
    if (inside && __any_sync(kFull, any)) {
      const int64_t at = (int64_t)phys * a.Hkv + h;
      if constexpr (FMT == kFmtBf16) {
        uint16_t* tile = reinterpret_cast<uint16_t*>(a.kc) + at * (kBlock * kHeadDim);
#pragma unroll
        for (int i0 = 0; i0 < 4; i0 += 2) {
          uint4 xa[2], xb[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint16_t* row = tile + ((i0 + u) * 4 + sub) * kHeadDim;
            xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
            if (by[i0 + u] != 0 && me.words) {
              xa[u] = *reinterpret_cast<const uint4*>(row + me.a * 8);
              xb[u] = *reinterpret_cast<const uint4*>(row + me.b * 8);
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int turned = by[i0 + u];
            if (__any_sync(kFull, turned != spun && turned != 0)) {
              sp.set(turns, a.rot.rot_dim, me, turned, 1.f, 1.f);
              spun = turned;
            }
            float f[16];
            const bool mine = turned != 0 && me.words;
            unpack16(xa[u], xb[u], f);
            if (MODE == kAny || mine) turn<MODE>(f, sp, me, a.rot.rot_dim, rows, sub);
            if (mine) {
              repack16(f, me.words, xa[u], xb[u]);
              uint16_t* row = tile + ((i0 + u) * 4 + sub) * kHeadDim;
              *reinterpret_cast<uint4*>(row + me.a * 8) = xa[u];
              *reinterpret_cast<uint4*>(row + me.b * 8) = xb[u];
            }
          }
        }
      } else {
        uint8_t* tile = a.kc + at * kInt8TileBytes;
        uint2 ca[4], cb[4];
        float scale[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int off = i * 4 + sub;
          ca[i] = cb[i] = make_uint2(0u, 0u);
          scale[i] = 0.f;
          if (by[i] != 0) {
            ca[i] = *reinterpret_cast<const uint2*>(tile + off * kHeadDim + me.a * 8);
            cb[i] = *reinterpret_cast<const uint2*>(tile + off * kHeadDim + me.b * 8);
            scale[i] = *(reinterpret_cast<const float*>(tile + kBlock * kHeadDim) + off);
          }
        }
        __syncwarp();  // every lane of a row has its scale before one of them writes the new one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (__any_sync(kFull, by[i] != spun && by[i] != 0)) {
            sp.set(turns, a.rot.rot_dim, me, by[i], 1.f, 1.f);
            spun = by[i];
          }
          float f[16];
          values_of8<FMT == kFmtFp8>(ca[i], f);
          values_of8<FMT == kFmtFp8>(cb[i], f + 8);
          turn<MODE>(f, sp, me, a.rot.rot_dim, rows, sub);
          store_turned<FMT == kFmtFp8>(f, scale[i], me.a, me.b, me.c, tile, i * 4 + sub,
                                       by[i] != 0);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

bool good_rotation(const pa_rotation* r) {
  return r && r->rot_dim >= 2 && r->rot_dim <= kHeadDim && r->rot_dim % 2 == 0 &&
         (r->interleaved == 0 || r->interleaved == 1) && r->magnitude - r->magnitude == 0.f;
}

// Whether a view's rows can be read (and, for `out`, written without one lying over another).
bool good_view(const pa_row_view* v, int64_t tokens, int64_t heads, bool out) {
  if (!v || !v->data || !aligned(v->data, 16)) return false;
  if (v->token_stride < 0 || v->head_stride < 0 || v->token_stride % 8 || v->head_stride % 8)
    return false;
  const int64_t lim = int64_t(1) << 56;
  if ((tokens > 1 && v->token_stride > lim / tokens) || (heads > 1 && v->head_stride > lim / heads))
    return false;
  if (!out) return true;
  const bool by_token = v->token_stride >= v->head_stride;
  const int64_t n_in = by_token ? heads : tokens, n_out = by_token ? tokens : heads;
  const int64_t s_in = by_token ? v->head_stride : v->token_stride;
  const int64_t s_out = by_token ? v->token_stride : v->head_stride;
  if (n_in > 1 && s_in < kHeadDim) return false;
  const int64_t run = n_in > 1 ? (n_in - 1) * s_in + kHeadDim : kHeadDim;
  return n_out <= 1 || s_out >= run;
}

bool same_view(const pa_row_view* a, const pa_row_view* b) {
  return a->data == b->data && a->token_stride == b->token_stride &&
         a->head_stride == b->head_stride;
}

View view_of(const pa_row_view* v) {
  View x;
  x.p = static_cast<uint16_t*>(v->data);
  x.ts = v->token_stride;
  x.hs = v->head_stride;
  return x;
}

int mode_of(const pa_rotation* r) {
  return r->interleaved ? kSide : (r->rot_dim % 16 == 0 ? kHalf : kAny);
}

template <int FMT>
cudaError_t launch_rows_of(int mode, unsigned blocks, cudaStream_t st, const RowsArgs& a) {
  const dim3 grid(blocks), block(kRotWarps * 32);
  if (mode == kHalf) return launch_dependent(rotate_rows_kernel<kHalf, FMT>, grid, block, 0, st, a);
  if (mode == kSide) return launch_dependent(rotate_rows_kernel<kSide, FMT>, grid, block, 0, st, a);
  return launch_dependent(rotate_rows_kernel<kAny, FMT>, grid, block, 0, st, a);
}

int launch_rows(RowsArgs a, int64_t tokens, int fmt, const pa_rotation* rot, int transpose,
                cudaStream_t st) {
  const int64_t total = (int64_t)a.Hq + 2 * (int64_t)a.Hkv;
  if (total > (1 << 24)) return PA_ERR_UNSUPPORTED;
  const int64_t per = (total + 4 * kIter - 1) / (4 * kIter);
  const int64_t warps = per * tokens;
  if (tokens > 0x7fffffff / per - kRotWarps) return PA_ERR_UNSUPPORTED;
  a.warps_per_token = (int)per;
  a.num_warps = (int)warps;
  a.sign = transpose ? -1.f : 1.f;
  a.rot = *rot;
  for (int i = rot->rot_dim / 2; i < 64; ++i) a.rot.turns[i] = 0;
  const unsigned blocks = (unsigned)((warps + kRotWarps - 1) / kRotWarps);
  const int mode = mode_of(rot);
  cudaError_t e;
  if (fmt == kFmtBf16)
    e = launch_rows_of<kFmtBf16>(mode, blocks, st, a);
  else if (fmt == kFmtInt8)
    e = launch_rows_of<kFmtInt8>(mode, blocks, st, a);
  else
    e = launch_rows_of<kFmtFp8>(mode, blocks, st, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

const void* cached_kernel(int mode, int fmt) {
#define PA_CACHED(M)                                                                         \
  (fmt == kFmtBf16 ? reinterpret_cast<const void*>(rotate_cached_kernel<M, kFmtBf16>)        \
   : fmt == kFmtInt8 ? reinterpret_cast<const void*>(rotate_cached_kernel<M, kFmtInt8>)      \
                     : reinterpret_cast<const void*>(rotate_cached_kernel<M, kFmtFp8>))
  return mode == kHalf ? PA_CACHED(kHalf) : mode == kSide ? PA_CACHED(kSide) : PA_CACHED(kAny);
#undef PA_CACHED
}

// theta as a fraction of a turn, in steps of 2^-64 and modulo one turn.
uint64_t turns_of(double radians) {
  const double two_pi = 6.283185307179586476925286766559;
  double x = fabs(radians) / two_pi;
  x -= floor(x);
  const double y = ldexp(x, 64);
  const uint64_t u = y >= 18446744073709551616.0 ? 0 : (uint64_t)y;
  return radians < 0 ? (uint64_t)0 - u : u;
}

}  // namespace

unsigned take_error_word_rotate(cudaStream_t stream, int* rc) {
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

extern "C" int pa_rotation_set(pa_rotation* rot, int rot_dim, int interleaved,
                               const double* radians, float magnitude) {
  if (!rot || !radians || rot_dim < 2 || rot_dim > kHeadDim || rot_dim % 2 != 0) return PA_ERR_ARG;
  if (!isfinite(magnitude)) return PA_ERR_ARG;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!isfinite(radians[i])) return PA_ERR_ARG;
  rot->rot_dim = rot_dim;
  rot->interleaved = interleaved ? 1 : 0;
  rot->magnitude = magnitude;
  for (int i = 0; i < 64; ++i) rot->turns[i] = i < rot_dim / 2 ? turns_of(radians[i]) : 0;
  return PA_OK;
}

extern "C" int pa_rotation_init(pa_rotation* rot, int rot_dim, int interleaved, double base,
                                int scaling, double factor, double original_len, double low,
                                double high) {
  if (!rot || rot_dim < 2 || rot_dim > kHeadDim || rot_dim % 2 != 0) return PA_ERR_ARG;
  if (scaling < PA_ROT_PLAIN || scaling > PA_ROT_RAMP) return PA_ERR_ARG;
  if (!(base > 0) || !isfinite(base)) return PA_ERR_ARG;
  if (scaling != PA_ROT_PLAIN && (!(factor > 0) || !isfinite(factor))) return PA_ERR_ARG;
  if (scaling == PA_ROT_BANDS || scaling == PA_ROT_RAMP) {
    if (!(original_len > 0) || !isfinite(original_len) || !(low > 0) || !isfinite(high))
      return PA_ERR_ARG;
    if (scaling == PA_ROT_BANDS ? !(low < high) : !(low <= high)) return PA_ERR_ARG;
    if (scaling == PA_ROT_RAMP && !(base > 1)) return PA_ERR_ARG;
  }
  const double two_pi = 6.283185307179586476925286766559;
  const int n = rot_dim / 2;
  if (scaling == PA_ROT_BASE && rot_dim > 2)
    base *= pow(factor, (double)rot_dim / (rot_dim - 2));
  double theta[64], magnitude = 1.0, a = 0, b = 0;
  if (scaling == PA_ROT_RAMP) {
    // the pair that makes `turns` turns over the original length
    auto pair_with = [&](double turns) {
      return rot_dim * log(original_len / (two_pi * turns)) / (2 * log(base));
    };
    auto clamped = [&](double x) { return x < 0 ? 0 : x > rot_dim - 1 ? rot_dim - 1 : x; };
    a = clamped(floor(pair_with(high)));
    b = clamped(ceil(pair_with(low)));
    magnitude = 0.1 * log(factor) + 1;
  }
  for (int i = 0; i < n; ++i) {
    double t = pow(base, -2.0 * i / rot_dim), s = 0;
    if (scaling == PA_ROT_LINEAR) {
      t /= factor;
    } else if (scaling == PA_ROT_BANDS) {
      s = (original_len * t / two_pi - low) / (high - low);
      s = s < 0 ? 0 : s > 1 ? 1 : s;
      t = t * s + t / factor * (1 - s);
    } else if (scaling == PA_ROT_RAMP) {
      s = b > a ? (i - a) / (b - a) : (i > a ? 1 : 0);
      s = s < 0 ? 0 : s > 1 ? 1 : s;
      t = t * (1 - s) + t / factor * s;
    }
    theta[i] = t;
  }
  return pa_rotation_set(rot, rot_dim, interleaved, theta, (float)magnitude);
}

extern "C" int pa_rotate(const pa_row_view* x, const int32_t* positions, int64_t num_tokens,
                         int num_heads, int head_dim, const pa_rotation* rot, int transpose,
                         const pa_row_view* y, void* stream) {
  pa::NvtxRange nvtx_range("pa_rotate");
  if (num_tokens < 0 || num_heads < 0 || head_dim <= 0) return PA_ERR_ARG;
  if (head_dim != kHeadDim) return PA_ERR_UNSUPPORTED;
  if (!good_rotation(rot)) return PA_ERR_ARG;
  if (num_tokens == 0 || num_heads == 0) return PA_OK;
  if (!positions || !aligned(positions, 4)) return PA_ERR_ARG;
  if (!good_view(x, num_tokens, num_heads, false) || !good_view(y, num_tokens, num_heads, true))
    return PA_ERR_ARG;
  if (x->data == y->data && !same_view(x, y)) return PA_ERR_ARG;
  RowsArgs a = {};
  a.q = view_of(x);
  a.qo = view_of(y);
  a.positions = positions;
  a.Hq = num_heads;
  a.Hkv = 0;
  return launch_rows(a, num_tokens, kFmtBf16, rot, transpose, static_cast<cudaStream_t>(stream));
}

extern "C" int pa_rotate_and_cache(const pa_row_view* q, const pa_row_view* k,
                                   const pa_row_view* v, const int32_t* positions,
                                   const int64_t* slot_mapping, int64_t num_tokens,
                                   const pa_rotation* rot, const pa_row_view* q_out,
                                   void* k_cache, void* v_cache, int kv_format,
                                   const pa_shape* shape, void* stream) {
  pa::NvtxRange nvtx_range("pa_rotate_and_cache");
  const int rc = check_shape_common(shape);
  if (rc != PA_OK) return rc;
  if (kv_format < PA_KV_BF16 || kv_format > PA_KV_FP8) return PA_ERR_ARG;
  if (num_tokens < 0 || !good_rotation(rot)) return PA_ERR_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return PA_ERR_ARG;
  if (num_tokens == 0) return PA_OK;
  const int Hq = q ? shape->num_q_heads : 0, Hkv = shape->num_kv_heads;
  if (!good_view(k, num_tokens, Hkv, false) || !good_view(v, num_tokens, Hkv, false))
    return PA_ERR_ARG;
  if (q) {
    if (!good_view(q, num_tokens, Hq, false) || !good_view(q_out, num_tokens, Hq, true))
      return PA_ERR_ARG;
    if (q->data == q_out->data && !same_view(q, q_out)) return PA_ERR_ARG;
  }
  if (!positions || !slot_mapping || !k_cache || !v_cache) return PA_ERR_ARG;
  if (!aligned(positions, 4) || !aligned(slot_mapping, 8) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16))
    return PA_ERR_ARG;
  RowsArgs a = {};
  if (q) {
    a.q = view_of(q);
    a.qo = view_of(q_out);
  }
  a.k = view_of(k);
  a.v = view_of(v);
  a.positions = positions;
  a.slots = slot_mapping;
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.num_slots = shape->num_blocks * shape->block_size;
  a.Hq = Hq;
  a.Hkv = Hkv;
  return launch_rows(a, num_tokens, kv_format, rot, 0, static_cast<cudaStream_t>(stream));
}

extern "C" int pa_rotate_cached(void* k_cache, int kv_format, const int32_t* block_tables,
                                const int32_t* context_lens, const int32_t* shifts, int first,
                                const int32_t* kept, int kept_len, const pa_rotation* rot,
                                const pa_shape* shape, void* stream) {
  pa::NvtxRange nvtx_range("pa_rotate_cached");
  const int rc = check_shape_common(shape);
  if (rc != PA_OK) return rc;
  if (kv_format < PA_KV_BF16 || kv_format > PA_KV_FP8 || !good_rotation(rot)) return PA_ERR_ARG;
  if ((shifts == nullptr) == (kept == nullptr)) return PA_ERR_ARG;
  if (first < 0 || kept_len < 0 || (kept && first != 0) || (shifts && kept_len != 0))
    return PA_ERR_ARG;
  if (shape->num_seqs == 0 || shape->max_blocks_per_seq == 0) return PA_OK;
  if (!k_cache || !block_tables || !context_lens) return PA_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(shifts, 4) || !aligned(kept, 4))
    return PA_ERR_ARG;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return PA_ERR_CUDA;
  const int mode = mode_of(rot);
  const size_t smem = sizeof(int) * (4 * (size_t)shape->num_seqs + 3 + 2 * kTurns) +
                      (mode == kAny ? sizeof(float) * kRotWarps * 4 * kRowPad : 0);
  if (smem > (size_t)dev.max_smem_optin) return PA_ERR_UNSUPPORTED;
  // flat tile indices are 32-bit
  if ((int64_t)shape->num_seqs * shape->max_blocks_per_seq * shape->num_kv_heads > 0x7fffffff)
    return PA_ERR_UNSUPPORTED;
  const void* kern = cached_kernel(mode, kv_format);
  int per_sm = 0;
  if (!kernel_occupancy(kern, kRotWarps * 32, smem, &per_sm) || per_sm <= 0) return PA_ERR_CUDA;
  CachedArgs a = {};
  a.kc = static_cast<uint8_t*>(k_cache);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.shifts = shifts;
  a.kept = kept;
  a.first = first;
  a.kept_len = kept_len;
  a.S = shape->num_seqs;
  a.Hkv = shape->num_kv_heads;
  a.max_blocks = shape->max_blocks_per_seq;
  a.num_blocks = shape->num_blocks;
  a.rot = *rot;
  for (int i = rot->rot_dim / 2; i < 64; ++i) a.rot.turns[i] = 0;
  const int64_t most = (int64_t)a.S * a.max_blocks * a.Hkv;
  const int64_t need = (most + kRotWarps - 1) / kRotWarps;
  const int64_t room = (int64_t)dev.num_sms * per_sm;
  const dim3 grid((unsigned)(need < room ? need : room)), block(kRotWarps * 32);
  typedef void (*Kernel)(const CachedArgs);
  if (launch_dependent(reinterpret_cast<Kernel>(const_cast<void*>(kern)), grid, block, smem,
                       static_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
