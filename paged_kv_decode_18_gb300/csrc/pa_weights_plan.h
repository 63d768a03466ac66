// pa_weights_plan.h -- what a window costs in the plan of the tcgen05 weights
// kernel; plain arithmetic, for the device and for a test on the host.
#pragma once

#ifdef __CUDACC__
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kWeightKeys = 128;  // keys per item (MMA M)

// Query tiles that key tile kt of a window meets: those from the first token
// that sees a key of it.
PA_HD int first_tile(int kt, int c, int lq, int QTb) {
  const int over = kt * kWeightKeys - (c - lq);
  return over > 0 ? over / QTb : 0;
}

// A window's cost over all heads: one and its query tiles for each of its nt key
// tiles. The costs of S sequences are summed in 32 bits. What the call announced
// (max_q_len, the table's width) stays within 2^30; a window longer than that may
// not, and counts as the S-th part of 2^30 (only the cut between CTAs follows costs).
PA_HD int window_cost(int nt, int c, int lq, int QTb, int Hkv, int S) {
  const int nq = lq > 0 ? (lq - 1) / QTb + 1 : 0;
  long long cost = 0;
  for (int kt = 0; kt < nt; ++kt) cost += 1 + (nq > 1 ? nq - first_tile(kt, c, lq, QTb) : nq);
  cost *= Hkv;
  const int most = (1 << 30) / S;
  return cost < most ? (int)cost : most;
}

}  // namespace pa
