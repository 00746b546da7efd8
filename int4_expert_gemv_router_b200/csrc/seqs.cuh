// Packed sequences: checking the caller's row ranges on the device and scanning over them.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMaxSeqs = 65536;
constexpr int kPlanThreads = 256;  // one CTA plans a call; more warps only take turns at the schedulers (1,024: 2-3 times as long)

// Exclusive prefix maximum and sum over the CTA's kPlanThreads threads, plus the running
// values of earlier rounds (carry_max, carry_sum, the same in every thread), which are moved
// on.  sh: one int per warp.  All threads call it.
__device__ __forceinline__ int block_excl_max(int v, int& carry, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int m = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, u);
  }
  if (lane == 31) sh[warp] = m;
  int before = __shfl_up_sync(0xffffffffu, m, 1);
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPlanThreads / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < kPlanThreads / 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = max(w, u);
    }
    if (lane < kPlanThreads / 32) sh[lane] = w;
  }
  __syncthreads();
  int r = carry;
  if (warp) r = max(r, sh[warp - 1]);
  if (lane) r = max(r, before);
  carry = max(carry, sh[kPlanThreads / 32 - 1]);
  __syncthreads();
  return r;
}
__device__ __forceinline__ int block_excl_sum(int v, int& carry, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPlanThreads / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < kPlanThreads / 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    if (lane < kPlanThreads / 32) sh[lane] = w;
  }
  __syncthreads();
  const int r = carry + (warp ? sh[warp - 1] : 0) + s - v;
  carry += sh[kPlanThreads / 32 - 1];
  __syncthreads();
  return r;
}

// The same over one warp, a lane a sequence: the largest v of the lanes before (0 at least), and the sum
// of v up to and with this lane.
__device__ __forceinline__ int warp_excl_max(int v, int lane) {
  v = __shfl_up_sync(0xffffffffu, v, 1);  // every lane shuffles: no lane may read one that does not
  v = lane ? max(v, 0) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = max(v, u);
  }
  return v;
}
__device__ __forceinline__ int warp_incl_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Sequence i's rows [a, b) are usable when the offsets are in order up to here and inside
// [0, T]: a at least every earlier offset (seen: their maximum, 0 at least), a <= b <= T.
// The usable sequences of a call are then disjoint.
__device__ __forceinline__ bool rows_ok(int a, int b, int seen, int T) { return a >= seen && b >= a && b <= T; }

}  // namespace moe
