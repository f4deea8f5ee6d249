// Prefix sums over sequences by one CTA, shared by the page plans and the forks of sequences.
#pragma once

#include "common.cuh"
#include "op_util.h"

namespace qw {
namespace {

constexpr int PLAN_MAX_SEQS = 16384;
constexpr int PLAN_THREADS = 512;

constexpr uint32_t PLAN_CAP = 0x7fffffffu;
__device__ __forceinline__ uint32_t cap_add(uint32_t a, uint32_t b) { return min(a + b, PLAN_CAP); }  // a, b <= PLAN_CAP
__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = cap_add(v, u);
  }
  return v;
}

// Exclusive prefix sums over n items of two counts (item(i, a, b) gives them) into sa[0 .. n] and sb[0 .. n]. A sum
// that reaches 2^31 - 1 stays there.
template <typename Item>
__device__ __forceinline__ void block_scan2(int n, int* sa, int* sb, Item item) {
  __shared__ uint32_t wa[32], wb[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + PLAN_THREADS - 1) / PLAN_THREADS, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  uint32_t a = 0, b = 0;  // of the thread's consecutive items
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    uint32_t x = 0, y = 0;
    item(i, x, y);
    a = cap_add(a, x);
    b = cap_add(b, y);
  }
  const uint32_t ia = warp_incl_scan(a), ib = warp_incl_scan(b);
  if (warp == 0) wa[lane] = wb[lane] = 0;
  __syncthreads();
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  const uint32_t ta = warp_incl_scan(wa[lane]), tb = warp_incl_scan(wb[lane]);  // every warp scans the warps' sums
  uint32_t oa = warp ? __shfl_sync(0xffffffffu, ta, warp - 1) : 0, ob = warp ? __shfl_sync(0xffffffffu, tb, warp - 1) : 0;
  const uint32_t pa = __shfl_up_sync(0xffffffffu, ia, 1), pb = __shfl_up_sync(0xffffffffu, ib, 1);
  if (lane) {
    oa = cap_add(oa, pa);
    ob = cap_add(ob, pb);
  }
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    uint32_t x = 0, y = 0;
    item(i, x, y);
    sa[i] = (int)oa;
    sb[i] = (int)ob;
    oa = cap_add(oa, x);
    ob = cap_add(ob, y);
  }
  if (tid == PLAN_THREADS - 1) {
    sa[n] = (int)ta;
    sb[n] = (int)tb;
  }
  __syncthreads();
}

// the last b in [0, n) with s[b] <= x (s ascending, s[0] = 0, x < s[n])
__device__ __forceinline__ int find_seq(const int* s, int n, int x) {
  int lo = 0, hi = n;  // s[lo] <= x < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(long long positions, int page) {
  return (int)(positions >> 31 ? (positions + page - 1) / page : ((uint32_t)positions + (uint32_t)page - 1u) / (uint32_t)page);
}

}  // namespace
}  // namespace qw
