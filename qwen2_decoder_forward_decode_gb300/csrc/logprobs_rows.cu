// Log probabilities of given tokens, with ranks, entropy and the likeliest tokens, of short rows ("LLM Speedrun:
// Architecture", Decoding: the softmax of the logits). The mathematics is logprobs.cu's.
//
// What bounds it: a CTA that shares a row meets about 40 barriers at the row's end, 8 us whatever the row's length. Here
// a warp has a row to itself and waits for no other. 4096 rows of 1000 bf16 logits take 6.6 us, with 20 top tokens
// 12.9 (by CTAs 43 and 79): the SMs' instructions, 930 and 1900 a row. A single row is a chain of latencies, 4 and
// 6.5 us.
//   - A lane loads two vectors of 16 bytes at a time, two batches ahead; 32 warps an SM cover the rest.
//   - Top tokens: each lane stores the maximum of each of up to 16 groups of its batches, as the upper 15 bits of its
//     ordered form. The top_k-th largest of these (up to 512) bounds the top_k-th logit from below; the groups that
//     reach it, hardly more than top_k, are read again, from the caches, and their logits at or above the bound
//     sorted. (The bound's search takes pairs of keys and skips the bits that all lanes' maxima share, what is read again
//     is compared as floats, divisions are multiplications: 1330 instructions a row became 560 for one top token.)
#include "../../include/qw.h"
#include "logprobs.cuh"

#include <algorithm>

namespace qw {
namespace {

constexpr int RW_NT = 256, RW_NW = RW_NT / 32, RW_VB = 2;  // threads, warps, a batch's vectors a lane
constexpr int RW_GROUPS = 16, RW_CAP = 224;                // groups of a lane's batches; keys in the list and the pushed ones

struct alignas(16) WarpShared {
  u64 buf[2][RW_CAP];
  uint32_t top[32][RW_GROUPS / 2];  // upper 15 bits of the ordered maxima, in pairs
  uint16_t work[32 * RW_GROUPS];    // groups that are read again: group * 32 + lane
  int n;                            // keys in the list
};

__device__ __forceinline__ int first_lanes(unsigned mask, int lane) { return __popc(mask & ((1u << lane) - 1u)); }

// The top_k largest of the n keys in `from`, sorted into `to`; returns their number. The whole warp.
__device__ __forceinline__ int keep_top(const u64* from, u64* to, int n, int top_k, int lane) {
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < n; i += 32) {
    const u64 key = from[i];
    int rank = 0;
#pragma unroll 4
    for (int x = 0; x < n; ++x) rank += from[x] > key;
    if (rank < top_k) to[rank] = key;
  }
  __syncwarp();
  return min(n, top_k);
}

template <typename T>
struct Row {
  using Lg = Logits<T>;
  static constexpr int N = Lg::N;
  const T* z;
  int vocab, shift;  // logits between the 16-byte boundary at or before the first one and that
  __device__ __forceinline__ int id(int vec) const { return vec * N - shift; }
  // vector `vec` of the row, -inf where it has none
  __device__ __forceinline__ uint4 load(int vec) const {
    const int j = id(vec);
    if (j >= 0 && j + N <= vocab) return ld_cached(z + j);
    const uint32_t none = Lg::minus_inf();
    uint4 r = make_uint4(none, none, none, none);
    if (j < vocab) {  // cut by one of the row's ends
      uint32_t u[4] = {none, none, none, none};
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (j + e < 0 || j + e >= vocab) continue;
        if constexpr (sizeof(T) == 4) u[e] = __float_as_uint(z[j + e]);
        else u[e / 2] = e % 2 ? (u[e / 2] & 0xffffu) | (uint32_t)bits16(z + j + e) << 16 : (u[e / 2] & 0xffff0000u) | bits16(z + j + e);
      }
      r = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return r;
  }
  static __device__ __forceinline__ uint32_t bits16(const T* p) { return *reinterpret_cast<const uint16_t*>(p); }
  static __device__ __forceinline__ uint4 ld_cached(const T* p) { return *reinterpret_cast<const uint4*>(p); }
};

// ln sum exp(z - most) and the entropy of a row with extreme values, from the definition. The whole warp.
template <typename T>
__device__ __noinline__ void slow_sums(const T* z, int vocab, float most, float& ln_s, float& entropy, bool& nan) {
  float s = 0.f, w = 0.f;
  bool bad = false;
#pragma unroll 1
  for (int j = threadIdx.x % 32; j < vocab; j += 32) {
    const float x = to_f32(z[j]), d = x - most, e = expf(d);
    bad |= x != x;
    s += e;
    if (e > 0.f) w = fmaf(d, e, w);
  }
  nan = __any_sync(0xffffffffu, bad);
  s = warp_sum(s);
  w = warp_sum(w);
  ln_s = logf(s);
  entropy = ln_s - w / s;
}

struct RowArgs {
  LogprobArgs a;
  int batches, per, groups;  // of a row; batches of a group
  uint32_t item_magic;       // 2^32 / (per * RW_VB), rounded up: divides by umulhi
};

// The largest 15-bit key that top_k of the row's groups reach (the lane's in pairs of sh.top, 2 * W or fewer), at least
// that of the lowest finite logit; `hits`: the lane's groups that reach it. The whole warp.
template <int W>
__device__ __forceinline__ uint32_t top_bound(const WarpShared& sh, int top_k, int lane, int& hits) {
  uint32_t keys[W];
#pragma unroll
  for (int i = 0; i < W; ++i) keys[i] = sh.top[lane][i];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) most = max(most, max(keys[i] & 0xffffu, keys[i] >> 16));
  const uint32_t bound = max(keys_bound<W>(keys, most, top_k), 0x40u);
  const uint32_t v = bound * 0x10001u;
  hits = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t n = (keys[i] - v) >> 15 & 0x10001u;
    hits |= ((n & 1u) | n >> 15) << 2 * i;
  }
  return bound;
}

// The sorted top_k (or fewer, of finite logits) of a row into sh.buf[side]; returns their number and sets side. The
// whole warp.
template <typename T>
__device__ __forceinline__ int select_top(WarpShared& sh, const Row<T>& rw, const RowArgs& ra, int lane, int& side) {
  constexpr int N = Row<T>::N;
  const int top_k = ra.a.top_k;
  int hits;
  __syncwarp();  // (the maxima were stored in halves)
  const uint32_t bound = ra.groups <= 2 ? top_bound<1>(sh, top_k, lane, hits)
                         : ra.groups <= 4 ? top_bound<2>(sh, top_k, lane, hits) : top_bound<RW_GROUPS / 2>(sh, top_k, lane, hits);
  int n_work = 0;
#pragma unroll 1
  for (int g = 0; g < ra.groups; ++g) {
    const bool hit = hits >> g & 1;
    const unsigned mask = __ballot_sync(0xffffffffu, hit);
    if (hit) sh.work[n_work + first_lanes(mask, lane)] = (uint16_t)(g * 32 + lane);
    n_work += __popc(mask);
  }
  if (lane == 0) sh.n = 0;
  __syncwarp();
  const float least = order_value(bound << 17);  // of the logits that the bound lets in
  const int items = n_work * ra.per * RW_VB;     // vectors
  u64 bar = 0;                                   // a key that is not above it cannot enter the list
#pragma unroll 1
  for (int i0 = 0; i0 < items; i0 += 32) {
    uint32_t take = 0;
    float x[N];
    int j = 0;
    const int item = i0 + lane;
    if (item < items) {
      const int w = __umulhi(item, ra.item_magic), v = item - w * ra.per * RW_VB, work = sh.work[w];
      const int batch = work / 32 * ra.per + v / RW_VB;
      j = rw.id((batch * RW_VB + v % RW_VB) * 32 + work % 32);
      if (batch < ra.batches) {
        unpack(rw.load((batch * RW_VB + v % RW_VB) * 32 + work % 32), x, T());  // (-inf where the row has none)
#pragma unroll
        for (int e = 0; e < N; ++e) take |= (x[e] >= least ? 1u : 0u) << e;
      }
    }
    bool more;
#pragma unroll 1
    do {  // (once, unless ties fill the list)
      int at = take ? atomicAdd(&sh.n, __popc(take)) : 0;
      uint32_t left = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (take >> e & 1) {
          if (at < RW_CAP) sh.buf[side][at] = order_key(x[e], j + e);
          else left |= 1u << e;
          ++at;
        }
      }
      more = __any_sync(0xffffffffu, left != 0);
      if (more) {  // the list is full: its best ones make room
        const int n = keep_top(sh.buf[side], sh.buf[side ^ 1], RW_CAP, top_k, lane);
        side ^= 1;
        bar = sh.buf[side][n - 1];
        if (lane == 0) sh.n = n;
        take = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) take |= ((left >> e & 1) && order_key(x[e], j + e) > bar ? 1u : 0u) << e;
        __syncwarp();
      }
    } while (more);
  }
  __syncwarp();
  const int n = keep_top(sh.buf[side], sh.buf[side ^ 1], sh.n, top_k, lane);
  side ^= 1;
  return n;
}
static_assert(RW_CAP >= 2 * LP_MAX_TOP, "a full list must shrink");

// A warp takes rows w, w + (warps of the grid), ...
template <typename T>
__global__ void __launch_bounds__(RW_NT, 4) logprob_rows_kernel(const __grid_constant__ RowArgs ra) {
  using Lg = Logits<T>;
  constexpr int N = Lg::N;
  const LogprobArgs& a = ra.a;
  __shared__ WarpShared all[RW_NW];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, top_k = a.top_k;
  WarpShared& sh = all[warp];
#pragma unroll 1
  for (int row = blockIdx.x * RW_NW + warp; row < a.n_rows; row += gridDim.x * RW_NW) {
    Row<T> rw;
    rw.z = (const T*)a.logits + (long long)row * a.row_stride;
    rw.vocab = a.vocab;
    rw.shift = (int)((uintptr_t)rw.z % 16) / (int)sizeof(T);
    uint4 r[RW_VB], next[RW_VB];
    auto load = [&](uint4* to, int batch) {
#pragma unroll
      for (int i = 0; i < RW_VB; ++i) to[i] = rw.load((batch * RW_VB + i) * 32 + lane);
    };
    load(r, 0);
    if (ra.batches > 1) load(next, 1);
    // lane q: id q of the row, its logit, how many logits stand before it. Equal logits before it in its vector are
    // counted here, since the passes count whole vectors.
    int t = -1, above = 0;
    float given = NAN;
    if (lane < a.n_ids) {
      t = a.ids[(size_t)row * a.n_ids + lane];
      if (t >= 0 && t < a.vocab) {
        given = to_f32(rw.z[t]);
        const int vec = (t + rw.shift) / N;
#pragma unroll 1
        for (int j = max(0, rw.id(vec)); j < t; ++j) above += to_f32(rw.z[j]) == given;
        if (given == -INFINITY && vec > 0) above -= rw.shift;  // what fills the first vector is counted too
      }
    }
    if (top_k) {
#pragma unroll
      for (int i = 0; i < RW_GROUPS / 8; ++i) reinterpret_cast<uint4*>(sh.top[lane])[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    // this lane's sums, in base 2: s = sum 2^(log2(e) z - m), w = sum (log2(e) z - m) 2^(..); m is the maximum's product
    // with log2(e) as it was rounded, so that its rounding is in no result
    float m = -INFINITY, s = 0.f, w = 0.f, most = -INFINITY, group_most = -INFINITY;
    int group = 0, in_group = 0;
#pragma unroll 1
    for (int batch = 0; batch < ra.batches; ++batch) {
      typename Lg::Top tops;
#pragma unroll
      for (int i = 0; i < RW_VB; ++i) tops.add(r[i]);
      const float top = tops.value();
      most = fmaxf(most, top);
      const float to = fmaxf(top, Lg::floor()) * LP_LOG2E;
      if (to > m) {
        const float d = m - to, f = ex2(d);
        if (m == -INFINITY) s = w = 0.f;
        else {
          w = fmaf(d, s, w) * f;
          s *= f;
        }
        m = to;
      }
      const f32x2 ref = pack2(-m, -m), l2e = pack2(LP_LOG2E, LP_LOG2E);
      f32x2 s2 = pack2(s, 0.f), w2 = pack2(w, 0.f);
#pragma unroll
      for (int i = 0; i < RW_VB; ++i) {
        f32x2 x[N / 2];
        Lg::pairs(r[i], x);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const f32x2 d = fma2_to(x[e], l2e, ref);
          const float2 v = unpack2(d);
          const f32x2 p = pack2(ex2(v.x), ex2(v.y));
          s2 = add2(s2, p);
          fma2(w2, d, p);
        }
      }
      s = unpack2(s2).x + unpack2(s2).y;
      w = unpack2(w2).x + unpack2(w2).y;
      if (a.ranks) {
        const int j0 = rw.id(batch * RW_VB * 32 + lane);
#pragma unroll 1
        for (int q = 0; q < a.n_ids; ++q) {
          const int tq = __shfl_sync(0xffffffffu, t, q);
          const float zq = __shfl_sync(0xffffffffu, given, q);
          if (!__any_sync(0xffffffffu, top >= zq)) continue;
          // whole vectors before t count from z on, the others from the next larger value on
          const typename Lg::Thr here = Lg::thr(zq), next_up = Lg::thr_above(zq);
          typename Lg::Count count;
#pragma unroll
          for (int i = 0; i < RW_VB; ++i) count.add(r[i], j0 + i * 32 * N + N <= tq ? here : next_up);
          const int n = __reduce_add_sync(0xffffffffu, count.total());
          if (lane == q) above += n;
        }
      }
      if (top_k) {
        group_most = fmaxf(group_most, top);
        if (++in_group == ra.per || batch + 1 == ra.batches) {
          reinterpret_cast<uint16_t*>(sh.top[lane])[group++] = (uint16_t)(order_bits(group_most) >> 17);
          group_most = -INFINITY;
          in_group = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < RW_VB; ++i) r[i] = next[i];
      if (batch + 2 < ra.batches) load(next, batch + 2);
    }
    int side = 0, n_top = 0;
    if (top_k) n_top = select_top<T>(sh, rw, ra, lane, side);
    bool nan = __any_sync(0xffffffffu, s != s);
    const float mm = warp_max(m);
    most = warp_max(most);
    {
      const float d = m == -INFINITY ? 0.f : m - mm, f = m == -INFINITY ? 0.f : ex2(d);
      w = warp_sum(fmaf(d, s, w) * f);
      s = warp_sum(s * f);
    }
    // log2(e) most - mm is exact, and brings ln s to most
    float ln_s = (log2f(s) - fmaf(most, LP_LOG2E, -mm)) * LP_LN2, entropy = (log2f(s) - w / s) * LP_LN2;
    if (fabsf(most) < INFINITY && extreme<T>(most)) slow_sums<T>(rw.z, a.vocab, most, ln_s, entropy, nan);
    const bool odd = nan || !(fabsf(most) < INFINITY);  // no distribution
    if (lane == 0) {
      if (odd) atomicOr(a.err, ERR_NONFINITE);
      if (a.entropy) a.entropy[row] = odd ? NAN : entropy;
    }
    if (lane < a.n_ids) {
      const bool in = t >= 0 && t < a.vocab;
      if (!in && t != -1) atomicOr(a.err, ERR_TOKEN);
      a.logprobs[(size_t)row * a.n_ids + lane] = t == -1 ? 0.f : odd || !in ? NAN : given - most - ln_s;
      if (a.ranks) a.ranks[(size_t)row * a.n_ids + lane] = odd || !in ? 0 : 1 + above;
    }
    if (lane < top_k && (odd || lane < n_top)) {
      const u64 key = odd ? 0 : sh.buf[side][lane];
      a.top_ids[(size_t)row * top_k + lane] = odd ? -1 : argmax_key_index(key);
      a.top_logprobs[(size_t)row * top_k + lane] = odd ? NAN : key_value(key) - most - ln_s;
    }
    if (!odd && n_top < top_k) {  // fewer finite logits: the lowest ids of probability 0
      int k = n_top;
#pragma unroll 1
      for (int j0 = 0; j0 < a.vocab && k < top_k; j0 += 32) {
        const bool none = j0 + lane < a.vocab && to_f32(rw.z[j0 + lane]) == -INFINITY;
        const unsigned mask = __ballot_sync(0xffffffffu, none);
        const int at = k + first_lanes(mask, lane);
        if (none && at < top_k) {
          a.top_ids[(size_t)row * top_k + at] = j0 + lane;
          a.top_logprobs[(size_t)row * top_k + at] = -INFINITY;
        }
        k += __popc(mask);
      }
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_logprobs_rows(int dtype, const LogprobArgs& a, int nsm, cudaStream_t s) {
  const int n = 32 * RW_VB * (dtype == QW_F32 ? 4 : 8), first = dtype == QW_F32 ? 3 : 7;  // (the first vector may begin before the row)
  RowArgs ra{a, (a.vocab + first + n - 1) / n, 0, 0, 0};
  ra.per = (ra.batches + RW_GROUPS - 1) / RW_GROUPS;
  ra.groups = (ra.batches + ra.per - 1) / ra.per;
  ra.item_magic = 0xffffffffu / (ra.per * RW_VB) + 1;
  const dim3 grid(std::min((a.n_rows + RW_NW - 1) / RW_NW, nsm * 4)), block(RW_NT);
  return dtype == QW_F32   ? launch_k(logprob_rows_kernel<float>, grid, block, 0, s, false, ra)
         : dtype == QW_F16 ? launch_k(logprob_rows_kernel<f16>, grid, block, 0, s, false, ra)
                           : launch_k(logprob_rows_kernel<bf16>, grid, block, 0, s, false, ra);
}

}  // namespace qw
