// Log probabilities of given tokens, with ranks, entropy and the likeliest tokens ("LLM Speedrun:
// Architecture", Decoding: the softmax of the logits).
//
// Mathematics: with m = max z, S = sum exp(z - m) and W = sum (z - m) exp(z - m), ln p_t = z_t - m - ln S and the
// entropy is ln S - W / S. A larger maximum m' turns S into S e^(m - m') and W into (W + (m - m') S) e^(m - m'),
// so one pass with running values does. Tokens are ordered by (logit, lower id first) as one 64-bit key.
//
// Precision: sums and differences are fp32, exponentials ex2's, good to 2^-22: a log probability is good to about a step of fp32 of
// itself (2e-9 to 1.1e-7 of a row's norm against 64 bits, a plain fp32 form 2e-9 to 5e-8), a near-certain token's to 1e-7 absolute.
//
// Times are in a CUDA graph; a lone call costs the host about 3 us from C, 10 to 14 from Python.
// What bounds it: each logit is read once, so HBM for fp32 logits (1024 rows of 151936: 131 us, 4.7 TB/s; without top
// tokens 106 us, 5.9 TB/s); 16-bit ones arrive twice as fast and are bound by the SMs' instructions, 9 to 14 a
// logit (1024 rows of 152064 bf16: 62 us for one likely id, 76 with a second, unlikely one whose rank counts
// every logit, 94 with 20 top tokens as well: 3.3 TB/s). One row takes 10 to 12 us, a chain of latencies: ids,
// batch, bound, second look, join.
// Short rows go to logprobs_rows.cu, whose row end has no barriers.
//   - All rows' batches (256 threads x 8 vectors of 16 bytes) form one list, cut into equal consecutive ranges,
//     one per CTA, three CTAs an SM. A row that a cut divides is joined by the last of its CTAs to arrive;
//     every sum's order is fixed, results repeat bit by bit.
//   - Each thread copies its own vectors (cp.async) into a ring of two batches and reads them back itself: no
//     barrier, and up to 96 KB in flight an SM. A batch is then in registers for its passes: maxima,
//     exponentials, counts for the ranks.
//   - Top tokens cost nothing while the row streams by but one stored maximum per thread and group of batches. At
//     the row's end the top_k-th largest thread maximum bounds the top_k-th logit from below; the groups whose
//     maximum reaches it, hardly more than top_k of them, are read again and their logits at or above the
//     bound sorted. (Lists that were kept while streaming, with a rising threshold, cost 50 us of 134 for
//     1024 rows of 152064: the warps met to raise it.)
//   - The join of a divided row takes one round trip to the L2 cache for all of its parts and a bound that about 2 top_k
//     of their keys reach (with the counts fetched id by id and a bound that let 400 keys in, 2 rows of 152064 fp32 and 32
//     top tokens took 23.5 us, not 12.4).
#include "logprobs.cuh"
#include "op_util.h"

#include <math.h>

#include <algorithm>

namespace qw {

constexpr int LP_NT = 256, LP_NW = LP_NT / 32, LP_VPT = 8, LP_NS = 2;  // threads, warps, a batch's 16-byte vectors a thread, ring
constexpr int LP_CTAS_PER_SM = 3, LP_MAX_CTAS = 640;
constexpr int LP_END = 5;         // what a row's end costs, in batches
constexpr int LP_CAP = 384;       // keys in the list and the pushed ones
constexpr int LP_EARLY = 3;       // keys of the parts that a thread fetches before it knows their bound

struct alignas(16) LogprobPart {  // of a row that several CTAs share
  float m, s, w, top;
  int above[LP_MAX_IDS];
  int nan, pad[3];
  u64 key[LP_MAX_TOP];  // its likeliest tokens, 0 behind the last
};

namespace {

constexpr int LP_GROUPS = 8;  // groups of a row's batches, of which each thread keeps a maximum
constexpr int LP_WORK = 128;   // groups that are read again at a time

struct Shared {
  u64 buf[2][LP_CAP];
  int n, side;                   // keys in buf[side]: the list, then what was pushed since
  u64 bar;                       // a key that is not above it cannot enter the list
  uint16_t top[LP_GROUPS][LP_NT];  // upper 16 bits of the ordered maxima
  uint16_t work[LP_WORK];        // group * LP_NT + thread
  int n_work;
  float red[4][LP_NW];
  int above[LP_MAX_IDS], nan;
  int id[2][LP_MAX_IDS], equal[2][LP_MAX_IDS];  // of the row and the next, by turns; equal: see fetch_ids
  float given[2][LP_MAX_IDS];
  bool last;
};

// Keeps the top_k largest of the n keys in buf[side], sorted, and their threshold. All threads; a barrier before.
__device__ __forceinline__ void compact(Shared& sh, int top_k) {
  const int n = min(sh.n, LP_CAP), side = sh.side, kept = min(n, top_k);
  const u64* from = sh.buf[side];
  u64* to = sh.buf[side ^ 1];
  // so many lanes count the keys above one
  const int log_lanes = n <= LP_NT / 8 ? 3 : n <= LP_NT / 4 ? 2 : n <= LP_NT / 2 ? 1 : 0, lanes = 1 << log_lanes;
#pragma unroll 1
  for (int i = threadIdx.x >> log_lanes; i < (n + 31 & ~31); i += LP_NT >> log_lanes) {  // (whole warps)
    const u64 key = i < n ? from[i] : ~0ull;
    int rank = 0;
#pragma unroll 4
    for (int x = threadIdx.x & (lanes - 1); x < n; x += lanes) rank += from[x] > key;
#pragma unroll 1
    for (int o = 1; o < lanes; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < n && rank < top_k) to[rank] = key;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    sh.n = kept;
    sh.side = side ^ 1;
    sh.bar = kept == top_k ? to[top_k - 1] : LP_NO_BAR;
  }
  __syncthreads();
}

// One batch of a row in registers: vector i of the thread is vector (batch * LP_VPT + i) * LP_NT + tid of the
// row, counted from the 16-byte boundary at or before its first logit.
template <typename T>
struct Batch {
  using Lg = Logits<T>;
  static constexpr int N = Lg::N;
  uint4 r[LP_VPT];
  int j0;            // id of vector 0's first logit (negative where the row begins inside a vector)
  __device__ __forceinline__ int id(int i) const { return j0 + i * LP_NT * N; }
  static __device__ __forceinline__ int first_id(const T* z, int batch) {
    return (batch * LP_NT * LP_VPT + (int)threadIdx.x) * N - (int)((uintptr_t)z % 16) / (int)sizeof(T);
  }

  // requests the thread's vectors of a batch into its places of a stage (place i: 16 bytes at i * LP_NT * 16)
  static __device__ __forceinline__ void request(const LogprobArgs& a, int row, int batch, unsigned char* stage) {
    const T* z = (const T*)a.logits + (long long)row * a.row_stride;
    const int j0 = first_id(z, batch);
    if (j0 >= 0 && j0 + (LP_VPT - 1) * LP_NT * N + N <= a.vocab) {
#pragma unroll
      for (int i = 0; i < LP_VPT; ++i) cp_async16(stage + i * LP_NT * 16, z + j0 + i * LP_NT * N);
      return;
    }
    const uint32_t none = Lg::minus_inf();
#pragma unroll 1
    for (int i = 0; i < LP_VPT; ++i) {
      const int j = j0 + i * LP_NT * N;
      unsigned char* to = stage + i * LP_NT * 16;
      if (j >= 0 && j + N <= a.vocab) {
        cp_async16(to, z + j);
      } else {  // behind the row, or cut by one of its ends
        *reinterpret_cast<uint4*>(to) = make_uint4(none, none, none, none);
#pragma unroll 1
        for (int e = max(0, -j); e < min(N, a.vocab - j); ++e) reinterpret_cast<T*>(to)[e] = z[j + e];
      }
    }
  }
  __device__ __forceinline__ void take(const LogprobArgs& a, int row, int batch, const unsigned char* stage) {
    j0 = first_id((const T*)a.logits + (long long)row * a.row_stride, batch);
#pragma unroll
    for (int i = 0; i < LP_VPT; ++i) r[i] = *reinterpret_cast<const uint4*>(stage + i * LP_NT * 16);
  }
};

// A bound on the top_k-th largest logit from the thread maxima, in steps of their upper 15 bits: the largest that
// top_k threads reach, at least the lowest finite logit's. By one warp: a search by all of them met at 16 barriers.
// All threads; the list is empty.
__device__ __forceinline__ uint32_t top_bound(Shared& sh, float tmax, int top_k) {
  uint16_t* all = reinterpret_cast<uint16_t*>(sh.buf[sh.side ^ 1]);
  all[threadIdx.x] = (uint16_t)(order_bits(tmax) >> 17);
  __syncthreads();
  if (threadIdx.x < 32) {
    const uint4 v = reinterpret_cast<const uint4*>(all)[threadIdx.x];
    uint32_t keys[4] = {v.x, v.y, v.z, v.w}, most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max(most, max(keys[i] & 0xffffu, keys[i] >> 16));
    const uint32_t bound = max(keys_bound<4>(keys, most, top_k), 0x40u);
    if (threadIdx.x == 0) sh.bar = bound;
  }
  __syncthreads();
  return (uint32_t)sh.bar;
}
static_assert(LP_NT == 32 * 8 && LP_MAX_TOP <= 32, "eight keys a lane");

// The sorted top_k (or fewer, of finite logits) of batches b0 .. b1 - 1 of a row, into the empty list. tmax: the
// thread's maximum of them; sh.top: its groups' (group: (batch - b0) / per). All threads.
template <typename T>
__device__ __forceinline__ void select_top(const LogprobArgs& a, Shared& sh, int row, int b0, int b1, int per, float tmax) {
  constexpr int N = Logits<T>::N;
  const int tid = threadIdx.x, top_k = a.top_k;
  const uint32_t bound = top_bound(sh, tmax, top_k);
  const T* z = (const T*)a.logits + (long long)row * a.row_stride;
  const int shift = (int)((uintptr_t)z % 16) / (int)sizeof(T);
  int hits = 0;  // the thread's groups that reach the bound
  for (int g = 0; g * per < b1 - b0; ++g) hits |= (sh.top[g][tid] >= 2 * bound) << g;
  u64 bar = ((u64)bound << 49) - 1;
#pragma unroll 1
  for (bool more = true; more;) {
    if (tid == 0) sh.n_work = 0;
    __syncthreads();
    while (hits) {
      const int at = atomicAdd(&sh.n_work, 1);
      if (at >= LP_WORK) break;
      sh.work[at] = (uint16_t)((__ffs(hits) - 1) * LP_NT + tid);
      hits &= hits - 1;
    }
    more = __syncthreads_or(hits);
    const int items = min(sh.n_work, LP_WORK) * per * LP_VPT;  // vectors
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += LP_NT) {
      float x[N];
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = -INFINITY;
      int j = 0;
      if (i0 + tid < items) {
        const int w = (i0 + tid) / (per * LP_VPT), v = (i0 + tid) - w * per * LP_VPT, g = sh.work[w] / LP_NT, th = sh.work[w] % LP_NT;
        const int batch = b0 + g * per + v / LP_VPT;
        j = ((batch * LP_VPT + v % LP_VPT) * LP_NT + th) * N - shift;
        if (batch < b1) {
          if (j >= 0 && j + N <= a.vocab) {
            unpack(ld_stream(z + j), x, T());
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (j + e >= 0 && j + e < a.vocab) x[e] = to_f32(z[j + e]);
          }
        }
      }
      uint32_t m = 0, left;
#pragma unroll
      for (int e = 0; e < N; ++e) m |= (x[e] == x[e] ? 1u : 0u) << e;
#pragma unroll 1
      do {  // (once, unless ties fill the list)
        uint32_t take = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) take |= (order_key(x[e], j + e) > bar ? 1u : 0u) << e;
        take &= m;
        int at = take ? atomicAdd(&sh.n, __popc(take)) : 0;
        left = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (take >> e & 1) {
            if (at < LP_CAP) sh.buf[sh.side][at] = order_key(x[e], j + e);
            else left |= 1u << e;
            ++at;
          }
        }
        m = left;
        left = __syncthreads_or(left);
        if (left) {
          compact(sh, top_k);
          bar = sh.bar > bar ? sh.bar : bar;
        }
      } while (left);
    }
  }
  __syncthreads();
  compact(sh, top_k);
}

// ln sum exp(z - most) and the entropy of a row with extreme values, from the definition. All threads.
template <typename T>
__device__ __noinline__ void slow_sums(const LogprobArgs& a, Shared& sh, int row, float most, float& ln_s, float& entropy, bool& nan) {
  const T* z = (const T*)a.logits + (long long)row * a.row_stride;
  float s = 0.f, w = 0.f;
  int bad = 0;
#pragma unroll 1
  for (int j = threadIdx.x; j < a.vocab; j += LP_NT) {
    const float x = to_f32(z[j]), d = x - most, e = expf(d);
    bad |= x != x;
    s += e;
    if (e > 0.f) w = fmaf(d, e, w);
  }
  nan = __syncthreads_or(bad);
  s = block_sum(s, sh.red[0]);
  w = block_sum(w, sh.red[0]);
  ln_s = logf(s);
  entropy = ln_s - w / s;
}

// Writes a row's results from its state (most: its largest logit; the list sorted in sh). All threads.
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobArgs& a, Shared& sh, int row, float most, float m, float s, float w, bool nan,
                                           int turn) {
  const int tid = threadIdx.x;
  // s and w are relative to m, the product log2(e) most as it was rounded: log2(e) most - m is exact, and brings
  // ln s to most
  float ln_s = (log2f(s) - fmaf(most, LP_LOG2E, -m)) * LP_LN2, entropy = (log2f(s) - w / s) * LP_LN2;
  if (fabsf(most) < INFINITY && extreme<T>(most)) slow_sums<T>(a, sh, row, most, ln_s, entropy, nan);
  const bool odd = nan || !(fabsf(most) < INFINITY);  // no distribution
  auto logprob = [&](float z) { return z - most - ln_s; };
  if (tid == 0) {
    if (odd) atomicOr(a.err, ERR_NONFINITE);
    if (a.entropy) a.entropy[row] = odd ? NAN : entropy;
  }
  if (tid < a.n_ids) {
    const int t = sh.id[turn][tid];
    const bool in = t >= 0 && t < a.vocab;
    if (!in && t != -1) atomicOr(a.err, ERR_TOKEN);
    a.logprobs[(size_t)row * a.n_ids + tid] = t == -1 ? 0.f : odd || !in ? NAN : logprob(sh.given[turn][tid]);
    if (a.ranks) a.ranks[(size_t)row * a.n_ids + tid] = odd || !in ? 0 : 1 + sh.above[tid];
  }
  if (tid < a.top_k && (odd || tid < sh.n)) {
    const u64 key = odd ? 0 : sh.buf[sh.side][tid];
    a.top_ids[(size_t)row * a.top_k + tid] = odd ? -1 : argmax_key_index(key);
    a.top_logprobs[(size_t)row * a.top_k + tid] = odd ? NAN : logprob(key_value(key));
  }
  if (!odd && sh.n < a.top_k && tid == 0) {  // fewer finite logits: the lowest ids of probability 0
    const T* z = (const T*)a.logits + (long long)row * a.row_stride;
    int k = sh.n;
#pragma unroll 1
    for (int j = 0; j < a.vocab && k < a.top_k; ++j) {
      if (to_f32(z[j]) == -INFINITY) {
        a.top_ids[(size_t)row * a.top_k + k] = j;
        a.top_logprobs[(size_t)row * a.top_k + k] = -INFINITY;
        ++k;
      }
    }
  }
}

// Reads one id of a row (this thread's), its logit, and how many equal logits stand before it in its vector (if that
// is in batches b0 .. b1 - 1: the passes count whole vectors), into place `turn`. Three loads that depend on one
// another: done a row ahead.
template <typename T>
__device__ __noinline__ void fetch_ids(const LogprobArgs& a, Shared& sh, int row, int b0, int b1, int turn) {
  constexpr int N = Logits<T>::N;
  const int t = a.ids[(size_t)row * a.n_ids + threadIdx.x];
  const T* z = (const T*)a.logits + (long long)row * a.row_stride;
  float given = NAN;
  int equal = 0;
  if (t >= 0 && t < a.vocab) {
    given = to_f32(z[t]);
    const int shift = (int)((uintptr_t)z % 16) / (int)sizeof(T), vec = (t + shift) / N, batch = vec / (LP_NT * LP_VPT);
    if (batch >= b0 && batch < b1)
#pragma unroll 1
      for (int j = max(0, vec * N - shift); j < t; ++j) equal += to_f32(z[j]) == given;
    if (given == -INFINITY && b0 == 0 && vec > 0) equal -= shift;  // what fills the first vector is counted too
  }
  sh.id[turn][threadIdx.x] = t;
  sh.equal[turn][threadIdx.x] = equal;
  sh.given[turn][threadIdx.x] = given;
}

// The list of all rows' batches, cut for the CTAs: into equal ranges (a range may end inside a row and go on with the
// next), or into ranges of whole row pieces.
struct Cuts {
  int batches, pieces, ctas, each, rest, items;
  __device__ __forceinline__ explicit Cuts(const LogprobArgs& a) : batches(a.batches), pieces(a.pieces), ctas(gridDim.x) {
    items = pieces ? a.n_rows * pieces : a.n_rows * batches;
    each = items / ctas;
    rest = items - each * ctas;
  }
  __device__ __forceinline__ int begin(int c) const {
    const int i = each * c + min(c, rest);
    return pieces ? i / pieces * batches + i % pieces * batches / pieces : i;
  }
  // the CTA that has batch x, the first or the last of a row
  __device__ __forceinline__ int cta_of(int x) const {
    const int i = pieces ? x / batches * pieces + (x % batches ? pieces - 1 : 0) : x, big = rest * (each + 1);
    return i < big ? i / (each + 1) : rest + (i - big) / each;
  }
};

// One CTA's range of the list of batches.
template <typename T>
__global__ void __launch_bounds__(LP_NT, LP_CTAS_PER_SM) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int N = Batch<T>::N;
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ __align__(16) unsigned char lp_ring[];
  const Cuts cuts(a);
  const int mine = cuts.begin(blockIdx.x), end = cuts.begin(blockIdx.x + 1);
  int at = mine;
  int ld_row = at / a.batches, ld_batch = at - ld_row * a.batches, to_load = end - at, ld_stage = 0, stage = 0;
  auto stage_ptr = [&](int i) { return lp_ring + (i * LP_NT * LP_VPT + tid) * 16; };
  auto load_next = [&]() {
    if (to_load > 0) {
      --to_load;
      Batch<T>::request(a, ld_row, ld_batch, stage_ptr(ld_stage));
      if (++ld_batch == a.batches) {
        ld_batch = 0;
        ++ld_row;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++ld_stage == LP_NS) ld_stage = 0;
  };
  int turn = 0;           // which of the two places has the row's ids
  int ahead = LP_NS - 1;  // batches still to be requested before the first is used
#pragma unroll 1
  while (at < end) {
    const int row = at / a.batches, b0 = at - row * a.batches, b1 = min(a.batches, b0 + end - at);
    if (tid < a.n_ids) {
      if (at == mine) fetch_ids<T>(a, sh, row, b0, b1, 0);
      sh.above[tid] = sh.equal[turn][tid];
    }
    if (tid == 0) {
      sh.n = 0;
      sh.side = 0;
      sh.bar = LP_NO_BAR;
      sh.nan = 0;
    }
    __syncthreads();
    // this thread's sums, in base 2 all: s = sum 2^(log2(e) z - m), w = sum (log2(e) z - m) 2^(..). m is the
    // maximum's product with log2(e) as it was rounded, so that its rounding is in no result.
    float m = -INFINITY, s = 0.f, w = 0.f, most = -INFINITY;
    bool nan = false;
    const int per = (b1 - b0 + LP_GROUPS - 1) / LP_GROUPS;  // batches of a group
    Batch<T> b;
#pragma unroll 1
    for (int batch = b0; batch < b1;) {
      load_next();  // into the stage that the last batch used
      if (ahead) {
        --ahead;
        continue;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(LP_NS - 1) : "memory");
      b.take(a, row, batch, stage_ptr(stage));
      if (++stage == LP_NS) stage = 0;
      typename Batch<T>::Lg::Top tops;
#pragma unroll
      for (int i = 0; i < LP_VPT; ++i) tops.add(b.r[i]);
      const float top = tops.value();
      most = fmaxf(most, top);
      const float to = fmaxf(top, Batch<T>::Lg::floor()) * LP_LOG2E;
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
      for (int i = 0; i < LP_VPT; ++i) {
        f32x2 x[N / 2];
        Batch<T>::Lg::pairs(b.r[i], x);
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
      nan |= s != s;
      if (a.ranks) {
#pragma unroll 1
        for (int q = 0; q < a.n_ids; ++q) {
          const int t = sh.id[turn][q];
          const float z = sh.given[turn][q];
          if (!__any_sync(0xffffffffu, top >= z)) continue;  // (none above a likely token in most batches)
          // whole vectors before t count from z on, the others from the next larger value on; equal logits
          // before t in its own vector were counted when the row began
          const typename Batch<T>::Lg::Thr here = Batch<T>::Lg::thr(z), next = Batch<T>::Lg::thr_above(z);
          typename Batch<T>::Lg::Count count;
          const int v = b.id(LP_VPT - 1) + N <= t ? LP_VPT : b.id(0) + N > t ? 0 : (t - b.j0 - N) / (LP_NT * N) + 1;  // vectors before t
#pragma unroll
          for (int i = 0; i < LP_VPT; ++i) count.add(b.r[i], i < v ? here : next);
          int above = count.total();
          above = __reduce_add_sync(0xffffffffu, above);
          if (lane == 0 && above) atomicAdd(&sh.above[q], above);
        }
      }
      if (a.top_k) {
        const int g = (batch - b0) / per;
        const uint32_t key = order_bits(top) >> 16;
        sh.top[g][tid] = (uint16_t)((batch - b0) % per ? max(key, (uint32_t)sh.top[g][tid]) : key);
      }
      // the next row's ids, by the first warp, while the others go on
      if (batch++ == b0 && tid < a.n_ids && at + b1 - b0 < end) fetch_ids<T>(a, sh, row + 1, 0, min(a.batches, end - at - (b1 - b0)), turn ^ 1);
    }
    // the CTA's state of the row
    if (a.top_k) select_top<T>(a, sh, row, b0, b1, per, most);
    float mm = warp_max(m);
    most = warp_max(most);
    if (lane == 0) {
      sh.red[0][warp] = mm;
      sh.red[3][warp] = most;
    }
    if (nan) sh.nan = 1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LP_NW; ++i) {
      mm = fmaxf(mm, sh.red[0][i]);
      most = fmaxf(most, sh.red[3][i]);
    }
    {
      const float d = m == -INFINITY ? 0.f : m - mm, f = m == -INFINITY ? 0.f : ex2(d);
      w = warp_sum(fmaf(d, s, w) * f);
      s = warp_sum(s * f);
    }
    if (lane == 0) {
      sh.red[1][warp] = s;
      sh.red[2][warp] = w;
    }
    __syncthreads();
    s = w = 0.f;
#pragma unroll
    for (int i = 0; i < LP_NW; ++i) {
      s += sh.red[1][i];
      w += sh.red[2][i];
    }
    nan = sh.nan;
    bool write = b1 - b0 == a.batches;
    if (!write) {
      // part slots as the list is cut: 2 c for the row a CTA begins with, 2 c + 1 for one that it begins itself
      const int r0 = row * a.batches;
      const int c0 = cuts.cta_of(r0), c1 = cuts.cta_of(r0 + a.batches - 1), first = 2 * c0 + (cuts.begin(c0) < r0 ? 1 : 0);
      auto slot_of = [&](int c) { return a.parts + (c == c0 ? first : 2 * c); };
      LogprobPart* mine = slot_of(blockIdx.x);
      if (tid == 0) {
        *reinterpret_cast<float4*>(&mine->m) = make_float4(mm, s, w, most);
        mine->nan = nan;
      }
      if (tid < a.n_ids) mine->above[tid] = sh.above[tid];
      if (tid < a.top_k) mine->key[tid] = tid < sh.n ? sh.buf[sh.side][tid] : 0;
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        sh.last = atomicAdd(a.counters + first, 1u) == (unsigned)(c1 - c0);
        if (sh.last) a.counters[first] = 0u;
        __threadfence();
        sh.n = 0;
        sh.nan = 0;
      }
      if (tid < a.n_ids) sh.above[tid] = 0;
      __syncthreads();
      write = sh.last;
      if (write) {
        // Everything of the parts is fetched at once. Every thread takes the parts c0 + tid, + LP_NT, ...: the same
        // order of sums at every run.
        const int parts = c1 - c0 + 1, top_k = a.top_k;
        u64 early[LP_EARLY];
#pragma unroll
        for (int k = 0; k < LP_EARLY; ++k) {
          const int i = tid + k * LP_NT, c = i / LP_MAX_TOP, e = i % LP_MAX_TOP;
          early[k] = c < parts && e < top_k ? __ldcg(&slot_of(c0 + c)->key[e]) : 0;
        }
        // j parts whose q-th keys reach a key have j q >= top_k keys that do: the j-th largest of all q-th keys bounds the
        // list from below. With q near twice the mean a part has, about 2 top_k keys reach it.
        const int asked = min(parts, LP_CAP), q = min(top_k, (2 * top_k + asked - 1) / asked), jth = q ? (top_k + q - 1) / q : 0;
        u64* qth = sh.buf[sh.side ^ 1];
        float pm = -INFINITY, ps = 0.f, pw = 0.f, pt = -INFINITY;
#pragma unroll 1
        for (int c = tid; c < parts; c += LP_NT) {
          const LogprobPart* p = slot_of(c0 + c);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(&p->m));
          const int4 n0 = __ldcg(reinterpret_cast<const int4*>(p->above)), n1 = __ldcg(reinterpret_cast<const int4*>(p->above) + 1);
          const int bad = __ldcg(&p->nan);
          if (q && c < asked) qth[c] = __ldcg(&p->key[q - 1]);
          const int n[LP_MAX_IDS] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
          for (int e = 0; e < LP_MAX_IDS; ++e)
            if (e < a.n_ids && n[e]) atomicAdd(&sh.above[e], n[e]);
          if (bad) sh.nan = 1;
          pt = fmaxf(pt, v.w);
          if (v.x > -INFINITY) {
            const float to = fmaxf(pm, v.x), d0 = pm == -INFINITY ? 0.f : pm - to, d1 = v.x - to, f0 = ex2(d0), f1 = ex2(d1);
            pw = fmaf(d0, ps, pw) * f0 + fmaf(d1, v.y, v.z) * f1;
            ps = fmaf(ps, f0, v.y * f1);
            pm = to;
          }
        }
        mm = warp_max(pm);
        most = warp_max(pt);
        if (lane == 0) {
          sh.red[0][warp] = mm;
          sh.red[3][warp] = most;
        }
        if (tid == 0) sh.bar = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LP_NW; ++i) {
          mm = fmaxf(mm, sh.red[0][i]);
          most = fmaxf(most, sh.red[3][i]);
        }
        {
          const float d = pm == -INFINITY ? 0.f : pm - mm, f = pm == -INFINITY ? 0.f : ex2(d);
          w = warp_sum(fmaf(d, ps, pw) * f);
          s = warp_sum(ps * f);
        }
        if (lane == 0) {
          sh.red[1][warp] = s;
          sh.red[2][warp] = w;
        }
        if (q) {
#pragma unroll 1
          for (int c = tid; c < asked; c += LP_NT) {
            const u64 key = qth[c];
            int larger = 0;
#pragma unroll 4
            for (int x = 0; x < asked; ++x) larger += qth[x] > key;
            if (key && larger == jth - 1) sh.bar = key;
          }
        }
        __syncthreads();
        s = w = 0.f;
#pragma unroll
        for (int i = 0; i < LP_NW; ++i) {
          s += sh.red[1][i];
          w += sh.red[2][i];
        }
        nan = sh.nan;
        if (q) {
          const u64 bar = sh.bar;
          auto push = [&](u64 key) {
            if (!key || key < bar) return;
            const int to = atomicAdd(&sh.n, 1);
            if (to < LP_CAP) sh.buf[sh.side][to] = key;
          };
#pragma unroll
          for (int k = 0; k < LP_EARLY; ++k) push(early[k]);
#pragma unroll 1
          for (int i = tid + LP_EARLY * LP_NT; i < parts * LP_MAX_TOP; i += LP_NT)
            if (i % LP_MAX_TOP < top_k) push(__ldcg(&slot_of(c0 + i / LP_MAX_TOP)->key[i % LP_MAX_TOP]));
          __syncthreads();
          const int listed = sh.n;
          __syncthreads();
          if (listed <= LP_CAP) {
            compact(sh, top_k);
          } else {  // more keys than have room: some parts at a time, next to the best ones
            if (tid == 0) sh.n = 0;
            __syncthreads();
            constexpr int step = (LP_CAP - LP_MAX_TOP) / LP_MAX_TOP;
#pragma unroll 1
            for (int c = 0; c < parts; c += step) {
              const int n = min(step, parts - c);
#pragma unroll 1
              for (int i = tid; i < n * LP_MAX_TOP; i += LP_NT)
                if (i % LP_MAX_TOP < top_k) push(__ldcg(&slot_of(c0 + c + i / LP_MAX_TOP)->key[i % LP_MAX_TOP]));
              __syncthreads();
              compact(sh, top_k);
            }
          }
        }
      }
    }
    if (write) finish_row<T>(a, sh, row, most, mm, s, w, nan, turn);
    __syncthreads();
    at += b1 - b0;
    turn ^= 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T>
cudaError_t launch_logprobs(LogprobArgs a, int nsm, cudaStream_t s) {
  constexpr int N = Logits<T>::N;
  // the first vector may begin before the row, by up to N - 1 logits
  a.batches = (int)(((long long)a.vocab + N - 1 + LP_NT * LP_VPT * N - 1) / (LP_NT * LP_VPT * N));
  const long long total = (long long)a.n_rows * a.batches;
  const int ctas = std::min(nsm * LP_CTAS_PER_SM, LP_MAX_CTAS);
  // The last CTA's time, in batches: equal ranges pay for one row end more than they have rows (about LP_END batches:
  // 8 us of latency against 1.5 us a batch), whole pieces for what the largest range has over the mean.
  const double equal = (double)total / ctas + LP_END * ((double)a.n_rows / ctas + 1);
  const int split = a.n_rows >= ctas ? 1 : std::min(ctas / a.n_rows, a.batches);
  const double whole = (double)(((long long)a.n_rows * split + ctas - 1) / ctas) * ((a.batches + split - 1) / split + LP_END);
  a.pieces = whole <= equal ? split : 0;
  const int grid = (int)std::min<long long>(a.pieces ? (long long)a.n_rows * a.pieces : total, ctas);
  constexpr int ring = LP_NS * LP_NT * LP_VPT * 16;
  const cudaError_t e = cudaFuncSetAttribute(logprob_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
  return e ? e : launch_k(logprob_kernel<T>, dim3(grid), dim3(LP_NT), ring, s, false, a);
}
static_assert(2 * LP_MAX_CTAS * sizeof(unsigned int) <= OP_COUNTER_BYTES, "counters");

// Whether a warp a row (logprobs_rows.cu) is faster. A warp takes 6 us and 0.8 a KB of row, for as many rows as the GPU
// has warps; the CTAs 9 us for every row that each of them gets, almost whatever its length. us here and there, 20 top
// tokens: 16 rows of 2 KB 8.9 and 7.0, of 4 KB 8.7 and 8.7, of 8 KB 8.8 and 12.5; 1024 rows of 8 KB 24 and 13, of 16 KB 25 and
// 20; 4096 rows of 2 KB 79 and 12.9, of 16 KB 84 and 40, of 32 KB 83 and 66 (without top tokens 43 and 47). The limit
// also keeps a lane's chain of additions short: 24 KB of 16-bit logits are 192 on a path.
bool rows_for_warps(int dtype, int n_rows, int vocab, int nsm) {
  const long long rounds = ((long long)n_rows + nsm * LP_CTAS_PER_SM - 1) / (nsm * LP_CTAS_PER_SM);
  return (long long)vocab * (long long)dtype_size(dtype) <= std::min(4096 * rounds, 24576ll);
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_token_logprobs_workspace(int32_t n_rows, int32_t vocab, int32_t top_k) {
  if (n_rows < 0 || vocab < 1 || top_k < 0 || top_k > LP_MAX_TOP) return 0;
  return OP_COUNTER_BYTES + 2 * LP_MAX_CTAS * sizeof(LogprobPart);
}

qw_status qw_op_token_logprobs(int32_t logits_dtype, int32_t n_rows, int32_t vocab, const void* logits,
                               int64_t row_stride, const int32_t* ids, int32_t n_ids, float* logprobs, int32_t* ranks,
                               float* entropy, int32_t top_k, int32_t* top_ids, float* top_logprobs, void* workspace,
                               size_t workspace_bytes, int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  if (!dtype_known(logits_dtype)) return op_fail(QW_ERR_INVALID_ARG, "unknown logits dtype");
  if (n_rows < 0 || vocab < 1) return op_fail(QW_ERR_INVALID_ARG, "bad row count or vocabulary");
  if (n_ids < 0 || n_ids > LP_MAX_IDS) return op_fail(QW_ERR_INVALID_ARG, "n_ids must be 0 .. 8");
  if (top_k < 0 || top_k > LP_MAX_TOP || top_k > vocab)
    return op_fail(QW_ERR_INVALID_ARG, "top_k must be 0 .. min(32, vocab)");
  if (row_stride < vocab || row_stride > (int64_t)1 << 40) return op_fail(QW_ERR_INVALID_ARG, "row_stride smaller than a row");
  // the list of batches (of at least 4096 logits) has 31-bit numbers, and so have ids with a batch's overhang
  if ((int64_t)n_rows * (vocab / 4096 + 2) > 0x7fffffffll || vocab > 0x7fff0000)
    return op_fail(QW_ERR_UNSUPPORTED, "n_rows * vocab too large");
  if (n_rows == 0) return QW_OK;
  if (!logits || !err_dev || !workspace || (n_ids && (!ids || !logprobs)) || (top_k && (!top_ids || !top_logprobs)))
    return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)logits % dtype_size(logits_dtype)) return op_fail(QW_ERR_INVALID_ARG, "logits misaligned");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_token_logprobs_workspace(n_rows, vocab, top_k))
    return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  const void* allocation = (const void*)((uintptr_t)logits & ~(uintptr_t)3);  // (16-bit rows may begin between)
  qw_status st = op_check_device({allocation, n_ids ? ids : nullptr, n_ids ? logprobs : nullptr, n_ids ? ranks : nullptr,
                                  entropy, top_k ? top_ids : nullptr, top_k ? top_logprobs : nullptr, workspace,
                                  err_dev});
  if (st) return st;
  int dev = 0, nsm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  const LogprobArgs a{logits, row_stride, n_rows, vocab, n_ids, top_k, 0, 0, ids, logprobs, ranks, entropy, top_ids,
                      top_logprobs, (unsigned int*)workspace, (LogprobPart*)((char*)workspace + OP_COUNTER_BYTES), err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  e = rows_for_warps(logits_dtype, n_rows, vocab, nsm) ? launch_logprobs_rows(logits_dtype, a, nsm, s)
      : logits_dtype == QW_F32 ? launch_logprobs<float>(a, nsm, s)
      : logits_dtype == QW_F16 ? launch_logprobs<f16>(a, nsm, s) : launch_logprobs<bf16>(a, nsm, s);
  if (e) return op_cuda_fail(e, "token logprobs launch");
  return QW_OK;
}

}  // extern "C"
