// Beam search's selection: the best candidates over the beams and the vocabulary of each group ("LLM Speedrun:
// Architecture", Decoding: the softmax of the logits), and the beams' token histories in their new order.
//
// Mathematics: beam w of score c goes on with token t at c + z_t - ln sum_j exp(z_j). One pass over the logits gives the sum
// and what can still be among the n_out best:
//   - The row is cut into pieces, a piece into chunks of 256 logits, a warp's load. A piece keeps every chunk's maximum; the
//     n_out-th largest of them bounds the n_out-th logit from below. Only chunks that reach the bound are looked at again
//     (from L2): all whose maximum lies above it, fewer than n_out, and of those that equal it the first n_out, since a
//     later one's equals come behind theirs. So rows full of equal logits cost no more than others.
//   - Candidates of different beams may lie closer than fp32 tells, and their order decides what the beams become. So the
//     order is that of scores in 64 bits, and the normaliser is summed for it: exponents are taken over an integer
//     power of two, 2^(z log2(e) - k), with log2(e) in two parts (one rounding of a small number each), so moving k is
//     exact; a lane's sum carries its rounding errors along in a second number, all sums of sums are whole numbers or 64-bit.
//   - ex2 is good to 2^-22 only. So a piece's logits above 2^-10 of its sum (at most 1024) are taken again in 64 bits, relative to
//     the piece's largest, in the place of what they were in the sum: a lane's share of a chunk is taken out as it went in, and
//     its other logits are put back. What remains are the smaller ones, whose errors mostly cancel once their mean is added back.
//     Against 64 bits the normaliser is off by 1e-10 where few tokens carry a row (by nothing where it is one), by 1e-9 to 2e-8
//     of wide rows, by 2e-7 at worst (thousands of equal logits that carry a row together).
//   - A second launch joins a group: pieces' sums, then the lists, of which only those with the n_out best heads count. A warp
//     holds a list a lane and takes the best head n_out times.
// What takes its time (no single resource is used up): the instructions of a logit (unpacking, two exponent products, a sum and
// its rounding in pairs, an exponential, a maximum), the second look and its 64-bit operations, then the groups' latency.
// 64 x 4 beams of 152064 logits, bf16: 33 us (2.4 TB/s); 4 beams 18, all latency; 8 x 32 beams, 32 candidates, fp32: 73 (2.1 TB/s).
// The sums' rounding costs 2.4 us of the 33, the logits that are taken again 3 to 4.
#include "common.cuh"
#include "op_util.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace qw {
namespace {

typedef unsigned long long u64;

constexpr int BS_MAX_BEAMS = 32, BS_MAX_OUT = 32, BS_NT = 256, BS_NW = BS_NT / 32;
constexpr int BS_CHUNK = 256, BS_MAX_CHUNKS = 1024;  // logits of a chunk; chunks of a piece
constexpr int BS_MAX_LISTS = 256;                    // beams * pieces of a group
constexpr int BS_MAX_VOCAB = 1 << 21;
constexpr int BS_CAP = 512;                          // candidates of a piece before they are ranked
constexpr float BS_LOG2E_HI = 1.44269502162933349609375f, BS_LOG2E_LO = 1.92596303e-8f;  // their sum is log2(e) to 2^-50
constexpr double BS_LN2 = 0.693147180559945309417232121458;
constexpr float BS_FAR = 1048576.f;  // maxima beyond it take the slow sum,
constexpr float BS_NEAR = BS_FAR - 128.f;  // and those below -BS_NEAR: chunks below -BS_FAR are left out of the other one

// Sums of 2^(z log2(e) - ref) are kept in units of 2^-38, which add and shift without rounding and fast (64-bit floating
// point costs 30 to 40 cycles an operation here).
constexpr double BS_REST = 0x1p-38 * (1. + 5.17e-8);  // ex2's results are 5.17e-8 too small on average over a factor of 2, 1.42e-7 at most (measured)
constexpr int BS_HOT = 1152;  // logits of a piece that are taken again: 1024 by the rule, whose bound is off by e^0.11 at most
// A piece's sum of exponentials: e^top exact + 2^ref rest, top its largest logit (-inf: none).
struct PieceState {
  double exact;
  long long rest;  // in units
  float top, ref;
};
struct BeamArgs {
  const void* logits;
  long long row_stride;
  int groups, beams, vocab, n_out, pieces, chunks, end_id, width;  // chunks: of a piece
  const float *scores, *weights;
  const int *ended, *history, *lens;
  int *parents, *tokens, *ended_out, *history_out, *lens_out;
  float* scores_out;
  PieceState* state;  // [rows][pieces]
  u64* cand;          // [rows][pieces][n_out], best first, 0 behind the last
  int* err;
};

// (logit, lower id first) as an integer; -0 counts as 0; a NaN's is any
__device__ __forceinline__ uint32_t value_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
constexpr uint32_t BS_NONE = 0x007fffffu;  // the key of -inf: every candidate's is above

// x, |x| <= 2^9, in units of 2^-38, rounded: its 2^-13ths first, what they leave is at most 2^-14 (conversions to 64 bits are slow: with
// them 4 beams took 42 us instead of 36, when a warp took a chunk's logits again)
__device__ __forceinline__ long long to_units(float x) {
  const float t = fmaf(x, 8192.f, 12582912.f), left = fmaf(t - 12582912.f, -1.f / 8192.f, x);
  return ((long long)(__float_as_int(t) - 0x4b400000) << 25) + __float2int_rn(left * 0x1p38f);
}

// units / 2^d for a whole number d >= 0 (or infinite)
__device__ __forceinline__ u64 shifted(u64 units, float d) { return d < 64.f ? units >> (int)d : 0ull; }

// 2^d of a whole number d <= 0, exactly; 0 below the normal numbers
__device__ __forceinline__ float power2(float d) { return d < -126.f ? 0.f : __uint_as_float((uint32_t)(127 + (int)d) << 23); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 8 logits of a lane. Wide: rows on 16-byte boundaries; 16-bit lanes hold logits lane * 8 .. + 7 of the chunk, fp32 ones
// lane * 4 .. + 3 and 128 behind. Else a logit at a time, lane + 32 e.
template <typename T, bool WIDE>
struct Chunk {
  static __device__ __forceinline__ int index(int lane, int e) {
    if (!WIDE) return e * 32 + lane;
    return sizeof(T) == 2 ? lane * 8 + e : (e >> 2) * 128 + lane * 4 + (e & 3);
  }
  static constexpr int WORDS = WIDE && sizeof(T) == 2 ? 4 : 8;
  uint32_t u[WORDS];
  __device__ __forceinline__ void load(const T* z, int left, int lane) {  // left: logits of the row from the chunk on
    if constexpr (WIDE) {
      constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
      for (int v = 0; v < WORDS / 4; ++v) {
        const int at = index(lane, v * V);
        uint4 r;
        if (at + V <= left) r = ld_stream(z + at);
        else r = edge(z, at, left);
        u[4 * v] = r.x; u[4 * v + 1] = r.y; u[4 * v + 2] = r.z; u[4 * v + 3] = r.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = e * 32 + lane < left ? __float_as_uint(to_f32(z[e * 32 + lane])) : 0xff800000u;
    }
  }
  static __device__ __noinline__ uint4 edge(const T* z, int at, int left) {  // cut by the row's end
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = at + i < left ? __float_as_uint(to_f32(z[at + i])) : 0xff800000u;
      } else {
        const uint32_t none = std::is_same<T, bf16>::value ? 0xff80u : 0xfc00u;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(z);
        const uint32_t lo = at + 2 * i < left ? p[at + 2 * i] : none, hi = at + 2 * i + 1 < left ? p[at + 2 * i + 1] : none;
        w[i] = lo | hi << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ float2 two(int i) const {  // logits 2 i, 2 i + 1
    if constexpr (WORDS == 4) {
      if constexpr (std::is_same<T, bf16>::value) return make_float2(bf_lo(u[i]), bf_hi(u[i]));
      else return __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    } else {
      return make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    }
  }
  __device__ __forceinline__ float at(int e) const { const float2 x = two(e >> 1); return e & 1 ? x.y : x.x; }
  __device__ __forceinline__ float top() const {  // NaN if there is one
    if constexpr (WORDS == 4 && std::is_same<T, bf16>::value) {
      auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&u[i]); };
      const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(0), h(1)), __hmax2_nan(h(2), h(3)));
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
      return max_nan(bf_lo(b), bf_hi(b));
    } else if constexpr (WORDS == 4) {
      auto h = [&](int i) { return *reinterpret_cast<const __half2*>(&u[i]); };
      const float2 m = __half22float2(__hmax2_nan(__hmax2_nan(h(0), h(1)), __hmax2_nan(h(2), h(3))));
      return max_nan(m.x, m.y);
    } else {
      float m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = max_nan(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
      return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
    }
  }
};

struct BeamShared {
  uint32_t top[BS_MAX_CHUNKS];       // maxima of the chunks
  uint32_t sub[64 * 32];             // of their lanes, where the candidates are many
  u64 key[BS_CAP + BS_MAX_OUT];
  int work[2 * BS_MAX_OUT + 2], equals[2 * BS_MAX_OUT + 2];
  u64 units[BS_NW];
  double sum[BS_NW];
  float ref[BS_NW];
  uint32_t most[BS_NW];
  int n, n_work;
  uint32_t bound;
  float chunk_ref[BS_MAX_CHUNKS];  // what a chunk was summed with
  uint16_t hot[BS_HOT];            // chunk * 32 + lane of logits that are taken again
  int n_hot;
  long long moved[BS_NW];  // what that changes in the sum, in units
  long long exact[BS_NW];  // their own sum in units of 2^-52
};

// The largest key that `k` of a warp's keys (NR a lane, of any number) reach, or one between it and the next larger; `least` if
// fewer than k are above it.
template <int NR>
__device__ __forceinline__ uint32_t key_bound(const uint32_t* keys, int k, uint32_t least) {
  uint32_t most = least, low = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    most = max(most, keys[i]);
    low = min(low, keys[i]);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  low = max(least, __reduce_min_sync(0xffffffffu, low));
  if (most <= low) return low;
  // common leading bits are the bound's, the others are tried from the top
  int bit = 31 - __clz(most ^ low);
  uint32_t v = bit == 31 ? 0u : most >> (bit + 1) << (bit + 1);
#pragma unroll 1
  for (; bit >= 0; --bit) {
    const uint32_t t = v | 1u << bit;
    int c = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) c += keys[i] >= t;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= k) v = t;
    if (c == k) break;
  }
  return max(v, least);
}

// The piece's bound and the chunks that reach it, in order: all above it, of those that equal it the first k. A warp.
template <int NR>
__device__ __noinline__ void choose_chunks(BeamShared& sh, int n, int k, int lane) {
  uint32_t keys[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) keys[i] = 32 * i + lane < n ? sh.top[32 * i + lane] : 0u;
  const uint32_t b = key_bound<NR>(keys, k, BS_NONE);
  int n_work = 0, same = 0;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (32 * i >= n) break;
    const uint32_t top = keys[i];
    const unsigned eq = __ballot_sync(0xffffffffu, top == b && b > BS_NONE);
    const bool take = top > b || (top == b && b > BS_NONE && same + __popc(eq & ((1u << lane) - 1u)) < k);
    const unsigned mask = __ballot_sync(0xffffffffu, take);
    if (take) sh.work[n_work + __popc(mask & ((1u << lane) - 1u))] = 32 * i + lane;
    n_work += __popc(mask);
    same += __popc(eq);
  }
  if (lane == 0) {
    sh.bound = b;
    sh.n_work = n_work;
    sh.n = 0;
  }
}
// A closer bound, of the lanes' maxima of those chunks (rare; more than a lane's registers should hold).
__device__ __noinline__ void closer_bound(BeamShared& sh, int n_work, int k, int lane) {
  uint32_t v = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = v | 1u << bit;
    int c = 0;
#pragma unroll 4
    for (int i = 0; i < n_work; ++i) c += sh.sub[i * 32 + lane] >= t;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= k) v = t;
    if (c == k) break;
  }
  if (lane == 0) {
    sh.bound = max(v, sh.bound);
    sh.n = 0;
  }
}

__device__ __forceinline__ long long warp_add(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The terms of a chunk over 2^ref, and their sums by halves of a pair
template <typename C>
__device__ __forceinline__ f32x2 chunk_terms(const C& x, float ref, f32x2* e) {
  const f32x2 hi2 = pack2(BS_LOG2E_HI, BS_LOG2E_HI), lo2 = pack2(BS_LOG2E_LO, BS_LOG2E_LO), r2 = pack2(-ref, -ref);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 z = x.two(i);
    const f32x2 z2 = pack2(z.x, z.y);
    const float2 y = unpack2(fma2_to(z2, lo2, fma2_to(z2, hi2, r2)));
    e[i] = pack2(ex2(y.x), ex2(y.y));
  }
  return add2(add2(e[0], e[1]), add2(e[2], e[3]));
}

// e^d of -700 < d <= 0 to 1e-10 of it, 1 of 0: d = n ln 2 + r, the series of e^r, from r^4 on in fp32 (at most 6e-4 of it). 64-bit
// operations are what bounds where it is used: 8 here, 17 in exp(); 256 x 4 beams of 4000 logits 31 -> 28 us.
__device__ __forceinline__ double exp_down(double d) {
  const float n = rintf((float)d * BS_LOG2E_HI);
  const double r = fma((double)n, -BS_LN2, d);
  const float f = (float)r;
  float q = fmaf(f, 1.f / 362880, 1.f / 40320);
  q = fmaf(f, q, 1.f / 5040);
  q = fmaf(f, q, 1.f / 720);
  q = fmaf(f, q, 1.f / 120);
  q = fmaf(f, q, 1.f / 24);
  double p = fma((double)q, r, 1. / 6.);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.);
  p = fma(p, r, 1.);
  return __hiloint2double(__double2hiint(p) + ((int)n << 20), __double2loint(p));
}

// The logits from the key `least` on of a lane's share of a chunk, taken out of the sum over 2^ref (what that changes in it, in
// units) and summed by themselves relative to `top` (in 2^-52).
template <typename C>
__device__ __forceinline__ void take_out(const C& x, float chunk_ref, uint32_t least, float ref, float top, long long& moved, long long& exact) {
  f32x2 e[4];
  const float2 sum = unpack2(chunk_terms(x, chunk_ref, e));
  const float unit = power2(chunk_ref - ref);
  float stays = 0.f;
  unsigned mask = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 two = unpack2(e[i >> 1]);
    if (value_key(x.at(i)) >= least) mask |= 1u << i;
    else stays += i & 1 ? two.y : two.x;
  }
  moved += to_units(stays * unit) - to_units(sum.x * unit) - to_units(sum.y * unit);
#pragma unroll 1
  for (; mask; mask &= mask - 1) {
    const int at = __ffs(mask) - 1;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v = at == i ? x.at(i) : v;
    exact += __double_as_longlong(1. + exp_down((double)v - (double)top)) - 0x3ff0000000000000ll;  // (in [1, 2] a number's bits count steps of 2^-52)
  }
}

// CTAs an SM: four of 16-bit rows, with 64 registers (64 x 4 beams 33 us; three, with 80, 38). fp32 rows as the compiler likes it: held to
// three CTAs, 8 x 32 beams take 69 us instead of 73, but 4 beams 19.0 instead of 17.8, and rows read a logit at a time 70 instead of 62.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(BS_NT, WIDE && sizeof(T) == 2 ? 4 : 1) beam_rows_kernel(const BeamArgs a) {
  using C = Chunk<T, WIDE>;
  __shared__ BeamShared sh;
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / a.pieces, piece = blockIdx.x - row * a.pieces;
  const float score = a.scores[row];
  if ((a.ended && a.ended[row]) || !(fabsf(score) < INFINITY)) return;  // no candidates of the row's logits
  const int k = a.n_out, from = piece * a.chunks * BS_CHUNK;
  const int n = min(a.chunks, (a.vocab - from + BS_CHUNK - 1) / BS_CHUNK);  // chunks of this piece; may be none
  const T* z = (const T*)a.logits + row * a.row_stride + from;
  const int left = a.vocab - from;
  const uint32_t far_low = value_key(-BS_FAR), far_high = value_key(BS_FAR);
  if (tid == 0) sh.n_hot = 0;

  float ref = 0.f;  // an integer; meaningful once `any`
  bool any = false;
  f32x2 acc = 0ull, rest = 0ull;  // a sum, and what its additions rounded off
  uint32_t most = 0;  // of the warp's chunks
  constexpr int U = 4;  // chunks requested at a time
  const f32x2 minus = pack2(-1.f, -1.f);
  C next[U];
#pragma unroll
  for (int q = 0; q < U; ++q) {
    const int c = warp + q * BS_NW;
    if (c < n) next[q].load(z + c * BS_CHUNK, left - c * BS_CHUNK, lane);
  }
#pragma unroll 1
  for (int c0 = warp; c0 < n; c0 += U * BS_NW) {
    C now[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      now[q] = next[q];
      const int c = c0 + (U + q) * BS_NW;
      if (c < n) next[q].load(z + c * BS_CHUNK, left - c * BS_CHUNK, lane);
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int c = c0 + q * BS_NW;
      if (c >= n) break;
      const float lane_top = now[q].top();
      const uint32_t top = __reduce_max_sync(0xffffffffu, lane_top == lane_top ? value_key(lane_top) : 0xffffffffu);  // (NaN above everything)
      if (lane == 0) sh.top[c] = top;
      most = max(most, top);
      if (top > far_low && top < far_high) {  // else e^-128 of the piece's largest and less, or the piece takes the slow sum
        const float need = ceilf(key_value(top) * BS_LOG2E_HI);
        if (!any || need > ref) {
          const float f = any ? power2(ref - need) : 0.f;
          const f32x2 f2 = pack2(f, f);
          mul2(acc, f2);
          mul2(rest, f2);
          ref = need;
          any = true;
        }
        if (lane == 0) sh.chunk_ref[c] = ref;
        f32x2 e[4];
        const f32x2 x = chunk_terms(now[q], ref, e), sum = add2(acc, x), part = fma2_to(acc, minus, sum);  // (a - b as -1 * b + a)
        rest = add2(rest, add2(fma2_to(fma2_to(part, minus, sum), minus, acc), fma2_to(part, minus, x)));
        acc = sum;
      }
    }
  }
  {
    // (a lane has at most 128 chunks, whose halves add 4 each: sums of 25 bits, those over the lanes fit 32)
    const float2 s0 = unpack2(acc), s1 = unpack2(rest);
    const u64 mine = any ? (u64)(to_units(s0.x) + to_units(s0.y) + to_units(s1.x) + to_units(s1.y)) : 0ull;
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)mine & 0x1ffffffu), hi = __reduce_add_sync(0xffffffffu, (uint32_t)(mine >> 25));
    if (lane == 0) {
      sh.units[warp] = ((u64)hi << 25) + lo;
      sh.ref[warp] = any ? ref : -INFINITY;
      sh.most[warp] = most;
    }
  }
  __syncthreads();
  uint32_t peak = 0;
#pragma unroll
  for (int w = 0; w < BS_NW; ++w) peak = max(peak, sh.most[w]);
  const bool far = peak <= value_key(-BS_NEAR) || peak >= far_high;
  const float m = peak >= 0xff800000u ? INFINITY : key_value(max(peak, BS_NONE));  // (+inf or NaN: the sum becomes NaN)
  u64 units = 0;  // the sum over 2^ref
  if (far) {
    // the largest logit is far out, or there is a NaN: the definition, on a few threads' patience
    double s = 0.;
    if (peak > BS_NONE)
#pragma unroll 1
      for (int j = tid; j < min(left, n * BS_CHUNK); j += BS_NT) s += (double)expf(to_f32(z[j]) - m);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane == 0) sh.sum[warp] = s;
  } else {
    ref = -INFINITY;
#pragma unroll
    for (int w = 0; w < BS_NW; ++w) ref = fmaxf(ref, sh.ref[w]);
#pragma unroll
    for (int w = 0; w < BS_NW; ++w) units += shifted(sh.units[w], ref - sh.ref[w]);
  }

  uint32_t least = 0xffffffffu;  // of the logits above 2^-10 of the sum
  if (!far) {
    const float y = fmaf(m, BS_LOG2E_LO, fmaf(m, BS_LOG2E_HI, -ref));  // the largest term's exponent
    least = value_key(m + (log2f((float)units) - (38.f + 10.f) - y) * (float)BS_LN2);
  }

  // ---- the piece's candidates; meanwhile the other warps look for those logits
  if (warp == 0) {
    if (n <= 256) choose_chunks<8>(sh, n, k, lane);
    else choose_chunks<BS_MAX_CHUNKS / 32>(sh, n, k, lane);
  } else if (!far) {
#pragma unroll 1
    for (int c0 = warp - 1; c0 < n; c0 += 32 * (BS_NW - 1)) {  // a chunk a lane; those found 8 at a time
      const int mine = c0 + lane * (BS_NW - 1);
      unsigned hot = __ballot_sync(0xffffffffu, mine < n && sh.top[mine] >= least);
#pragma unroll 1
      while (hot) {
        C x[8];
        int at[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          at[q] = hot ? c0 + (__ffs(hot) - 1) * (BS_NW - 1) : -1;
          hot &= hot - 1;
          if (at[q] >= 0) x[q].load(z + at[q] * BS_CHUNK, left - at[q] * BS_CHUNK, lane);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (at[q] >= 0 && value_key(x[q].top()) >= least) {
            const int i = atomicAdd(&sh.n_hot, 1);
            if (i < BS_HOT) sh.hot[i] = (uint16_t)(at[q] * 32 + lane);
          }
      }
    }
  }
  __syncthreads();
  {  // a share a thread, from the last thread on: the first ones have more to do
    const int n_hot = min(sh.n_hot, BS_HOT);
    long long moved = 0, exact = 0;
#pragma unroll 1
    for (int i = BS_NT - 1 - tid; i < n_hot; i += BS_NT) {
      const int c = sh.hot[i] >> 5;
      C x;
      x.load(z + c * BS_CHUNK, left - c * BS_CHUNK, sh.hot[i] & 31);
      take_out(x, sh.chunk_ref[c], least, ref, m, moved, exact);
    }
    if (__any_sync(0xffffffffu, exact != 0)) {
      moved = warp_add(moved);
      exact = warp_add(exact);
    }
    if (lane == 0) {
      sh.moved[warp] = moved;
      sh.exact[warp] = exact;
    }
  }
  const int n_work = sh.n_work;  // at most 2 k
  uint32_t bound = sh.bound;
  // keys above the bound into the list, the equals counted; again with a closer bound if they are too many
#pragma unroll 1
  for (int turn = 0;; ++turn) {
#pragma unroll 1
    for (int i = warp; i < n_work; i += BS_NW) {
      const int c = sh.work[i];
      C x;
      x.load(z + c * BS_CHUNK, left - c * BS_CHUNK, lane);
      int eq = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = value_key(x.at(e));
        if (v > bound) {
          const int at = atomicAdd(&sh.n, 1);
          if (at < BS_CAP) sh.key[at] = (u64)v << 32 | (0xffffffffu - (uint32_t)(from + c * BS_CHUNK + C::index(lane, e)));
        }
        eq += v == bound;
      }
      if (turn == 0) sh.sub[i * 32 + lane] = value_key(x.top());
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) sh.equals[i] = eq;
    }
    __syncthreads();
    if (sh.n <= BS_CAP) break;  // (the second bound: fewer than k lanes of 8 logits lie above it)
    __syncthreads();
    if (warp == 0) closer_bound(sh, n_work, k, lane);
    __syncthreads();
    bound = sh.bound;
  }
  if (tid == BS_NT - 1) {
    PieceState st{0., (long long)units, m, far ? -INFINITY : ref};
    long long exact = 0;
#pragma unroll
    for (int w = 0; w < BS_NW; ++w) {
      if (far) st.exact += sh.sum[w];
      st.rest += sh.moved[w];
      exact += sh.exact[w];
    }
    if (!far) st.exact = (double)exact * 0x1p-52;
    st.rest = max(st.rest, 0ll);  // (negative by its rounding only)
    a.state[(size_t)row * a.pieces + piece] = st;
  }
  int n_key = sh.n;
  const int want = bound > BS_NONE ? k - n_key : 0;  // equals that may still count, those with the lowest ids
  if (want > 0) {
#pragma unroll 1
    for (int i = warp; i < n_work; i += BS_NW) {
      int before = 0;
#pragma unroll 1
      for (int j = 0; j < i; ++j) before += sh.equals[j];
      if (before >= want || sh.equals[i] == 0) continue;
      const int c = sh.work[i];
      C x;
      x.load(z + c * BS_CHUNK, left - c * BS_CHUNK, lane);
      // a lane's logits in the order of their ids: all of a lane before the next one's, or, a step at a time, across the lanes
      constexpr int RUN = !WIDE ? 1 : sizeof(T) == 2 ? 8 : 4;
#pragma unroll
      for (int e0 = 0; e0 < 8; e0 += RUN) {
        int mine = 0;
#pragma unroll
        for (int e = e0; e < e0 + RUN; ++e) mine += value_key(x.at(e)) == bound;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        int at = before + incl - mine;
#pragma unroll
        for (int e = e0; e < e0 + RUN; ++e)
          if (value_key(x.at(e)) == bound) {
            if (at < want) sh.key[n_key + at] = (u64)bound << 32 | (0xffffffffu - (uint32_t)(from + c * BS_CHUNK + C::index(lane, e)));
            ++at;
          }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    int all = 0;
#pragma unroll 1
    for (int j = 0; j < n_work; ++j) all += sh.equals[j];
    n_key += min(want, all);
  }
  __syncthreads();
  u64* out = a.cand + ((size_t)row * a.pieces + piece) * k;
#pragma unroll 1
  for (int i = tid; i < n_key; i += BS_NT) {
    const u64 key = sh.key[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n_key; ++j) rank += sh.key[j] > key;
    if (rank < k) out[rank] = key;
  }
  for (int i = n_key + tid; i < k; i += BS_NT) out[i] = 0;
}

// ---- a group's selection -----------------------------------------------------------------------------------

__device__ __forceinline__ u64 order64(double v) {
  const u64 u = (u64)__double_as_longlong(v + 0.);
  return u >> 63 ? ~u : u | 1ull << 63;
}
struct Best {
  u64 score, key;  // weighed score in its order, logit and id; 0: none
};
// equal scores: the lower beam, then the larger logit, then the lower id
__device__ __forceinline__ bool wins(int row, u64 key, int row2, u64 key2) { return row != row2 ? row < row2 : key > key2; }

// ln x of x >= 1, to 1e-12, 0 of 1: x = 2^e y with y in [0.70, 1.42), and ln y = 2 atanh(t) = 2 (t + t^3 / 3 + ...) with
// t = (y - 1) / (y + 1), |t| < 0.172, from an fp32 reciprocal and a Newton step. About 15 operations of 64 bits.
__device__ __forceinline__ double ln_sum(double x) {
  const long long bits = __double_as_longlong(x), digits = bits & 0xfffffffffffffll;
  int e = (int)(bits >> 52) - 1023;
  const bool high = digits > 0x6a09e667f3bccll;  // above sqrt(2)
  e += high;
  const double y = __longlong_as_double(digits | (long long)(high ? 1022 : 1023) << 52), d = y + 1.;
  double r = (double)__frcp_rn((float)d);
  r = r * (2. - d * r);
  const double t = (y - 1.) * r, q = t * t;
  double p = 1. / 13.;
  p = p * q + 1. / 11.;
  p = p * q + 1. / 9.;
  p = p * q + 1. / 7.;
  p = p * q + 1. / 5.;
  p = p * q + 1. / 3.;
  return 2. * (t + t * q * p) + (double)e * BS_LN2;
}

__global__ void __launch_bounds__(BS_NT) beam_groups_kernel(const BeamArgs a) {
  __shared__ double s_norm[BS_MAX_BEAMS], s_score[BS_MAX_BEAMS], s_weight[BS_MAX_BEAMS];  // norm: ln of the sum of exp(z - top)
  __shared__ float s_top[BS_MAX_BEAMS];
  __shared__ int s_kind[BS_MAX_BEAMS];  // 0: no candidates, 1: the row's logits, 2: ended
  __shared__ Best s_head[BS_MAX_LISTS], s_run[32][BS_MAX_OUT];
  __shared__ alignas(16) uint32_t s_high[BS_MAX_LISTS];  // upper halves of the heads' scores
  __shared__ int s_pick[BS_MAX_OUT];
  __shared__ int s_surv[32], s_row[BS_MAX_OUT], s_token[BS_MAX_OUT], s_len[BS_MAX_OUT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x, k = a.n_out, P = a.pieces;
  pdl_wait();
  // Every row's sum of exp(z - top), a few lanes a row: one for each of its pieces and one for what they leave
  const int L = P >= 16 ? 32 : P >= 8 ? 16 : P >= 4 ? 8 : P >= 2 ? 4 : 2, sub = lane & (L - 1);
#pragma unroll 1
  for (int w0 = warp * (32 / L); w0 < a.beams; w0 += BS_NW * (32 / L)) {
    const int w = w0 + lane / L, row = g * a.beams + min(w, a.beams - 1);
    const float c = a.scores[row], weight = a.weights ? a.weights[row] : 1.f;
    const bool ended = a.ended && a.ended[row];
    const PieceState* st = a.state + (size_t)row * P;
    const PieceState first = sub < P ? st[sub] : PieceState{0., 0, -INFINITY, -INFINITY};  // (nothing that is used where the row has no candidates)
    const bool bad = c != c || c == INFINITY || !(weight > 0.f && weight < INFINITY);
    const int kind = bad || c == -INFINITY ? 0 : ended ? 2 : 1;
    float top = first.top, ref = first.ref;
#pragma unroll 1
    for (int p = sub + L; p < P; p += L) {
      top = fmaxf(top, st[p].top);
      ref = fmaxf(ref, st[p].ref);
    }
#pragma unroll 1
    for (int o = L / 2; o; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    }
    u64 rest = shifted((u64)first.rest, ref - first.ref);
#pragma unroll 1
    for (int p = sub + L; p < P; p += L) rest += shifted((u64)st[p].rest, ref - st[p].ref);
#pragma unroll 1
    for (int o = L / 2; o; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
    double s = 0.;
#pragma unroll 1
    for (int p = sub; p <= P; p += L) {
      const double x = p == P ? (double)rest * BS_REST : p == sub ? first.exact : st[p].exact;
      const double of = p == P ? (double)ref * BS_LN2 : (double)(p == sub ? first.top : st[p].top);
      if (x != 0.) s += x * exp(of == (double)top ? 0. : of - (double)top);
    }
#pragma unroll 1
    for (int o = L / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (sub == 0 && w < a.beams) {
      if (bad) atomicOr(a.err, ERR_NONFINITE);
      s_kind[w] = kind;
      s_norm[w] = s;
      s_top[w] = top;
      s_score[w] = c;
      s_weight[w] = weight;
    }
  }
  if (tid < 32) s_surv[tid] = -1;
  __syncthreads();
  if (tid < a.beams && s_kind[tid] == 1) {  // one logarithm for all rows
    const double sum = s_norm[tid];
    if (sum > 0. && sum < INFINITY) {
      s_norm[tid] = ln_sum(sum);
      if (fabsf(s_top[tid]) >= BS_FAR) {  // far out the normaliser is one number of 64 bits, whose step may exceed ln of the sum
        s_norm[tid] += (double)s_top[tid];
        s_top[tid] = 0.f;
      }
    } else {  // nothing but -inf, or a NaN
      s_kind[tid] = 0;
      atomicOr(a.err, ERR_NONFINITE);
    }
  }
  __syncthreads();
  auto score_of = [&](int w, u64 key) {  // in 64 bits
    return s_kind[w] == 2 ? s_score[w] : s_score[w] + (((double)key_value((uint32_t)(key >> 32)) - (double)s_top[w]) - s_norm[w]);
  };
  auto best_of = [&](int list, int r) {
    const int w = list / P, p = list - w * P;
    Best b{0, 0};
    if (s_kind[w] == 2) {
      if (p == 0 && r == 0) b.key = 1;
    } else if (s_kind[w] == 1) {
      b.key = a.cand[((size_t)(g * a.beams + w) * P + p) * k + r];
    }
    if (b.key) b.score = order64(s_weight[w] * score_of(w, b.key));
    return b;
  };
  const int lists = a.beams * P;
  if (lists <= 32) {
    if (tid < lists) s_surv[tid] = tid;
  } else {  // the lists with the n_out best heads
    if (tid < BS_MAX_LISTS) {
      s_head[tid] = tid < lists ? best_of(tid, 0) : Best{0, 0};
      s_high[tid] = (uint32_t)(s_head[tid].score >> 32);
    }
    __syncthreads();
    static_assert(BS_MAX_LISTS <= BS_NT, "a list a thread");
    const int l = tid;
    const Best b = s_head[l];
    if (b.key) {
      const uint32_t mine = s_high[l];
      int rank = 0, same = 0;
#pragma unroll 2
      for (int j = 0; j < lists; j += 4) {  // (behind the last list are zeros)
        const uint4 h = *reinterpret_cast<const uint4*>(s_high + j);
        rank += (h.x > mine) + (h.y > mine) + (h.z > mine) + (h.w > mine);
        same += (h.x == mine) + (h.y == mine) + (h.z == mine) + (h.w == mine);
      }
      if (same > 1) {  // before it: better, or equal and of a lower beam, or of this one with a better key
        const int l0 = l / P * P;
#pragma unroll 1
        for (int j = 0; j < lists; ++j) {
          const Best o = s_head[j];
          rank += s_high[j] == mine && (o.score > b.score || (o.score == b.score && o.key && (j < l0 || (j < l0 + P && o.key > b.key))));
        }
      }
      if (rank < k) s_surv[rank] = l;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int x = tid; x < 32 * k; x += BS_NT) {
    const int i = x / k, r = x - i * k, list = s_surv[i];
    // a list behind i better heads has k - i candidates
    s_run[i][r] = list >= 0 && (lists <= 32 || i + r < k) ? best_of(list, r) : Best{0, 0};
  }
  if (tid < k) s_pick[tid] = -1;
  __syncthreads();
  if (warp == 0) {  // a list a lane, the best head taken n_out times
    const int list = s_surv[lane], w = list >= 0 ? list / P : 0;
    int at = 0;
    Best b = s_run[lane][0];
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
      const uint32_t hi = (uint32_t)(b.score >> 32), top = __reduce_max_sync(0xffffffffu, hi);
      const uint32_t lo = hi == top ? (uint32_t)b.score : 0u, top2 = __reduce_max_sync(0xffffffffu, lo);
      if (top == 0 && top2 == 0) break;
      unsigned mask = __ballot_sync(0xffffffffu, hi == top && lo == top2);
      int best = __ffs(mask) - 1;
#pragma unroll 1
      while (mask &= mask - 1) {  // equal scores
        const int other = __ffs(mask) - 1;
        if (wins(__shfl_sync(0xffffffffu, w, other), __shfl_sync(0xffffffffu, b.key, other), __shfl_sync(0xffffffffu, w, best),
                 __shfl_sync(0xffffffffu, b.key, best)))
          best = other;
      }
      if (lane == best) {
        s_pick[i] = lane * BS_MAX_OUT + at;
        b = ++at < k ? s_run[lane][at] : Best{0, 0};
      }
    }
  }
  __syncthreads();
  if (tid < k) {  // a candidate a thread
    const int pick = s_pick[tid], o = g * k + tid;
    int row = -1, token = -1;
    if (pick >= 0) {
      const int i = pick / BS_MAX_OUT, w = s_surv[i] / P;
      const u64 key = s_run[i][pick % BS_MAX_OUT].key;
      const bool old = s_kind[w] == 2;
      row = g * a.beams + w;
      token = old ? a.end_id : (int)(0xffffffffu - (uint32_t)key);
      a.scores_out[o] = (float)score_of(w, key);
      if (a.ended_out) a.ended_out[o] = old || token == a.end_id;
      s_token[tid] = old ? -1 : token;
    } else {  // fewer candidates than places
      a.scores_out[o] = -INFINITY;
      if (a.ended_out) a.ended_out[o] = 1;
    }
    a.parents[o] = row;
    a.tokens[o] = token;
    s_row[tid] = row;
  }
  if (!a.history) return;
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < k; i += BS_NT) {
    const int row = s_row[i], held = row >= 0 ? a.lens[row] : 0, len = max(0, min(held, a.width));
    s_len[i] = len;
    if (row < 0) {
      a.lens_out[g * k + i] = 0;
      continue;
    }
    const bool grows = s_token[i] >= 0, fits = len < a.width;
    if (grows && fits) a.history_out[(size_t)(g * k + i) * a.width + len] = s_token[i];
    a.lens_out[g * k + i] = len + (grows && fits);
    if (held != len || (grows && !fits)) atomicOr(a.err, ERR_CAPACITY);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = warp; i < k; i += BS_NW) {  // a history a warp, 512 tokens in flight
    const int n = s_len[i];
    const int* src = a.history + (size_t)max(s_row[i], 0) * a.width;
    int* dst = a.history_out + (size_t)(g * k + i) * a.width;
#pragma unroll 1
    for (int j0 = lane; j0 < n; j0 += 512) {
      int x[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q] = j0 + 32 * q < n ? src[j0 + 32 * q] : 0;
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (j0 + 32 * q < n) dst[j0 + 32 * q] = x[q];
    }
  }
}

// ---- host ------------------------------------------------------------------------------------------------------

// How rows are cut: enough pieces for about four CTAs an SM, none of fewer than 64 chunks, lists and chunks within the
// kernels' limits.
struct Cut {
  int pieces, chunks;
};
Cut cut_rows(int64_t rows, int beams, int vocab) {
  const int chunks = (vocab + BS_CHUNK - 1) / BS_CHUNK;
  int64_t p = (608 + rows - 1) / rows;
  p = std::min<int64_t>(p, (chunks + 63) / 64);
  p = std::max<int64_t>(std::min<int64_t>(p, BS_MAX_LISTS / beams), (chunks + BS_MAX_CHUNKS - 1) / BS_MAX_CHUNKS);
  const int per = (int)((chunks + p - 1) / p);
  return Cut{(chunks + per - 1) / per, per};
}
static_assert((BS_MAX_VOCAB / BS_CHUNK + BS_MAX_CHUNKS - 1) / BS_MAX_CHUNKS * BS_MAX_BEAMS <= BS_MAX_LISTS, "lists");

template <typename T>
cudaError_t launch_beams(const BeamArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.groups * a.beams;
  const bool wide = aligned16(a.logits) && a.row_stride * sizeof(T) % 16 == 0;
  const dim3 grid((unsigned)(rows * a.pieces));
  const cudaError_t e = wide ? launch_k(beam_rows_kernel<T, true>, grid, dim3(BS_NT), 0, s, false, a)
                             : launch_k(beam_rows_kernel<T, false>, grid, dim3(BS_NT), 0, s, false, a);
  return e ? e : launch_k(beam_groups_kernel, dim3(a.groups), dim3(BS_NT), 0, s, true, a);
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_beam_select_workspace(int32_t n_groups, int32_t n_beams, int32_t vocab, int32_t n_out) {
  if (n_groups < 0 || n_beams < 1 || n_beams > BS_MAX_BEAMS || vocab < 1 || vocab > BS_MAX_VOCAB || n_out < 1 || n_out > BS_MAX_OUT ||
      n_groups > 65535)
    return 0;
  const int64_t rows = (int64_t)std::max(n_groups, 1) * n_beams;
  return (size_t)(rows * cut_rows(rows, n_beams, vocab).pieces) * (sizeof(PieceState) + n_out * sizeof(u64));
}

qw_status qw_op_beam_select(int32_t logits_dtype, int32_t n_groups, int32_t n_beams, int32_t vocab, const void* logits,
                            int64_t row_stride, const float* scores, const float* weights, const int32_t* ended,
                            int32_t end_id, int32_t n_out, int32_t* parents, int32_t* tokens, float* scores_out,
                            int32_t* ended_out, int32_t width, const int32_t* history, const int32_t* lens,
                            int32_t* history_out, int32_t* lens_out, void* workspace, size_t workspace_bytes,
                            int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  if (!dtype_known(logits_dtype)) return op_fail(QW_ERR_INVALID_ARG, "unknown logits dtype");
  if (n_groups < 0 || n_beams < 1 || vocab < 1 || n_out < 1) return op_fail(QW_ERR_INVALID_ARG, "bad beam selection dimension");
  if (n_groups > 65535 || n_beams > BS_MAX_BEAMS || n_out > BS_MAX_OUT || vocab > BS_MAX_VOCAB)
    return op_fail(QW_ERR_UNSUPPORTED, "more than 65535 groups, 32 beams, 32 candidates or 2^21 tokens");
  if (row_stride < vocab || row_stride > (int64_t)1 << 40) return op_fail(QW_ERR_INVALID_ARG, "rows must not overlap");
  if (end_id < -1 || end_id >= vocab) return op_fail(QW_ERR_INVALID_ARG, "end_id must be a token or -1");
  if (!history != !lens || !history != !history_out || !history != !lens_out)
    return op_fail(QW_ERR_INVALID_ARG, "history, lens, history_out and lens_out: all or none");
  if (history && (width < 1 || width > 1 << 30)) return op_fail(QW_ERR_INVALID_ARG, "bad history width");
  if (history && (history_out == history || lens_out == lens))
    return op_fail(QW_ERR_INVALID_ARG, "history_out and lens_out must not be the old ones");
  if (n_groups == 0) return QW_OK;
  if (!logits || !scores || !parents || !tokens || !scores_out || !workspace || !err_dev)
    return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (scores_out == scores || (ended && ended_out == ended))
    return op_fail(QW_ERR_INVALID_ARG, "scores_out and ended_out must not be the old ones");
  if ((uintptr_t)logits % dtype_size(logits_dtype)) return op_fail(QW_ERR_INVALID_ARG, "logits misaligned");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_beam_select_workspace(n_groups, n_beams, vocab, n_out))
    return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  qw_status st = op_check_device({(const void*)((uintptr_t)logits & ~(uintptr_t)3), scores, weights, ended, parents, tokens, scores_out, ended_out,
                                  history, lens, history_out, lens_out, workspace, err_dev});
  if (st) return st;
  const int64_t rows = (int64_t)n_groups * n_beams;
  const Cut cut = cut_rows(rows, n_beams, vocab);
  PieceState* state = (PieceState*)workspace;
  const BeamArgs a{logits, row_stride, n_groups, n_beams, vocab, n_out, cut.pieces, cut.chunks, end_id, width,
                   scores, weights, ended, history, lens, parents, tokens, ended_out, history_out, lens_out, scores_out,
                   state, (u64*)(state + rows * cut.pieces), err_dev};
  const cudaError_t e = logits_dtype == QW_F32 ? launch_beams<float>(a, (cudaStream_t)cuda_stream)
                        : logits_dtype == QW_F16 ? launch_beams<f16>(a, (cudaStream_t)cuda_stream)
                                                 : launch_beams<bf16>(a, (cudaStream_t)cuda_stream);
  if (e) return op_cuda_fail(e, "beam selection launch");
  return QW_OK;
}

}  // extern "C"
