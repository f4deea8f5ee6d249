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
//     exact; a lane's sums are fp32 over at most some hundred logits, all sums of sums 64-bit. Against 64 bits
//     the normaliser is off by 1e-8 where fp32 sums of fp32 exponents give 1e-7.
//   - A second launch joins a group: pieces' sums, then the lists, of which only those with the n_out best heads count. A warp
//     holds a list a lane and takes the best head n_out times.
// What bounds it: the instructions of a logit (unpacking, two exponent products and a sum in pairs, an exponential, a maximum), at
// 57% of the issue slots, then the groups' latency. 64 x 4 beams of 152064 logits, bf16: 27 us (2.9 TB/s; rows 20, groups 7);
// 4 beams 13.5, all latency; 8 x 32 beams, 32 candidates, fp32: 65 (2.4 TB/s).
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

// The sum of a piece: of 2^(z log2(e) - ref) in units of 2^-38, which add and shift without rounding and fast (64-bit floating
// point costs 30 to 40 cycles an operation here), or, where the largest logit lies far out, of exp(z - ref), a double.
constexpr int BS_UNIT = 38;
struct PieceState {
  union {
    u64 units;
    double sum;
  };
  float ref;
  int slow;  // which of the two
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

template <typename T, bool WIDE>
__global__ void __launch_bounds__(BS_NT) beam_rows_kernel(const BeamArgs a) {
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

  float ref = 0.f;  // an integer; meaningful once `any`
  bool any = false;
  f32x2 acc[2] = {0ull, 0ull};
  uint32_t most = 0;  // of the warp's chunks
  constexpr int U = 4;  // chunks requested at a time
  const f32x2 hi2 = pack2(BS_LOG2E_HI, BS_LOG2E_HI), lo2 = pack2(BS_LOG2E_LO, BS_LOG2E_LO);
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
          mul2(acc[0], f2);
          mul2(acc[1], f2);
          ref = need;
          any = true;
        }
        const f32x2 r2 = pack2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = now[q].two(i);
          const f32x2 x2 = pack2(x.x, x.y);
          const float2 e = unpack2(fma2_to(x2, lo2, fma2_to(x2, hi2, r2)));
          acc[i & 1] = add2(acc[i & 1], pack2(ex2(e.x), ex2(e.y)));
        }
      }
    }
  }
  {
    // (a lane's sum is below 2^11: halves of 25 bits, whose sums over the lanes fit 32)
    const float2 s0 = unpack2(acc[0]), s1 = unpack2(acc[1]);
    const u64 mine = any ? (u64)__float2ull_rn(s0.x * 0x1p38f) + __float2ull_rn(s0.y * 0x1p38f) + __float2ull_rn(s1.x * 0x1p38f) + __float2ull_rn(s1.y * 0x1p38f) : 0ull;
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
  PieceState* state = a.state + (size_t)row * a.pieces + piece;
  if (peak <= value_key(-BS_NEAR) || peak >= far_high) {
    // the largest logit is far out, or there is a NaN: the definition, on a few threads' patience
    const float m = peak >= 0xff800000u ? INFINITY : key_value(max(peak, BS_NONE));  // (+inf or NaN: the sum becomes NaN)
    double s = 0.;
    if (peak > BS_NONE)
#pragma unroll 1
      for (int j = tid; j < min(left, n * BS_CHUNK); j += BS_NT) s += (double)expf(to_f32(z[j]) - m);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (lane == 0) sh.sum[warp] = s;
    __syncthreads();
    if (tid == 0) {
      double t = 0.;
#pragma unroll
      for (int w = 0; w < BS_NW; ++w) t += sh.sum[w];
      PieceState st;
      st.sum = t;
      st.ref = peak > BS_NONE ? m : -INFINITY;
      st.slow = 1;
      *state = st;
    }
  } else if (tid == 0) {
    float r = -INFINITY;
#pragma unroll
    for (int w = 0; w < BS_NW; ++w) r = fmaxf(r, sh.ref[w]);
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < BS_NW; ++w) t += shifted(sh.units[w], r - sh.ref[w]);
    PieceState st;
    st.units = t;
    st.ref = r;
    st.slow = 0;
    *state = st;
  }

  // ---- the piece's candidates
  if (warp == 0) {
    if (n <= 256) choose_chunks<8>(sh, n, k, lane);
    else choose_chunks<BS_MAX_CHUNKS / 32>(sh, n, k, lane);
  }
  __syncthreads();
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

// ln(units 2^(ref - 38)), to 1e-12: units = 2^e x with x in [0.70, 1.42), and ln x = 2 atanh(t) = 2 (t + t^3 / 3 + ...) with
// t = (x - 1) / (x + 1), |t| < 0.172, from an fp32 reciprocal and a Newton step. About 15 operations of 64 bits.
__device__ __forceinline__ double ln_units(u64 units, float ref) {
  if (units == 0) return -INFINITY;
  int e = 63 - __clzll((long long)units);
  u64 bits = units << (63 - e);  // the leading bit at the top
  if (bits > 0xb504f333f9de6484ull) ++e;  // above sqrt(2)
  const double x = (double)units * __longlong_as_double((long long)(1023 - e) << 52), y = x + 1.;
  double r = (double)__frcp_rn((float)y);
  r = r * (2. - y * r);
  const double t = (x - 1.) * r, q = t * t;
  double p = 1. / 13.;
  p = p * q + 1. / 11.;
  p = p * q + 1. / 9.;
  p = p * q + 1. / 7.;
  p = p * q + 1. / 5.;
  p = p * q + 1. / 3.;
  return 2. * (t + t * q * p) + ((double)ref + (double)(e - BS_UNIT)) * BS_LN2;
}

// ln of a row's sum of exponentials, with pieces that were summed from the definition; NaN if there is one. A warp.
__device__ __noinline__ double far_norm(const PieceState* st, int n, int lane) {
  double m = -INFINITY, s = 0.;
  bool nan = false;
#pragma unroll 1
  for (int p = lane; p < n; p += 32) {
    if (st[p].ref == -INFINITY) continue;  // nothing but -inf
    const double x = st[p].slow ? (double)st[p].ref + log(st[p].sum) : (double)st[p].ref * BS_LN2 + log((double)st[p].units * 0x1p-38);
    if (x != x) {
      nan = true;
      continue;
    }
    const double hi = fmax(m, x);
    s = s * exp(m - hi) + exp(x - hi);
    m = hi;
  }
#pragma unroll 1
  for (int o = 16; o; o >>= 1) {
    const double m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const double hi = fmax(m, m2);
    s = (m > -INFINITY ? s * exp(m - hi) : 0.) + (m2 > -INFINITY ? s2 * exp(m2 - hi) : 0.);
    m = hi;
  }
  return __any_sync(0xffffffffu, nan) ? (double)NAN : m + log(s);
}

__global__ void __launch_bounds__(BS_NT) beam_groups_kernel(const BeamArgs a) {
  __shared__ double s_norm[BS_MAX_BEAMS], s_score[BS_MAX_BEAMS], s_weight[BS_MAX_BEAMS];
  __shared__ float s_ref[BS_MAX_BEAMS];
  __shared__ u64 s_units[BS_MAX_BEAMS];
  __shared__ int s_kind[BS_MAX_BEAMS];  // 0: no candidates, 1: the row's logits, 2: ended
  __shared__ Best s_head[BS_MAX_LISTS], s_run[32][BS_MAX_OUT];
  __shared__ alignas(16) uint32_t s_high[BS_MAX_LISTS];  // upper halves of the heads' scores
  __shared__ int s_pick[BS_MAX_OUT];
  __shared__ int s_surv[32], s_row[BS_MAX_OUT], s_token[BS_MAX_OUT], s_len[BS_MAX_OUT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x, k = a.n_out, P = a.pieces;
  pdl_wait();
#pragma unroll 1
  for (int w = warp; w < a.beams; w += BS_NW) {
    const int row = g * a.beams + w;
    const float c = a.scores[row], weight = a.weights ? a.weights[row] : 1.f;
    const bool ended = a.ended && a.ended[row];
    const bool bad = c != c || c == INFINITY || !(weight > 0.f && weight < INFINITY);
    const int kind = bad || c == -INFINITY ? 0 : ended ? 2 : 1;
    double far_s = 0.;
    u64 s = 0;
    float ref = NAN;  // NaN: far_s is the normaliser already
    if (kind == 1) {
      const PieceState* st = a.state + (size_t)row * P;
      bool far = false;
      ref = -INFINITY;
#pragma unroll 1
      for (int p = lane; p < P; p += 32) {
        far |= st[p].slow;
        ref = fmaxf(ref, st[p].ref);
      }
      if (__any_sync(0xffffffffu, far)) {
        far_s = far_norm(st, P, lane);
        ref = NAN;
      } else {
        ref = warp_max(ref);
#pragma unroll 1
        for (int p = lane; p < P; p += 32) s += shifted(st[p].units, ref - st[p].ref);
#pragma unroll 1
        for (int o = P > 16 ? 16 : P > 8 ? 8 : P > 4 ? 4 : P > 2 ? 2 : P > 1 ? 1 : 0; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      }
    }
    if (lane == 0) {
      if (bad) atomicOr(a.err, ERR_NONFINITE);
      s_kind[w] = kind;
      s_norm[w] = far_s;
      s_units[w] = s;
      s_ref[w] = ref;
      s_score[w] = c;
      s_weight[w] = weight;
    }
  }
  if (tid < 32) s_surv[tid] = -1;
  __syncthreads();
  if (tid < a.beams && s_kind[tid] == 1) {  // one logarithm for all rows
    const float ref = s_ref[tid];
    const double norm = ref == ref ? ln_units(s_units[tid], ref) : s_norm[tid];
    s_norm[tid] = norm;
    if (!(fabs(norm) < INFINITY)) {
      s_kind[tid] = 0;
      atomicOr(a.err, ERR_NONFINITE);
    }
  }
  __syncthreads();
  auto score_of = [&](int w, u64 key) {  // in 64 bits
    return s_kind[w] == 2 ? s_score[w] : s_score[w] + ((double)key_value((uint32_t)(key >> 32)) - s_norm[w]);
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
