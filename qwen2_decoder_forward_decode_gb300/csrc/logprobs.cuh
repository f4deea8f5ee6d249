// What both kernels of the token log probabilities share: arguments, the order of logits, 16 bytes of logits in
// registers.
#pragma once

#include "common.cuh"

#include <type_traits>

namespace qw {

constexpr int LP_MAX_IDS = 8, LP_MAX_TOP = 32;
constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
typedef unsigned long long u64;

struct LogprobPart;
struct LogprobArgs {
  const void* logits;
  long long row_stride;
  int n_rows, vocab, n_ids, top_k, batches;  // batches of a row
  int pieces;  // > 0: rows are cut into so many pieces of their own and CTAs take whole pieces; 0: see Cuts
  const int* ids;
  float* logprobs;
  int* ranks;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  unsigned int* counters;  // of the workspace, zero between calls
  LogprobPart* parts;
  int* err;
};

// logprobs_rows.cu: short rows, a warp each
cudaError_t launch_logprobs_rows(int dtype, const LogprobArgs& a, int nsm, cudaStream_t s);

namespace {

// (logit, lower id first) as an integer; -0 counts as 0
__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ u64 order_key(float z, int j) { return (u64)order_bits(z) << 32 | (0xffffffffu - (uint32_t)j); }
__device__ __forceinline__ float key_value(u64 k) { return order_value((uint32_t)(k >> 32)); }

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr u64 LP_NO_BAR = 0x007fffffffffffffull;  // the key of (-inf, id 0): every finite logit's is above

// ---- 16 bytes of logits ------------------------------------------------------------------------------------
//
// pair(u): the logits of word u (two for 16-bit types) as packed fp32, with -inf raised to a finite value whose
// exponential is 0 (so that d * exp(d) is 0 as well); a NaN stays.
// Rows whose maximum lies so low that the floor would count, or so high that products with log2(e) overflow (masks
// of the type's lowest value that leave nothing), are summed again, slowly.
constexpr float LP_FLOOR = -1e28f;  // (times log2(e), and that times 2^31 logits, is finite)
template <typename T>
__device__ __forceinline__ bool extreme(float most) {
  return !(most < 5e27f && most > (std::is_same<T, f16>::value ? -65000.f : -5e27f));
}
template <typename T> struct Logits;
template <> struct Logits<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint32_t minus_inf() { return 0xff800000u; }
  static __device__ __forceinline__ float floor() { return LP_FLOOR; }
  // maximum of the vectors that were added
  struct Top {
    float m = -INFINITY;
    __device__ __forceinline__ void add(const uint4& r) {
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w))));
    }
    __device__ __forceinline__ float value() const { return m; }
  };
  static __device__ __forceinline__ void pairs(const uint4& r, f32x2* p) {
    p[0] = pack2(max_nan(__uint_as_float(r.x), LP_FLOOR), max_nan(__uint_as_float(r.y), LP_FLOOR));
    p[1] = pack2(max_nan(__uint_as_float(r.z), LP_FLOOR), max_nan(__uint_as_float(r.w), LP_FLOOR));
  }
  // counts of logits at or above a threshold, a vector at a time
  struct Count {
    int n = 0;
    __device__ __forceinline__ void add(const uint4& r, float thr) {
      n += (__uint_as_float(r.x) >= thr) + (__uint_as_float(r.y) >= thr) + (__uint_as_float(r.z) >= thr) + (__uint_as_float(r.w) >= thr);
    }
    __device__ __forceinline__ int total() const { return n; }
  };
  typedef float Thr;
  static __device__ __forceinline__ Thr thr(float z) { return z; }
  static __device__ __forceinline__ Thr thr_above(float z) {  // the next larger value
    const uint32_t bits = order_bits(z);
    return order_value(bits == 0x80000000u ? 0x80000001u : bits + 1);
  }
};
template <typename T2>
__device__ __forceinline__ T2 as_pair(uint32_t u) { return *reinterpret_cast<const T2*>(&u); }
// the next larger value of a 16-bit float's bits (0 and -0: the smallest positive one)
__device__ __forceinline__ uint32_t next16(uint32_t b) { return (b & 0x7fff) == 0 ? 1u : b & 0x8000 ? b - 1 : b + 1; }
template <typename T, typename T2>
struct Logits16 {
  static constexpr int N = 8;
  struct Top {
    T2 m = as_pair<T2>(std::is_same<T, bf16>::value ? 0xff80ff80u : 0xfc00fc00u);  // -inf
    __device__ __forceinline__ void add(const uint4& r) {
      m = __hmax2(m, __hmax2(__hmax2(as_pair<T2>(r.x), as_pair<T2>(r.y)), __hmax2(as_pair<T2>(r.z), as_pair<T2>(r.w))));
    }
    __device__ __forceinline__ float value() const { return fmaxf(__low2float(m), __high2float(m)); }
  };
  // Counts of both halves in one sum of masks: a true half adds 0xffff, so the sum of lo low and hi high ones is
  // (lo - hi) 2^16 - lo.
  struct Count {
    uint32_t n = 0;
    __device__ __forceinline__ void add(const uint4& r, T2 thr) {
      n += __hge2_mask(as_pair<T2>(r.x), thr) + __hge2_mask(as_pair<T2>(r.y), thr);
      n += __hge2_mask(as_pair<T2>(r.z), thr) + __hge2_mask(as_pair<T2>(r.w), thr);
    }
    __device__ __forceinline__ int total() const {
      const uint32_t lo = -n & 0xffffu;
      return (int)(2 * lo) - (int16_t)((n + lo) >> 16);
    }
  };
  typedef T2 Thr;
  static __device__ __forceinline__ uint32_t bits(float z) {
    const T h = from_f32<T>(z);
    return *reinterpret_cast<const uint16_t*>(&h);
  }
  static __device__ __forceinline__ T2 thr(float z) { return as_pair<T2>(bits(z) * 0x10001u); }
  static __device__ __forceinline__ T2 thr_above(float z) { return as_pair<T2>(next16(bits(z)) * 0x10001u); }
};
template <> struct Logits<bf16> : Logits16<bf16, __nv_bfloat162> {
  static __device__ __forceinline__ uint32_t minus_inf() { return 0xff80ff80u; }
  static __device__ __forceinline__ float floor() { return to_f32(__float2bfloat16_rn(LP_FLOOR)); }
  static __device__ __forceinline__ f32x2 pair(uint32_t u) {
    const __nv_bfloat162 h = __hmax2_nan(as_pair<__nv_bfloat162>(u), __float2bfloat162_rn(floor()));
    const uint32_t v = *reinterpret_cast<const uint32_t*>(&h);
    return pack2(bf_lo(v), bf_hi(v));
  }
  static __device__ __forceinline__ void pairs(const uint4& r, f32x2* p) {
    p[0] = pair(r.x); p[1] = pair(r.y); p[2] = pair(r.z); p[3] = pair(r.w);
  }
};
template <> struct Logits<f16> : Logits16<f16, __half2> {
  static __device__ __forceinline__ uint32_t minus_inf() { return 0xfc00fc00u; }
  static __device__ __forceinline__ float floor() { return -65504.f; }
  static __device__ __forceinline__ f32x2 pair(uint32_t u) {
    const float2 t = __half22float2(__hmax2_nan(as_pair<__half2>(u), __float2half2_rn(floor())));
    return pack2(t.x, t.y);
  }
  static __device__ __forceinline__ void pairs(const uint4& r, f32x2* p) {
    p[0] = pair(r.x); p[1] = pair(r.y); p[2] = pair(r.z); p[3] = pair(r.w);
  }
};

// the logits of a vector
__device__ __forceinline__ void unpack(const uint4& r, float* x, float) {
  x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float* x, bf16) {
  x[0] = bf_lo(r.x); x[1] = bf_hi(r.x); x[2] = bf_lo(r.y); x[3] = bf_hi(r.y);
  x[4] = bf_lo(r.z); x[5] = bf_hi(r.z); x[6] = bf_lo(r.w); x[7] = bf_hi(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float* x, f16) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(as_pair<__half2>(u[i]));
    x[2 * i] = t.x;
    x[2 * i + 1] = t.y;
  }
}

// The largest 15-bit key that top_k of a warp's keys reach. keys: the lane's, in pairs (their upper bits are set here);
// most: the largest of them. top_k <= 32. The whole warp.
template <int W>
__device__ __forceinline__ uint32_t keys_bound(uint32_t* keys, uint32_t most, int top_k) {
  // top_k <= 32 lanes reach the least of the lanes' maxima: what it has in common with the largest is the bound's
  const uint32_t lo = __reduce_min_sync(0xffffffffu, most), hi = __reduce_max_sync(0xffffffffu, most);
  uint32_t bit = lo == hi ? 0u : 0x80000000u >> __clz(lo ^ hi), bound = bit ? hi & ~(2u * bit - 1u) : hi;
#pragma unroll
  for (int i = 0; i < W; ++i) keys[i] |= 0x80008000u;
#pragma unroll 1
  for (; bit; bit >>= 1) {
    // a half's top bit outlasts the subtraction if the half reaches the candidate
    const uint32_t v = (bound | bit) * 0x10001u;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) n += (keys[i] - v) >> 15 & 0x10001u;
    if ((int)__reduce_add_sync(0xffffffffu, (n & 0xffffu) + (n >> 16)) >= top_k) bound |= bit;
  }
  return bound;
}

}  // namespace
}  // namespace qw
