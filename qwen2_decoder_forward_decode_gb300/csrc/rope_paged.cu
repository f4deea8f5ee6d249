// Rotary positions of queries and keys, fused with the append of keys and values to a paged cache
// ("LLM Speedrun: Architecture": RoPE, Split-half RoPE implementation, KV cache).
//
// Pair i of a head turns by positions[t] * w_i. The frequency comes as a fraction of a turn in units of
// 2^-64, so the angle modulo a turn is the low 64 bits of an integer product: exact at every position,
// where an fp32 angle is off by 2^-24 p radians. The two top bits (after adding an eighth of a turn)
// give the quadrant, the rest an angle of at most pi/4 in fp32 for sincospif.
#include "common.cuh"
#include "op_util.h"

#include <cmath>

namespace qw {
namespace {

struct RopeArgs {
  int n_tokens, nq, nkv, hd, rot, adjacent, page, n_pages;
  float mscale;
  long long page_stride, head_stride, pos_stride;
  const int* positions;
  const long long* slots;
  const unsigned long long* turns;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride, qo_stride;
  void *q_out, *kc, *vc;
  int* err;
};

__device__ __forceinline__ void turn_sincos(unsigned long long turns, int pos, float& c, float& s) {
  const unsigned long long u = turns * (unsigned long long)(long long)pos + (1ull << 61);
  const long long r = (long long)(u & ((1ull << 62) - 1)) - (1ll << 61);  // [-1/8, 1/8) turn
  const int quadrant = (int)(u >> 62);
  float s0, c0;
  sincospif((float)r * 0x1p-63f, &s0, &c0);
  s = quadrant & 1 ? c0 : s0;
  c = quadrant & 1 ? s0 : c0;
  if (quadrant == 1 || quadrant == 2) c = -c;
  if (quadrant >= 2) s = -s;
}

// W elements as they lie in memory
template <typename T, int W>
struct alignas(W * sizeof(T) >= 16 ? 16 : W * sizeof(T)) Raw {
  T x[W];
};

// fp16 values that overflow, or are not finite, set bad
__device__ __forceinline__ float cast_io(float v, bool&, float) { return v; }
__device__ __forceinline__ bf16 cast_io(float v, bool&, bf16) { return __float2bfloat16_rn(v); }
__device__ __forceinline__ f16 cast_io(float v, bool& bad, f16) {
  bad |= !(fabsf(v) < 65520.f);
  return __float2half_rn(v);
}
template <int W, typename T>
__device__ __forceinline__ void store_w(T* p, const float* x, bool& bad) {
  Raw<T, W> y;
#pragma unroll
  for (int i = 0; i < W; ++i) y.x[i] = cast_io(x[i], bad, T());
  *reinterpret_cast<Raw<T, W>*>(p) = y;
}

// A CTA takes every gridDim-th token. An item is W elements of a head, with their partners rot / 2 further where the
// pairs are halves; a thread has the same items of every token, so their places are worked out once. It copies
// them itself (cp.async) into its places of a ring, ROPE_STAGES - 1 tokens ahead, and reads them back itself. The
// rot / 2 (cos, sin) pairs, which all heads share, are computed a token ahead.
// What bounds it: every element is read and written once, HBM for long prefills and latency for decode steps.
// In a CUDA graph (a lone call costs the host about 3 us from C, 10 to 14 from Python) 16 tokens take 2.7 us, 8191 tokens of 36
// bf16 heads of 128, half of each rotated in adjacent pairs, 25.5 us, 5.9 TB/s. The 16-bit instances of pairs in halves hold two
// vectors an item and spill (144 bytes a thread, fp16 128): the same tokens take 37.7 us, rotated as a whole 36.0 (adjacent
// 29.1); fp32 to fp16, without spills, 50.3 and 52.4 us for 42.1 us of traffic. A CTA a token, with the same angles and vectors, took
// 46 us (the chain position - angle - barrier - store, 4 us, is not hidden); tokens ahead in registers
// instead of the ring 35 us (spills); three stages with three CTAs an SM 26.5 us.
constexpr int ROPE_THREADS = 256, ROPE_ITEMS = 3, ROPE_STAGES = 2, ROPE_CTAS_PER_SM = 4;

template <typename IO, typename KV, int W, bool ADJACENT>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_CTAS_PER_SM) rope_append_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) unsigned char rope_ring[];  // [stage][item][half][thread] of 16 bytes
  __shared__ float2 s_cs[2][128];
  __shared__ long long s_row[2];  // the token's row in the caches, -1: none
  const int tid = threadIdx.x;
  const int rotated = ADJACENT ? a.rot / W : a.rot / 2 / W, per_head = rotated + (a.hd - a.rot) / W;
  const int qk = (a.nq + a.nkv) * per_head, items = qk + a.nkv * (a.hd / W);
  bool bad = false;

  struct Item {
    const IO* src;       // token 0's
    long long stride;    // from token to token
    void* dst;           // q_out's token 0, or the caches' row 0
    int d;               // dimension; -1: not rotated, -2: no item
    bool is_q;
  };
  auto item = [&](int it) {
    Item m{nullptr, 0, nullptr, -2, false};
    if (it < qk) {
      const int h = it / per_head, i = it - h * per_head, d = i < rotated ? i * W : a.rot + (i - rotated) * W;
      m.d = i < rotated ? d : -1;
      m.is_q = h < a.nq;
      if (m.is_q) {
        m.src = (const IO*)a.q + h * a.hd + d;
        m.stride = a.q_stride;
        m.dst = (IO*)a.q_out + h * a.hd + d;
      } else {
        m.src = (const IO*)a.k + (h - a.nq) * a.hd + d;
        m.stride = a.k_stride;
        m.dst = (KV*)a.kc + (h - a.nq) * a.head_stride + d;
      }
    } else if (it < items) {
      const int e = (it - qk) * W, h = e / a.hd;
      m.src = (const IO*)a.v + e;
      m.stride = a.v_stride;
      m.dst = (KV*)a.vc + h * a.head_stride + (e - h * a.hd);
      m.d = -1;
    }
    return m;
  };
  typedef Raw<IO, W> R;
  auto place = [&](int stage, int k, int half) {
    return reinterpret_cast<R*>(rope_ring + (((stage * ROPE_ITEMS + k) * 2 + half) * ROPE_THREADS + tid) * 16);
  };
  auto copy = [&](R* to, const IO* from) {
    if constexpr (sizeof(R) == 2) *to = *reinterpret_cast<const R*>(from);
    else if constexpr (sizeof(R) == 16) cp_async16(to, from);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from), "n"(sizeof(R)) : "memory");
  };
  auto write = [&](const Item& m, int t, const R* r, const float2* cs, long long row) {
    if (m.d == -2 || (!m.is_q && row < 0)) return;
    float x[2][W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      x[0][e] = to_f32(r[0].x[e]);
      if (!ADJACENT) x[1][e] = to_f32(r[1].x[e]);
    }
    if (m.d >= 0) {
      if constexpr (ADJACENT) {
#pragma unroll
        for (int e = 0; e + 1 < W; e += 2) {
          const float2 c = cs[(m.d + e) / 2];
          const float u = x[0][e], v = x[0][e + 1];
          x[0][e] = u * c.x - v * c.y;
          x[0][e + 1] = u * c.y + v * c.x;
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 c = cs[m.d + e];
          const float u = x[0][e], v = x[1][e];
          x[0][e] = u * c.x - v * c.y;
          x[1][e] = u * c.y + v * c.x;
        }
      }
    }
    if (m.is_q) {
      IO* dst = (IO*)m.dst + t * a.qo_stride;
      store_w<W>(dst, x[0], bad);
      if (!ADJACENT && m.d >= 0) store_w<W>(dst + a.rot / 2, x[1], bad);
    } else {
      KV* dst = (KV*)m.dst + row;
      store_w<W>(dst, x[0], bad);
      if (!ADJACENT && m.d >= 0) store_w<W>(dst + a.rot / 2, x[1], bad);
    }
  };
  // positions and slots are read a token before they are used
  const bool turns = tid < a.rot / 2, slots = tid == ROPE_THREADS - 1;
  const unsigned long long my_turns = turns ? a.turns[tid] : 0;
  int pos = 0;
  long long slot = -1;
  auto look = [&](int t) {
    if (turns && t < a.n_tokens) pos = a.positions[t];
    if (slots && t < a.n_tokens) slot = a.slots[t];
  };
  auto angles = [&](int side) {  // the pairs and the cache row of the token looked at last
    if (turns) {
      float c, s;
      turn_sincos(my_turns, pos, c, s);
      s_cs[side][tid] = make_float2(c * a.mscale, s * a.mscale);
    }
    if (slots) {
      long long row = -1;
      if (slot >= 0 && slot < (long long)a.n_pages * a.page) {
        const long long page = slot >> 32 ? slot / a.page : (long long)((uint32_t)slot / (uint32_t)a.page);
        row = page * a.page_stride + (slot - page * a.page) * a.pos_stride;
      } else if (slot != -1) {
        atomicOr(a.err, ERR_PAGE);
      }
      s_row[side] = row;
    }
  };

  Item mine[ROPE_ITEMS];
#pragma unroll
  for (int k = 0; k < ROPE_ITEMS; ++k) mine[k] = item(tid + k * ROPE_THREADS);
  int ahead = blockIdx.x, ld_stage = 0, stage = 0, side = 0;
  auto load_next = [&]() {
    if (ahead < a.n_tokens) {
#pragma unroll
      for (int k = 0; k < ROPE_ITEMS; ++k) {
        if (mine[k].d == -2) continue;
        const IO* src = mine[k].src + ahead * mine[k].stride;
        copy(place(ld_stage, k, 0), src);
        if (!ADJACENT && mine[k].d >= 0) copy(place(ld_stage, k, 1), src + a.rot / 2);
      }
      ahead += gridDim.x;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++ld_stage == ROPE_STAGES) ld_stage = 0;
  };
  look(blockIdx.x);
#pragma unroll 1
  for (int i = 0; i < ROPE_STAGES - 1; ++i) load_next();
  angles(0);
  look(blockIdx.x + gridDim.x);
  __syncthreads();
#pragma unroll 1
  for (int t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
    load_next();
    asm volatile("cp.async.wait_group %0;" ::"n"(ROPE_STAGES - 1) : "memory");
    const long long row = s_row[side];
#pragma unroll
    for (int k = 0; k < ROPE_ITEMS; ++k) {
      R r[2];
      r[0] = *place(stage, k, 0);
      if (!ADJACENT) r[1] = *place(stage, k, 1);
      write(mine[k], t, r, s_cs[side], row);
    }
#pragma unroll 1
    for (int it = tid + ROPE_ITEMS * ROPE_THREADS; it < items; it += ROPE_THREADS) {  // of very many heads
      const Item m = item(it);
      if (!m.is_q && row < 0) continue;
      R r[2];
      const IO* src = m.src + t * m.stride;
      r[0] = *reinterpret_cast<const R*>(src);
      if (!ADJACENT && m.d >= 0) r[1] = *reinterpret_cast<const R*>(src + a.rot / 2);
      write(m, t, r, s_cs[side], row);
    }
    if (++stage == ROPE_STAGES) stage = 0;
    side ^= 1;
    angles(side);
    look(t + 2 * gridDim.x);
    __syncthreads();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (bad) atomicOr(a.err, ERR_RANGE);
}

template <typename IO, typename KV, int W>
cudaError_t launch_rope_w(const RopeArgs& a, cudaStream_t s) {
  int dev = 0, nsm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev))) return e;
  const dim3 grid(a.n_tokens < nsm * ROPE_CTAS_PER_SM ? a.n_tokens : nsm * ROPE_CTAS_PER_SM);
  constexpr int ring = ROPE_STAGES * ROPE_ITEMS * 2 * ROPE_THREADS * 16;
  auto kernel = a.adjacent ? rope_append_kernel<IO, KV, W, true> : rope_append_kernel<IO, KV, W, false>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring))) return e;
  return launch_k(kernel, grid, dim3(ROPE_THREADS), ring, s, false, a);
}
// W: 16 bytes of io where the rotated halves (or pairs) and the rest divide into such vectors, half of that (16-bit
// types) or single pairs else.
template <typename IO, typename KV>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const int unit = a.adjacent ? a.rot : a.rot / 2;
  auto fits = [&](int w) { return unit % w == 0 && (a.hd - a.rot) % w == 0; };
  if constexpr (sizeof(IO) == 2)
    if (fits(8)) return launch_rope_w<IO, KV, 8>(a, s);
  if (fits(4)) return launch_rope_w<IO, KV, 4>(a, s);
  return a.adjacent ? launch_rope_w<IO, KV, 2>(a, s) : launch_rope_w<IO, KV, 1>(a, s);
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

qw_status qw_rope_turns(int32_t rot_dim, double theta, int32_t scaling, double factor, double orig_len, double low,
                        double high, uint64_t* turns, float* mscale) {
  set_error_message("");
  if (!turns || !mscale) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (rot_dim < 2 || rot_dim % 2) return op_fail(QW_ERR_INVALID_ARG, "rot_dim must be even and positive");
  if (scaling < QW_ROPE_NONE || scaling > QW_ROPE_BANDS) return op_fail(QW_ERR_INVALID_ARG, "unknown rope scaling");
  if (!(theta > 1.0) || !std::isfinite(theta)) return op_fail(QW_ERR_INVALID_ARG, "theta must be above 1");
  if (scaling != QW_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return op_fail(QW_ERR_INVALID_ARG, "rope factor must be at least 1");
  const bool bands = scaling == QW_ROPE_YARN || scaling == QW_ROPE_BANDS;
  if (bands && (!(orig_len > 0) || !std::isfinite(orig_len) || !(low > 0) || !(high > low) || !std::isfinite(high)))
    return op_fail(QW_ERR_INVALID_ARG, "rope scaling needs orig_len > 0 and 0 < low < high");
  const double turn = 6.283185307179586476925286766559;
  const int r = rot_dim;
  if (scaling == QW_ROPE_NTK && r > 2) theta *= std::pow(factor, (double)r / (r - 2));
  double first = 0, last = 1;
  if (scaling == QW_ROPE_YARN) {
    // theta^(-2i/r) orig_len / 2 pi = n turns at i = r ln(orig_len / (2 pi n)) / (2 ln theta)
    const double k = r / (2.0 * std::log(theta));
    first = std::fmax(std::floor(k * std::log(orig_len / (turn * high))), 0.0);
    last = std::fmin(std::ceil(k * std::log(orig_len / (turn * low))), (double)(r - 1));
  }
  for (int i = 0; i < r / 2; ++i) {
    double w = std::pow(theta, -2.0 * i / r);
    if (scaling == QW_ROPE_LINEAR) {
      w /= factor;
    } else if (scaling == QW_ROPE_YARN) {
      const double c = std::fmin(std::fmax((i - first) / std::fmax(last - first, 1e-3), 0.0), 1.0);
      w = (1.0 - c) * w + c * (w / factor);
    } else if (scaling == QW_ROPE_BANDS) {
      const double c = std::fmin(std::fmax((orig_len * w / turn - low) / (high - low), 0.0), 1.0);
      w = c * w + (1.0 - c) * (w / factor);
    }
    // w <= 1, so the fraction is below 0.16 of a turn and the product below 2^62
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(w / turn, 64));
  }
  *mscale = scaling == QW_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return QW_OK;
}

qw_status qw_op_rope_append(const qw_paged_kv* cache, int32_t n_tokens, int32_t n_heads, int32_t io_dtype,
                            const int32_t* positions, const int64_t* slots, const uint64_t* turns, int32_t rot_dim,
                            int32_t adjacent, float mscale, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride,
                            int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  qw_paged_kv c;
  qw_status st = op_check_cache(cache, &c);
  if (st) return st;
  if ((st = op_check_io(io_dtype, c.dtype))) return st;
  if (n_tokens < 0 || n_heads < 1) return op_fail(QW_ERR_INVALID_ARG, "bad token or head count");
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > c.head_dim)
    return op_fail(QW_ERR_INVALID_ARG, "rot_dim must be even, between 2 and head_dim");
  if (adjacent != 0 && adjacent != 1) return op_fail(QW_ERR_INVALID_ARG, "adjacent must be 0 or 1");
  if (!std::isfinite(mscale)) return op_fail(QW_ERR_INVALID_ARG, "mscale not finite");
  if (n_heads > 4096 || c.n_kv_heads > 4096) return op_fail(QW_ERR_UNSUPPORTED, "more than 4096 heads");
  if (n_tokens > 1 << 30) return op_fail(QW_ERR_UNSUPPORTED, "more than 2^30 tokens");
  if (n_tokens == 0) return QW_OK;
  if (!positions || !slots || !turns || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (((uintptr_t)slots | (uintptr_t)turns) & 7) return op_fail(QW_ERR_INVALID_ARG, "slots or turns not 8-byte aligned");
  const int64_t wq = (int64_t)n_heads * c.head_dim, wk = (int64_t)c.n_kv_heads * c.head_dim;
  if ((st = op_check_rows(q, q_stride, wq, io_dtype, "q"))) return st;
  if ((st = op_check_rows(k, k_stride, wk, io_dtype, "k"))) return st;
  if ((st = op_check_rows(v, v_stride, wk, io_dtype, "v"))) return st;
  if ((st = op_check_rows(q_out, q_out_stride, wq, io_dtype, "q_out"))) return st;
  if (q_out == q && q_out_stride != q_stride) return op_fail(QW_ERR_INVALID_ARG, "q_out may be q with the same stride only");
  if ((st = op_check_device({c.k, c.v, positions, slots, turns, q, k, v, q_out, err_dev}))) return st;
  RopeArgs a{n_tokens, n_heads, c.n_kv_heads, c.head_dim, rot_dim, adjacent, c.page_size, c.n_pages, mscale,
             c.page_stride, c.head_stride, c.pos_stride, positions, (const long long*)slots,
             (const unsigned long long*)turns, q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_out, c.k, c.v,
             err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  cudaError_t e;
  if (io_dtype == QW_F32)
    e = c.dtype == QW_F32 ? launch_rope<float, float>(a, s)
        : c.dtype == QW_F16 ? launch_rope<float, f16>(a, s) : launch_rope<float, bf16>(a, s);
  else
    e = io_dtype == QW_F16 ? launch_rope<f16, f16>(a, s) : launch_rope<bf16, bf16>(a, s);
  if (e) return op_cuda_fail(e, "rope append launch");
  return QW_OK;
}

}  // extern "C"
