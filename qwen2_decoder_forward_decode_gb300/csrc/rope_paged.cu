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

template <typename T> __device__ __forceinline__ T store_io(float v, int* err);
template <> __device__ __forceinline__ float store_io<float>(float v, int*) { return v; }
template <> __device__ __forceinline__ bf16 store_io<bf16>(float v, int*) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ f16 store_io<f16>(float v, int* err) { return to_half_checked(v, err); }

// One thread per (token, pair or value): heads q, then k, then v.
template <typename IO, typename KV>
__global__ void rope_append_kernel(const RopeArgs a) {
  const int half = a.rot / 2;
  const int per_head = half + (a.hd - a.rot);  // rotated pairs, then single dimensions
  const int items = (a.nq + a.nkv) * per_head + a.nkv * a.hd;
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int t = (int)(idx / items);
  if (t >= a.n_tokens) return;
  const int it = (int)(idx - (long long)t * items);
  const long long slot = a.slots[t];
  const bool open = slot >= 0 && slot < (long long)a.n_pages * a.page;
  if (!open && slot != -1 && it == 0) atomicOr(a.err, ERR_PAGE);
  const long long page = open ? slot / a.page : 0;
  const long long row = page * a.page_stride + (open ? slot - page * a.page : 0) * a.pos_stride;
  if (it >= (a.nq + a.nkv) * per_head) {  // a value
    if (!open) return;
    const int e = it - (a.nq + a.nkv) * per_head, h = e / a.hd;
    const float x = to_f32(((const IO*)a.v)[t * a.v_stride + e]);
    ((KV*)a.vc)[row + h * a.head_stride + (e - h * a.hd)] = store_io<KV>(x, a.err);
    return;
  }
  const int h = it / per_head, i = it - h * per_head;
  const bool is_q = h < a.nq;
  if (!is_q && !open) return;
  const IO* src = is_q ? (const IO*)a.q + t * a.q_stride + h * a.hd : (const IO*)a.k + t * a.k_stride + (h - a.nq) * a.hd;
  int d0, d1 = -1;
  float y0, y1 = 0.f;
  if (i < half) {
    d0 = a.adjacent ? 2 * i : i;
    d1 = a.adjacent ? 2 * i + 1 : i + half;
    float c, s;
    turn_sincos(a.turns[i], a.positions[t], c, s);
    c *= a.mscale;
    s *= a.mscale;
    const float x0 = to_f32(src[d0]), x1 = to_f32(src[d1]);
    y0 = x0 * c - x1 * s;
    y1 = x0 * s + x1 * c;
  } else {
    d0 = a.rot + (i - half);
    y0 = to_f32(src[d0]);
  }
  if (is_q) {
    IO* dst = (IO*)a.q_out + t * a.qo_stride + h * a.hd;
    dst[d0] = store_io<IO>(y0, a.err);
    if (d1 >= 0) dst[d1] = store_io<IO>(y1, a.err);
  } else {
    KV* dst = (KV*)a.kc + row + (h - a.nq) * a.head_stride;
    dst[d0] = store_io<KV>(y0, a.err);
    if (d1 >= 0) dst[d1] = store_io<KV>(y1, a.err);
  }
}

template <typename IO, typename KV>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const long long items = (long long)(a.nq + a.nkv) * (a.rot / 2 + a.hd - a.rot) + (long long)a.nkv * a.hd;
  const long long blocks = (a.n_tokens * items + 255) / 256;
  return launch_k(rope_append_kernel<IO, KV>, dim3((unsigned)blocks), dim3(256), 0, s, false, a);
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
