// Decode attention over a paged key-value cache: one query token per sequence ("LLM Speedrun:
// Architecture": Attention, Grouped Query Attention).
//
// One pass over the positions with a running maximum m, sum l and output o per query head: a new score
// s moves them to m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') V.
#include "common.cuh"
#include "op_util.h"

#include <math.h>

#include <cmath>

namespace qw {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_MAX_HD = 256;

struct PagedAttnArgs {
  const void *k, *v;
  long long page_stride, head_stride, pos_stride;
  int n_seqs, nq, nkv, hd, page, n_pages, max_blocks;
  const int *table, *lens;
  const void* q;
  void* out;
  long long q_stride, out_stride;
  float scale;
  float* lse;
  int* err;
};

// One CTA per (KV head, sequence); warp w takes the group's query heads w, w + 4, ...
template <typename IO, typename KV>
__global__ void __launch_bounds__(PA_WARPS * 32) paged_attn_kernel(const PagedAttnArgs a) {
  const int g = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = a.nq / a.nkv;
  const long long room = (long long)a.max_blocks * a.page;
  int len = a.lens[b];
  if (len < 0 || len > room) {
    if (threadIdx.x == 0) atomicOr(a.err, ERR_PAGE);
    len = len < 0 ? 0 : (int)room;
  }
  constexpr int E = PA_MAX_HD / 32;
  for (int h = g * group + warp; h < (g + 1) * group; h += PA_WARPS) {
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      q[e] = d < a.hd ? to_f32(((const IO*)a.q)[b * a.q_stride + (long long)h * a.hd + d]) : 0.f;
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < len; ++j) {
      const int blk = j / a.page, id = a.table[(size_t)b * a.max_blocks + blk];
      if (id < 0 || id >= a.n_pages) {
        if (lane == 0) atomicOr(a.err, ERR_PAGE);
        continue;
      }
      const long long at = id * a.page_stride + g * a.head_stride + (long long)(j - blk * a.page) * a.pos_stride;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane + 32 * e;
        if (d < a.hd) s = fmaf(q[e], to_f32(((const KV*)a.k)[at + d]), s);
      }
      s = warp_sum(s) * a.scale;
      const float mn = fmaxf(m, s);
      const float ref = mn == -INFINITY ? 0.f : mn;  // no score above -inf yet
      const float c = expf(m - ref), p = expf(s - ref);
      l = fmaf(l, c, p);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane + 32 * e;
        if (d < a.hd) o[e] = fmaf(o[e], c, p * to_f32(((const KV*)a.v)[at + d]));
      }
      m = s != s ? s : mn;  // a NaN stays
    }
    const float inv = len == 0 ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      if (d < a.hd) ((IO*)a.out)[b * a.out_stride + (long long)h * a.hd + d] = from_f32<IO>(o[e] * inv);
    }
    if (lane == 0 && a.lse) a.lse[(size_t)b * a.nq + h] = m + logf(l);
  }
}

template <typename IO, typename KV>
cudaError_t launch_paged(const PagedAttnArgs& a, cudaStream_t s) {
  return launch_k(paged_attn_kernel<IO, KV>, dim3(a.nkv, a.n_seqs), dim3(PA_WARPS * 32), 0, s, false, a);
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 8 || head_dim % 8 || head_dim > PA_MAX_HD) return 0;
  return 256;
}

qw_status qw_op_paged_attention(const qw_paged_kv* cache, int32_t n_seqs, int32_t n_heads, const int32_t* block_table,
                                int32_t max_blocks, const int32_t* lens, int32_t io_dtype, const void* q,
                                int64_t q_stride, float scale, void* out, int64_t out_stride, float* lse,
                                void* workspace, size_t workspace_bytes, int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  qw_paged_kv c;
  qw_status st = op_check_cache(cache, &c);
  if (st) return st;
  if ((st = op_check_io(io_dtype, c.dtype))) return st;
  if (n_seqs < 0 || max_blocks < 1 || n_heads < 1 || n_heads % c.n_kv_heads)
    return op_fail(QW_ERR_INVALID_ARG, "bad attention shape");
  if (n_seqs > 65535 || n_heads > 4096) return op_fail(QW_ERR_UNSUPPORTED, "more than 65535 sequences or 4096 heads");
  if ((int64_t)max_blocks * c.page_size > 0x7fffffffll)
    return op_fail(QW_ERR_UNSUPPORTED, "max_blocks * page_size above 2^31 - 1");
  if (!std::isfinite(scale)) return op_fail(QW_ERR_INVALID_ARG, "scale not finite");
  if (n_seqs == 0) return QW_OK;
  if (!block_table || !lens || !workspace || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  const int64_t width = (int64_t)n_heads * c.head_dim;
  if ((st = op_check_rows(q, q_stride, width, io_dtype, "q"))) return st;
  if ((st = op_check_rows(out, out_stride, width, io_dtype, "out"))) return st;
  if (out == q && out_stride != q_stride) return op_fail(QW_ERR_INVALID_ARG, "out may be q with the same stride only");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_paged_attention_workspace(n_heads, c.n_kv_heads, c.head_dim))
    return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  if ((st = op_check_device({c.k, c.v, block_table, lens, q, out, lse, workspace, err_dev}))) return st;
  PagedAttnArgs a{c.k, c.v, c.page_stride, c.head_stride, c.pos_stride, n_seqs, n_heads, c.n_kv_heads, c.head_dim,
                  c.page_size, c.n_pages, max_blocks, block_table, lens, q, out, q_stride, out_stride, scale, lse,
                  err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  cudaError_t e;
  if (io_dtype == QW_F32)
    e = c.dtype == QW_F32 ? launch_paged<float, float>(a, s)
        : c.dtype == QW_F16 ? launch_paged<float, f16>(a, s) : launch_paged<float, bf16>(a, s);
  else
    e = io_dtype == QW_F16 ? launch_paged<f16, f16>(a, s) : launch_paged<bf16, bf16>(a, s);
  if (e) return op_cuda_fail(e, "paged attention launch");
  return QW_OK;
}

}  // extern "C"
