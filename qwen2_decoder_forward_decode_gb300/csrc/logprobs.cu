// Log probabilities of given tokens, with ranks, entropy and the likeliest tokens ("LLM Speedrun:
// Architecture", Decoding: the softmax of the logits).
//
// With m = max z, S = sum exp(z - m) and W = sum (z - m) exp(z - m): ln p_t = z_t - m - ln S and the
// entropy is ln S - W / S. Tokens are ordered by (logit, lower id first) as one 64-bit key.
#include "common.cuh"
#include "op_util.h"

#include <math.h>

namespace qw {
namespace {

constexpr int LP_THREADS = 512;
constexpr int LP_MAX_IDS = 8, LP_MAX_TOP = 32;

struct LogprobArgs {
  const void* logits;
  long long row_stride;
  int n_rows, vocab, n_ids, top_k;
  const int* ids;
  float* logprobs;
  int* ranks;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  int* err;
};

// (logit, lower id first) as an integer; -0 counts as 0
__device__ __forceinline__ unsigned long long order_key(float z, int j) { return argmax_key(z + 0.f, j); }
__device__ __forceinline__ float order_key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS) logprob_kernel(const LogprobArgs a) {
  __shared__ float red[32];
  __shared__ unsigned long long kred[32];
  __shared__ int ired[32];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = LP_THREADS / 32;
  const T* z = (const T*)a.logits + (size_t)row * a.row_stride;
  float m = -INFINITY;
  int odd = 0;  // a NaN or +inf in the row
  for (int j = tid; j < a.vocab; j += LP_THREADS) {
    const float x = to_f32(z[j]);
    if (!(x < INFINITY)) odd = 1;
    m = fmaxf(m, x);
  }
  m = warp_max(m);
  odd = __syncthreads_or(odd);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int w = 0; w < nw; ++w) m = fmaxf(m, red[w]);
  if (odd || m == -INFINITY) {  // no distribution
    if (tid == 0) atomicOr(a.err, ERR_NONFINITE);
    for (int i = tid; i < a.n_ids; i += LP_THREADS) {
      const int t = a.ids[(size_t)row * a.n_ids + i];
      a.logprobs[(size_t)row * a.n_ids + i] = t == -1 ? 0.f : NAN;
      if (a.ranks) a.ranks[(size_t)row * a.n_ids + i] = 0;
      if (t < -1 || t >= a.vocab) atomicOr(a.err, ERR_TOKEN);
    }
    if (tid == 0 && a.entropy) a.entropy[row] = NAN;
    for (int i = tid; i < a.top_k; i += LP_THREADS) {
      a.top_ids[(size_t)row * a.top_k + i] = -1;
      a.top_logprobs[(size_t)row * a.top_k + i] = NAN;
    }
    return;
  }
  float S = 0.f, W = 0.f;
  for (int j = tid; j < a.vocab; j += LP_THREADS) {
    const float d = to_f32(z[j]) - m;
    const float e = expf(d);
    S += e;
    if (e > 0.f) W = fmaf(d, e, W);
  }
  S = block_sum(S, red);
  W = block_sum(W, red);
  const float ln_s = logf(S);
  if (tid == 0 && a.entropy) a.entropy[row] = ln_s - W / S;
  for (int i = 0; i < a.n_ids; ++i) {
    const int t = a.ids[(size_t)row * a.n_ids + i];
    if (t < 0 || t >= a.vocab) {
      if (tid == 0) {
        if (t != -1) atomicOr(a.err, ERR_TOKEN);
        a.logprobs[(size_t)row * a.n_ids + i] = t == -1 ? 0.f : NAN;
        if (a.ranks) a.ranks[(size_t)row * a.n_ids + i] = 0;
      }
      continue;
    }
    const float zt = to_f32(z[t]);
    if (tid == 0) a.logprobs[(size_t)row * a.n_ids + i] = zt - m - ln_s;
    if (!a.ranks) continue;
    int above = 0;
    for (int j = tid; j < a.vocab; j += LP_THREADS) {
      const float x = to_f32(z[j]);
      above += x > zt || (x == zt && j < t);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    __syncthreads();
    if (lane == 0) ired[warp] = above;
    __syncthreads();
    if (tid == 0) {
      int r = 1;
      for (int w = 0; w < nw; ++w) r += ired[w];
      a.ranks[(size_t)row * a.n_ids + i] = r;
    }
  }
  unsigned long long last = ~0ull;  // the key taken before: the next is the largest below it
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int j = tid; j < a.vocab; j += LP_THREADS) {
      const unsigned long long key = order_key(to_f32(z[j]), j);
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    __syncthreads();
    if (lane == 0) kred[warp] = best;
    __syncthreads();
    best = kred[0];
    for (int w = 1; w < nw; ++w) best = kred[w] > best ? kred[w] : best;
    last = best;
    if (tid == 0) {
      a.top_ids[(size_t)row * a.top_k + k] = argmax_key_index(best);
      a.top_logprobs[(size_t)row * a.top_k + k] = order_key_value(best) - m - ln_s;
    }
  }
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_token_logprobs_workspace(int32_t n_rows, int32_t vocab, int32_t top_k) {
  if (n_rows < 0 || vocab < 1 || top_k < 0 || top_k > LP_MAX_TOP) return 0;
  return 256;
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
  if (n_rows == 0) return QW_OK;
  if (!logits || !err_dev || !workspace || (n_ids && (!ids || !logprobs)) || (top_k && (!top_ids || !top_logprobs)))
    return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)logits % dtype_size(logits_dtype)) return op_fail(QW_ERR_INVALID_ARG, "logits misaligned");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_token_logprobs_workspace(n_rows, vocab, top_k))
    return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  qw_status st = op_check_device({logits, n_ids ? ids : nullptr, n_ids ? logprobs : nullptr, n_ids ? ranks : nullptr,
                                  entropy, top_k ? top_ids : nullptr, top_k ? top_logprobs : nullptr, workspace,
                                  err_dev});
  if (st) return st;
  LogprobArgs a{logits, row_stride, n_rows, vocab, n_ids, top_k, ids, logprobs, ranks, entropy, top_ids,
                top_logprobs, err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  const dim3 grid(n_rows), block(LP_THREADS);
  const cudaError_t e = logits_dtype == QW_F32   ? launch_k(logprob_kernel<float>, grid, block, 0, s, false, a)
                        : logits_dtype == QW_F16 ? launch_k(logprob_kernel<f16>, grid, block, 0, s, false, a)
                                                 : launch_k(logprob_kernel<bf16>, grid, block, 0, s, false, a);
  if (e) return op_cuda_fail(e, "token logprobs launch");
  return QW_OK;
}

}  // extern "C"
