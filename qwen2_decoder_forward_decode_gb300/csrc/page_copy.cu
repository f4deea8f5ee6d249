// Copies of pages inside the caches of all layers: the partly filled last pages of forked sequences, and the pages that a
// compaction moves.
//
// What bounds it: HBM, every byte once in and once out. A unit is a page of one layer's keys or values, and a CTA's; there are CTAs
// enough that the last ones even out (64 an SM; 8 an SM, of which 5 fit at a time, took units in turn in 123 us where this takes
// 119). 128 threads, each eight vectors of 16 bytes at a time; 512 threads 127. 256 pages of 12 layers, 64 positions of 4 heads of 128,
// bf16: 119 us (6.4 TB/s of the copy's 6.8); 16 last pages of 28 layers 3.2 us.
#include "common.cuh"
#include "op_util.h"

#include <algorithm>

namespace qw {
namespace {

constexpr int COPY_MAX_CACHES = 128, COPY_THREADS = 128, COPY_VECS = 8;

struct CopyArgs {
  int n, n_caches, n_pages, page, nkv, row;  // row: vectors of a head's dimensions
  long long page_stride, head_stride, pos_stride;  // in vectors
  const int *src, *dst, *len;
  int* err;
  uint4* base[2 * COPY_MAX_CACHES];  // keys, values of each cache
};

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int per = 2 * a.n_caches;
  const long long units = (long long)a.n * per;
  int old = -1, from = -1, to = -1, len = 0;
#pragma unroll 1
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / per), k = (int)(u - (long long)i * per);
    if (i != old) {
      old = i;
      from = a.src[i];
      to = a.dst[i];
      len = a.len ? a.len[i] : a.page;
      bool ok = from >= 0 && from < a.n_pages && to >= 0 && to < a.n_pages && len >= 0 && len <= a.page;
      if (!ok && from != -1 && k == 0 && threadIdx.x == 0) atomicOr(a.err, ERR_PAGE);
      if (!ok || from == to) len = 0;
    }
    if (len == 0) continue;
    const uint4* x = a.base[k] + from * a.page_stride;
    uint4* y = a.base[k] + to * a.page_stride;
    const int head = len * a.row, n = a.nkv * head;  // (the host bounds n)
#pragma unroll 1
    for (int v0 = threadIdx.x; v0 < n; v0 += COPY_VECS * COPY_THREADS) {
      uint4 r[COPY_VECS];
      long long at[COPY_VECS];
#pragma unroll
      for (int q = 0; q < COPY_VECS; ++q) {
        const int v = v0 + q * COPY_THREADS;
        if (v >= n) continue;
        const int h = v / head, w = v - h * head, p = w / a.row;
        at[q] = h * a.head_stride + p * a.pos_stride + (w - p * a.row);
        r[q] = ld_stream(x + at[q]);
      }
#pragma unroll
      for (int q = 0; q < COPY_VECS; ++q)
        if (v0 + q * COPY_THREADS < n) y[at[q]] = r[q];
    }
  }
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" qw_status qw_op_page_copy(const qw_paged_kv* caches, int32_t n_caches, int32_t n, const int32_t* src,
                                     const int32_t* dst, const int32_t* len, int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  if (n_caches < 0 || n < 0) return op_fail(QW_ERR_INVALID_ARG, "bad page copy dimension");
  if (n_caches > COPY_MAX_CACHES) return op_fail(QW_ERR_UNSUPPORTED, "more than 128 caches");
  if (n_caches == 0) return QW_OK;
  if (!caches) return op_fail(QW_ERR_INVALID_ARG, "null cache");
  CopyArgs a{};
  qw_paged_kv c0{};
  qw_status st;
  for (int i = 0; i < n_caches; ++i) {
    qw_paged_kv c;
    if ((st = op_check_cache(caches + i, &c))) return st;
    if (i == 0) c0 = c;
    else if (c.dtype != c0.dtype || c.n_pages != c0.n_pages || c.page_size != c0.page_size || c.n_kv_heads != c0.n_kv_heads ||
             c.head_dim != c0.head_dim || c.page_stride != c0.page_stride || c.head_stride != c0.head_stride ||
             c.pos_stride != c0.pos_stride)
      return op_fail(QW_ERR_UNSUPPORTED, "the caches of one call have the same type, extents and strides");
    a.base[2 * i] = (uint4*)c.k;
    a.base[2 * i + 1] = (uint4*)c.v;
  }
  const int unit = 16 / (int)dtype_size(c0.dtype);
  if ((int64_t)c0.n_kv_heads * c0.page_size * (c0.head_dim / unit) > 1 << 30)
    return op_fail(QW_ERR_UNSUPPORTED, "a page of more than 2^30 vectors");
  if (n == 0) return QW_OK;
  if (!src || !dst || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  const void* ptrs[4 + 2 * COPY_MAX_CACHES] = {src, dst, len, err_dev};
  std::copy(a.base, a.base + 2 * n_caches, ptrs + 4);
  if ((st = op_check_device(OpPointers{ptrs, 4 + 2 * (size_t)n_caches}))) return st;
  a.n = n;
  a.n_caches = n_caches;
  a.n_pages = c0.n_pages;
  a.page = c0.page_size;
  a.nkv = c0.n_kv_heads;
  a.row = c0.head_dim / unit;
  a.page_stride = c0.page_stride / unit;
  a.head_stride = c0.head_stride / unit;
  a.pos_stride = c0.pos_stride / unit;
  a.src = src;
  a.dst = dst;
  a.len = len;
  a.err = err_dev;
  int dev = 0, nsm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  const int64_t units = (int64_t)n * 2 * n_caches;
  const int ctas = (int)(units < 64 * nsm ? units : 64 * nsm);
  if ((e = launch_k(page_copy_kernel, dim3(ctas), dim3(COPY_THREADS), 0, (cudaStream_t)cuda_stream, false, a)))
    return op_cuda_fail(e, "page copy launch");
  return QW_OK;
}
