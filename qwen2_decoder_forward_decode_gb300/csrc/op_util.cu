// Argument checks of the single-operation entry points of a paged cache.
#include "op_util.h"

#include <cuda.h>

namespace qw {

namespace {
typedef CUresult (*AttributesFn)(unsigned int, CUpointer_attribute*, void**, CUdeviceptr);
AttributesFn attributes_fn() {
  static const AttributesFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &p, 12000, cudaEnableDefault, &q);
    if (e) cudaGetLastError();
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? (AttributesFn)p : (AttributesFn) nullptr;
  }();
  return fn;
}
}  // namespace

qw_status op_check_device(OpPointers ptrs) {
  for (const void* p : ptrs)
    if ((uintptr_t)p & 3) return op_fail(QW_ERR_INVALID_ARG, "a pointer is not aligned to 4 bytes");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e) return op_cuda_fail(e, "cudaGetDevice");
  // Pointers into an allocation that this call has looked up already need no look of their own: callers' tensors mostly lie
  // in a few, and a look costs 0.1 to 0.4 us (a page copy has 56 pointers of 28 layers).
  struct { uintptr_t lo, hi; } seen[4];
  int n_seen = 0;
  for (const void* p : ptrs) {
    if (!p) continue;
    bool known = false;
    for (int i = 0; i < n_seen; ++i) known |= (uintptr_t)p - seen[i].lo < seen[i].hi - seen[i].lo;
    if (known) continue;
    int where = -1;  // the memory's device
    unsigned int type = 0, managed = 0;
    CUdeviceptr start = 0;
    size_t size = 0;
    CUpointer_attribute what[] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL, CU_POINTER_ATTRIBUTE_IS_MANAGED,
                                  CU_POINTER_ATTRIBUTE_RANGE_START_ADDR, CU_POINTER_ATTRIBUTE_RANGE_SIZE};
    void* into[] = {&type, &where, &managed, &start, &size};
    const AttributesFn f = attributes_fn();
    if (!f || f(5, what, into, (CUdeviceptr)p) != CUDA_SUCCESS) {
      cudaPointerAttributes a;
      if ((e = cudaPointerGetAttributes(&a, p))) return op_cuda_fail(e, "cudaPointerGetAttributes");
      type = a.type == cudaMemoryTypeDevice ? CU_MEMORYTYPE_DEVICE : 0;
      managed = a.type == cudaMemoryTypeManaged;
      where = a.device;
      size = 0;
    }
    if (managed) continue;
    if (type != CU_MEMORYTYPE_DEVICE) return op_fail(QW_ERR_INVALID_ARG, "a pointer is not device memory");
    if (where != dev) return op_fail(QW_ERR_INVALID_ARG, "a pointer belongs to another device than the current one");
    if (n_seen < 4 && (uintptr_t)p - start < size) {
      seen[n_seen].lo = start;
      seen[n_seen++].hi = start + size;
    }
  }
  return QW_OK;
}

qw_status op_check_cache(const qw_paged_kv* c, qw_paged_kv* norm) {
  if (!c) return op_fail(QW_ERR_INVALID_ARG, "null cache");
  if (!c->k || !c->v) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (!dtype_known(c->dtype)) return op_fail(QW_ERR_INVALID_ARG, "unknown cache dtype");
  if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1)
    return op_fail(QW_ERR_INVALID_ARG, "non-positive cache dimension");
  if (c->head_dim % 8 || c->head_dim > 256)
    return op_fail(QW_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 256");
  if (!aligned16(c->k) || !aligned16(c->v)) return op_fail(QW_ERR_INVALID_ARG, "cache not 16-byte aligned");
  qw_paged_kv n = *c;
  if (n.n_pages == 1) n.page_stride = 0;
  if (n.n_kv_heads == 1) n.head_stride = 0;
  if (n.page_size == 1) n.pos_stride = 0;
  const int64_t unit = 16 / (int64_t)dtype_size(c->dtype);
  const int64_t far = (int64_t)1 << 40;  // elements: keeps every product below in 64 bits
  for (int64_t s : {n.page_stride, n.head_stride, n.pos_stride}) {
    if (s < 0 || s > far) return op_fail(QW_ERR_INVALID_ARG, "bad cache stride");
    if (s % unit) return op_fail(QW_ERR_INVALID_ARG, "cache strides must be multiples of 16 bytes");
  }
  // the extent that each order's inner rows cover must fit the next stride
  auto fits = [&](int64_t s1, int n1, int64_t s2, int n2) {  // n1 rows s1 apart inside n2 blocks s2 apart
    int64_t cover = n.head_dim;
    if (n1 > 1) {
      if (s1 < cover) return false;
      cover += (int64_t)(n1 - 1) * s1;
    }
    if (n2 > 1) {
      if (s2 < cover) return false;
      cover += (int64_t)(n2 - 1) * s2;
    }
    return n.n_pages == 1 || n.page_stride >= cover;
  };
  if (!fits(n.pos_stride, n.page_size, n.head_stride, n.n_kv_heads) &&
      !fits(n.head_stride, n.n_kv_heads, n.pos_stride, n.page_size))
    return op_fail(QW_ERR_INVALID_ARG, "cache strides overlap, or pages are not the outer dimension");
  *norm = n;
  return QW_OK;
}

qw_status op_check_io(int32_t io_dtype, int32_t cache_dtype) {
  if (!dtype_known(io_dtype)) return op_fail(QW_ERR_INVALID_ARG, "unknown io dtype");
  if (io_dtype != QW_F32 && io_dtype != cache_dtype)
    return op_fail(QW_ERR_UNSUPPORTED, "io dtype must be QW_F32 or the cache's");
  return QW_OK;
}

qw_status op_check_rows(const void* p, int64_t stride, int64_t width, int32_t t, const char* what) {
  if (!p) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  const int64_t unit = 16 / (int64_t)dtype_size(t);
  if (!aligned16(p) || stride % unit || stride < width || stride > (int64_t)1 << 40) {
    set_error_message(what, "rows must be 16-byte aligned, their stride a multiple of 16 bytes that covers a row");
    return QW_ERR_INVALID_ARG;
  }
  return QW_OK;
}

}  // namespace qw
