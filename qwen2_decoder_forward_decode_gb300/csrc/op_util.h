// Host-side checks shared by the single-operation entry points of a paged cache.
#pragma once

#include "../../include/qw.h"
#include "internal.h"

#include <initializer_list>

namespace qw {

inline qw_status op_fail(qw_status s, const char* msg) {
  set_error_message(msg);
  return s;
}
inline qw_status op_cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();  // reported here: the next launch that asks for the last error must not find it
  set_error_message(where, cudaGetErrorString(e));
  return QW_ERR_CUDA;
}

inline size_t dtype_size(int32_t t) { return t == QW_F32 ? 4 : 2; }
inline bool dtype_known(int32_t t) { return t == QW_F32 || t == QW_F16 || t == QW_BF16; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Both operators with a workspace keep their counters (zero between calls) in its first bytes, so that one workspace
// can serve them in turn.
constexpr size_t OP_COUNTER_BYTES = 16384;

// Every pointer must be memory of the current device: a host pointer or another device's would
// fault in the kernel. Managed memory passes. Null pointers are skipped (optional arguments). A pointer that is not
// aligned to 4 bytes would fault too: all elements but 16-bit ones have 4 or 8.
qw_status op_check_device(std::initializer_list<const void*> ptrs);

// Shape, strides and alignment of a paged cache; on success *norm is the cache with the strides
// along extents of 1 set to 0.
qw_status op_check_cache(const qw_paged_kv* c, qw_paged_kv* norm);

// io_dtype against the cache's type.
qw_status op_check_io(int32_t io_dtype, int32_t cache_dtype);

// Rows of `width` elements of dtype t, `stride` apart: 16-byte aligned and not overlapping.
qw_status op_check_rows(const void* p, int64_t stride, int64_t width, int32_t t, const char* what);

}  // namespace qw
