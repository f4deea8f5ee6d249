// Page plans of a paged key-value cache: block tables, slot maps and positions built on the GPU from
// the sequences' lengths, and the return of finished sequences' pages.
//
// With have_b = ceil(len_b / page) and need_b = ceil((len_b + new_b) / page), sequence b takes
// need_b - have_b pages. Two exclusive prefix sums over the sequences (tokens and pages) place every
// token and every page: token t belongs to the last b with cu[b] <= t, page i of the step to the last
// b with pg[b] <= i, and that page is free[n_free - 1 - i]. The sums live in shared memory; tokens and
// pages are then independent (a binary search each).
#include "common.cuh"
#include "op_util.h"

namespace qw {
namespace {

constexpr int PLAN_MAX_SEQS = 16384;
constexpr int PLAN_THREADS = 1024;

struct PlanArgs {
  int n, page, n_pages, max_blocks, max_tokens;
  const int *lens, *n_new, *free_pages, *n_free;
  int *table, *lens_out, *n_free_out, *cu, *positions;
  long long* slots;
  int* err;
};
struct ReleaseArgs {
  int n, page, n_pages, max_blocks;
  const int *lens, *done, *table, *n_free;
  int *free_pages, *lens_out, *n_free_out, *err;
};

__device__ __forceinline__ long long warp_incl_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive prefix sums over n items of two non-negative counts (item(i, a, b) gives them) into
// sa[0 .. n] and sb[0 .. n]. Sums above 2^31 - 1 are cut there and returned as they are in tot.
template <typename Item>
__device__ void block_scan2(int n, int* sa, int* sb, long long* tot, Item item) {
  __shared__ long long wa[PLAN_THREADS / 32], wb[PLAN_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const long long cap = 0x7fffffffll;
  long long ca = 0, cb = 0;  // sums of the items before this chunk
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + tid;
    long long a = 0, b = 0;
    if (i < n) item(i, a, b);
    const long long ia = warp_incl_scan(a), ib = warp_incl_scan(b);
    if (lane == 31) {
      wa[warp] = ia;
      wb[warp] = ib;
    }
    __syncthreads();
    long long oa = ca, ob = cb;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) {
        oa += wa[w];
        ob += wb[w];
      }
      ca += wa[w];
      cb += wb[w];
    }
    if (i < n) {
      const long long xa = oa + ia - a, xb = ob + ib - b;
      sa[i] = (int)(xa < cap ? xa : cap);
      sb[i] = (int)(xb < cap ? xb : cap);
    }
    __syncthreads();
  }
  if (tid == 0) {
    sa[n] = (int)(ca < cap ? ca : cap);
    sb[n] = (int)(cb < cap ? cb : cap);
  }
  tot[0] = ca;
  tot[1] = cb;
  __syncthreads();
}

// the last b in [0, n) with s[b] <= x (s ascending, s[0] = 0, x < s[n])
__device__ __forceinline__ int find_seq(const int* s, int n, int x) {
  int lo = 0, hi = n;  // s[lo] <= x < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_sm[];
  int* cu = plan_sm;           // [n + 1] tokens before a sequence
  int* pg = plan_sm + a.n + 1;  // [n + 1] pages taken before it
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int n_free = *a.n_free;
  const long long room = (long long)a.max_blocks * a.page;
  long long tot[2];
  block_scan2(a.n, cu, pg, tot, [&](int i, long long& t, long long& p) {
    const int len = a.lens[i], add = a.n_new ? a.n_new[i] : 1;
    if (len < 0 || add < 0 || (long long)len + add > room) {
      s_bad = 1;
      return;
    }
    t = add;
    p = ((long long)len + add + a.page - 1) / a.page - (len + (long long)a.page - 1) / a.page;
  });
  const bool bad = s_bad || n_free < 0 || n_free > a.n_pages || tot[0] > a.max_tokens || tot[1] > n_free;
  if (bad && tid == 0) atomicOr(a.err, ERR_CAPACITY);
  const int n_tok = bad ? 0 : (int)tot[0], n_take = bad ? 0 : (int)tot[1];
  for (int i = tid; i < n_take; i += blockDim.x) {
    const int b = find_seq(pg, a.n, i);
    const int have = (int)((a.lens[b] + (long long)a.page - 1) / a.page);
    a.table[(size_t)b * a.max_blocks + have + (i - pg[b])] = a.free_pages[n_free - 1 - i];
  }
  for (int t = tid; t < a.max_tokens; t += blockDim.x) {
    int pos = 0;
    long long slot = -1;
    if (t < n_tok) {
      const int b = find_seq(cu, a.n, t);
      const int len = a.lens[b];
      pos = len + (t - cu[b]);
      const int have = (int)((len + (long long)a.page - 1) / a.page);
      const int j = pos / a.page;
      const int id = j < have ? a.table[(size_t)b * a.max_blocks + j] : a.free_pages[n_free - 1 - (pg[b] + j - have)];
      if (id >= 0 && id < a.n_pages) slot = (long long)id * a.page + (pos - j * a.page);
      else atomicOr(a.err, ERR_PAGE);
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  __syncthreads();  // lens_out may be lens
  for (int i = tid; i <= a.n; i += blockDim.x) {
    a.cu[i] = bad ? 0 : cu[i];
    if (i < a.n) a.lens_out[i] = a.lens[i] + (bad ? 0 : cu[i + 1] - cu[i]);
  }
  if (tid == 0) *a.n_free_out = n_free - n_take;
}

__global__ void __launch_bounds__(PLAN_THREADS) page_release_kernel(const ReleaseArgs a) {
  extern __shared__ int plan_sm[];
  int* pg = plan_sm;               // [n + 1] pages given back before a sequence
  int* gone = plan_sm + a.n + 1;   // [n + 1] sequences finished before it
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int n_free = *a.n_free;
  const long long room = (long long)a.max_blocks * a.page;
  long long tot[2];
  block_scan2(a.n, pg, gone, tot, [&](int i, long long& p, long long& g) {
    const int len = a.lens[i];
    if (len < 0 || len > room) {
      s_bad = 1;
      return;
    }
    if (!a.done[i]) return;
    p = (len + (long long)a.page - 1) / a.page;
    g = 1;
  });
  const bool bad = s_bad || n_free < 0 || n_free > a.n_pages || tot[0] > a.n_pages - n_free;
  if (bad && tid == 0) atomicOr(a.err, ERR_CAPACITY);
  const int n_give = bad ? 0 : (int)tot[0];
  for (int i = tid; i < n_give; i += blockDim.x) {
    const int b = find_seq(pg, a.n, i);
    const int id = a.table[(size_t)b * a.max_blocks + (i - pg[b])];
    if (id < 0 || id >= a.n_pages) atomicOr(a.err, ERR_PAGE);
    a.free_pages[n_free + i] = id;
  }
  __syncthreads();  // lens_out may be lens
  for (int i = tid; i < a.n; i += blockDim.x) a.lens_out[i] = !bad && gone[i + 1] > gone[i] ? 0 : a.lens[i];
  if (tid == 0) *a.n_free_out = n_free + n_give;
}

template <typename K>
cudaError_t plan_smem(K kernel, int n, size_t* bytes) {
  *bytes = (size_t)2 * (n + 1) * sizeof(int);
  return *bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)*bytes)
                            : cudaSuccess;
}

qw_status plan_dims(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks) {
  if (n_seqs < 0 || page_size < 1 || n_pages < 1 || max_blocks < 1)
    return op_fail(QW_ERR_INVALID_ARG, "bad page plan dimension");
  if (n_seqs > PLAN_MAX_SEQS) return op_fail(QW_ERR_UNSUPPORTED, "more than 16384 sequences");
  return QW_OK;
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

qw_status qw_op_page_plan(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks, int32_t max_tokens,
                          const int32_t* lens, const int32_t* n_new, const int32_t* free_pages,
                          const int32_t* n_free, int32_t* block_table, int32_t* lens_out, int32_t* n_free_out,
                          int32_t* cu_tokens, int32_t* positions, int64_t* slots, int32_t* err_dev,
                          void* cuda_stream) {
  set_error_message("");
  qw_status st = plan_dims(n_seqs, page_size, n_pages, max_blocks);
  if (st) return st;
  if (max_tokens < 0) return op_fail(QW_ERR_INVALID_ARG, "negative max_tokens");
  if (!free_pages || !n_free || !n_free_out || !cu_tokens || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_seqs > 0 && (!lens || !block_table || !lens_out)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (max_tokens > 0 && (!positions || !slots)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)slots & 7) return op_fail(QW_ERR_INVALID_ARG, "slots not 8-byte aligned");
  if ((st = op_check_device({lens, n_new, free_pages, n_free, block_table, lens_out, n_free_out, cu_tokens, positions,
                             slots, err_dev})))
    return st;
  PlanArgs a{n_seqs, page_size, n_pages, max_blocks, max_tokens, lens, n_new, free_pages, n_free, block_table,
             lens_out, n_free_out, cu_tokens, positions, (long long*)slots, err_dev};
  size_t smem;
  cudaError_t e = plan_smem(page_plan_kernel, n_seqs, &smem);
  if (e) return op_cuda_fail(e, "page plan attributes");
  if ((e = launch_k(page_plan_kernel, dim3(1), dim3(PLAN_THREADS), smem, (cudaStream_t)cuda_stream, false, a)))
    return op_cuda_fail(e, "page plan launch");
  return QW_OK;
}

qw_status qw_op_page_release(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks,
                             const int32_t* lens, const int32_t* done, const int32_t* block_table,
                             int32_t* free_pages, const int32_t* n_free, int32_t* lens_out, int32_t* n_free_out,
                             int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  qw_status st = plan_dims(n_seqs, page_size, n_pages, max_blocks);
  if (st) return st;
  if (!free_pages || !n_free || !n_free_out || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_seqs > 0 && (!lens || !done || !block_table || !lens_out)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((st = op_check_device({lens, done, block_table, free_pages, n_free, lens_out, n_free_out, err_dev}))) return st;
  ReleaseArgs a{n_seqs, page_size, n_pages, max_blocks, lens, done, block_table, n_free, free_pages, lens_out,
                n_free_out, err_dev};
  size_t smem;
  cudaError_t e = plan_smem(page_release_kernel, n_seqs, &smem);
  if (e) return op_cuda_fail(e, "page release attributes");
  if ((e = launch_k(page_release_kernel, dim3(1), dim3(PLAN_THREADS), smem, (cudaStream_t)cuda_stream, false, a)))
    return op_cuda_fail(e, "page release launch");
  return QW_OK;
}

}  // extern "C"
