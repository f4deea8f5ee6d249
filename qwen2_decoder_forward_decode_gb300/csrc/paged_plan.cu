// Page plans of a paged key-value cache: block tables, slot maps and positions built on the GPU from
// the sequences' lengths, and the return of finished sequences' pages.
//
// With have_b = ceil(len_b / page) and need_b = ceil((len_b + new_b) / page), sequence b takes
// need_b - have_b pages. Two exclusive prefix sums over the sequences (tokens and pages) place every
// token and every page: token t belongs to the last b with cu[b] <= t, page i of the step to the last
// b with pg[b] <= i, and that page is free[n_free - 1 - i]. Every CTA computes the sums into its shared
// memory (at most 16384 sequences); tokens, up to four to a thread, and pages are then independent, with
// a binary search each.
// What bounds it: latency (two dependent loads, a scan, a search, one more load). A step of at most
// PLAN_SMALL tokens, or a release of as many table entries, takes one CTA; more are spread over the SMs.
// Outputs that alias inputs (lengths and the free count) are then written by a second, small kernel, since
// a CTA may still be reading when another writes. Measured in a CUDA graph (a lone call costs the host about 3 us from C, 10 to 12
// from Python): 512 sequences with one token each 5.1 us (in place no more), 64 prompts of 117 000 tokens together 6.2 us (in
// place, with the second kernel, 8.2), 512 sequences of which a third give 37 000 pages back 4.3 us (in place 5.6);
// one CTA for everything took 117 us for the prompts.
#include "common.cuh"
#include "op_util.h"

namespace qw {
namespace {

constexpr int PLAN_MAX_SEQS = 16384;
constexpr int PLAN_THREADS = 512;
constexpr int PLAN_SMALL = 8192;

struct PlanArgs {
  int n, page, n_pages, max_blocks, max_tokens;
  const int *lens, *n_new, *free_pages, *n_free;
  int *table, *lens_out, *n_free_out, *cu, *positions;
  long long* slots;
  int* err;
  bool items, counts;  // what this launch writes: tokens and pages; the lengths and the free count
};
struct ReleaseArgs {
  int n, page, n_pages, max_blocks;
  const int *lens, *done, *table, *n_free;
  int *free_pages, *lens_out, *n_free_out, *err;
  bool items, counts;
};

constexpr uint32_t PLAN_CAP = 0x7fffffffu;
__device__ __forceinline__ uint32_t cap_add(uint32_t a, uint32_t b) { return min(a + b, PLAN_CAP); }  // a, b <= PLAN_CAP
__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = cap_add(v, u);
  }
  return v;
}

// Exclusive prefix sums over n items of two counts (item(i, a, b) gives them) into sa[0 .. n] and sb[0 .. n]. A sum
// that reaches 2^31 - 1 stays there.
template <typename Item>
__device__ __forceinline__ void block_scan2(int n, int* sa, int* sb, Item item) {
  __shared__ uint32_t wa[32], wb[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + PLAN_THREADS - 1) / PLAN_THREADS, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  uint32_t a = 0, b = 0;  // of the thread's consecutive items
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    uint32_t x = 0, y = 0;
    item(i, x, y);
    a = cap_add(a, x);
    b = cap_add(b, y);
  }
  const uint32_t ia = warp_incl_scan(a), ib = warp_incl_scan(b);
  if (warp == 0) wa[lane] = wb[lane] = 0;
  __syncthreads();
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  const uint32_t ta = warp_incl_scan(wa[lane]), tb = warp_incl_scan(wb[lane]);  // every warp scans the warps' sums
  uint32_t oa = warp ? __shfl_sync(0xffffffffu, ta, warp - 1) : 0, ob = warp ? __shfl_sync(0xffffffffu, tb, warp - 1) : 0;
  const uint32_t pa = __shfl_up_sync(0xffffffffu, ia, 1), pb = __shfl_up_sync(0xffffffffu, ib, 1);
  if (lane) {
    oa = cap_add(oa, pa);
    ob = cap_add(ob, pb);
  }
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    uint32_t x = 0, y = 0;
    item(i, x, y);
    sa[i] = (int)oa;
    sb[i] = (int)ob;
    oa = cap_add(oa, x);
    ob = cap_add(ob, y);
  }
  if (tid == PLAN_THREADS - 1) {
    sa[n] = (int)ta;
    sb[n] = (int)tb;
  }
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

__device__ __forceinline__ int pages_of(long long positions, int page) {
  return (int)(positions >> 31 ? (positions + page - 1) / page : ((uint32_t)positions + (uint32_t)page - 1u) / (uint32_t)page);
}

__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_sm[];
  int* cu = plan_sm;           // [n + 1] tokens before a sequence
  int* pg = plan_sm + a.n + 1;  // [n + 1] pages taken before it
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (!a.items) pdl_wait();  // (the launch that reads what this one overwrites)
  if (tid == 0) s_bad = 0;
  const int n_free = *a.n_free;
  const long long room = min((long long)a.max_blocks * a.page, 0x7fffffffll);  // (lengths are 32-bit)
  __syncthreads();
  block_scan2(a.n, cu, pg, [&](int i, uint32_t& t, uint32_t& p) {
    const int len = a.lens[i], add = a.n_new ? a.n_new[i] : 1;
    if (len < 0 || add < 0 || (long long)len + add > room) {
      s_bad = 1;
      return;
    }
    t = (uint32_t)add;
    p = (uint32_t)(pages_of((long long)len + add, a.page) - pages_of(len, a.page));
  });
  // (a capped sum is 2^31 - 1; so many pages are never free, and a step of so many tokens is refused too)
  const bool bad = s_bad || n_free < 0 || n_free > a.n_pages || cu[a.n] > a.max_tokens || (uint32_t)cu[a.n] == PLAN_CAP || pg[a.n] > n_free;
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(a.err, ERR_CAPACITY);
  const int n_tok = bad ? 0 : cu[a.n], n_take = bad ? 0 : pg[a.n];
  const int first = blockIdx.x * PLAN_THREADS + tid, step = gridDim.x * PLAN_THREADS;
  const int run = a.max_tokens > step ? 4 : 1;  // tokens a thread maps in a row: one search, mostly one page
  if (a.items) {
#pragma unroll 1
    for (int i = first; i < n_take; i += step) {
      const int b = find_seq(pg, a.n, i);
      a.table[(size_t)b * a.max_blocks + pages_of(a.lens[b], a.page) + (i - pg[b])] = a.free_pages[n_free - 1 - i];
    }
#pragma unroll 1
    for (int t0 = run * first; t0 < a.max_tokens; t0 += run * step) {
      int b = t0 < n_tok ? find_seq(cu, a.n, t0) : 0, in = -1, id = 0, len = 0, have = 0;  // in: page of the sequence that id is
      if (t0 < n_tok) {
        len = a.lens[b];
        have = pages_of(len, a.page);
      }
#pragma unroll 1
      for (int t = t0; t < min(t0 + run, a.max_tokens); ++t) {
        int pos = 0;
        long long slot = -1;
        if (t < n_tok) {
          while (t >= cu[b + 1]) {
            ++b;
            in = -1;
            len = a.lens[b];
            have = pages_of(len, a.page);
          }
          pos = len + (t - cu[b]);
          const int j = (int)((uint32_t)pos / (uint32_t)a.page);
          if (j != in) {
            in = j;
            id = j < have ? a.table[(size_t)b * a.max_blocks + j] : a.free_pages[n_free - 1 - (pg[b] + j - have)];
          }
          if (id >= 0 && id < a.n_pages) slot = (long long)id * a.page + (pos - j * a.page);
          else atomicOr(a.err, ERR_PAGE);
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
      }
    }
    if (blockIdx.x == 0)
      for (int i = tid; i <= a.n; i += PLAN_THREADS) a.cu[i] = bad ? 0 : cu[i];
  }
  if (a.counts && blockIdx.x == 0) {
    __syncthreads();  // lens_out may be lens
    for (int i = tid; i < a.n; i += PLAN_THREADS) a.lens_out[i] = a.lens[i] + (bad ? 0 : cu[i + 1] - cu[i]);
    if (tid == 0) *a.n_free_out = n_free - n_take;
  }
}

__global__ void __launch_bounds__(PLAN_THREADS) page_release_kernel(const ReleaseArgs a) {
  extern __shared__ int plan_sm[];
  int* pg = plan_sm;               // [n + 1] pages given back before a sequence
  int* gone = plan_sm + a.n + 1;   // [n + 1] sequences finished before it
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (!a.items) pdl_wait();
  if (tid == 0) s_bad = 0;
  const int n_free = *a.n_free;
  const long long room = (long long)a.max_blocks * a.page;
  __syncthreads();
  block_scan2(a.n, pg, gone, [&](int i, uint32_t& p, uint32_t& g) {
    const int len = a.lens[i];
    if (len < 0 || len > room) {
      s_bad = 1;
      return;
    }
    if (!a.done[i]) return;
    p = (uint32_t)pages_of(len, a.page);
    g = 1;
  });
  const bool bad = s_bad || n_free < 0 || n_free > a.n_pages || pg[a.n] > a.n_pages - n_free;
  if (bad && tid == 0 && blockIdx.x == 0) atomicOr(a.err, ERR_CAPACITY);
  const int n_give = bad ? 0 : pg[a.n];
  if (a.items) {
#pragma unroll 1
    for (int i = blockIdx.x * PLAN_THREADS + tid; i < n_give; i += gridDim.x * PLAN_THREADS) {
      const int b = find_seq(pg, a.n, i);
      const int id = a.table[(size_t)b * a.max_blocks + (i - pg[b])];
      if (id < 0 || id >= a.n_pages) atomicOr(a.err, ERR_PAGE);
      a.free_pages[n_free + i] = id;
    }
  }
  if (a.counts && blockIdx.x == 0) {
    __syncthreads();  // lens_out may be lens
    for (int i = tid; i < a.n; i += PLAN_THREADS) a.lens_out[i] = !bad && gone[i + 1] > gone[i] ? 0 : a.lens[i];
    if (tid == 0) *a.n_free_out = n_free + n_give;
  }
}

// One launch, or, where several CTAs read what the call overwrites, a second one for the counts.
template <typename K, typename Args>
cudaError_t launch_plan(K kernel, Args a, int64_t items, bool aliased, cudaStream_t s) {
  const size_t smem = (size_t)2 * (a.n + 1) * sizeof(int);
  cudaError_t e = cudaSuccess;
  int dev = 0, nsm = 0, ctas = 1;
  // the same limit in every call: it is the kernel's, and a smaller one could come between another thread's setting and launch
  constexpr int most = 2 * (PLAN_MAX_SEQS + 1) * (int)sizeof(int);
  if (smem > 40 * 1024 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most))) return e;
  if (items > PLAN_SMALL) {
    if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev))) return e;
    const int64_t want = (items + 4 * PLAN_THREADS - 1) / (4 * PLAN_THREADS);
    ctas = want < nsm ? (int)want : nsm;
  }
  a.items = true;
  a.counts = ctas == 1 || !aliased;
  if ((e = launch_k(kernel, dim3(ctas), dim3(PLAN_THREADS), smem, s, false, a)) || a.counts) return e;
  a.items = false;
  a.counts = true;
  return launch_k(kernel, dim3(1), dim3(PLAN_THREADS), smem, s, true, a);
}

qw_status plan_dims(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks) {
  if (n_seqs < 0 || page_size < 1 || n_pages < 1 || max_blocks < 1)
    return op_fail(QW_ERR_INVALID_ARG, "bad page plan dimension");
  if (n_seqs > PLAN_MAX_SEQS) return op_fail(QW_ERR_UNSUPPORTED, "more than 16384 sequences");
  if (n_pages > 1 << 30) return op_fail(QW_ERR_UNSUPPORTED, "more than 2^30 pages");
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
  if (max_tokens > 1 << 30) return op_fail(QW_ERR_UNSUPPORTED, "more than 2^30 tokens");
  if (!free_pages || !n_free || !n_free_out || !cu_tokens || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_seqs > 0 && (!lens || !block_table || !lens_out)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (max_tokens > 0 && (!positions || !slots)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)slots & 7) return op_fail(QW_ERR_INVALID_ARG, "slots not 8-byte aligned");
  if ((st = op_check_device({lens, n_new, free_pages, n_free, block_table, lens_out, n_free_out, cu_tokens, positions,
                             slots, err_dev})))
    return st;
  const PlanArgs a{n_seqs, page_size, n_pages, max_blocks, max_tokens, lens, n_new, free_pages, n_free, block_table,
                   lens_out, n_free_out, cu_tokens, positions, (long long*)slots, err_dev, true, true};
  const cudaError_t e =
      launch_plan(page_plan_kernel, a, max_tokens, lens_out == lens || n_free_out == n_free, (cudaStream_t)cuda_stream);
  if (e)
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
  const ReleaseArgs a{n_seqs, page_size, n_pages, max_blocks, lens, done, block_table, n_free, free_pages, lens_out,
                      n_free_out, err_dev, true, true};
  const int64_t entries = (int64_t)n_seqs * max_blocks;
  const cudaError_t e = launch_plan(page_release_kernel, a, entries < n_pages ? entries : n_pages,
                                    lens_out == lens || n_free_out == n_free, (cudaStream_t)cuda_stream);
  if (e)
    return op_cuda_fail(e, "page release launch");
  return QW_OK;
}

}  // extern "C"
