// Forks of sequences over a paged cache: sequences that go on in several continuations share their pages, and a page
// goes back to the free list when nobody holds it any more.
//
// With kids_p the children of the old sequence p, every full page of p gains kids_p - 1 holders, and a last page that is
// partly filled loses its only one where kids_p is 0: its first child keeps it, the others get fresh pages, since each
// will write there. All changes are sums, so their order does not matter:
//   1. fork_tables: every CTA counts the children in shared memory (at most 16384 sequences) and numbers the copies by
//      a prefix sum; warps then copy the children's tables and add the parents' changes to delta[page] (atomics on
//      whole numbers; rows that go on with one child add 0 and are skipped). shares + delta < 0 means that a page's
//      last holder left. A page crosses that line back and forth while others add to it, so the pages below the line
//      are counted per range of the pool as they cross it (in shared memory, then in the workspace), and the counts are right at
//      the end.
//   2. fork_pool: a CTA a range. The counts of the ranges before give the place in the free list, ballots the order
//      within the range: ascending page ids, the same in every run.
// What bounds it: latency (parents, length, table entry, count: four loads in a chain, then a second launch that
// programmatic dependent launch has waiting): 16 children of one prompt 6.7 us, 64 x 4 beams over 73000 pages 15.
#include "page_scan.cuh"

namespace qw {
namespace {

constexpr int FORK_RANGES = 1024, FORK_RANGE_MIN = 2048;  // ranges of the pool, pages of one at least
constexpr int FORK_POOL_THREADS = 256, FORK_SEG = 128;    // table entries that a warp takes: one round of loads
constexpr int FORK_PAD = 8;                               // a range's counter has a sector of its own
constexpr size_t FORK_HEAD = 64 + FORK_RANGES * FORK_PAD * 4;  // bytes before delta

struct ForkHead {  // of the workspace
  int bad, n_free, n_copies;
  unsigned int ticket;   // zero between calls
  int pad[12];
  int gone[FORK_RANGES * FORK_PAD];  // pages that lost their last holder, by range; zero between calls
};
static_assert(sizeof(ForkHead) <= FORK_HEAD, "head");

struct ForkArgs {
  int n, n_out, page, n_pages, max_blocks, range, segs;
  const int *lens, *table, *parents, *shares, *free_pages, *n_free;
  int *lens_out, *table_out, *shares_out, *free_out, *n_free_out, *copy_src, *copy_dst, *copy_len;
  ForkHead* head;
  int* delta;  // [n_pages], zero between calls
  int* err;
};

// (a negative count is taken as 0: so a page's crossings of the line sum to what its end says, and every place in the list is
// inside it)
__device__ __forceinline__ int shares_of(const ForkArgs& a, int id) { return max(a.shares[id], 0); }

__device__ __forceinline__ void hold(const ForkArgs& a, int* gone, int id, int d) {
  if (id < 0 || id >= a.n_pages) {
    atomicOr(a.err, ERR_PAGE);
    return;
  }
  const int was = shares_of(a, id) + atomicAdd(a.delta + id, d), is = was + d;
  if ((was < 0) != (is < 0)) atomicAdd(gone + id / a.range, is < 0 ? 1 : -1);
}

__global__ void __launch_bounds__(PLAN_THREADS) fork_tables_kernel(const ForkArgs a) {
  extern __shared__ int fork_sm[];
  int* kids = fork_sm;        // [n] children
  int* first = kids + a.n;    // [n] the lowest of them
  int* fresh = first + a.n;   // [n_out] number of the page that a child takes, -1: none
  __shared__ uint32_t w_sum[PLAN_THREADS / 32];
  __shared__ int s_bad, s_gone[FORK_RANGES];  // (the CTA's pages that crossed the line; thousands would meet at few counters)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  for (int i = tid; i < FORK_RANGES; i += PLAN_THREADS) s_gone[i] = 0;
  const int n_free = *a.n_free;
  const long long room = min((long long)a.max_blocks * a.page, 0x7fffffffll);
  if (tid == 0) s_bad = n_free < 0 || n_free > a.n_pages;
  for (int p = tid; p < a.n; p += PLAN_THREADS) {
    kids[p] = 0;
    first[p] = 0x7fffffff;
  }
  __syncthreads();
  for (int p = tid; p < a.n; p += PLAN_THREADS) {
    const int len = a.lens[p];
    if (len < 0 || len > room) s_bad = 1;
  }
  for (int i = tid; i < a.n_out; i += PLAN_THREADS) {
    const int p = a.parents[i];
    if (p >= 0 && p < a.n) {
      atomicAdd(kids + p, 1);
      atomicMin(first + p, i);
    } else if (p != -1 && blockIdx.x == 0) {
      atomicOr(a.err, ERR_PAGE);
    }
  }
  __syncthreads();
  auto parent = [&](int i) {
    const int p = a.parents[i];
    return p >= 0 && p < a.n ? p : -1;
  };
  auto takes = [&](int i, int p) { return p >= 0 && first[p] != i && a.lens[p] % a.page != 0; };
  const int per = (a.n_out + PLAN_THREADS - 1) / PLAN_THREADS, i0 = min(a.n_out, tid * per), i1 = min(a.n_out, i0 + per);
  uint32_t mine = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) mine += takes(i, parent(i));
  const uint32_t incl = warp_incl_scan(mine);
  if (lane == 31) w_sum[warp] = incl;
  __syncthreads();
  uint32_t at = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < PLAN_THREADS / 32; ++w) {
    if (w < warp) at += w_sum[w];
    total += w_sum[w];
  }
#pragma unroll 1
  for (int i = i0; i < i1; ++i) fresh[i] = takes(i, parent(i)) ? (int)at++ : -1;
  __syncthreads();
  const bool bad = s_bad || (int)total > n_free;
  if (blockIdx.x == 0 && tid == 0) {
    a.head->bad = bad;
    a.head->n_free = n_free;
    a.head->n_copies = (int)total;
    if (bad) atomicOr(a.err, ERR_CAPACITY);
  }
  for (int i = blockIdx.x * PLAN_THREADS + tid; i < a.n_out; i += gridDim.x * PLAN_THREADS) {
    const int p = bad ? -1 : parent(i), len = p >= 0 ? a.lens[p] : 0, no = bad ? -1 : fresh[i];
    a.lens_out[i] = len;
    const int from = no >= 0 ? a.table[(size_t)p * a.max_blocks + len / a.page] : -1;
    const int to = no >= 0 ? a.free_pages[n_free - 1 - no] : -1;
    if (no >= 0 && (from < 0 || from >= a.n_pages || to < 0 || to >= a.n_pages)) atomicOr(a.err, ERR_PAGE);
    a.copy_src[i] = from;
    a.copy_dst[i] = to;
    a.copy_len[i] = no >= 0 ? len % a.page : 0;
  }
  if (bad) return;
  // a warp takes FORK_SEG entries of a child's table, or of a parent's
  const int n_tasks = (a.n_out + a.n) * a.segs;  // (the host bounds it)
#pragma unroll 1
  for (int t = blockIdx.x * (PLAN_THREADS / 32) + warp; t < n_tasks; t += gridDim.x * (PLAN_THREADS / 32)) {
    const int r = t / a.segs, j0 = (t - r * a.segs) * FORK_SEG;
    if (r < a.n_out) {
      const int p = parent(r);
      if (p < 0) continue;
      const int have = pages_of(a.lens[p], a.page), end = min(have, j0 + FORK_SEG), no = fresh[r];
      const int *src = a.table + (size_t)p * a.max_blocks, *pick = a.free_pages + (n_free - 1 - no);
      int* dst = a.table_out + (size_t)r * a.max_blocks;
#pragma unroll 4
      for (int j = j0 + lane; j < end; j += 32) dst[j] = no >= 0 && j == have - 1 ? *pick : src[j];
    } else {
      const int p = r - a.n_out, d = kids[p] - 1;
      if (d == 0) continue;
      const int len = a.lens[p], end = min(d > 0 ? len / a.page : pages_of(len, a.page), j0 + FORK_SEG);
      const int* src = a.table + (size_t)p * a.max_blocks;
#pragma unroll 4
      for (int j = j0 + lane; j < end; j += 32) hold(a, s_gone, src[j], d);
    }
  }
  __syncthreads();
  for (int i = tid; i < FORK_RANGES; i += PLAN_THREADS)
    if (s_gone[i]) atomicAdd(&a.head->gone[i * FORK_PAD], s_gone[i]);
}

__global__ void __launch_bounds__(FORK_POOL_THREADS) fork_pool_kernel(const ForkArgs a) {
  constexpr int NW = FORK_POOL_THREADS / 32, STEPS = 8, CHUNK = STEPS * FORK_POOL_THREADS;
  __shared__ int s_before[NW], s_total[NW], s_count[STEPS * NW], s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  pdl_wait();
  const int bad = a.head->bad, n_free = a.head->n_free, keep = bad ? n_free : n_free - a.head->n_copies;
  int before = 0, total = 0;
  for (int i = tid; i < gridDim.x; i += FORK_POOL_THREADS) {
    const int n = a.head->gone[i * FORK_PAD];
    total += n;
    if (i < c) before += n;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    s_before[warp] = before;
    s_total[warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    before += s_before[w];
    total += s_total[w];
  }
  if (tid == 0) {
    if (c == 0) {
      *a.n_free_out = bad ? n_free : min(keep + total, a.n_pages);
      if (!bad && keep + total > a.n_pages) atomicOr(a.err, ERR_PAGE);  // pages that were held and on the list
    }
    s_last = atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;  // (every CTA has read the counts by then)
  }
  const long long first = (long long)c * a.range, end = min((long long)a.n_pages, first + a.range);
  int place = keep + before;
#pragma unroll 1
  for (long long base = first; base < end; base += CHUNK) {
    uint32_t gone = 0;
    unsigned lanes[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const long long id = base + s * FORK_POOL_THREADS + tid;
      bool g = false;
      if (id < end) {
        const int d = a.delta[id], now = shares_of(a, (int)id) + d;
        g = d != 0 && now < 0;
        if (d) a.delta[id] = 0;
        if (d || a.shares_out != a.shares) a.shares_out[id] = g ? 0 : now;
        if (a.free_out != a.free_pages && id < keep) a.free_out[id] = a.free_pages[id];
      }
      lanes[s] = __ballot_sync(0xffffffffu, g);
      gone |= (uint32_t)g << s;
      if (lane == 0) s_count[s * NW + warp] = __popc(lanes[s]);
    }
    __syncthreads();
    if (total) {
      int sum = 0, at[STEPS];
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          if (w == warp) at[s] = sum;
          sum += s_count[s * NW + w];
        }
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int to = place + at[s] + __popc(lanes[s] & ((1u << lane) - 1u));
        if ((gone >> s & 1) && to < a.n_pages) a.free_out[to] = (int)(base + s * FORK_POOL_THREADS + tid);
      }
      place += sum;
    }
    __syncthreads();
  }
  if (s_last) {
    for (int i = tid; i < gridDim.x; i += FORK_POOL_THREADS) a.head->gone[i * FORK_PAD] = 0;
    if (tid == 0) a.head->ticket = 0;
  }
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_page_fork_workspace(int32_t n_pages) {
  if (n_pages < 1 || n_pages > 1 << 30) return 0;
  return FORK_HEAD + (size_t)n_pages * sizeof(int);
}

qw_status qw_op_page_fork(int32_t n_seqs, int32_t n_out, int32_t page_size, int32_t n_pages, int32_t max_blocks,
                          const int32_t* lens, const int32_t* block_table, const int32_t* parents, const int32_t* shares,
                          const int32_t* free_pages, const int32_t* n_free, int32_t* lens_out, int32_t* table_out,
                          int32_t* shares_out, int32_t* free_out, int32_t* n_free_out, int32_t* copy_src,
                          int32_t* copy_dst, int32_t* copy_len, void* workspace, size_t workspace_bytes,
                          int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  if (n_seqs < 0 || n_out < 0 || page_size < 1 || n_pages < 1 || max_blocks < 1)
    return op_fail(QW_ERR_INVALID_ARG, "bad page fork dimension");
  if (n_seqs > PLAN_MAX_SEQS || n_out > PLAN_MAX_SEQS) return op_fail(QW_ERR_UNSUPPORTED, "more than 16384 sequences");
  if (n_pages > 1 << 30) return op_fail(QW_ERR_UNSUPPORTED, "more than 2^30 pages");
  const int segs = (int)(((int64_t)max_blocks + FORK_SEG - 1) / FORK_SEG);
  if ((int64_t)(n_seqs + n_out) * segs > 0x7fffffff - (1 << 20))
    return op_fail(QW_ERR_UNSUPPORTED, "(n_seqs + n_out) * max_blocks too large");
  if (!shares || !free_pages || !n_free || !shares_out || !free_out || !n_free_out || !workspace || !err_dev)
    return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_seqs > 0 && (!lens || !block_table)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_out > 0 && (!parents || !lens_out || !table_out || !copy_src || !copy_dst || !copy_len))
    return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if ((lens_out && lens_out == lens) || (table_out && table_out == block_table))
    return op_fail(QW_ERR_INVALID_ARG, "lens_out and table_out must not be the old ones");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_page_fork_workspace(n_pages)) return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  qw_status st = op_check_device({lens, block_table, parents, shares, free_pages, n_free, lens_out, table_out, shares_out,
                                  free_out, n_free_out, copy_src, copy_dst, copy_len, workspace, err_dev});
  if (st) return st;
  const int64_t least = ((int64_t)n_pages + FORK_RANGES - 1) / FORK_RANGES;
  const int range = least < FORK_RANGE_MIN ? FORK_RANGE_MIN : (int)least;
  const ForkArgs a{n_seqs,     n_out,    page_size, n_pages,    max_blocks, range,     segs,
                   lens,       block_table, parents, shares,    free_pages, n_free,    lens_out,
                   table_out,  shares_out, free_out, n_free_out, copy_src,  copy_dst,  copy_len,
                   (ForkHead*)workspace, (int*)((char*)workspace + FORK_HEAD), err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  cudaError_t e;
  int dev = 0, nsm = 0;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  const size_t smem = (size_t)(2 * n_seqs + n_out) * sizeof(int);
  // the same limit in every call: it is the kernel's, and a smaller one could come between another thread's setting and launch
  constexpr int most = 3 * PLAN_MAX_SEQS * (int)sizeof(int);
  static_assert(most + FORK_RANGES * 4 + 256 <= 232448, "shared memory");
  if (smem > 40 * 1024 && (e = cudaFuncSetAttribute(fork_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most)))
    return op_cuda_fail(e, "page fork launch");
  const int64_t want = ((int64_t)(n_seqs + n_out) * segs + PLAN_THREADS / 32 - 1) / (PLAN_THREADS / 32);
  const int ctas = want < 1 ? 1 : want < nsm ? (int)want : nsm;
  if ((e = launch_k(fork_tables_kernel, dim3(ctas), dim3(PLAN_THREADS), smem, s, false, a)) ||
      (e = launch_k(fork_pool_kernel, dim3((unsigned)(((int64_t)n_pages + range - 1) / range)), dim3(FORK_POOL_THREADS), 0, s, true, a)))
    return op_cuda_fail(e, "page fork launch");
  return QW_OK;
}

}  // extern "C"
