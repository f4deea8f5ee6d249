// Compaction of a paged cache's pool: the live pages with the highest ids move into the lowest free ones, so that the
// pool's upper end becomes free.
//
// With n pages of which f are free, L = n - f pages are live. Holes are free ids below L, movers live ids from L on; there
// are as many of one as of the other. The i-th mover from above goes into the i-th hole from below, i < M = min(holes,
// max_moves). With F(id) the free ids below id, all numbers are local: a hole's is F(id); a mover's is the live ids above
// it, n - 1 - id - (f - F(id)); and the place of a page that is free afterwards, counted from above, is
//   f - F(id + 1)  (free before)  - max(0, M - F(id + 1)) below L  (filled)  + min(M, live ids above), below L + M  (moved).
// Three launches, each with the next one waiting (programmatic dependent launch):
//   1. marks: a bit for every page of the free list, counts per range of the pool, the lengths checked.
//   2. moves: a CTA a range sums the counts before it and ranks its pages by population counts.
//   3. tables: the entries of moved pages rewritten, their holders' counts carried along, the marks taken back.
// What bounds it: latency, three launches' chains of loads (4096 pages 11 us); a million pages 28 us, of which 2.5 are traffic: marks
// by atomics 9, ranks 11, table entries 10, each of a few loads that wait for one another.
#include "page_scan.cuh"

namespace qw {
namespace {

constexpr int CP_MARK_THREADS = 1024;  // few CTAs: each adds its counts to every range's
constexpr int CP_RANGES = 1024, CP_RANGE_MIN = 2048, CP_THREADS = 256, CP_SEG = 128;
constexpr int CP_PAD = 8;  // a range's counter has a sector of its own
constexpr size_t CP_HEAD = 64 + CP_RANGES * CP_PAD * 4;

struct CompactHead {  // of the workspace, zero between calls
  int bad;
  unsigned int ticket;
  int n_moves;  // written before it is read
  int pad[13];
  int free_in[CP_RANGES * CP_PAD];  // free pages by range
};
static_assert(sizeof(CompactHead) <= CP_HEAD, "head");

struct CompactArgs {
  int n, page, n_pages, max_blocks, max_moves, range, ranges, segs;
  const int *lens, *table, *shares, *free_pages, *n_free;
  int *table_out, *shares_out, *free_out, *src, *dst, *n_moves;
  CompactHead* head;
  uint32_t* bits;  // [n_pages / 32, rounded up] free pages, zero between calls
  int* number;     // [n_pages] a mover's number, -1 for other pages from L on
  int* err;
};

__global__ void __launch_bounds__(CP_MARK_THREADS) compact_marks_kernel(const CompactArgs a) {
  __shared__ int s_free[CP_RANGES];  // the CTA's pages by range: a million would meet at few counters
  pdl_trigger();
  for (int i = threadIdx.x; i < a.ranges; i += CP_MARK_THREADS) s_free[i] = 0;
  __syncthreads();
  const int n_free = *a.n_free, first = blockIdx.x * CP_MARK_THREADS + threadIdx.x, step = gridDim.x * CP_MARK_THREADS;
  const long long room = min((long long)a.max_blocks * a.page, 0x7fffffffll);
  int bad = 0;
  if (n_free < 0 || n_free > a.n_pages) {
    bad = ERR_CAPACITY;
  } else {
#pragma unroll 1
    for (long long i0 = first; i0 < n_free; i0 += 4ll * step) {
      int id[4];
      uint32_t was[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) id[q] = i0 + (long long)q * step < n_free ? a.free_pages[i0 + (long long)q * step] : -2;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        was[q] = 0;
        if (id[q] >= 0 && id[q] < a.n_pages) {
          was[q] = atomicOr(a.bits + (id[q] >> 5), 1u << (id[q] & 31)) >> (id[q] & 31) & 1;
          atomicAdd(s_free + id[q] / a.range, 1);
        } else if (i0 + (long long)q * step < n_free) {
          bad |= ERR_PAGE;
        }
      }
      if (was[0] | was[1] | was[2] | was[3]) bad |= ERR_PAGE;  // twice on the list
    }
  }
#pragma unroll 1
  for (int b = first; b < a.n; b += step) {
    const int len = a.lens[b];
    if (len < 0 || len > room) bad |= ERR_CAPACITY;
  }
  if (bad) {
    atomicOr(&a.head->bad, 1);
    atomicOr(a.err, bad);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.ranges; i += CP_MARK_THREADS)
    if (s_free[i]) atomicAdd(&a.head->free_in[i * CP_PAD], s_free[i]);
}

__global__ void __launch_bounds__(CP_THREADS) compact_moves_kernel(const CompactArgs a) {
  constexpr int NW = CP_THREADS / 32;
  __shared__ int s_sum[2][NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  pdl_trigger();
  pdl_wait();
  const int n = a.n_pages, n_free = *a.n_free;
  const long long first = (long long)c * a.range, end = min((long long)n, first + a.range);
  if (a.head->bad) {  // nothing moves
#pragma unroll 1
    for (long long id = first + tid; id < end; id += CP_THREADS) {
      if (a.shares && a.shares_out != a.shares) a.shares_out[id] = a.shares[id];
      if (a.free_out != a.free_pages && id < n_free) a.free_out[id] = a.free_pages[id];
    }
#pragma unroll 1
    for (int i = c * CP_THREADS + tid; i < a.max_moves; i += gridDim.x * CP_THREADS) a.src[i] = a.dst[i] = -1;
    if (c == 0 && tid == 0) *a.n_moves = a.head->n_moves = 0;
    return;
  }
  const int live = n - n_free, live_range = live / a.range;
  int before = 0, holes = 0;  // free ids before the range, below `live`
  for (int i = tid; i < a.ranges; i += CP_THREADS) {
    const int k = a.head->free_in[i * CP_PAD];
    if (i < c) before += k;
    if (i < live_range) holes += k;
  }
  for (long long w = ((long long)live_range * a.range >> 5) + tid; w <= live >> 5 && w < (n + 31) >> 5; w += CP_THREADS)
    holes += __popc(a.bits[w] & (w == live >> 5 ? (1u << (live & 31)) - 1u : 0xffffffffu));
  before = __reduce_add_sync(0xffffffffu, before);
  holes = __reduce_add_sync(0xffffffffu, holes);
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = holes;
  }
  __syncthreads();
  before = holes = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    before += s_sum[0][w];
    holes += s_sum[1][w];
  }
  const int moves = min(holes, a.max_moves);
  if (c == 0 && tid == 0) *a.n_moves = a.head->n_moves = moves;
#pragma unroll 1
  for (int i = moves + c * CP_THREADS + tid; i < a.max_moves; i += gridDim.x * CP_THREADS) a.src[i] = a.dst[i] = -1;
  // CP_WORDS words of 32 pages a warp at a time, one word a lane; the warps' counts in front
  constexpr int CP_WORDS = CP_RANGE_MIN / (32 * NW);
#pragma unroll 1
  for (long long base = first; base < end; base += CP_RANGE_MIN) {
    const long long w0 = (base >> 5) + warp * CP_WORDS;
    const uint32_t mine = lane < CP_WORDS && (w0 + lane) * 32 < end ? a.bits[w0 + lane] : 0u;
    const int count = __popc(mine);
    int incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) s_sum[0][warp] = incl;
    __syncthreads();
    int at = before;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) at += s_sum[0][w];
      before += s_sum[0][w];
    }
#pragma unroll 1
    for (int k = 0; k < CP_WORDS && (w0 + k) * 32 < end; ++k) {  // a page a lane: stores side by side
      const uint32_t word = __shfl_sync(0xffffffffu, mine, k);
      const int below = at + __shfl_sync(0xffffffffu, incl - count, k);
      const long long id64 = (w0 + k) * 32 + lane;
      if (id64 >= end) continue;
      const int id = (int)id64;
      const bool is_free = word >> lane & 1;
      const int F = below + __popc(word & ((1u << lane) - 1u));          // free ids below
      const int free_above = n_free - F - is_free, live_above = n - 1 - id - free_above;
      const bool filled = id < live && is_free && F < moves, moved = id >= live && !is_free && live_above < moves;
      if (filled) a.dst[F] = id;
      if (moved) a.src[live_above] = id;
      if (id >= live) a.number[id] = moved ? live_above : -1;
      if ((is_free && !filled) || moved) {
        const int r = free_above - (id < live ? max(0, moves - F - is_free) : 0) + (id >= live ? min(moves, live_above) : moves);
        a.free_out[r] = id;
      }
      if (a.shares && a.shares_out != a.shares && !filled) a.shares_out[id] = moved ? 0 : a.shares[id];
    }
  }
}

__global__ void __launch_bounds__(CP_THREADS) compact_tables_kernel(const CompactArgs a) {
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  const bool bad = a.head->bad;
  const int n = a.n_pages, live = bad ? n : n - *a.n_free, moves = a.head->n_moves;
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;  // (every CTA has read the head by then)
  const int first = blockIdx.x * CP_THREADS + tid, step = gridDim.x * CP_THREADS;
  for (int w = first; w < (n + 31) >> 5; w += step) a.bits[w] = 0u;
  if (a.shares)
    for (int i = first; i < moves; i += step) {
      const int from = a.src[i];
      a.shares_out[a.dst[i]] = a.shares[from];
      if (a.shares_out == a.shares) a.shares_out[from] = 0;
    }
  const bool apart = a.table_out != a.table;  // (in place, entries are checked even where nothing moves)
  const int n_tasks = a.n * a.segs;  // (the host bounds it)
#pragma unroll 1
  for (int t = blockIdx.x * (CP_THREADS / 32) + warp; t < n_tasks; t += gridDim.x * (CP_THREADS / 32)) {
    const int b = t / a.segs, j0 = (t - b * a.segs) * CP_SEG;
    const int have = bad ? 0 : pages_of(a.lens[b], a.page), end = min(apart ? a.max_blocks : have, j0 + CP_SEG);
    const size_t row = (size_t)b * a.max_blocks;
    static_assert(CP_SEG == 128, "four entries a lane");
    int id[4], k[4];  // (the three loads of an entry wait for each other, those of four entries do not)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = j0 + lane + 32 * q;
      id[q] = j < end ? a.table[row + j] : 0;
      if (j < min(have, end) && (id[q] < 0 || id[q] >= n)) atomicOr(a.err, ERR_PAGE);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) k[q] = j0 + lane + 32 * q < min(have, end) && id[q] >= live && id[q] < n ? a.number[id[q]] : -1;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (k[q] >= 0) id[q] = a.dst[k[q]];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if ((apart && j0 + lane + 32 * q < end) || k[q] >= 0) a.table_out[row + j0 + lane + 32 * q] = id[q];
  }
  __syncthreads();
  if (s_last) {
    for (int i = tid; i < a.ranges; i += CP_THREADS) a.head->free_in[i * CP_PAD] = 0;
    if (tid == 0) {
      a.head->bad = 0;
      a.head->ticket = 0;
    }
  }
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_page_compact_workspace(int32_t n_pages) {
  if (n_pages < 1 || n_pages > 1 << 30) return 0;
  const size_t words = ((size_t)n_pages + 127) / 128 * 4;
  return CP_HEAD + (words + (size_t)n_pages) * sizeof(int);
}

qw_status qw_op_page_compact(int32_t n_seqs, int32_t page_size, int32_t n_pages, int32_t max_blocks, int32_t max_moves,
                             const int32_t* lens, const int32_t* block_table, const int32_t* shares,
                             const int32_t* free_pages, const int32_t* n_free, int32_t* table_out, int32_t* shares_out,
                             int32_t* free_out, int32_t* move_src, int32_t* move_dst, int32_t* n_moves, void* workspace,
                             size_t workspace_bytes, int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  if (n_seqs < 0 || page_size < 1 || n_pages < 1 || max_blocks < 1 || max_moves < 0)
    return op_fail(QW_ERR_INVALID_ARG, "bad page compaction dimension");
  if (n_pages > 1 << 30 || max_moves > 1 << 30) return op_fail(QW_ERR_UNSUPPORTED, "more than 2^30 pages or moves");
  const int segs = (int)(((int64_t)max_blocks + CP_SEG - 1) / CP_SEG);
  if ((int64_t)n_seqs * segs > 0x7fffffff - (1 << 20)) return op_fail(QW_ERR_UNSUPPORTED, "n_seqs * max_blocks too large");
  if (!free_pages || !n_free || !free_out || !n_moves || !workspace || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (n_seqs > 0 && (!lens || !block_table || !table_out)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (max_moves > 0 && (!move_src || !move_dst)) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  if (!shares != !shares_out) return op_fail(QW_ERR_INVALID_ARG, "shares and shares_out: both or none");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  if (workspace_bytes < qw_op_page_compact_workspace(n_pages)) return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  qw_status st = op_check_device({lens, block_table, shares, free_pages, n_free, table_out, shares_out, free_out, move_src,
                                  move_dst, n_moves, workspace, err_dev});
  if (st) return st;
  int64_t range = ((int64_t)n_pages + CP_RANGES - 1) / CP_RANGES;
  range = range < CP_RANGE_MIN ? CP_RANGE_MIN : (range + 31) / 32 * 32;  // whole words
  const int ranges = (int)(((int64_t)n_pages + range - 1) / range);
  const size_t words = ((size_t)n_pages + 127) / 128 * 4;
  uint32_t* bits = (uint32_t*)((char*)workspace + CP_HEAD);
  const CompactArgs a{n_seqs, page_size, n_pages, max_blocks, max_moves, (int)range, ranges, segs,
                      lens, block_table, shares, free_pages, n_free, table_out, shares_out, free_out, move_src, move_dst, n_moves,
                      (CompactHead*)workspace, bits, (int*)(bits + words), err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  cudaError_t e;
  int dev = 0, nsm = 0;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  auto grid = [&](int64_t threads) {  // CTAs for so many threads' items
    const int64_t want = (threads + CP_THREADS - 1) / CP_THREADS;
    return dim3((unsigned)(want < 1 ? 1 : want < 4 * nsm ? want : 4 * nsm));
  };
  const int64_t most = n_pages > n_seqs ? n_pages : n_seqs, marks = (most + 2 * CP_MARK_THREADS - 1) / (2 * CP_MARK_THREADS), rows = (int64_t)n_seqs * segs * 32;
  if ((e = launch_k(compact_marks_kernel, dim3((unsigned)(marks < nsm ? marks : nsm)), dim3(CP_MARK_THREADS), 0, s, false, a)) ||
      (e = launch_k(compact_moves_kernel, dim3(ranges), dim3(CP_THREADS), 0, s, true, a)) ||
      (e = launch_k(compact_tables_kernel, grid(rows > n_pages / 32 ? rows : n_pages / 32), dim3(CP_THREADS), 0, s, true, a)))
    return op_cuda_fail(e, "page compaction launch");
  return QW_OK;
}

}  // extern "C"
