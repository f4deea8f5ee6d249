// Common parts of the attention of groups that share a beginning (attn_shared.cu, attn_shared_tc.cu, attn_shared_simt.cu):
// the list of tiles and its cuts, the places of partial results.
#pragma once

#include "attn_paged.cuh"

namespace qw {
namespace shared_attn {

using paged::comb_stride;
using paged::cta_of;
using paged::cut;
using paged::PA_BIAS;
using paged::OwnAttnArgs;
using paged::Range;

constexpr int SH_MAX_CTAS = 160;  // of the tensor-core kernel, one an SM; the CUDA cores' kernel takes two

// The own positions of 16-bit caches, see attn_shared_own.cu: positions of a tile, a unit's weight in tiles, units of so many
// tiles are not split, head dimensions and heads of a part. (Weights of 1 to 6 are within 1%; units of up to 4 or 8 tiles kept whole
// cost 48 sequences of 1 to 200 own positions 2 and 20%.)
constexpr int OWN_WEIGHT = 4, OWN_WHOLE = 2, OWN_WARPS = 8;
__host__ __device__ constexpr int own_rows(int hd) { return hd <= 64 ? 32 : 16; }

struct SharedHead {  // of the workspace
  int bad, each, rest, total;
};
struct SharedArgs {
  OwnAttnArgs p;  // skip: the shared positions of each sequence; state: of the positions behind them
  int n_groups;
  const int* cu;
  SharedHead* head;
  int* at;       // [n_groups] where the list has the group
  SharedHead* own_head;  // the same for the list of own positions (16-bit caches)
  int* own_at;           // [n_seqs]
  float* whole;  // [2][n_seqs][nq][comb_stride(hd)] states of units that one CTA covers, see state_of
  float* parts;  // [2 * CTAs][rows of a tile][comb_stride(HD)] of the others
};

// A unit is a tile of MT rows (sequence, head of the KV head) of one group and KV head, over the group's shared positions in
// blocks of BK. Neighbouring units read the same keys and values. A block counts as many numbers of the list as the unit has
// halves of MT rows where the kernel takes 256 rows (their products are what bounds it), else one.
struct Unit {
  int g, lo, rows, nt, pre, nb;  // the group: first sequence, rows of a KV head, their tiles, shared positions, their blocks
  int u, t, v, c;                // unit kv * nt + tile of the group, block, where the list has the unit, numbers a block
};
template <int MT>
__host__ __device__ __forceinline__ int block_cost(int rows, int tile) { return MT == 256 && rows - tile * MT > MT / 2 ? 2 : 1; }
// A unit's ends (queries, first products, states) count like 4 blocks before it, 2 where a block is long (the CUDA cores). Measured
// with 2, 4 and 8: 256 sequences of 16383 shared positions 94, 92, 89 us (bf16, blocks of cost 2), 136, 134, 136 (fp32 callers);
// 256 prompts of one sequence 231, 226, 235 (cost 1); an fp32 cache 32.6, 32.9, 34.7. (bf16 with probabilities of one piece; with
// two, at these weights, 101 and 248.)
template <int MT>
__host__ __device__ constexpr int unit_weight(int cost) { return MT == 64 ? 2 : 4 * cost; }
// numbers of one KV head's units
template <int MT>
__host__ __device__ __forceinline__ int head_numbers(int rows, int nt, int nb) {
  const int full = block_cost<MT>(MT, 0), last = block_cost<MT>(rows, nt - 1);
  return (nt - 1) * (unit_weight<MT>(full) + full * nb) + unit_weight<MT>(last) + last * nb;
}

// The group g; its numbers in the list, 0 if it has nothing to do. bad: its bounds or its length are out of range.
template <int MT, int BK>
__device__ __forceinline__ int load_group(const SharedArgs& a, int g, Unit& p, bool& bad) {
  const int lo = __ldg(a.cu + g), hi = __ldg(a.cu + g + 1);
  bad = lo < 0 || hi < lo || hi > a.p.n_seqs;
  p.g = g;
  if (bad || hi == lo) return 0;
  const long long room = (long long)a.p.max_blocks * a.p.page;
  int pre = __ldg(a.p.skip + lo);
  if (pre < 0 || pre > room) pre = 0;  // (the kernel of the other positions reports it)
  p.lo = lo;
  p.rows = (hi - lo) * (a.p.nq / a.p.nkv);
  p.nt = (p.rows + MT - 1) / MT;
  p.pre = pre;
  p.nb = (pre + BK - 1) / BK;
  p.c = block_cost<MT>(p.rows, 0);
  return p.nb ? a.p.nkv * head_numbers<MT>(p.rows, p.nt, p.nb) : 0;
}

// The next unit; false behind the list's end `end`.
template <int MT, int BK>
__device__ __forceinline__ bool next_unit(const SharedArgs& a, int end, Unit& p) {
  p.t = 0;
  p.v += unit_weight<MT>(p.c) + p.c * p.nb;
  if (p.v >= end) return false;
  if (++p.u < a.p.nkv * p.nt) {
    p.c = block_cost<MT>(p.rows, p.u % p.nt);
    return true;
  }
  p.u = 0;
  bool bad;
  int g = p.g;
  while (++g < a.n_groups && !load_group<MT, BK>(a, g, p, bad)) {}
  return true;
}

// the unit's blocks from p.t on that lie before the list's end `end`
template <int MT>
__device__ __forceinline__ int blocks_of(const Unit& p, int end) { return min(p.nb, (end - p.v - unit_weight<MT>(p.c) + p.c - 1) / p.c) - p.t; }

// The CTA's range of the list and its first unit; CTA 0 leaves the cuts and the groups' places for the join. A cut that
// falls on a unit's weight moves to the unit's beginning, one inside a block to the next block. scratch: shared memory, free
// again when the call returns.
constexpr int SH_SCRATCH = 256;
template <int MT, int BK, int NT>
__device__ __forceinline__ Range find_groups(const SharedArgs& a, Unit& first, void* scratch) {
  Unit* s_at = (Unit*)scratch;
  int* w_sum = (int*)(s_at + 2);
  static_assert(2 * sizeof(Unit) + NT / 32 * sizeof(int) <= SH_SCRATCH, "scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_groups + NT - 1) / NT, g0 = min(a.n_groups, tid * per), g1 = min(a.n_groups, g0 + per);
  int mine = 0, bad = tid == 0 && (a.cu[0] != 0 || a.cu[a.n_groups] != a.p.n_seqs);
  Unit p{};
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    bool b;
    mine += load_group<MT, BK>(a, g, p, b);
    bad |= b;
  }
  bad = __syncthreads_or(bad);
  if (bad) mine = 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) w_sum[warp] = incl;
  __syncthreads();
  int base = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += w_sum[w];
    total += w_sum[w];
  }
  // Every range has a number of each half of a block: a range of the second half alone would be empty, and the join adds the
  // parts of all ranges between a unit's first block and its last.
  const int ctas = min((int)gridDim.x, MT == 256 ? total / 2 : total), c = blockIdx.x;  // (a list that is not empty has 5 numbers)
  Range r{0, 0, 0, 0};
  if (ctas) {
    r.each = total / ctas;
    r.rest = total - r.each * ctas;
  }
  if (c == 0 && tid == 0) {
    *a.head = SharedHead{bad, r.each, r.rest, total};
    if (bad) atomicOr(a.p.err, ERR_PAGE);
  }
  if (mine) {
    int at = base;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      bool b;
      const int n = load_group<MT, BK>(a, g, p, b);
      if (c == 0) a.at[g] = at;
      if (c < ctas)
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const int x = cut(r, c + k);
          if (x < at || x >= at + n) continue;
          const int per_head = n / a.p.nkv, kv = (x - at) / per_head, big = unit_weight<MT>(block_cost<MT>(MT, 0)) + block_cost<MT>(MT, 0) * p.nb;
          const int in = x - at - kv * per_head, tile = min(in / big, p.nt - 1);
          p.u = kv * p.nt + tile;
          p.v = at + kv * per_head + tile * big;
          p.c = block_cost<MT>(p.rows, tile);
          p.t = (max(0, x - p.v - unit_weight<MT>(p.c)) + p.c - 1) / p.c;
          s_at[k] = p;
        }
      at += n;
    }
  }
  __syncthreads();
  if (c < ctas) {
    first = s_at[0];
    auto place = [](const Unit& x) { return x.v + (x.t ? unit_weight<MT>(x.c) + x.c * x.t : 0); };
    r.begin = place(first);
    r.end = c + 1 == ctas ? total : place(s_at[1]);
    if (first.t == first.nb) next_unit<MT, BK>(a, r.end, first);
  }
  __syncthreads();
  return r;
}

// Row i of the group's KV head: its sequence and head, and whether the sequence takes part: it shares what the group's first
// one does, and is no shorter.
struct Row {
  int b, h;
  bool in;
};
__device__ __forceinline__ Row row_of(const SharedArgs& a, const Unit& p, int kv, int i) {
  Row r{0, 0, false};
  if (i >= p.rows) return r;
  const int grp = a.p.nq / a.p.nkv, s = i / grp;
  r.b = p.lo + s;
  r.h = kv * grp + (i - s * grp);
  r.in = __ldg(a.p.skip + r.b) == p.pre && __ldg(a.p.lens + r.b) >= p.pre;
  return r;
}

// Where a row's state goes, i its number in the tile: part slots are 2 c for the unit that CTA c begins with, 2 c + 1 for
// one that it begins later and does not finish. second: the state of the odd blocks, where a tile's halves take the even and
// the odd blocks of the same rows (i is then of the upper half, too).
template <int MT, int HD>
__device__ __forceinline__ float* state_of(const SharedArgs& a, const Range& r, const Unit& p, bool whole, const Row& row, int i, bool second = false) {
  if (whole) return a.whole + ((size_t)((second ? a.p.n_seqs : 0) + row.b) * a.p.nq + row.h) * comb_stride(a.p.hd);
  const int slot = 2 * blockIdx.x + (cut(r, blockIdx.x) < p.v ? 1 : 0);
  return a.parts + ((size_t)slot * MT + i) * comb_stride(HD);
}

// Byte offset in the caches of position pos of the unit's shared part, or -1: none, or a bad page.
template <typename T>
__device__ __forceinline__ long long position_of(const SharedArgs& a, const Unit& p, int kv, int pos) {
  if (pos >= p.pre) return -1;
  const int blk = pos / a.p.page, id = __ldg(a.p.table + (size_t)p.lo * a.p.max_blocks + blk);
  if (id < 0 || id >= a.p.n_pages) {
    atomicOr(a.p.err, ERR_PAGE);
    return -1;
  }
  return (id * a.p.page_stride + kv * a.p.head_stride + (long long)(pos - blk * a.p.page) * a.p.pos_stride) * (int)sizeof(T);
}

// rows of a tile, positions of a block and padded head dimensions of the kernel that a shape takes
struct Geometry {
  int mt, bk, hd, ctas;
};
inline Geometry geometry(int cache_dtype, int io_dtype, int hd, int nsm) {
  const int n = nsm < SH_MAX_CTAS ? nsm : SH_MAX_CTAS;
  if (cache_dtype != QW_F32 && hd <= 128) return Geometry{io_dtype == QW_F32 ? 128 : 256, 128, hd <= 64 ? 64 : 128, n};
  return Geometry{64, 64, hd <= 64 ? 64 : hd <= 128 ? 128 : 256, hd <= 128 ? 2 * n : n};
}

// 16-bit caches, heads of at most 128 dimensions: attn_shared_tc.cu for fp32 callers, attn_shared_pair.cu for 16-bit ones;
// attn_shared_simt.cu: the others
cudaError_t launch_shared_tc(const qw_paged_kv& cache, int ctas, const SharedArgs& a, cudaStream_t s);
cudaError_t launch_shared_pair(const qw_paged_kv& cache, int ctas, const SharedArgs& a, cudaStream_t s);
cudaError_t launch_own(int cache_dtype, int io_dtype, int ctas, const SharedArgs& a, cudaStream_t s);
cudaError_t launch_shared_simt(int cache_dtype, int io_dtype, int ctas, const SharedArgs& a, cudaStream_t s);

}  // namespace shared_attn
}  // namespace qw
