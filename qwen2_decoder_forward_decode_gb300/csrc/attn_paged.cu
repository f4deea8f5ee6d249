// Decode attention over a paged key-value cache: one query token per sequence ("LLM Speedrun:
// Architecture": Attention, Grouped Query Attention).
//
// Mathematics: one pass over the positions with a running maximum m, sum l and output o per query head.
// A tile of scores s (in base 2) moves them to m' = max(m, s), l' = l 2^(m - m') + sum 2^(s - m'),
// o' = o 2^(m - m') + sum 2^(s - m') V. States of disjoint position sets merge the same way, so the
// positions may be split at will: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// What bounds it: every key and value is used by the few query heads of its group only, about 2 flops
// per byte and head, so HBM. Everything else serves to keep loads in flight on every SM:
//   - One CTA per SM. The tiles of all sequences and KV heads form one list (sequence, unit, tile),
//     cut into equal consecutive ranges, one per CTA, from the lengths on the device: ragged batches
//     and single long sequences load every SM alike, and a captured graph follows the lengths.
//   - Each of the CTA's 8 warps owns the same rows of every tile and copies them itself (cp.async,
//     16 bytes a lane) into its own ring of stages, looking the rows' pages up one tile ahead. Warps
//     meet only where a unit ends; the ring runs on into the next unit meanwhile.
//   - A unit that one CTA covers is finished there. The parts of a split unit go to the workspace; the
//     last CTA to arrive merges them, in groups of PA_GROUP CTAs first where there are more (a single
//     CTA reading every part of a long sequence would be bound by latency). The order of every sum is
//     fixed by the lengths, so results repeat bit by bit.
#include "common.cuh"
#include "op_util.h"

#include <math.h>

#include <cmath>
#include <type_traits>

namespace qw {
namespace {

constexpr int PA_MAX_HD = 256;
constexpr int PA_MAX_CTAS = 160;   // persistent CTAs the workspace has room for
constexpr int PA_WHOLE = 3;         // units of at most so many tiles are not split
constexpr int PA_GROUP = 10;       // parts merged at once: 152 CTAs are at most 16 groups
constexpr int PA_JOIN = 20;        // states a join holds: two groups, or the group sums of two units (18)
constexpr float PA_BIAS = 10.f;    // probabilities are kept times 2^10: their fp16 halves stay normal
                                   // numbers down to 2^-24 of the largest
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

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
  unsigned int* counters;  // [2][2 * PA_MAX_CTAS], zero between calls
  float* part;             // [2 * PA_MAX_CTAS][HB][HD + 8]
  int* err;
};

__host__ __device__ constexpr int comb_stride(int hd) { return hd + 8; }  // o, then m and l

// two elements at an even index
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const f16* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
__device__ __forceinline__ float2 load2(const bf16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(bf_lo(u), bf_hi(u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
// 16 bytes into shared memory; zeros instead where !ok
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldmatrix_x4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_t(float* c, const uint32_t* a, uint32_t b0, uint32_t b1, f16) { mma16816(c, a, b0, b1); }
__device__ __forceinline__ void mma_t(float* c, const uint32_t* a, uint32_t b0, uint32_t b1, bf16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T> struct Pair;
template <> struct Pair<f16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_half2(a, b); }
  static __device__ __forceinline__ float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
};
template <> struct Pair<bf16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) { return make_float2(bf_lo(u), bf_hi(u)); }
};
template <typename IO>
__device__ __forceinline__ void store4(IO* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(Pair<IO>::pack(v.x, v.y), Pair<IO>::pack(v.z, v.w));
}
// a, b as a sum of N pieces of type T, most significant first; each piece rounds what the ones before
// left, so N pieces carry N times T's digits
template <typename T, int N>
__device__ __forceinline__ void split(float a, float b, uint32_t* piece) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    piece[i] = Pair<T>::pack(a, b);
    const float2 r = Pair<T>::unpack(piece[i]);
    a -= r.x;
    b -= r.y;
  }
}

// ---- the list of tiles ---------------------------------------------------------------------------------

__device__ __forceinline__ int seq_len(const PagedAttnArgs& a, int b, bool& bad) {
  const long long room = (long long)a.max_blocks * a.page;
  const int len = __ldg(a.lens + b);
  bad = len < 0 || len > room;
  return len < 0 ? 0 : len > room ? (int)room : len;
}
__device__ __forceinline__ int seq_len(const PagedAttnArgs& a, int b) {
  bool bad;
  return seq_len(a, b, bad);
}

// The list weighs a unit's end (the merge of the warps, the next queries) like V tiles, in front of its own.
// A place is tile t of nt of unit u of sequence b; v: where the list has the unit. All numbers of the
// list fit 31 bits (the host refuses shapes that could hold more).
struct Place {
  int b, u, t, nt, len, v;
};

// The next tile; false behind the list's end `end` (as a number of the list).
template <int TILE, int V>
__device__ __forceinline__ bool advance(const PagedAttnArgs& a, int n_units, int end, Place& p) {
  if (++p.t < p.nt) return p.v + V + p.t < end;
  p.t = 0;
  p.v += V + p.nt;
  if (p.v >= end) return false;
  if (++p.u < n_units) return true;
  p.u = 0;
  do {
    p.len = seq_len(a, ++p.b);
    p.nt = (p.len + TILE - 1) / TILE;
  } while (p.nt == 0 && p.b + 1 < a.n_seqs);
  return true;
}

// The list cut into `ctas` consecutive ranges: the first `rest` of them have each + 1 numbers. A cut that
// falls on a unit's weight, or inside a unit of at most PA_WHOLE tiles, moves to the unit's beginning:
// short units are never split, since joining the parts costs about 3 us, a tile more in one CTA
// less than 1 us.
struct Range {
  int each, rest, begin, end;  // begin, end: this CTA's range, moved
};
__device__ __forceinline__ int cut(const Range& r, int c) { return r.each * c + min(c, r.rest); }
// the last CTA c with cut(c) <= x
__device__ __forceinline__ int cta_of(const Range& r, int x) {
  const int big = r.rest * (r.each + 1), from = x < big ? 0 : r.rest;
  return from + (x - (x < big ? 0 : big)) / (r.each + (x < big ? 1 : 0));
}

// The CTA's range and its first place. Every CTA sums the sequences' tiles itself (L2 serves the lengths).
template <typename IO, int TILE, int V, int NT>
__device__ __forceinline__ Range find_range(const PagedAttnArgs& a, int n_units, Place& first) {
  __shared__ int w_sum[NT / 32];
  __shared__ Place s_at[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + NT - 1) / NT, b0 = min(a.n_seqs, tid * per), b1 = min(a.n_seqs, b0 + per);
  int mine = 0, empty = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    bool bad;
    const int len = seq_len(a, b, bad);
    if (len) mine += V + (len + TILE - 1) / TILE;
    empty |= len == 0;
    if (bad && blockIdx.x == 0) atomicOr(a.err, ERR_PAGE);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) w_sum[warp] = incl;
  empty = __syncthreads_or(empty);
  if (empty) {  // sequences of length 0 have no tile: out 0, lse -inf, spread over the CTAs
    const int width = a.nq * a.hd;
#pragma unroll 1
    for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
      if (seq_len(a, b) > 0) continue;
#pragma unroll 1
      for (int i = 4 * tid; i < width; i += 4 * NT) store4((IO*)a.out + b * a.out_stride + i, make_float4(0.f, 0.f, 0.f, 0.f));
      if (a.lse)
#pragma unroll 1
        for (int h = tid; h < a.nq; h += NT) a.lse[(size_t)b * a.nq + h] = -INFINITY;
    }
  }
  int base = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += w_sum[w];
    total += w_sum[w];
  }
  base *= n_units;
  mine *= n_units;
  total *= n_units;
  const int ctas = min((int)gridDim.x, total), c = blockIdx.x;
  Range r{0, 0, 0, 0};
  if (c < ctas) {
    r.each = total / ctas;
    r.rest = total - r.each * ctas;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {  // the places of the range's two cuts
      const int x = cut(r, c + k);
      int at = base;
      if (x < base || x >= base + mine) continue;
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const int len = seq_len(a, b), nt = (len + TILE - 1) / TILE, unit = nt ? V + nt : 0;
        if (x < at + unit * n_units) {
          const int u = (x - at) / unit, v = at + u * unit;
          s_at[k] = Place{b, u, nt <= PA_WHOLE ? 0 : max(0, x - v - V), nt, len, v};
          break;
        }
        at += unit * n_units;
      }
    }
  }
  __syncthreads();
  if (c < ctas) {
    first = s_at[0];
    r.begin = first.v + (first.t ? V + first.t : 0);
    r.end = c + 1 == ctas ? total : s_at[1].v + (s_at[1].t ? V + s_at[1].t : 0);
  }
  return r;
}

// ---- the rows of a tile ----------------------------------------------------------------------------------

// Each warp's rows of a tile, requested by the warp itself. Stage layout: K [RW][HD], V [RW][HD] of T, the
// 16-byte chunks of row r permuted by chunk ^ (r & 7), so that 8 rows' same chunk lie in distinct banks.
template <typename T, int HD, int RW, int NW>
struct Loader {
  static constexpr int TILE = RW * NW, CH = HD * (int)sizeof(T) / 16, CE = 16 / (int)sizeof(T);
  static constexpr int STAGE = 2 * RW * HD * (int)sizeof(T);
  static constexpr int V = NW * STAGE >= 65536 ? 1 : 65536 / (NW * STAGE);  // a unit's end costs about what 64 KB do
  static __device__ __forceinline__ uint32_t at(int row, int chunk) { return (uint32_t)(row * CH + (chunk ^ (row & 7 & (CH - 1)))) * 16; }
  static_assert((CH & (CH - 1)) == 0, "chunks are permuted by exclusive or");
  // byte offset of the lane's row (lanes 0 .. RW - 1) in the caches, or -1: no such row
  static __device__ __forceinline__ long long row(const PagedAttnArgs& a, const Place& p, int n_hb, int warp, int lane) {
    const int j = p.t * TILE + warp * RW + lane;
    if (lane >= RW || j >= p.len) return -1;
    const int blk = j / a.page, id = __ldg(a.table + (size_t)p.b * a.max_blocks + blk);
    if (id < 0 || id >= a.n_pages) {
      if (p.u == 0) atomicOr(a.err, ERR_PAGE);
      return -1;
    }
    return (id * a.page_stride + (p.u / n_hb) * a.head_stride + (long long)(j - blk * a.page) * a.pos_stride) * (int)sizeof(T);
  }
  // Requests the rows of mask (a bit per row; zeros for the others). The lane copies chunk lane % CH of
  // every (32 / CH)-th row of K and V; k, v: the caches at the lane's chunk; col: whether the head has it.
  static __device__ __forceinline__ void request(const char* k, const char* v, long long row_off, uint32_t mask, uint32_t stage, int lane,
                                                 bool col, int hd) {
    constexpr int RP = CH >= 32 ? 1 : 32 / CH, CP = CH >= 32 ? CH / 32 : 1;  // rows a step, chunks a row and lane
    const int ch0 = CH >= 32 ? lane : lane % CH, r0 = CH >= 32 ? 0 : lane / CH;
    if (row_off < 0) row_off = 0;
#pragma unroll
    for (int i = 0; i < RW / RP; ++i) {
      const int r = i * RP + r0;
      const long long off = __shfl_sync(0xffffffffu, row_off, r);
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const bool ok = (mask >> r & 1) && (CP > 1 ? (ch0 + 32 * c) * CE < hd : col);
        const uint32_t dst = stage + at(r, ch0 + 32 * c);
        cp_async16_or_zero(dst, k + off + 512 * c, ok);
        cp_async16_or_zero(dst + RW * CH * 16, v + off + 512 * c, ok);
      }
    }
  }
};

// ---- the end of a unit -------------------------------------------------------------------------------------

// All code that runs once per unit or per CTA is kept short (loops, one out-of-line join): a first version
// with everything inlined and unrolled was 130 KB per kernel, and its instruction misses cost 8 us at
// every unit's end and 10 us in the join.
template <typename IO, int HB, int HD, int NT>
struct Finish {
  static constexpr int CS = comb_stride(HD), N4 = HB * HD / 4;

  struct Acc {  // 4 output elements of one head
    float4 o;
    float m, l;
  };
  // Sum of n states [HB][CS] in shared memory at elements d .. d + 3 of head h, in their order.
  static __device__ __noinline__ Acc sum(const float* s, int n, int h, int d) {
    s += h * CS;
    float top = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < n; ++i) top = fmaxf(top, s[i * HB * CS + HD]);
    const float ref = top == -INFINITY ? 0.f : top;
    Acc a{make_float4(0.f, 0.f, 0.f, 0.f), top, 0.f};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(s + i * HB * CS + d);
      const float2 ml = *reinterpret_cast<const float2*>(s + i * HB * CS + HD);
      const float w = ex2(ml.x - ref);
      a.o.x = fmaf(w, x.x, a.o.x);
      a.o.y = fmaf(w, x.y, a.o.y);
      a.o.z = fmaf(w, x.z, a.o.z);
      a.o.w = fmaf(w, x.w, a.o.w);
      a.l = fmaf(w, ml.y, a.l);
    }
    return a;
  }

  static __device__ __forceinline__ void write_out(const PagedAttnArgs& a, const Place& p, int n_hb, int h, int d, const Acc& s) {
    const int group = a.nq / a.nkv, g = p.u / n_hb, hg = (p.u - g * n_hb) * HB + h;
    if (hg >= group || d >= a.hd) return;
    const int head = g * group + hg;
    const float inv = 1.f / s.l;  // (l = 0: every score was -inf, and 0 / 0 is the formula's NaN)
    store4((IO*)a.out + p.b * a.out_stride + head * a.hd + d, make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv));
    if (d == 0 && a.lse) a.lse[(size_t)p.b * a.nq + head] = (s.m - PA_BIAS + log2f(s.l)) * LN2;
  }
  static __device__ __forceinline__ void put(float* slot, int h, int d, const Acc& s) {
    *reinterpret_cast<float4*>(slot + h * CS + d) = s.o;
    if (d == 0) *reinterpret_cast<float2*>(slot + h * CS + HD) = make_float2(s.m, s.l);
  }

  // Part slots: a CTA's range cuts at most two units, the one it begins with (slot 2 c) and the one that it
  // begins itself and does not finish (slot 2 c + 1, or 2 c if its range begins with it).
  static __device__ __forceinline__ int slot_of(const Range& r, const Place& p, int c) { return 2 * c + (cut(r, c) < p.v ? 1 : 0); }
  static __device__ __forceinline__ float* slot_ptr(const PagedAttnArgs& a, int slot) { return a.part + (size_t)slot * HB * CS; }

  // The CTA's state of the unit at p (comb: [NW][HB][CS] in shared memory, one per warp), covering tiles
  // [t0, t1) of it. All threads call it; comb may be written again afterwards. True if the unit is split:
  // its part then lies in the workspace, for join().
  template <int NW>
  static __device__ __forceinline__ bool unit(const PagedAttnArgs& a, const Range& r, const Place& p, int n_hb, const float* comb,
                                              int t0, int t1) {
    __syncthreads();
    const bool whole = t0 == 0 && t1 == p.nt;
    float* slot = slot_ptr(a, slot_of(r, p, blockIdx.x));
#pragma unroll 1
    for (int i4 = threadIdx.x; i4 < N4; i4 += NT) {
      const int h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
      const Acc s = sum(comb, NW, h, d);
      if (whole) write_out(a, p, n_hb, h, d, s);
      else put(slot, h, d, s);
    }
    __syncthreads();
    return !whole;
  }

  // Joins the CTA's split units (at most two, places pend[0 .. n)), both at once: announces its parts, and
  // merges a unit's parts if it is the last to: first those of PA_GROUP consecutive CTAs, then the groups'
  // sums. The parts are fetched into shared memory (buf, all of the kernel's) together. Done once at
  // the CTA's end: an announcement takes a memory fence and an atomic's round trip, about 1 us, the merge
  // of a level 2 us.
  template <int V>
  static __device__ __forceinline__ void join(const PagedAttnArgs& a, const Range& r, const Place* pend, int n, int n_hb, float* buf) {
    constexpr int S4 = HB * CS / 4;
    // what is merged next: states of CTAs from, from + step, ...; the unit's first slot; its CTAs and groups
    __shared__ int s_from[2], s_step[2], s_count[2], s_first[2], s_c0[2], s_groups[2], s_last[2];
    const int c = blockIdx.x, w = threadIdx.x / 32;
    const bool speaker = threadIdx.x % 32 == 0 && w < n;
    if (threadIdx.x < 2) s_last[threadIdx.x] = s_count[threadIdx.x] = 0;
    __syncthreads();
    if (speaker) {
      const Place& p = pend[w];
      const int c0 = cta_of(r, p.v + V), c1 = cta_of(r, p.v + V + p.nt - 1), g0 = c - (c - c0) % PA_GROUP;
      s_c0[w] = c0;
      s_from[w] = g0;
      s_step[w] = 1;
      s_count[w] = min(PA_GROUP, c1 - g0 + 1);
      s_first[w] = slot_of(r, p, c0);
      s_groups[w] = (c1 - c0) / PA_GROUP + 1;
    }
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
      if (speaker && (level == 0 || s_last[w])) {
        const int slot = level || s_from[w] == s_c0[w] ? s_first[w] : 2 * s_from[w];
        if (level) {
          s_from[w] = s_c0[w];
          s_step[w] = PA_GROUP;
          s_count[w] = s_groups[w];
        }
        unsigned int* counter = a.counters + level * 2 * PA_MAX_CTAS + slot;
        __threadfence();  // (the CTA's parts, written before the last barrier)
        s_last[w] = atomicAdd(counter, 1u) == (unsigned)s_count[w] - 1u;
        if (s_last[w]) *counter = 0u;
        __threadfence();
      }
      __syncthreads();
      const int n0 = s_last[0] ? s_count[0] : 0, n1 = s_last[1] ? s_count[1] : 0;
      if (n0 + n1 == 0) return;
#pragma unroll 1
      for (int part = w; part < n0 + n1; part += NT / 32) {  // a warp a state
        const int k = part >= n0, cta = s_from[k] + (part - (k ? n0 : 0)) * s_step[k];
        const float* src = slot_ptr(a, cta == s_c0[k] ? s_first[k] : 2 * cta);
        float* dst = buf + part * HB * CS;
#pragma unroll 4
        for (int i = threadIdx.x % 32; i < S4; i += 32) cp_async16(dst + i * 4, src + i * 4);
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
      const bool done0 = level || s_groups[0] == 1, done1 = n1 == 0 || level || s_groups[1] == 1;
#pragma unroll 1
      for (int i = n0 ? threadIdx.x : N4 + threadIdx.x; i < (n1 ? 2 * N4 : N4); i += NT) {
        const int k = i >= N4, i4 = i - k * N4, h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
        const Acc s = sum(buf + (k ? n0 * HB * CS : 0), k ? n1 : n0, h, d);
        if (k ? done1 : done0) write_out(a, pend[k], n_hb, h, d, s);
        else put(slot_ptr(a, s_from[k] == s_c0[k] ? s_first[k] : 2 * s_from[k]), h, d, s);  // the group's first slot
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        if (done0) s_last[0] = 0;
        if (done1) s_last[1] = 0;
      }
      __syncthreads();
    }
  }
};

// ---- 16-bit caches on the tensor cores -----------------------------------------------------------------------
//
// A unit is a KV head with HB of its query heads. S = Q K^T and O += P V by mma.sync m16n8k16 with the
// query heads as the 16 rows: the bound is HBM (tcgen05's M = 64 rows would idle for groups of at most
// 16), and the products must not lose an fp32 caller's digits. Queries and probabilities are therefore
// fed as sums of pieces of the cache's type: with HB = 8, rows 0 - 7 hold the first piece and rows
// 8 - 15 the second, so two pieces cost what one does; bf16 caches of fp32 callers take a third piece
// (8 digits each) as a second product. Groups of more than 8 heads use HB = 16, one product per piece.
template <typename T, int HD, int HB, typename IO>
struct MmaCfg {
  static constexpr bool F32IO = std::is_same<IO, float>::value;
  static constexpr int NW = 8, RW = 16, NT = NW * 32;
  static constexpr bool three = F32IO && sizeof(T) == 2 && !std::is_same<T, f16>::value;
  static constexpr int NQ = !F32IO ? 1 : three ? 3 : 2, NP = three ? 3 : 2;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB) / (NW * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;  // stages of a warp's ring
  static constexpr int SMEM = NS * NW * Ld::STAGE + COMB;
};

template <typename T, int HD, int HB, typename IO>
__global__ void __launch_bounds__(256, 1) paged_mma_kernel(const PagedAttnArgs a) {
  using C = MmaCfg<T, HD, HB, IO>;
  using Ld = typename C::Ld;
  using Fin = Finish<IO, HB, HD, C::NT>;
  constexpr int NW = C::NW, NS = C::NS, NQ = C::NQ, NP = C::NP, CS = comb_stride(HD), TILE = Ld::TILE, V = Ld::V;
  using Raw = typename std::conditional<C::F32IO, float2, uint32_t>::type;  // two query elements
  constexpr int NKK = HD / 16, NA = HB == 8 ? (NQ + 1) / 2 : NQ, NPA = HB == 8 ? (NP + 1) / 2 : NP;  // products per step
  static_assert(NS >= 2 && C::SMEM >= PA_JOIN * HB * CS * 4, "the ring, and the parts of a join in its place");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[NW][NS];  // rows of a stage that exist
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * NW * Ld::STAGE);
  const uint32_t ring = smem_addr(pa_smem) + warp * NS * Ld::STAGE;
  Place ld;
  const Range r = find_range<IO, TILE, V, C::NT>(a, n_units, ld);
  if (r.begin >= r.end) return;
  Place p = ld;
  bool more = true;  // tiles to request
  long long row_off = Ld::row(a, ld, n_hb, warp, lane);
  int ld_stage = 0;
  const bool col = lane % Ld::CH * Ld::CE < a.hd;
  const char *kl = (const char*)a.k + lane % Ld::CH * 16, *vl = (const char*)a.v + lane % Ld::CH * 16;
  auto load_next = [&]() {  // requests the tile at ld and looks up the rows of the one after it
    if (more) {
      const uint32_t mask = __ballot_sync(0xffffffffu, row_off >= 0);
      Ld::request(kl, vl, row_off, mask, ring + ld_stage * Ld::STAGE, lane, col, a.hd);
      if (lane == 0) s_mask[warp][ld_stage] = mask;
      more = advance<TILE, V>(a, n_units, r.end, ld);
      if (more) row_off = Ld::row(a, ld, n_hb, warp, lane);
    }
    cp_commit();
    if (++ld_stage == NS) ld_stage = 0;
  };
  int stage = 0, ahead = NS - 1;  // tiles still to be requested before the first is used
  Place pend[2];
  int n_pend = 0;
  for (bool left = true; left;) {
    const int t0 = p.t, t1 = min(p.nt, r.end - p.v - V);
    // the unit's queries, columns 2 tig, 2 tig + 1 and 2 tig + 8, 2 tig + 9 of every 16: requested here, used
    // after the first tile's requests
    Raw xq[HB / 8][NKK][2];
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      const int g = p.u / n_hb, h = (p.u - g * n_hb) * HB + gid + 8 * half;
      const IO* q = (const IO*)a.q + p.b * a.q_stride + (g * group + h) * a.hd + 2 * tig;
#pragma unroll
      for (int i = 0; i < 2 * NKK; ++i)
        xq[half][i / 2][i % 2] = h < group && i * 8 < a.hd ? *reinterpret_cast<const Raw*>(q + i * 8) : Raw{};
    }
    bool fresh = true;
    uint32_t qa[NA][NKK][4];  // A fragments: pieces of rows gid and gid + 8
    float sc[2];
    float o[HD / 8][4], m[HB / 8], l[HB / 8];
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
    for (int h = 0; h < HB / 8; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll 1
    for (int t = t0; t < t1;) {
      load_next();  // into the stage that the last tile used
      if (ahead) {
        --ahead;
        continue;
      }
      ++t;
      cp_wait<NS - 1>();
      __syncwarp();
      if (fresh) {
        fresh = false;
#pragma unroll
        for (int half = 0; half < HB / 8; ++half) {
          float up = 1.f, down = 1.f;
          if constexpr (C::F32IO) {
            // fp32 queries times a power of two that puts the row's largest at 2^10: the pieces stay normal
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NKK; ++i) top = fmaxf(top, fmaxf(fabsf(xq[half][i / 2][i % 2].x), fabsf(xq[half][i / 2][i % 2].y)));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = (int)(__float_as_uint(top) >> 23) - 127;
            if (ex > -100 && ex < 100) {
              up = __uint_as_float((uint32_t)(127 + 10 - ex) << 23);
              down = __uint_as_float((uint32_t)(127 - 10 + ex) << 23);
            }
          }
          sc[half] = a.scale * LOG2E * down;
#pragma unroll
          for (int kk = 0; kk < NKK; ++kk)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t piece[4];
              if constexpr (C::F32IO) split<T, NQ>(xq[half][kk][c].x * up, xq[half][kk][c].y * up, piece);
              else piece[0] = xq[half][kk][c];
#pragma unroll
              for (int i = 0; i < NQ; ++i) qa[HB == 8 ? i / 2 : i][kk][2 * c + (HB == 8 ? i & 1 : half)] = piece[i];
              if (HB == 8 && NQ & 1) qa[NA - 1][kk][2 * c + 1] = 0u;
            }
        }
        if (HB == 8) sc[1] = sc[0];
      }
      const uint32_t mask = s_mask[warp][stage];
      if (mask) {
        const uint32_t ks = ring + stage * Ld::STAGE, vs = ks + Ld::STAGE / 2;
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
          uint32_t b[4];  // keys 0 - 7 and 8 - 15, dimensions kk * 16 .. + 15
          ldmatrix_x4(b, ks + Ld::at((mi >> 1) * 8 + r8, kk * 2 + (mi & 1)));
#pragma unroll
          for (int n = 0; n < NA; ++n) {
            mma_t(c[0], qa[n][kk], b[0], b[1], T());
            mma_t(c[1], qa[n][kk], b[2], b[3], T());
          }
        }
        uint32_t pa[NPA][4];
#pragma unroll
        for (int half = 0; half < HB / 8; ++half) {
          float s[4];  // positions 2 tig, 2 tig + 1, and + 8
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = HB == 8 ? c[i >> 1][i & 1] + c[i >> 1][2 + (i & 1)] : c[i >> 1][2 * half + (i & 1)];
            s[i] = (mask >> (2 * tig + (i & 1) + 8 * (i >> 1))) & 1 ? x * sc[half] : -INFINITY;
          }
          float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float mn = fmaxf(m[half], top);
          if (__any_sync(0xffffffffu, mn > m[half])) {
            const float f = mn == -INFINITY ? 1.f : ex2(m[half] - mn);
            l[half] *= f;
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
              if (HB == 8) {
                o[n][0] *= f; o[n][1] *= f; o[n][2] *= f; o[n][3] *= f;
              } else {
                o[n][2 * half] *= f; o[n][2 * half + 1] *= f;
              }
            }
            m[half] = mn;
          }
          const float ref = (mn == -INFINITY ? 0.f : mn) - PA_BIAS;
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2(s[i] - ref);
          l[half] += (e[0] + e[1]) + (e[2] + e[3]);
          uint32_t lo[4], hi[4];
          split<T, NP>(e[0], e[1], lo);
          split<T, NP>(e[2], e[3], hi);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int n = HB == 8 ? i / 2 : i, rw = HB == 8 ? i & 1 : half;
            pa[n][rw] = lo[i];
            pa[n][2 + rw] = hi[i];
          }
          if (HB == 8 && NP & 1) pa[NPA - 1][1] = pa[NPA - 1][3] = 0u;
        }
#pragma unroll
        for (int dd = 0; dd < NKK; ++dd) {
          uint32_t b[4];  // dimensions dd * 16 .. + 7 and + 8 .. + 15
          ldmatrix_x4_t(b, vs + Ld::at((mi & 1) * 8 + r8, dd * 2 + (mi >> 1)));
#pragma unroll
          for (int n = 0; n < NPA; ++n) {
            mma_t(o[2 * dd], pa[n], b[0], b[1], T());
            mma_t(o[2 * dd + 1], pa[n], b[2], b[3], T());
          }
        }
      }
      __syncwarp();
      if (++stage == NS) stage = 0;
    }
    // the warp's state: o, m, l of its rows
    float* cw = comb + (size_t)warp * HB * CS;
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      float sum = l[half];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float* row = cw + (gid + 8 * half) * CS;
#pragma unroll
      for (int n = 0; n < HD / 8; ++n) {
        const float2 v = HB == 8 ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]) : make_float2(o[n][2 * half], o[n][2 * half + 1]);
        *reinterpret_cast<float2*>(row + n * 8 + 2 * tig) = v;
      }
      if (tig == 0) {
        row[HD] = m[half];
        row[HD + 1] = sum;
      }
    }
    if (Fin::template unit<NW>(a, r, p, n_hb, comb, t0, t1)) {
      pend[n_pend] = p;
      ++n_pend;
    }
    p.t = t1 - 1;
    left = advance<TILE, V>(a, n_units, r.end, p);
  }
  cp_wait<0>();
  if (n_pend) Fin::template join<V>(a, r, pend, n_pend, n_hb, reinterpret_cast<float*>(pa_smem));
}

// ---- CUDA cores: fp32 caches, and heads of more than 128 dimensions -------------------------------------------
//
// A warp takes RW positions of a tile, LPR = 32 / RW lanes each. Scores: lane (position lane % RW, part
// lane / RW) sums every LPR-th group of 4 dimensions for all 8 heads (q in shared memory), shuffles add the
// parts, and the lane then keeps 8 / LPR heads of its position. Values: a lane owns groups of 4 dimensions
// (several lanes share one where the head is short, each taking every PG-th position); the 8 probabilities
// of a position come from shared memory. Products are packed pairs (f32x2): two dimensions in the
// scores, two heads in the values.
template <typename T, int HD>
struct SimtCfg {
  static constexpr int HB = 8, RW = HD <= 32 ? 32 : HD <= 64 ? 16 : 8, NW = HD * sizeof(T) > 512 ? 4 : 8, NT = NW * 32;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4, QS = HB * HD * 4, PS = NW * (RW + 1) * HB * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB - QS - PS) / (NW * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;
  static constexpr int SMEM = NS * NW * Ld::STAGE + COMB + QS + PS;
};

// 4 elements as two pairs
__device__ __forceinline__ ulonglong2 lds4(const unsigned char* p, float) { return *reinterpret_cast<const ulonglong2*>(p); }
__device__ __forceinline__ ulonglong2 lds4(const unsigned char* p, f16) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 x = Pair<f16>::unpack(u.x), y = Pair<f16>::unpack(u.y);
  return make_ulonglong2(pack2(x.x, x.y), pack2(y.x, y.y));
}
__device__ __forceinline__ ulonglong2 lds4(const unsigned char* p, bf16) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_ulonglong2(pack2(bf_lo(u.x), bf_hi(u.x)), pack2(bf_lo(u.y), bf_hi(u.y)));
}

template <typename T, int HD, typename IO>
__global__ void __launch_bounds__(SimtCfg<T, HD>::NT, 1) paged_simt_kernel(const PagedAttnArgs a) {
  using C = SimtCfg<T, HD>;
  using Ld = typename C::Ld;
  using Fin = Finish<IO, C::HB, HD, C::NT>;
  constexpr int NW = C::NW, NS = C::NS, HB = C::HB, RW = C::RW, CS = comb_stride(HD), TILE = Ld::TILE, V = Ld::V;
  constexpr int LPR = 32 / RW, HPL = HB / LPR;  // lanes of a position, heads a lane keeps
  constexpr int G4 = HD / 4;                    // groups of 4 dimensions
  constexpr int PG = G4 >= 32 ? 1 : 32 / G4;    // lanes that share a group, by position
  constexpr int GL = G4 >= 32 ? G4 / 32 : 1;    // groups a lane owns
  static_assert(NS >= 2 && C::SMEM >= PA_JOIN * HB * CS * 4, "the ring, and the parts of a join in its place");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[NW][NS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * NW * Ld::STAGE);
  float* qs = comb + NW * HB * CS;                  // [HB][HD]
  float* ps = qs + HB * HD + warp * (RW + 1) * HB;  // [RW][HB] probabilities, then [HB] factors
  unsigned char* ring_p = pa_smem + warp * NS * Ld::STAGE;
  const uint32_t ring = smem_addr(ring_p);
  Place ld;
  const Range r = find_range<IO, TILE, V, C::NT>(a, n_units, ld);
  if (r.begin >= r.end) return;
  Place p = ld;
  bool more = true;  // tiles to request
  long long row_off = Ld::row(a, ld, n_hb, warp, lane);
  int ld_stage = 0;
  const bool col = lane % Ld::CH * Ld::CE < a.hd;
  const char *kl = (const char*)a.k + lane % Ld::CH * 16, *vl = (const char*)a.v + lane % Ld::CH * 16;
  auto load_next = [&]() {  // requests the tile at ld and looks up the rows of the one after it
    if (more) {
      const uint32_t mask = __ballot_sync(0xffffffffu, row_off >= 0);
      Ld::request(kl, vl, row_off, mask, ring + ld_stage * Ld::STAGE, lane, col, a.hd);
      if (lane == 0) s_mask[warp][ld_stage] = mask;
      more = advance<TILE, V>(a, n_units, r.end, ld);
      if (more) row_off = Ld::row(a, ld, n_hb, warp, lane);
    }
    cp_commit();
    if (++ld_stage == NS) ld_stage = 0;
  };
  int stage = 0, ahead = NS - 1;  // tiles still to be requested before the first is used
  Place pend[2];
  int n_pend = 0;
  const int pos = lane % RW, part = lane / RW;
  const int vg = G4 >= 32 ? lane : lane % G4, vp = G4 >= 32 ? 0 : lane / G4;
  const float sc = a.scale * LOG2E;
  auto grp = [&](const unsigned char* half, int row, int g4) {  // 4 dimensions of a row
    constexpr int B4 = 4 * (int)sizeof(T);
    const int byte = g4 * B4;
    return lds4(half + Ld::at(row, byte / 16) + byte % 16, T());
  };
  for (bool left = true; left;) {
    const int t0 = p.t, t1 = min(p.nt, r.end - p.v - V);
    const int g = p.u / n_hb, h0 = (p.u - g * n_hb) * HB;
#pragma unroll 1
    for (int i = 2 * tid; i < HB * HD; i += 2 * C::NT) {
      const int h = i / HD, d = i - h * HD;
      *reinterpret_cast<float2*>(qs + i) =
          h0 + h < group && d < a.hd ? load2((const IO*)a.q + p.b * a.q_stride + (g * group + h0 + h) * a.hd + d) : make_float2(0.f, 0.f);
    }
    bool fresh = true;
    f32x2 o[GL][4][HB / 2];  // pairs of heads
#pragma unroll
    for (int i = 0; i < GL; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int h = 0; h < HB / 2; ++h) o[i][d][h] = 0ull;
    float m[HPL], l[HPL];  // heads part * HPL + i; l: this lane's positions
#pragma unroll
    for (int i = 0; i < HPL; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll 1
    for (int t = t0; t < t1;) {
      load_next();  // into the stage that the last tile used
      if (ahead) {
        --ahead;
        continue;
      }
      ++t;
      cp_wait<NS - 1>();
      __syncwarp();
      if (fresh) {
        fresh = false;
        __syncthreads();  // q
      }
      const uint32_t mask = s_mask[warp][stage];
      if (mask) {
        const unsigned char *ks = ring_p + stage * Ld::STAGE, *vs = ks + Ld::STAGE / 2;
        f32x2 dot[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) dot[h] = 0ull;
#pragma unroll
        for (int i = 0; i < G4 / LPR; ++i) {
          const int g4 = part + LPR * i;
          const ulonglong2 k4 = grp(ks, pos, g4);
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            const ulonglong2 q4 = *reinterpret_cast<const ulonglong2*>(qs + h * HD + g4 * 4);
            fma2(dot[h], q4.x, k4.x);
            fma2(dot[h], q4.y, k4.y);
          }
        }
        float s[HPL];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          const float2 two = unpack2(dot[h]);
          float d = two.x + two.y;
#pragma unroll
          for (int x = RW; x < 32; x <<= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
          if (LPR == 1 || h / HPL == part) s[h % HPL] = d;
        }
        const bool there = (mask >> pos) & 1;
        float f[HPL], e[HPL];
        bool moved = false;
#pragma unroll
        for (int i = 0; i < HPL; ++i) {
          const float x = there ? s[i] * sc : -INFINITY;
          float top = x;
#pragma unroll
          for (int y = 1; y < RW; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
          const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
          f[i] = mn > m[i] ? ex2(m[i] - ref) : 1.f;
          moved |= mn > m[i];
          e[i] = ex2(x - (ref - PA_BIAS));
          l[i] = fmaf(l[i], f[i], e[i]);
          m[i] = mn;
        }
#pragma unroll
        for (int i = 0; i < HPL; i += 2) {
          *reinterpret_cast<float2*>(ps + pos * HB + HPL * part + i) = make_float2(e[i], e[i + 1]);
          if (pos == 0) *reinterpret_cast<float2*>(ps + RW * HB + HPL * part + i) = make_float2(f[i], f[i + 1]);
        }
        moved = __any_sync(0xffffffffu, moved);
        __syncwarp();
        auto pairs = [&](int row, f32x2* w) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(ps + row * HB), y = *reinterpret_cast<const ulonglong2*>(ps + row * HB + 4);
          w[0] = x.x; w[1] = x.y; w[2] = y.x; w[3] = y.y;
        };
        f32x2 w[HB / 2];
        if (moved) {
          pairs(RW, w);
#pragma unroll
          for (int i = 0; i < GL; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int h = 0; h < HB / 2; ++h) mul2(o[i][d][h], w[h]);
        }
#pragma unroll
        for (int j = 0; j < RW; j += PG) {
          const int row = j + vp;
          pairs(row, w);
#pragma unroll
          for (int i = 0; i < GL; ++i) {
            const ulonglong2 v4 = grp(vs, row, vg + 32 * i);
            const float2 a01 = unpack2(v4.x), a23 = unpack2(v4.y);
            const f32x2 v[4] = {pack2(a01.x, a01.x), pack2(a01.y, a01.y), pack2(a23.x, a23.x), pack2(a23.y, a23.y)};
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int h = 0; h < HB / 2; ++h) fma2(o[i][d][h], w[h], v[d]);
          }
        }
      }
      __syncwarp();
      if (++stage == NS) stage = 0;
    }
    float* cw = comb + (size_t)warp * HB * CS;
#pragma unroll
    for (int i = 0; i < GL; ++i)
#pragma unroll
      for (int h = 0; h < HB; h += 2) {
        float x[2][4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float2 two = unpack2(o[i][d][h / 2]);
          x[0][d] = two.x;
          x[1][d] = two.y;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int y = G4; y < 32; y <<= 1) x[k][d] += __shfl_xor_sync(0xffffffffu, x[k][d], y);  // the lanes that share the group
          if (vp == 0)
            *reinterpret_cast<float4*>(cw + (h + k) * CS + (vg + 32 * i) * 4) = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
        }
      }
#pragma unroll
    for (int i = 0; i < HPL; ++i) {
      float sum = l[i];
#pragma unroll
      for (int y = 1; y < RW; y <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
      if (pos == 0) {
        cw[(part * HPL + i) * CS + HD] = m[i];
        cw[(part * HPL + i) * CS + HD + 1] = sum;
      }
    }
    if (Fin::template unit<NW>(a, r, p, n_hb, comb, t0, t1)) {
      pend[n_pend] = p;
      ++n_pend;
    }
    p.t = t1 - 1;
    left = advance<TILE, V>(a, n_units, r.end, p);
  }
  cp_wait<0>();
  if (n_pend) Fin::template join<V>(a, r, pend, n_pend, n_hb, reinterpret_cast<float*>(pa_smem));
}

// ---- host ------------------------------------------------------------------------------------------------------

template <typename K>
cudaError_t launch(K kernel, int threads, int smem, int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e ? e : launch_k(kernel, dim3(ctas), dim3(threads), smem, s, false, a);
}
template <typename T, int HD, int HB, typename IO>
cudaError_t launch_mma(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  using C = MmaCfg<T, HD, HB, IO>;
  return launch(paged_mma_kernel<T, HD, HB, IO>, C::NT, C::SMEM, ctas, a, s);
}
template <typename T, int HD, typename IO>
cudaError_t launch_simt(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  using C = SimtCfg<T, HD>;
  return launch(paged_simt_kernel<T, HD, IO>, C::NT, C::SMEM, ctas, a, s);
}
// Heads of sizes between the instances are padded with zeros in shared memory to the next one.
template <typename T, typename IO>
cudaError_t launch_16bit(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  if (a.hd > 128) return launch_simt<T, 256, IO>(ctas, a, s);
  if (a.nq / a.nkv <= 8)
    return a.hd <= 32   ? launch_mma<T, 32, 8, IO>(ctas, a, s)
           : a.hd <= 64 ? launch_mma<T, 64, 8, IO>(ctas, a, s) : launch_mma<T, 128, 8, IO>(ctas, a, s);
  return a.hd <= 64 ? launch_mma<T, 64, 16, IO>(ctas, a, s) : launch_mma<T, 128, 16, IO>(ctas, a, s);
}

// floats of one part: the largest instance that the shape may take
size_t part_floats(int n_heads, int n_kv_heads, int head_dim) {
  const int hb = n_heads / n_kv_heads <= 8 ? 8 : 16, hd = head_dim <= 32 ? 32 : head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  return (size_t)hb * comb_stride(hd);
}
constexpr size_t COUNTER_BYTES = 4 * PA_MAX_CTAS * sizeof(unsigned int);

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t qw_op_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 8 || head_dim % 8 || head_dim > PA_MAX_HD) return 0;
  return COUNTER_BYTES + 2 * PA_MAX_CTAS * part_floats(n_heads, n_kv_heads, head_dim) * sizeof(float);
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
  if ((int64_t)max_blocks * c.page_size > (int64_t)1 << 30)
    return op_fail(QW_ERR_UNSUPPORTED, "max_blocks * page_size above 2^30");
  // the tile list's numbers are 31-bit: tiles of at least 64 positions, and a weight of at most 5 a unit
  if ((int64_t)n_seqs * n_heads * ((int64_t)max_blocks * c.page_size / 64 + 6) > 0x7fffffffll)
    return op_fail(QW_ERR_UNSUPPORTED, "n_seqs * n_heads * max_blocks * page_size too large");
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
  int dev = 0, nsm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  PagedAttnArgs a{c.k, c.v, c.page_stride, c.head_stride, c.pos_stride, n_seqs, n_heads, c.n_kv_heads, c.head_dim,
                  c.page_size, c.n_pages, max_blocks, block_table, lens, q, out, q_stride, out_stride, scale, lse,
                  (unsigned int*)workspace, (float*)((char*)workspace + COUNTER_BYTES), err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  const int ctas = nsm < PA_MAX_CTAS ? nsm : PA_MAX_CTAS;
  if (c.dtype == QW_F32)
    e = c.head_dim <= 32    ? launch_simt<float, 32, float>(ctas, a, s)
        : c.head_dim <= 64  ? launch_simt<float, 64, float>(ctas, a, s)
        : c.head_dim <= 128 ? launch_simt<float, 128, float>(ctas, a, s) : launch_simt<float, 256, float>(ctas, a, s);
  else if (c.dtype == QW_F16)
    e = io_dtype == QW_F32 ? launch_16bit<f16, float>(ctas, a, s) : launch_16bit<f16, f16>(ctas, a, s);
  else
    e = io_dtype == QW_F32 ? launch_16bit<bf16, float>(ctas, a, s) : launch_16bit<bf16, bf16>(ctas, a, s);
  if (e) return op_cuda_fail(e, "paged attention launch");
  return QW_OK;
}

}  // extern "C"
