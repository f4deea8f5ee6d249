// Common parts of the decode attention over a paged key-value cache (attn_paged.cu, attn_paged_simt.cu): the list of
// tiles and its cuts, the rows of a tile, the end of a unit.
#pragma once

#include "common.cuh"
#include "op_util.h"

#include <cfloat>
#include <math.h>

#include <cmath>
#include <type_traits>

namespace qw {
namespace paged {

constexpr int PA_MAX_HD = 256;
constexpr int PA_MAX_CTAS = 320;   // CTAs the workspace has room for
constexpr int PA_WHOLE = 3;        // units of at most so many tiles are not split
constexpr int PA_LEVELS = 4;       // of a join
constexpr int PA_MAX_WEIGHT = 4;   // of a unit's end in the list of tiles, in tiles
// positions of the kernels' tiles, at least: bounds the length of the list of tiles (each kernel asserts both)
__host__ __device__ constexpr int least_tile(bool f32_cache, int head_dim) { return f32_cache && head_dim > 128 ? 16 : 32; }
constexpr int PA_FLUSH = 16;         // products that the tensor cores sum up for an fp32 caller (their additions cut,
                                   // so a long sum's error grows with its length: 1.6e-6 for 100)
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
  unsigned int* counters;  // [PA_LEVELS][2 * PA_MAX_CTAS], zero between calls
  float* part;             // [2 * PA_MAX_CTAS][HB][comb_stride(HD)]
  int* err;
};

__host__ __device__ constexpr int comb_stride(int hd) { return hd + 4; }  // o, then m and l

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
// 16-byte chunks of row r permuted by chunk ^ (r & 7), so that 8 rows' same chunk lie in distinct banks. (Rows of 64 bytes,
// 16-bit heads of at most 32 dimensions, have 4 chunks only: rows r and r + 4 share banks, and an ldmatrix takes twice the
// accesses. 100 sequences of up to 8000 positions, 8 and 2 heads of 32, bf16: 38 us for 16 us of traffic.)
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

// The maximum of a warp's state: -inf for no position at all (pages outside the cache), the lowest finite number, which
// weighs as little next to others, for positions whose scores are all -inf.
__device__ __forceinline__ float state_max(float m, bool any) { return any ? fmaxf(m, -FLT_MAX) : m; }

// All code that runs once per unit or per CTA is kept short: loops, one out-of-line sum of states.
template <typename IO, int HB, int HD, int NT, int SMEM>
struct Finish {
  static constexpr int CS = comb_stride(HD), N4 = HB * HD / 4;
  // parts merged at once: of two units, they fit the kernel's shared memory
  static constexpr int GROUP_FIT = SMEM / (2 * HB * CS * 4), GROUP = GROUP_FIT > 10 ? 10 : GROUP_FIT;
  static_assert(GROUP * GROUP * GROUP * GROUP >= PA_MAX_CTAS, "levels");

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
    // l = 0: no position was left, and out is 0 as for length 0; or every score was -inf, and 0 / 0 is the formula's NaN
    const float inv = s.l == 0.f && s.m == -INFINITY ? 1.f : 1.f / s.l;
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

  // Joins the CTA's split units (at most two, places pend[0 .. n)), both at once, in a tree: at level 0 the parts of
  // GROUP consecutive CTAs, counted from the unit's first, at level 1 the sums of GROUP groups, and so on. A CTA
  // announces its part and merges the group if it is the last to; the group's first slot takes the sum. The
  // parts are fetched into shared memory (buf, all of the kernel's) together. Done once at the CTA's
  // end: an announcement takes a memory fence and an atomic's round trip, about 1 us, a level 2 us.
  template <int V>
  static __device__ __forceinline__ void join(const PagedAttnArgs& a, const Range& r, const Place* pend, int n, int n_hb, float* buf) {
    constexpr int S4 = HB * CS / 4;
    // what is merged next: states of CTAs from, from + step, ...; the unit's first slot and its CTAs
    __shared__ int s_from[2], s_count[2], s_first[2], s_c0[2], s_c1[2], s_last[2];
    const int c = blockIdx.x, w = threadIdx.x / 32;
    const bool speaker = threadIdx.x % 32 == 0 && w < n;
    if (threadIdx.x < 2) s_last[threadIdx.x] = s_count[threadIdx.x] = 0;
    __syncthreads();
    if (speaker) {
      const Place& p = pend[w];
      s_c0[w] = cta_of(r, p.v + V);
      s_c1[w] = cta_of(r, p.v + V + p.nt - 1);
      s_first[w] = slot_of(r, p, s_c0[w]);
      s_last[w] = 1;
    }
    int step = 1;
#pragma unroll 1
    for (int level = 0; level < PA_LEVELS; ++level, step *= GROUP) {
      if (speaker && s_last[w]) {
        const int c0 = s_c0[w], from = c - (c - c0) % (step * GROUP), count = min(GROUP, (s_c1[w] - from) / step + 1);
        s_from[w] = from;
        s_count[w] = count;
        unsigned int* counter = a.counters + level * 2 * PA_MAX_CTAS + (from == c0 ? s_first[w] : 2 * from);
        __threadfence();  // (the CTA's parts, written before the last barrier)
        const bool last = atomicAdd(counter, 1u) == (unsigned)count - 1u;
        if (last) *counter = 0u;
        s_last[w] = last;
        __threadfence();
      }
      __syncthreads();
      const int n0 = s_last[0] ? s_count[0] : 0, n1 = s_last[1] ? s_count[1] : 0;
      if (n0 + n1 == 0) return;
#pragma unroll 1
      for (int part = w; part < n0 + n1; part += NT / 32) {  // a warp a state
        const int k = part >= n0, cta = s_from[k] + (part - (k ? n0 : 0)) * step;
        const float* src = slot_ptr(a, cta == s_c0[k] ? s_first[k] : 2 * cta);
        float* dst = buf + part * HB * CS;
#pragma unroll 4
        for (int i = threadIdx.x % 32; i < S4; i += 32) cp_async16(dst + i * 4, src + i * 4);
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
      const bool done0 = n0 == 0 || s_c1[0] - s_c0[0] < step * GROUP, done1 = n1 == 0 || s_c1[1] - s_c0[1] < step * GROUP;
#pragma unroll 1
      for (int i = n0 ? threadIdx.x : N4 + threadIdx.x; i < (n1 ? 2 * N4 : N4); i += NT) {
        const int k = i >= N4, i4 = i - k * N4, h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
        const Acc s = sum(buf + (k ? n0 * HB * CS : 0), k ? n1 : n0, h, d);
        if (k ? done1 : done0) write_out(a, pend[k], n_hb, h, d, s);
        else put(slot_ptr(a, s_from[k] == s_c0[k] ? s_first[k] : 2 * s_from[k]), h, d, s);
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

// attn_paged_simt.cu: fp32 caches, and heads of more than 128 dimensions
cudaError_t launch_simt(int cache_dtype, int io_dtype, int ctas, const PagedAttnArgs& a, cudaStream_t s);

template <typename K>
cudaError_t launch(K kernel, int threads, int smem, int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e ? e : launch_k(kernel, dim3(ctas), dim3(threads), smem, s, false, a);
}

}  // namespace paged
}  // namespace qw
