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
constexpr int PA_MAX_CTAS = 192;   // persistent CTAs the workspace has room for
constexpr int PA_GROUP = 12;       // parts merged at once: 152 CTAs are at most 13 groups
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
  int io;                  // qw_dtype of q and out
};

__host__ __device__ constexpr int comb_stride(int hd) { return hd + 8; }  // o, then m and l

__device__ __forceinline__ float load_io(const void* p, long long i, int io) {
  return io == QW_F32 ? ((const float*)p)[i] : io == QW_F16 ? __half2float(((const f16*)p)[i]) : __bfloat162float(((const bf16*)p)[i]);
}
__device__ __forceinline__ void store_out(void* p, long long i, float v, int io) {
  if (io == QW_F32) ((float*)p)[i] = v;
  else if (io == QW_F16) ((f16*)p)[i] = __float2half_rn(v);
  else ((bf16*)p)[i] = __float2bfloat16_rn(v);
}

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

// A place in the list: tile t of nt of unit u of sequence b; base: the sequence's first tile in units of
// one unit's tiles (the list holds base * n_units tiles before it).
struct Place {
  int b, u, t, nt, len;
  long long base;
};

template <int TILE>
__device__ __forceinline__ void advance(const PagedAttnArgs& a, int n_units, Place& p) {  // only while tiles are left
  if (++p.t < p.nt) return;
  p.t = 0;
  if (++p.u < n_units) return;
  p.u = 0;
  p.base += p.nt;
  do {
    p.len = seq_len(a, ++p.b);
    p.nt = (p.len + TILE - 1) / TILE;
  } while (p.nt == 0 && p.b + 1 < a.n_seqs);
}

struct Range {
  long long total, begin, end;  // tiles in the list, this CTA's range
  int ctas;                     // CTAs that have one
};

// The CTA's range and its first place. Every CTA sums the sequences' tiles itself (L2 serves the lengths).
template <int TILE, int NT>
__device__ Range find_range(const PagedAttnArgs& a, int n_units, Place& first) {
  __shared__ long long w_sum[NT / 32];
  __shared__ Place s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + NT - 1) / NT, b0 = min(a.n_seqs, tid * per), b1 = min(a.n_seqs, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    bool bad;
    mine += (seq_len(a, b, bad) + TILE - 1) / TILE;
    if (bad && blockIdx.x == 0) atomicOr(a.err, ERR_PAGE);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) w_sum[warp] = incl;
  __syncthreads();
  long long base = incl - mine, tiles = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += w_sum[w];
    tiles += w_sum[w];
  }
  Range r;
  r.total = tiles * n_units;
  r.ctas = (int)min((long long)gridDim.x, r.total);
  r.begin = r.end = 0;
  if ((int)blockIdx.x < r.ctas) {
    r.begin = r.total * blockIdx.x / r.ctas;
    r.end = r.total * (blockIdx.x + 1) / r.ctas;
    if (base * n_units <= r.begin && r.begin < (base + mine) * n_units) {
      for (int b = b0; b < b1; ++b) {
        const int len = seq_len(a, b), nt = (len + TILE - 1) / TILE;
        if (r.begin < (base + nt) * n_units) {
          const long long in = r.begin - base * n_units;
          s_first = Place{b, (int)(in / nt), (int)(in % nt), nt, len, base};
          break;
        }
        base += nt;
      }
    }
  }
  __syncthreads();
  first = s_first;
  return r;
}

// CTA whose range holds tile x of the list: the last c with floor(total c / ctas) <= x
__device__ __forceinline__ int cta_of(const Range& r, long long x) { return (int)(((x + 1) * r.ctas - 1) / r.total); }
__device__ __forceinline__ long long begin_of(const Range& r, int c) { return r.total * c / r.ctas; }

// Sequences of length 0 have no tile: out 0, lse -inf.
__device__ void write_empty(const PagedAttnArgs& a) {
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    if (seq_len(a, b) > 0) continue;
    const int width = a.nq * a.hd;
    for (int i = threadIdx.x; i < width; i += blockDim.x) store_out(a.out, b * a.out_stride + i, 0.f, a.io);
    if (a.lse)
      for (int h = threadIdx.x; h < a.nq; h += blockDim.x) a.lse[(size_t)b * a.nq + h] = -INFINITY;
  }
}

// ---- the rows of a tile ----------------------------------------------------------------------------------

// Each warp's rows of a tile, requested by the warp itself. Stage layout: K [RW][HD], V [RW][HD] of T, the
// 16-byte chunks of row r permuted by chunk ^ (r & 7), so that 8 rows' same chunk lie in distinct banks.
template <typename T, int HD, int RW, int NW>
struct Loader {
  static constexpr int TILE = RW * NW, CH = HD * (int)sizeof(T) / 16, CE = 16 / (int)sizeof(T);
  static constexpr int STAGE = 2 * RW * HD * (int)sizeof(T);
  static __device__ __forceinline__ uint32_t at(int row, int chunk) { return (uint32_t)(row * CH + (chunk ^ (row & 7 & (CH - 1)))) * 16; }
  static_assert((CH & (CH - 1)) == 0, "chunks are permuted by exclusive or");
  // element offset of the lane's row (lanes 0 .. RW - 1) in the caches, or -1: no such row
  static __device__ __forceinline__ long long row(const PagedAttnArgs& a, const Place& p, int n_hb, int warp, int lane) {
    const int j = p.t * TILE + warp * RW + lane;
    if (lane >= RW || j >= p.len) return -1;
    const int blk = j / a.page, id = __ldg(a.table + (size_t)p.b * a.max_blocks + blk);
    if (id < 0 || id >= a.n_pages) {
      if (p.u == 0) atomicOr(a.err, ERR_PAGE);
      return -1;
    }
    return id * a.page_stride + (p.u / n_hb) * a.head_stride + (long long)(j - blk * a.page) * a.pos_stride;
  }
  static __device__ __forceinline__ void request(const PagedAttnArgs& a, long long row_off, uint32_t stage, int lane) {
    constexpr int N = RW * CH;  // chunks of K (and of V)
#pragma unroll
    for (int i = 0; i < (N + 31) / 32; ++i) {
      const int c = i * 32 + lane, r = c / CH, ch = c - r * CH;
      const long long off = __shfl_sync(0xffffffffu, row_off, r < RW ? r : 0);
      if (N % 32 == 0 || c < N) {
        const bool ok = off >= 0 && ch * CE < a.hd;
        const long long e = ok ? off + ch * CE : 0;
        cp_async16_or_zero(stage + at(r, ch), (const T*)a.k + e, ok);
        cp_async16_or_zero(stage + N * 16 + at(r, ch), (const T*)a.v + e, ok);
      }
    }
  }
};

// ---- the end of a unit -------------------------------------------------------------------------------------

// State of one thread in a merge: up to MAXE groups of 4 output elements.
template <int HB, int HD, int NT>
struct Finish {
  static constexpr int CS = comb_stride(HD), N4 = HB * HD / 4, E = (N4 + NT - 1) / NT;

  static __device__ __forceinline__ void write_out(const PagedAttnArgs& a, const Place& p, int n_hb, const float4* o, const float* M,
                                                   const float* L) {
    const int group = a.nq / a.nkv, g = p.u / n_hb, h0 = (p.u - g * n_hb) * HB;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i4 = threadIdx.x + e * NT, h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
      if (i4 >= N4 || h0 + h >= group) continue;
      const int head = g * group + h0 + h;
      if (d < a.hd) {
        const float inv = 1.f / L[e];  // (l = 0: every score was -inf, and 0 / 0 is the formula's NaN)
        const long long at = p.b * a.out_stride + (long long)head * a.hd + d;
        store_out(a.out, at, o[e].x * inv, a.io);
        store_out(a.out, at + 1, o[e].y * inv, a.io);
        store_out(a.out, at + 2, o[e].z * inv, a.io);
        store_out(a.out, at + 3, o[e].w * inv, a.io);
      }
      if (d == 0 && a.lse) a.lse[(size_t)p.b * a.nq + head] = (M[e] - PA_BIAS + log2f(L[e])) * LN2;
    }
  }

  // Sum of n states (state(i): [HB][CS] in shared or global memory) at this thread's elements.
  template <typename State>
  static __device__ __forceinline__ void gather(int n, State state, float4* o, float* M, float* L) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i4 = threadIdx.x + e * NT, h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
      o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      M[e] = -INFINITY;
      L[e] = 0.f;
      if (i4 >= N4) continue;
      for (int i0 = 0; i0 < n; i0 += PA_GROUP) {  // (one round: n <= PA_GROUP + 1 but for odd grids)
        float m[PA_GROUP], l[PA_GROUP];
        float4 x[PA_GROUP];
#pragma unroll
        for (int i = 0; i < PA_GROUP; ++i) {
          m[i] = -INFINITY;
          l[i] = 0.f;
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + i < n) {
            const float* s = state(i0 + i) + h * CS;
            x[i] = *reinterpret_cast<const float4*>(s + d);
            m[i] = s[HD];
            l[i] = s[HD + 1];
          }
        }
        float top = M[e];
#pragma unroll
        for (int i = 0; i < PA_GROUP; ++i) top = fmaxf(top, m[i]);
        const float ref = top == -INFINITY ? 0.f : top;
        const float c = exp2f(M[e] - ref);
        o[e].x *= c; o[e].y *= c; o[e].z *= c; o[e].w *= c;
        L[e] *= c;
#pragma unroll
        for (int i = 0; i < PA_GROUP; ++i) {
          const float w = exp2f(m[i] - ref);
          o[e].x = fmaf(w, x[i].x, o[e].x);
          o[e].y = fmaf(w, x[i].y, o[e].y);
          o[e].z = fmaf(w, x[i].z, o[e].z);
          o[e].w = fmaf(w, x[i].w, o[e].w);
          L[e] = fmaf(w, l[i], L[e]);
        }
        M[e] = top;
      }
    }
  }

  static __device__ __forceinline__ void put(float* slot, const float4* o, const float* M, const float* L) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i4 = threadIdx.x + e * NT, h = i4 / (HD / 4), d = (i4 - h * (HD / 4)) * 4;
      if (i4 >= N4) continue;
      *reinterpret_cast<float4*>(slot + h * CS + d) = o[e];
      if (d == 0) {
        slot[h * CS + HD] = M[e];
        slot[h * CS + HD + 1] = L[e];
      }
    }
  }

  // One arrival of n at a counter, after this CTA's writes; true for the last, which sees all writes.
  static __device__ __forceinline__ bool arrive(unsigned int* counter, int n) {
    __shared__ bool s_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = atomicAdd(counter, 1u) == (unsigned)(n - 1);
      if (s_last) *counter = 0u;
    }
    __syncthreads();
    const bool last = s_last;
    if (last) __threadfence();
    __syncthreads();  // (s_last is used again)
    return last;
  }

  // The CTA's state of the unit at p (comb: [NW][HB][CS] in shared memory, one per warp), covering tiles
  // [t0, t1) of it. All threads call it; comb may be written again afterwards.
  static __device__ void unit(const PagedAttnArgs& a, const Range& r, const Place& p, int n_units, int n_hb, int nw, const float* comb, int t0,
                              int t1) {
    __syncthreads();
    float4 o[E];
    float M[E], L[E];
    gather(nw, [&](int i) { return comb + (size_t)i * HB * CS; }, o, M, L);
    if (t0 == 0 && t1 == p.nt) {
      write_out(a, p, n_hb, o, M, L);
      __syncthreads();
      return;
    }
    const long long u0 = p.base * n_units + (long long)p.u * p.nt;  // the unit's tiles in the list
    const int c0 = cta_of(r, u0), c1 = cta_of(r, u0 + p.nt - 1), c = blockIdx.x;
    // a CTA's range cuts at most two units: slot 0 the one it begins with, slot 1 the one it ends with
    auto slot_of = [&](int cta) { return 2 * cta + (cta == c0 && begin_of(r, c0) != u0 ? 1 : 0); };
    auto slot_ptr = [&](int s) { return a.part + (size_t)s * HB * CS; };
    const int mine = slot_of(c);
    put(slot_ptr(mine), o, M, L);
    const int g = (c - c0) / PA_GROUP, n_groups = (c1 - c0) / PA_GROUP + 1;
    const int g0 = c0 + g * PA_GROUP, gn = min(PA_GROUP, c1 - g0 + 1);
    if (!arrive(a.counters + slot_of(g0), gn)) return;
    gather(gn, [&](int i) { return (const float*)slot_ptr(slot_of(g0 + i)); }, o, M, L);
    if (n_groups > 1) {
      __syncthreads();  // every thread has read the parts: the group's first slot takes their sum
      put(slot_ptr(slot_of(g0)), o, M, L);
      if (!arrive(a.counters + 2 * PA_MAX_CTAS + slot_of(c0), n_groups)) return;
      gather(n_groups, [&](int i) { return (const float*)slot_ptr(slot_of(c0 + i * PA_GROUP)); }, o, M, L);
    }
    write_out(a, p, n_hb, o, M, L);
    __syncthreads();
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
template <typename T, int HD, int HB, bool F32IO>
struct MmaCfg {
  static constexpr int NW = 8, RW = 16, NT = NW * 32;
  static constexpr bool three = F32IO && sizeof(T) == 2 && !std::is_same<T, f16>::value;
  static constexpr int NQ = !F32IO ? 1 : three ? 3 : 2, NP = three ? 3 : 2;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB) / (NW * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;  // stages of a warp's ring
  static constexpr int SMEM = NS * NW * Ld::STAGE + COMB;
};

template <typename T, int HD, int HB, bool F32IO>
__global__ void __launch_bounds__(256, 1) paged_mma_kernel(const PagedAttnArgs a) {
  using C = MmaCfg<T, HD, HB, F32IO>;
  using Ld = typename C::Ld;
  constexpr int NW = C::NW, NS = C::NS, NQ = C::NQ, NP = C::NP, CS = comb_stride(HD), TILE = Ld::TILE;
  constexpr int NKK = HD / 16, NA = HB == 8 ? (NQ + 1) / 2 : NQ, NPA = HB == 8 ? (NP + 1) / 2 : NP;  // products per step
  static_assert(NS >= 2, "ring");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[NW][NS];  // rows of a stage that exist
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * NW * Ld::STAGE);
  const uint32_t ring = smem_addr(pa_smem) + warp * NS * Ld::STAGE;
  write_empty(a);
  Place ld;
  const Range r = find_range<TILE, C::NT>(a, n_units, ld);
  if (r.begin >= r.end) return;
  Place p = ld;
  long long to_load = r.end - r.begin, left = to_load;
  long long row_off = Ld::row(a, ld, n_hb, warp, lane);
  int ld_stage = 0;
  auto load_next = [&]() {  // requests the tile at ld and looks up the rows of the one after it
    if (to_load > 0) {
      Ld::request(a, row_off, ring + ld_stage * Ld::STAGE, lane);
      const uint32_t mask = __ballot_sync(0xffffffffu, row_off >= 0);
      if (lane == 0) s_mask[warp][ld_stage] = mask;
      if (--to_load > 0) {
        advance<TILE>(a, n_units, ld);
        row_off = Ld::row(a, ld, n_hb, warp, lane);
      }
    }
    cp_commit();
    if (++ld_stage == NS) ld_stage = 0;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load_next();
  int stage = 0;
  while (left > 0) {
    const int t0 = p.t, t1 = (int)min((long long)p.nt, t0 + left);
    // queries of the unit: A fragments (rows gid and gid + 8 at columns 2 tig and 2 tig + 8)
    uint32_t qa[NA][NKK][4];
    float sc[2];
    {
      const int g = p.u / n_hb, h0 = (p.u - g * n_hb) * HB;
#pragma unroll
      for (int half = 0; half < HB / 8; ++half) {
        const int h = h0 + gid + 8 * half;
        const long long at = p.b * a.q_stride + (long long)(g * group + h) * a.hd;
        float x[NKK][4];
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = kk * 16 + 2 * tig + (i & 1) + 8 * (i >> 1);
            x[kk][i] = h < group && d < a.hd ? load_io(a.q, at + d, a.io) : 0.f;
            top = fmaxf(top, fabsf(x[kk][i]));
          }
        float up = 1.f, down = 1.f;
        if (F32IO) {
          // fp32 queries times a power of two that puts the row's largest at 2^10: the pieces stay normal
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
        for (int kk = 0; kk < NKK; ++kk) {
          uint32_t lo[4], hi[4];  // pieces at columns 2 tig and 2 tig + 8
          split<T, NQ>(x[kk][0] * up, x[kk][1] * up, lo);
          split<T, NQ>(x[kk][2] * up, x[kk][3] * up, hi);
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const int n = HB == 8 ? i / 2 : i, rw = HB == 8 ? i & 1 : half;
            qa[n][kk][rw] = lo[i];
            qa[n][kk][2 + rw] = hi[i];
          }
          if (HB == 8 && NQ & 1) qa[NA - 1][kk][1] = qa[NA - 1][kk][3] = 0u;
        }
      }
      if (HB == 8) sc[1] = sc[0];
    }
    float o[HD / 8][4], m[HB / 8], l[HB / 8];
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
    for (int h = 0; h < HB / 8; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
      cp_wait<NS - 2>();
      __syncwarp();
      load_next();  // into the stage that the last tile used
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
            const float f = mn == -INFINITY ? 1.f : exp2f(m[half] - mn);
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
          for (int i = 0; i < 4; ++i) e[i] = exp2f(s[i] - ref);
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
    Finish<HB, HD, C::NT>::unit(a, r, p, n_units, n_hb, NW, comb, t0, t1);
    left -= t1 - t0;
    p.t = t1 - 1;
    if (left > 0) advance<TILE>(a, n_units, p);
  }
  cp_wait<0>();
}

// ---- CUDA cores: fp32 caches, and heads of more than 128 dimensions -------------------------------------------
//
// 8 positions a warp and tile. Scores: lane (position lane % 8, quarter lane / 8) sums every fourth group of
// 4 dimensions for all 8 heads (q in shared memory), two shuffles add the quarters, and the lane then keeps
// heads 2 (lane / 8) and + 1. Values: a lane owns groups of 4 dimensions (several lanes share one where
// the head is short, each taking every PG-th position) and the 8 probabilities of a position come from
// shared memory as two vectors. About 600 warp instructions per 8 KB of an fp32 tile, a third of what
// an SM issues while HBM delivers it.
template <typename T, int HD>
struct SimtCfg {
  static constexpr int HB = 8, RW = 8, NW = HD * sizeof(T) > 512 ? 4 : 8, NT = NW * 32;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4, QS = HB * HD * 4, PS = NW * (RW + 1) * HB * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB - QS - PS) / (NW * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;
  static constexpr int SMEM = NS * NW * Ld::STAGE + COMB + QS + PS;
};

__device__ __forceinline__ float4 lds4(const unsigned char* p, float) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 lds4(const unsigned char* p, f16) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 x = Pair<f16>::unpack(u.x), y = Pair<f16>::unpack(u.y);
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 lds4(const unsigned char* p, bf16) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}

template <typename T, int HD>
__global__ void __launch_bounds__(SimtCfg<T, HD>::NT, 1) paged_simt_kernel(const PagedAttnArgs a) {
  using C = SimtCfg<T, HD>;
  using Ld = typename C::Ld;
  constexpr int NW = C::NW, NS = C::NS, HB = C::HB, RW = C::RW, CS = comb_stride(HD), TILE = Ld::TILE;
  constexpr int G4 = HD / 4;                    // groups of 4 dimensions
  constexpr int PG = G4 >= 32 ? 1 : 32 / G4;    // lanes that share a group, by position
  constexpr int GL = G4 >= 32 ? G4 / 32 : 1;    // groups a lane owns
  static_assert(NS >= 2, "ring");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[NW][NS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * NW * Ld::STAGE);
  float* qs = comb + NW * HB * CS;                           // [HB][HD]
  float* ps = qs + HB * HD + warp * (RW + 1) * HB;           // [RW][HB] probabilities, then [HB] factors
  unsigned char* ring_p = pa_smem + warp * NS * Ld::STAGE;
  const uint32_t ring = smem_addr(ring_p);
  write_empty(a);
  Place ld;
  const Range r = find_range<TILE, C::NT>(a, n_units, ld);
  if (r.begin >= r.end) return;
  Place p = ld;
  long long to_load = r.end - r.begin, left = to_load;
  long long row_off = Ld::row(a, ld, n_hb, warp, lane);
  int ld_stage = 0;
  auto load_next = [&]() {
    if (to_load > 0) {
      Ld::request(a, row_off, ring + ld_stage * Ld::STAGE, lane);
      const uint32_t mask = __ballot_sync(0xffffffffu, row_off >= 0);
      if (lane == 0) s_mask[warp][ld_stage] = mask;
      if (--to_load > 0) {
        advance<TILE>(a, n_units, ld);
        row_off = Ld::row(a, ld, n_hb, warp, lane);
      }
    }
    cp_commit();
    if (++ld_stage == NS) ld_stage = 0;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load_next();
  int stage = 0;
  const int pos = lane & 7, quarter = lane >> 3;
  const int vg = G4 >= 32 ? lane : lane % G4, vp = G4 >= 32 ? 0 : lane / G4;
  const float sc = a.scale * LOG2E;
  auto grp = [&](const unsigned char* half, int row, int g4) {  // 4 dimensions of a row
    constexpr int B4 = 4 * (int)sizeof(T);
    const int byte = g4 * B4;
    return lds4(half + Ld::at(row, byte / 16) + byte % 16, T());
  };
  while (left > 0) {
    const int t0 = p.t, t1 = (int)min((long long)p.nt, t0 + left);
    {
      const int g = p.u / n_hb, h0 = (p.u - g * n_hb) * HB;
      for (int i = tid; i < HB * HD; i += C::NT) {
        const int h = i / HD, d = i - h * HD;
        qs[i] = h0 + h < group && d < a.hd ? load_io(a.q, p.b * a.q_stride + (long long)(g * group + h0 + h) * a.hd + d, a.io) : 0.f;
      }
    }
    __syncthreads();
    float4 o[HB][GL];
#pragma unroll
    for (int h = 0; h < HB; ++h)
#pragma unroll
      for (int i = 0; i < GL; ++i) o[h][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2 quarter, 2 quarter + 1
    for (int t = t0; t < t1; ++t) {
      cp_wait<NS - 2>();
      __syncwarp();
      load_next();  // into the stage that the last tile used
      const uint32_t mask = s_mask[warp][stage];
      if (mask) {
        const unsigned char *ks = ring_p + stage * Ld::STAGE, *vs = ks + Ld::STAGE / 2;
        float dot[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) dot[h] = 0.f;
#pragma unroll
        for (int i = 0; i < G4 / 4; ++i) {
          const float4 k4 = grp(ks, pos, quarter + 4 * i);
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            const float4 q4 = *reinterpret_cast<const float4*>(qs + h * HD + (quarter + 4 * i) * 4);
            dot[h] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, dot[h]))));
          }
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          float d = dot[h];
          d += __shfl_xor_sync(0xffffffffu, d, 8);
          d += __shfl_xor_sync(0xffffffffu, d, 16);
          if ((h >> 1) == quarter) s[h & 1] = d;
        }
        const bool there = (mask >> pos) & 1;
        float2 f, e;
        {
          float fe[2], ee[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = there ? s[i] * sc : -INFINITY;
            float top = x;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
            fe[i] = exp2f(m[i] - ref);
            if (m[i] == -INFINITY) fe[i] = mn == -INFINITY ? 1.f : 0.f;
            ee[i] = exp2f(x - (ref - PA_BIAS));
            l[i] = fmaf(l[i], fe[i], ee[i]);  // this lane's position only
            m[i] = mn;
          }
          f = make_float2(fe[0], fe[1]);
          e = make_float2(ee[0], ee[1]);
        }
        *reinterpret_cast<float2*>(ps + pos * HB + 2 * quarter) = e;
        if (pos == 0) *reinterpret_cast<float2*>(ps + RW * HB + 2 * quarter) = f;
        const bool moved = __any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f);
        __syncwarp();
        if (moved) {
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            const float w = ps[RW * HB + h];
#pragma unroll
            for (int i = 0; i < GL; ++i) {
              o[h][i].x *= w; o[h][i].y *= w; o[h][i].z *= w; o[h][i].w *= w;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < RW; j += PG) {
          const int row = j + vp;
          const float4 pa = *reinterpret_cast<const float4*>(ps + row * HB), pb = *reinterpret_cast<const float4*>(ps + row * HB + 4);
          const float w[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
          for (int i = 0; i < GL; ++i) {
            const float4 v4 = grp(vs, row, vg + 32 * i);
#pragma unroll
            for (int h = 0; h < HB; ++h) {
              o[h][i].x = fmaf(w[h], v4.x, o[h][i].x);
              o[h][i].y = fmaf(w[h], v4.y, o[h][i].y);
              o[h][i].z = fmaf(w[h], v4.z, o[h][i].z);
              o[h][i].w = fmaf(w[h], v4.w, o[h][i].w);
            }
          }
        }
      }
      __syncwarp();
      if (++stage == NS) stage = 0;
    }
    float* cw = comb + (size_t)warp * HB * CS;
#pragma unroll
    for (int h = 0; h < HB; ++h)
#pragma unroll
      for (int i = 0; i < GL; ++i) {
        float4 x = o[h][i];
#pragma unroll
        for (int s = G4; s < 32; s <<= 1) {  // the lanes that share the group
          x.x += __shfl_xor_sync(0xffffffffu, x.x, s);
          x.y += __shfl_xor_sync(0xffffffffu, x.y, s);
          x.z += __shfl_xor_sync(0xffffffffu, x.z, s);
          x.w += __shfl_xor_sync(0xffffffffu, x.w, s);
        }
        if (vp == 0) *reinterpret_cast<float4*>(cw + h * CS + (vg + 32 * i) * 4) = x;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      if (pos == 0) {
        cw[(2 * quarter + i) * CS + HD] = m[i];
        cw[(2 * quarter + i) * CS + HD + 1] = sum;
      }
    }
    Finish<HB, HD, C::NT>::unit(a, r, p, n_units, n_hb, NW, comb, t0, t1);
    left -= t1 - t0;
    p.t = t1 - 1;
    if (left > 0) advance<TILE>(a, n_units, p);
  }
  cp_wait<0>();
}

// ---- host ------------------------------------------------------------------------------------------------------

template <typename K>
cudaError_t launch(K kernel, int threads, int smem, int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e ? e : launch_k(kernel, dim3(ctas), dim3(threads), smem, s, false, a);
}
template <typename T, int HD, int HB, bool F32IO>
cudaError_t launch_mma(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  using C = MmaCfg<T, HD, HB, F32IO>;
  return launch(paged_mma_kernel<T, HD, HB, F32IO>, C::NT, C::SMEM, ctas, a, s);
}
template <typename T, bool F32IO>
cudaError_t pick_mma(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  // heads of other sizes are padded with zeros in shared memory to the next instance
  if (a.nq / a.nkv <= 8)
    return a.hd <= 32   ? launch_mma<T, 32, 8, F32IO>(ctas, a, s)
           : a.hd <= 64 ? launch_mma<T, 64, 8, F32IO>(ctas, a, s) : launch_mma<T, 128, 8, F32IO>(ctas, a, s);
  return a.hd <= 64 ? launch_mma<T, 64, 16, F32IO>(ctas, a, s) : launch_mma<T, 128, 16, F32IO>(ctas, a, s);
}
template <typename T, int HD>
cudaError_t launch_simt(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  using C = SimtCfg<T, HD>;
  return launch(paged_simt_kernel<T, HD>, C::NT, C::SMEM, ctas, a, s);
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
                  (unsigned int*)workspace, (float*)((char*)workspace + COUNTER_BYTES), err_dev, io_dtype};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  const int ctas = nsm < PA_MAX_CTAS ? nsm : PA_MAX_CTAS;
  if (c.dtype == QW_F32)
    e = c.head_dim <= 32    ? launch_simt<float, 32>(ctas, a, s)
        : c.head_dim <= 64  ? launch_simt<float, 64>(ctas, a, s)
        : c.head_dim <= 128 ? launch_simt<float, 128>(ctas, a, s) : launch_simt<float, 256>(ctas, a, s);
  else if (c.dtype == QW_F16)
    e = c.head_dim > 128     ? launch_simt<f16, 256>(ctas, a, s)
        : io_dtype == QW_F32 ? pick_mma<f16, true>(ctas, a, s) : pick_mma<f16, false>(ctas, a, s);
  else
    e = c.head_dim > 128     ? launch_simt<bf16, 256>(ctas, a, s)
        : io_dtype == QW_F32 ? pick_mma<bf16, true>(ctas, a, s) : pick_mma<bf16, false>(ctas, a, s);
  if (e) return op_cuda_fail(e, "paged attention launch");
  return QW_OK;
}

}  // extern "C"
