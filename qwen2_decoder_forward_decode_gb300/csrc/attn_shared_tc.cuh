// What the two tensor-core kernels of attn_shared.cu have in common: the producers that fill a ring of key and value tiles.
#pragma once

#include "attn_shared.cuh"
#include "tc_common.cuh"

namespace qw {
namespace shared_attn {

constexpr int TC_BK = 128, TC_PRODUCERS = 4, TC_MASKS = 16;

// Every launch meets these kernels' code cold, and fetching it costs about a cycle a byte: what does not run in the main loop is
// kept short (loops, one place for a piece of code, functions of their own).

// Bounded wait, as tc::mbar_wait, with the waiting out of line.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, int* err) { return tc::mbar_wait(bar, parity, err); }
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int* err) { return mbar_test(bar, parity) || wait_long(bar, parity, err); }

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 16 columns of this thread's TMEM lane, completed by tmem_wait_st
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Products with operands in shared memory given by the lower halves of their descriptors (address and leading offset, see
// tc_common.cuh; the upper halves are constants). One thread issues all products, and its instructions set the pace: a descriptor
// is an addition here, where building each from its address took 60 to 90 cycles a product.
constexpr uint32_t DESC_HI = 1024u >> 4 | 1u << 14 | 2u << 29;  // 8-row atoms 1024 bytes apart, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo = 16) { return addr >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DESC_HI)
      : "memory");
}
// the A operand in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DESC_HI)
      : "memory");
}

// The caches as tensor maps, with boxes of `rows` positions; rows 0: no maps.
struct PageMaps {
  CUtensorMap k, v;
  int rows;
};

// Boxes lie within a page and within a warp's 32 positions, and begin on the swizzle's 8-row pattern: pages of multiples of 8.
inline void make_page_maps(const qw_paged_kv& c, PageMaps& m) {
  int rows = 32;
  while (rows >= 8 && c.page_size % rows) rows /= 2;
  m.rows = rows >= 8 && make_map_pages(&m.k, c.k, c, rows) && make_map_pages(&m.v, c.v, c, rows) ? rows : 0;
}

// Four warps fill a ring of NS tiles [128 positions][HD] (HD / 64 boxes of 64 columns, 128-byte swizzle) in the order
// K_0, K_1, V_0, K_2, V_1, ..., V_{n-1} of every unit; a warp owns 32 positions of each tile.
//   - Where pages hold multiples of 8 positions, TMA copies them, a box a page or part of one.
//   - Else, and where a block is cut by the shared part's end or has a bad page, cp.async does, 16 bytes a lane, with zeros for
//     positions that are not there. It moves about 26 bytes a cycle and SM where TMA keeps up with L2 (16383 positions, 256
//     sequences: 4200 cycles a block of 128 rows and positions against 1300 of products).
// full[NS] expects TC_PRODUCERS arrivals, empty[NS] what the caller set. masks [TC_MASKS][4]: the positions of a block that exist.
template <typename T, int MT, int HD, int NS>
__device__ __forceinline__ void produce(const SharedArgs& a, const PageMaps& maps, const Range& r, Unit p, uint32_t ring, uint32_t full0,
                                        uint32_t empty0, uint32_t* masks, volatile int* s_abort) {
  constexpr int CH = HD / 8, RP = 32 / CH, TILE = TC_BK * HD * 2;  // chunks of a row, rows a step
  constexpr int AHEAD = NS - 1 < 4 ? NS - 1 : 4;                   // tiles in flight by cp.async
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane % CH, r0 = lane / CH;
  const bool col = ch * 8 < a.p.hd;
  const bool mine = maps.rows && lane * maps.rows < 32;  // this lane asks for a box
  int n = 0, told = 0, block = 0;                        // tiles requested, tiles announced, blocks begun
  bool ok = true;
  auto announce = [&](int upto) {  // (their copies have landed)
    fence_proxy_async();
    __syncwarp();
    if (lane == 0)
      for (int i = told; i < upto; ++i) mbar_arrive(full0 + 8 * (i % NS));
    told = upto;
  };
  struct Rows {
    bool boxes;
    int id, at;      // a lane's box: page and position in it
    long long off;   // a lane's row
    uint32_t mask;
  };
  // the entry of the table that the lane's box of block t needs
  auto entry = [&](int t) {
    const int pos = t * TC_BK + warp * 32 + lane * maps.rows;
    return mine && pos < p.pre ? __ldg(a.p.table + (size_t)p.lo * a.p.max_blocks + pos / a.p.page) : -1;
  };
  auto find = [&](int kv, int t, int id) {
    Rows x{false, id, 0, 0, 0xffffffffu};
    const int first = t * TC_BK + warp * 32;
    if (maps.rows && first + 32 <= p.pre) {
      x.at = (first + lane * maps.rows) % a.p.page;
      x.boxes = __all_sync(0xffffffffu, !mine || (id >= 0 && id < a.p.n_pages));
    }
    if (!x.boxes) {
      x.off = position_of<T>(a, p, kv, first + lane);
      x.mask = __ballot_sync(0xffffffffu, x.off >= 0);
      if (x.off < 0) x.off = 0;
    }
    return x;
  };
  auto request = [&](bool values, int kv, const Rows& x) {
    const void* cache = values ? a.p.v : a.p.k;
    const CUtensorMap* map = values ? &maps.v : &maps.k;
    const int s = n % NS;
    const uint32_t full = full0 + 8 * s;
    if (n >= NS) {
      const uint32_t par = (n / NS & 1) ^ 1;
      if (!__all_sync(0xffffffffu, mbar_test(empty0 + 8 * s, par))) {  // (one answer for the warp: it announces together)
        if (told < n) {
          paged::cp_wait<0>();
          announce(n);
        }
        if (!wait_long(empty0 + 8 * s, par, a.p.err)) *s_abort = 1;
      }
    }
    if (*s_abort) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    const uint32_t dst = ring + s * TILE + warp * 32 * 128;
    if (x.boxes) {
      if (told < n) {  // (announced in order)
        paged::cp_wait<0>();
        announce(n);
      }
      if (lane == 0) mbar_expect_tx(full, 32 * HD * 2);
      __syncwarp();
      if (mine) {
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) tma_load_4d(dst + c * (TC_BK * 128) + lane * maps.rows * 128, map, full, c * 64, x.at, kv, x.id);
      }
      told = ++n;
      return;
    }
    const char* src = (const char*)cache + ch * 16;
#pragma unroll 4
    for (int i = 0; i < 32 / RP; ++i) {
      const int row = i * RP + r0;
      const long long o = __shfl_sync(0xffffffffu, x.off, row);
      paged::cp_async16_or_zero(dst + (ch >> 3) * (TC_BK * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), src + o, (x.mask >> row & 1) && col);
    }
    paged::cp_commit();
    ++n;
    if (n - told > AHEAD) {
      paged::cp_wait<AHEAD>();
      announce(n - AHEAD);
    }
  };
  do {
    const int kv = p.u / p.nt, t1 = p.t + blocks_of<MT>(p, r.end);
    int id = entry(p.t), t = p.t;
    Rows now{}, last{};
#pragma unroll 1
    for (int i = 0, end = 2 * (t1 - p.t); i < end && ok; ++i) {  // K_0, K_1, V_0, ..., V_{n-1}
      const bool values = i > 0 && (i % 2 == 0 || i + 1 == end);
      if (!values) {
        last = now;
        now = find(kv, t, id);
        if (t + 1 < t1) id = entry(t + 1);
        ++t;
        if (lane == 0) masks[(block % TC_MASKS) * 4 + warp] = now.mask;
        ++block;
      }
      request(values, kv, values && i + 1 < end ? last : now);
    }
  } while (ok && next_unit<MT, TC_BK>(a, r.end, p));
  paged::cp_wait<0>();
  if (told < n) announce(n);
  // every copy lands before the shared memory is released
  if (lane == 0)
    for (int i = n > NS ? n - NS : 0; i < n; ++i) tc::mbar_wait(full0 + 8 * (i % NS), i / NS & 1, a.p.err);
}

}  // namespace shared_attn
}  // namespace qw
