// The shared positions of attn_shared.cu on the 5th-generation tensor cores (tcgen05, TMEM) for 16-bit callers, heads of at
// most 128 dimensions.
//
// Two chains of products run side by side, so that one's products fill the time of the other's softmax: S = Q K^T (128 rows x
// 128 positions), P = 2^(S - m) in two pieces written over it, O += P V, all in TMEM. A unit of more than 128 rows has its first 128 in
// chain A and the others in chain B, over the same blocks of keys and values; one of fewer rows has its even blocks in A and
// its odd ones in B, with a state each.
//   warps 0 .. 3     producers (attn_shared_tc.cuh)
//   warps 12, 13     issue the products of a chain each: S, then in turn P V and the next S. A step's products take the tensor
//                    cores' queue as a whole, so that the chains stay half a step apart; mixed, both wait for the
//                    products at the same time and then for the softmax (4000 cycles a block of 256 rows). (One warp for both
//                    chains is in their way, too: a step's waits and commits take it as long as the products themselves,
//                    4200 cycles.)
//   warps 4 .. 7     softmax of chain A, 8 .. 11 of chain B: one row a lane, 64 of its 128 scores in registers at a time, once for the
//                    maximum, once for the probabilities (one pass, with the maximum of the block before, was within 2%)
// O stays in TMEM. Its reference m moves only when a row's maximum exceeds it by more than 2^5; then the warp rescales its
// rows of O, which is safe: S of a block is issued after the chain's last P V, so that is done when S arrives. P is at most
// 2^15 then, in fp16's range, and keeps its digits down to 2^-24 of the row's largest (PA_BIAS).
//
// Precision: probabilities are sums of two pieces of the cache's type, as over own positions and in attn_paged.cu (22 bits, bf16
// 16, so that the output's own rounding is what remains); their sum l takes them before that. One piece would save 8 of a step's
// 24 products, 13 us of 256 sequences behind 16383 positions, and raises bf16's error against 64 bits by a third. The tensor
// cores' additions cut: over 1000 products of 16 positions about 1e-5 of the norm, next to the output's 2^-9 or 2^-12.
// What bounds it: of many rows the chain of one block, S, softmax, P V, that the two chains fill to 53% of the tensor cores' time.
// 256 sequences, 28 and 4 heads of 128 behind 16383 positions: 72 us, 1260 TFLOP/s of products (840 of the formula's). Of few
// rows HBM and L2: 16 groups of 8 behind 512 to 4096 positions 30 us, 86 MB. The shares of 72 and 56 registers spill in the
// producers and issuers, 324 to 336 bytes of stores a thread.
//
// Every wait is bounded: on expiry ERR_TIMEOUT is set, the CTA stops issuing work, waits (bounded) for what it issued, and
// releases its TMEM.
#include <math.h>

#include "attn_shared_tc.cuh"

namespace qw {
namespace shared_attn {
namespace {

using paged::split;

constexpr int MT = 256, BK = TC_BK, THREADS = 512, MMA_WARP = 12, TMEM_WARP = 15;  // (a warp whose lanes never part allocates and frees TMEM)
constexpr float MOVE_AT = 5.f;  // base-2 growth of a row's maximum that moves its reference

template <int HD>
struct Cfg {
  static constexpr int TILE = BK * HD * 2;            // bytes of a tile; HD / 64 boxes [128 rows][64 columns]
  static constexpr int Q_BYTES = 2 * 128 * HD * 2;    // of both halves
  // q_full, s_full[2], p_full[2], o_full[2], done[2], idle, full[8], empty[8]
  static constexpr int NBAR = 10;                     // (with the ring's an even number: the masks behind are read 16 bytes at a time)
  static constexpr int SMALL = (NBAR + 2 * 8) * 8 + 16 + TC_MASKS * 16;
  static constexpr int NS_FIT = (232448 - Q_BYTES - SMALL) / TILE, NS = NS_FIT > 8 ? 8 : NS_FIT;
  static constexpr int OFF_RING = Q_BYTES, OFF_SMALL = OFF_RING + NS * TILE, SMEM = OFF_SMALL + SMALL;
  static constexpr int O_COL = 256;                   // TMEM columns: S of both chains (P over them), then O of both
  static_assert(NS >= 4, "ring");
  static_assert((OFF_SMALL + (NBAR + 16) * 8 + 16) % 16 == 0, "masks");
};

// The tiles of a unit of nb blocks in the ring's order K_0, K_1, V_0, K_2, V_1, ..., V_{nb-1}
__device__ __forceinline__ int k_tile(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_tile(int j, int nb) { return j + 1 < nb ? 2 * j + 2 : 2 * nb - 1; }

template <typename T, int HD>
__global__ void __launch_bounds__(THREADS, 1) shared_pair_kernel(const __grid_constant__ PageMaps maps, const SharedArgs a) {
  using C = Cfg<HD>;
  constexpr int NS = C::NS;
  constexpr bool BF = std::is_same<T, bf16>::value;
  extern __shared__ __align__(1024) unsigned char sh_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  const uint32_t base = smem_addr(sh_smem);
  uint64_t* bars = (uint64_t*)(sh_smem + C::OFF_SMALL);
  const uint32_t q_full = smem_addr(bars), s_full0 = q_full + 8, p_full0 = q_full + 24, o_full0 = q_full + 40, done = q_full + 56,
                 idle = q_full + 72, full0 = q_full + 80, empty0 = full0 + 64;
  uint32_t* tmem_slot = (uint32_t*)(bars + C::NBAR + 16);
  volatile int* s_abort = (volatile int*)(tmem_slot + 1);
  volatile int* s_turn = (volatile int*)(tmem_slot + 2);  // 1: a chain's products are being issued
  uint32_t* masks = tmem_slot + 4;  // [block % TC_MASKS][4] positions that exist
  if (base & 1023) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(a.p.err, ERR_LAYOUT);
    pdl_wait();
    return;
  }
  Unit p;
  const Range r = find_groups<MT, BK, THREADS>(a, p, sh_smem);
  if (r.begin >= r.end) {
    pdl_wait();  // (this grid ends after the one before it)
    return;
  }
  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_turn = 0;
    mbar_init(q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(p_full0 + 8 * i, 4);
      mbar_init(o_full0 + 8 * i, 1);
    }
    mbar_init(done, 1);
    mbar_init(done + 8, 1);
    mbar_init(idle, 10);  // the softmax warps and the issuers
    for (int i = 0; i < NS; ++i) {
      mbar_init(full0 + 8 * i, TC_PRODUCERS);
      mbar_init(empty0 + 8 * i, 2);
    }
    mbar_fence_init();
  }
  if (warp == TMEM_WARP) tc::tmem_alloc(smem_addr(tmem_slot), 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int* err = a.p.err;

  if (warp < TC_PRODUCERS) {
    setmaxnreg_dec<72>();
    produce<T, MT, HD, NS>(a, maps, r, p, base + C::OFF_RING, full0, empty0, masks, s_abort);
  } else if (warp >= 12) {
    setmaxnreg_dec<56>();
    if (warp < MMA_WARP + 2 && lane == 0) {
      // ---- issues the products of chain c
      constexpr uint32_t kind = BF ? 1u << 7 | 1u << 10 : 0u;
      constexpr uint32_t idS = tc::idesc_f16(128, BK) | kind, idO = tc::idesc_f16_bmn(128, HD) | kind;
      const int c = warp - MMA_WARP;
      const uint32_t s_full = s_full0 + 8 * c, p_full = p_full0 + 8 * c, s_col = tmem + c * 128, o_col = tmem + C::O_COL + c * 128;
      int tile0 = 0, units = 0, steps = 0;  // tiles before the unit, units, steps so far
      bool ok = true;
      auto turn = [&]() {  // the tensor cores' queue for a whole step: false if the other chain does not give it up
        if (atomicCAS((int*)s_turn, 0, 1) == 0) return true;
        const long long t0 = clock64();
        while (atomicCAS((int*)s_turn, 0, 1) != 0)
          if (clock64() - t0 > tc::WAIT_BUDGET) {
            atomicOr(err, ERR_TIMEOUT);
            return false;
          }
        return true;
      };
      do {
        const int nb = blocks_of<MT>(p, r.end);
        const bool two = p.c == 2;  // both halves have rows
        if (!(ok = wait_for(q_full, units & 1, err))) break;
        ++units;
        // Tile i of the unit. A wait names a phase by its parity only, so that a chain sees every tile of a slot land, and no slot is
        // filled again before both have: a tile of the other chain is waited for in its turn, too, and given back at once.
        auto landed = [&](int i, uint32_t& addr) {
          const uint32_t n = tile0 + i, s = n % NS;
          addr = base + C::OFF_RING + s * C::TILE;
          return wait_for(full0 + 8 * s, n / NS & 1, err);
        };
        auto release = [&](int i) { tc::mma_commit(empty0 + 8 * ((uint32_t)(tile0 + i) % NS)); };
        int seen = 0;  // where the halves take even and odd blocks: tiles before it are used or passed by
        auto pass_to = [&](int i) {
          if (two) return true;
          for (; seen < i; ++seen) {
            uint32_t addr;
            if (!landed(seen, addr)) return false;
            mbar_arrive(empty0 + 8 * ((uint32_t)(tile0 + seen) % NS));
          }
          ++seen;
          return true;
        };
        const uint32_t ql = desc_lo(base) + (two ? c * (128 * HD * 2 >> 4) : 0);
        auto products_s = [&](uint32_t k) {
          const uint32_t kl = desc_lo(k);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const int at = ((kk >> 2) * 128 * 128 + (kk & 3) * 32) >> 4;
            mma_ss(s_col, ql + at, kl + at, idS, kk > 0);
          }
          tc::mma_commit(s_full);
        };
        const int step = two ? 1 : 2;
        int j = two ? 0 : c;
        bool first = true;
        uint32_t k, v;
        if (j < nb && (ok = pass_to(k_tile(j)) && landed(k_tile(j), k))) {
          tc::tc_fence_after();
          if ((ok = turn())) {
            products_s(k);
            *s_turn = 0;
            release(k_tile(j));
          }
        }
        for (; j < nb && ok; j += step) {
          const bool more = j + step < nb;
          // (the tiles landed long ago, mostly: their waits pass while the softmax is at work)
          ok = !*s_abort && pass_to(v_tile(j, nb)) && landed(v_tile(j, nb), v) && (!more || (pass_to(k_tile(j + step)) && landed(k_tile(j + step), k))) &&
               wait_for(p_full, steps & 1, err) && turn();
          if (!ok) break;
          ++steps;
          tc::tc_fence_after();
          const uint32_t vl = desc_lo(v, BK * 128);
#pragma unroll
          for (int piece = 1; piece >= 0; --piece)  // the lower one first
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_ts(o_col, s_col + (kk >> 2) * 64 + piece * 32 + (kk & 3) * 8, vl + kk * (2048 >> 4), idO, !first || piece == 0 || kk > 0);
          first = false;
          if (more) products_s(k);
          else tc::mma_commit(o_full0 + 8 * c);
          *s_turn = 0;
          release(v_tile(j, nb));
          if (more) release(k_tile(j + step));
        }
        if (ok) ok = pass_to(2 * nb);
        mbar_arrive(idle);  // (so that no issuer is a unit behind)
        tile0 += 2 * nb;
      } while (ok && next_unit<MT, BK>(a, r.end, p));
      if (!ok) *s_abort = 1;
      tc::mma_commit(done + 8 * c);  // arrives once all products issued above are done
      wait_for(done + 8 * c, 0, err);
    }
  } else {
    setmaxnreg_inc<192>();
    // ---- softmax: chain c, row `row` of its 128
    const int c = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), s_at = lanes + c * 128, o_at = lanes + C::O_COL + c * 128;
    // (the scale's sign goes to the queries; 0 becomes the least positive number, with which masked scores stay -inf and no
    // finite score lies further than 1e-6 from 0)
    const float sc = fmaxf(fabsf(a.p.scale) * paged::LOG2E, __uint_as_float(1u));
    int block0 = 0, units = 0, steps = 0, segments = 0;
    bool ok = true;
    do {
      const int kv = p.u / p.nt, tile = p.u - kv * p.nt, nb = blocks_of<MT>(p, r.end);
      const bool two = p.c == 2;
      if (units > 0 && !wait_for(idle, (units - 1) & 1, err)) ok = false;  // (all products of the last unit are done)
      const Row mine = row_of(a, p, kv, tile * MT + (two ? c * 128 : 0) + row);
      if (two || c == 0) {  // the queries of the warp's rows, all requested at once; zeros for rows that take no part
        constexpr int CH = HD / 8, RP = 32 / CH;  // chunks of a row, rows a step
        const int ch = lane % CH, w0 = (warp & 3) * 32;
        const uint32_t at = base + c * (128 * HD * 2) + (ch >> 3) * (128 * 128);
        const long long q_row = mine.in ? mine.b * a.p.q_stride + mine.h * a.p.hd : -1;
#pragma unroll 4
        for (int i = 0; i < 32; i += RP) {
          const int rr = i + lane / CH;
          const long long off = __shfl_sync(0xffffffffu, q_row, rr);
          const bool there = off >= 0 && ch * 8 < a.p.hd;
          paged::cp_async16_or_zero(at + (w0 + rr) * 128 + (((ch & 7) ^ (rr & 7)) << 4), (const T*)a.p.q + (there ? off + ch * 8 : 0), there);
        }
        paged::cp_commit();
        paged::cp_wait<0>();
        if (a.p.scale < 0.f) {  // (the scale's sign goes to the queries: each lane's own chunks)
#pragma unroll 1
          for (int i = 0; i < 32; i += RP) {
            const int rr = i + lane / CH;
            uint4* x = reinterpret_cast<uint4*>(sh_smem + (at - base) + (w0 + rr) * 128 + (((ch & 7) ^ (rr & 7)) << 4));
            uint4 v = *x;
            v.x ^= 0x80008000u; v.y ^= 0x80008000u; v.z ^= 0x80008000u; v.w ^= 0x80008000u;
            *x = v;
          }
        }
        fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      const int n = two ? nb : c == 0 ? (nb + 1) / 2 : nb / 2;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        if (*s_abort || !wait_for(s_full0 + 8 * c, steps & 1, err)) ok = false;
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++steps;
        tc::tc_fence_after();
        const uint32_t* mask = masks + ((block0 + (two ? i : 2 * i + c)) % TC_MASKS) * 4;
        // the block's maximum, 64 positions at a time; scores of positions that are not there become -inf in TMEM
        float mx = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t u[64];
          tc::tmem_ld32_nowait(s_at + 64 * h, u);
          tc::tmem_ld32_nowait(s_at + 64 * h + 32, u + 32);
          tc::tmem_wait_ld();
          const uint2 there = *reinterpret_cast<const uint2*>(mask + 2 * h);
          any |= (there.x | there.y) != 0u;
          if ((there.x & there.y) != 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              if (!(there.x >> q & 1)) u[q] = 0xff800000u;
              if (!(there.y >> q & 1)) u[32 + q] = 0xff800000u;
            }
            tc::tmem_st32(s_at + 64 * h, u);
            tc::tmem_st32(s_at + 64 * h + 32, u + 32);
            tc::tmem_wait_st();
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 32; ++q) top[q & 3] = max3(top[q & 3], __uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1]));
          mx = fmaxf(mx, fmaxf(max3(top[0], top[1], top[2]), top[3]));
        }
        mx *= sc;
        const bool move = mx > m + MOVE_AT || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? ex2(m - mx) : 1.f;  // (0 where m is -inf)
          if (i > 0) {
#pragma unroll 1
            for (int d = 0; d < HD; d += 32) {
              uint32_t o[32];
              tc::tmem_ld32_nowait(o_at + d, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
              tc::tmem_st32(o_at + d, o);
            }
          }
          if (move) {
            l *= f;
            m = mx;
          }
          __syncwarp();
        }
        const float ref = (m == -INFINITY ? 0.f : m) - PA_BIAS;
        const f32x2 c2 = pack2(sc, sc), r2 = pack2(-ref, -ref);
        f32x2 acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // (both pieces of a half's probabilities go over its scores)
          uint32_t u[64], w[2][32];
          tc::tmem_ld32_nowait(s_at + 64 * h, u);
          tc::tmem_ld32_nowait(s_at + 64 * h + 32, u + 32);
          tc::tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float2 e = unpack2(fma2_to(pack2(__uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1])), c2, r2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            acc[q & 3] = add2(acc[q & 3], pack2(p0, p1));
            uint32_t pieces[2];
            split<T, 2>(p0, p1, pieces);
            w[0][q] = pieces[0];
            w[1][q] = pieces[1];
          }
          tc::tmem_st32(s_at + 64 * h, w[0]);
          tc::tmem_st32(s_at + 64 * h + 32, w[1]);
        }
        const float2 s0 = unpack2(add2(acc[0], acc[1])), s1 = unpack2(add2(acc[2], acc[3]));
        l += (s0.x + s0.y) + (s1.x + s1.y);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full0 + 8 * c);
      }
      if (ok && n > 0 && !wait_for(o_full0 + 8 * c, segments & 1, err)) ok = false;
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (n > 0) ++segments;
      tc::tc_fence_after();
      __syncwarp();
      if (lane == 0) mbar_arrive(idle);
      block0 += nb;
      ++units;
      const bool whole = nb == p.nb;
      float* dst = mine.in ? state_of<MT, HD>(a, r, p, whole, mine, c * 128 + row, !two && c) : nullptr;
      const int width = whole ? a.p.hd : HD;
      if (n > 0) {
#pragma unroll 1
        for (int d = 0; d < HD; d += 32) {
          float o[32];
          __syncwarp();  // (the lanes' stores part them; TMEM is read by whole warps)
          tc::tmem_ld32(o_at + d, o);
          if (dst)
#pragma unroll
            for (int q = 0; q < 32; q += 4)
              if (d + q < width) *reinterpret_cast<float4*>(dst + d + q) = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
        }
      }
      tc::tc_fence_before();
      if (dst) *reinterpret_cast<float2*>(dst + width) = make_float2(paged::state_max(m, any), l);
    } while (next_unit<MT, BK>(a, r.end, p));
    if (!ok) *s_abort = 1;
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == TMEM_WARP) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  pdl_wait();  // (this grid ends after the one before it)
}

template <typename T, int HD>
cudaError_t run(int ctas, const PageMaps& m, const SharedArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(shared_pair_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::SMEM);
  return e ? e : launch_k(shared_pair_kernel<T, HD>, dim3(ctas), dim3(THREADS), Cfg<HD>::SMEM, s, true, m, a);
}

}  // namespace

cudaError_t launch_shared_pair(const qw_paged_kv& cache, int ctas, const SharedArgs& a, cudaStream_t s) {
  PageMaps m{};
  make_page_maps(cache, m);
  if (cache.dtype == QW_F16) return a.p.hd <= 64 ? run<f16, 64>(ctas, m, a, s) : run<f16, 128>(ctas, m, a, s);
  return a.p.hd <= 64 ? run<bf16, 64>(ctas, m, a, s) : run<bf16, 128>(ctas, m, a, s);
}

}  // namespace shared_attn
}  // namespace qw
