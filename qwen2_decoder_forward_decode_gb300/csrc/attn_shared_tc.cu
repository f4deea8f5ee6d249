// The shared positions of attn_shared.cu on the 5th-generation tensor cores (tcgen05, TMEM) for fp32 callers over 16-bit caches,
// heads of at most 128 dimensions.
//
// A unit is 128 rows (sequence, head) of one group and KV head. Blocks of 128 positions stream past them:
//   warps 0 .. 3    producers (attn_shared_tc.cuh): tiles of keys and values in the order in which they are consumed.
//   warp 12         issues the products: S_j = Q K_j^T into buffer j % 2, a block ahead, and O_j = P_j V_j with P_j from TMEM.
//   warps 4 .. 11   softmax. Warps w and w + 4 share TMEM lanes, one row a lane: the first takes positions 0 .. 63 of every
//                   block, the other 64 .. 127, and they trade maxima through shared memory. They write P_j over S_j, and
//                   then add O_{j-1} to their half of the row's output in registers, a fp32 sum that rounds (the tensor
//                   cores' additions cut: over thousands of positions 1e-6 of the norm) and needs no rescaling in TMEM.
// The warps meet at a unit's ends only: there the softmax warps put the rows' queries into shared memory.
//
// Precision: queries and probabilities are sums of pieces of the cache's type, two of fp16 (22 bits of the row's largest
// element), three of bf16, whose products are added up lowest piece first. Exponentials are ex2's, good to 2^-22.
//
// What bounds it: the softmax and the fold of O, 128 rows by 8 warps, and of bf16 caches the products of three pieces. 256 sequences,
// 28 and 4 heads of 128 behind 16383 positions: 132 us with the fp16 cache, 173 with bf16; behind 8000 88. The registers' shares spill:
// 236 to 376 bytes of stores a thread.
//
// Every wait is bounded: on expiry ERR_TIMEOUT is set, the CTA stops issuing work, waits (bounded) for what it issued, and
// releases its TMEM.
#include <math.h>

#include "attn_shared_tc.cuh"

namespace qw {
namespace shared_attn {
namespace {

using paged::Pair;
using paged::split;

constexpr int MT = 128, BK = TC_BK, THREADS = 512, MMA_WARP = 12, TMEM_WARP = 15;  // (a warp whose lanes never part allocates and frees TMEM)

template <typename T, int HD>
struct Cfg {
  static constexpr bool BF = std::is_same<T, bf16>::value, three = BF;
  static constexpr int NQ = three ? 3 : 2, NP = NQ;  // pieces of queries and probabilities
  static constexpr int TILE = BK * HD * 2;                        // bytes of a tile; HD / 64 boxes [128 rows][64 columns]
  static constexpr int Q_BYTES = NQ * MT * HD * 2;
  // q_full, s_full[2], p_full[2], o_full[2], done, pair[4], full[NS], empty[NS]
  static constexpr int NBAR = 12;
  static constexpr int SMALL = (NBAR + 2 * 8) * 8 + 16 + MT * 4 + 2 * 2 * MT * 4 + TC_MASKS * 16;
  static constexpr int NS_FIT = (232448 - Q_BYTES - SMALL) / TILE, NS = NS_FIT > 8 ? 8 : NS_FIT;
  static constexpr int OFF_RING = Q_BYTES, OFF_SMALL = OFF_RING + NS * TILE, SMEM = OFF_SMALL + SMALL;
  // TMEM columns: S buffers (P pieces 0 and 1 over them), third pieces, O
  static constexpr int P3 = 256, O_COL = three ? 384 : 256, NO = three ? 1 : 2;
  static_assert(NS >= 4, "ring");
  static_assert(O_COL + NO * 128 <= 512, "TMEM");
};

template <typename T, int HD>
__global__ void __launch_bounds__(THREADS, 1) shared_tc_kernel(const __grid_constant__ PageMaps maps, const SharedArgs a) {
  using C = Cfg<T, HD>;
  constexpr int NS = C::NS, NQ = C::NQ, NP = C::NP;
  extern __shared__ __align__(1024) unsigned char sh_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  const uint32_t base = smem_addr(sh_smem);
  uint64_t* bars = (uint64_t*)(sh_smem + C::OFF_SMALL);
  const uint32_t q_full = smem_addr(bars), s_full0 = q_full + 8, p_full0 = q_full + 24, o_full0 = q_full + 40, done = q_full + 56,
                 pair0 = q_full + 64, full0 = q_full + 96, empty0 = full0 + 64;
  uint32_t* tmem_slot = (uint32_t*)(bars + C::NBAR + 16);
  volatile int* s_abort = (volatile int*)(tmem_slot + 1);
  float* undo = (float*)(tmem_slot + 4);                    // [MT] of the queries' power of two
  float* xch = undo + MT;                                   // [block parity][half][row]
  uint32_t* masks = (uint32_t*)(xch + 4 * MT);              // [block % TC_MASKS][4] positions that exist
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
    mbar_init(q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full0 + 8 * i, 1);
      mbar_init(p_full0 + 8 * i, 8);
      mbar_init(o_full0 + 8 * i, 1);
    }
    mbar_init(done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(pair0 + 8 * i, 2);
    for (int i = 0; i < NS; ++i) {
      mbar_init(full0 + 8 * i, TC_PRODUCERS);
      mbar_init(empty0 + 8 * i, 1);
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
    if (warp == MMA_WARP && lane == 0) {
      // ---- issues the products
      constexpr uint32_t kind = C::BF ? 1u << 7 | 1u << 10 : 0u;
      constexpr uint32_t idS = tc::idesc_f16(MT, BK) | kind, idO = tc::idesc_f16_bmn(MT, HD) | kind;
      int n = 0, block = 0, units = 0;  // tiles, blocks and units so far
      bool ok = true;
      do {
        const int nb = blocks_of<MT>(p, r.end);
        if (!(ok = wait_for(q_full, units & 1, err))) break;
        ++units;
        auto tile = [&](uint32_t& addr) {
          const int s = n % NS;
          if (!wait_for(full0 + 8 * s, n / NS & 1, err)) return false;
          tc::tc_fence_after();
          addr = base + C::OFF_RING + s * C::TILE;
          return true;
        };
        auto release = [&]() { tc::mma_commit(empty0 + 8 * (n++ % NS)); };
        auto issue_s = [&](int j) {  // j: block of all
          uint32_t k;
          if (!tile(k)) return false;
          const uint32_t ql = desc_lo(base), kl = desc_lo(k);
#pragma unroll
          for (int i = NQ - 1; i >= 0; --i)  // the lowest piece first
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const int at = ((kk >> 2) * MT * 128 + (kk & 3) * 32) >> 4;
              mma_ss(tmem + (j & 1) * 128, ql + (i * MT * HD * 2 >> 4) + at, kl + at, idS, i < NQ - 1 || kk > 0);
            }
          tc::mma_commit(s_full0 + 8 * (j & 1));
          release();
          return true;
        };
        ok = issue_s(block);
        for (int j = 0; j < nb && ok; ++j, ++block) {
          if (*s_abort) ok = false;
          // S of the next block goes where P of the last one was, whose product was issued before
          if (ok && j + 1 < nb) ok = issue_s(block + 1);
          if (!ok || !(ok = wait_for(p_full0 + 8 * (block & 1), block >> 1 & 1, err))) break;
          uint32_t v;
          if (!(ok = tile(v))) break;
          const uint32_t vl = desc_lo(v, BK * 128), o = tmem + C::O_COL + (block & 1) * (C::NO - 1) * 128;
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) {
            const uint32_t pc = tmem + (i < 2 ? (block & 1) * 128 + i * 64 : C::P3 + (block & 1) * 64);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) mma_ts(o, pc + kk * 8, vl + kk * (2048 >> 4), idO, i < NP - 1 || kk > 0);
          }
          tc::mma_commit(o_full0 + 8 * (block & 1));
          release();
        }
      } while (ok && next_unit<MT, BK>(a, r.end, p));
      if (!ok) *s_abort = 1;
      tc::mma_commit(done);  // arrives once all products issued above are done
      wait_for(done, 0, err);
    }
  } else {
    setmaxnreg_inc<192>();
    // ---- softmax
    constexpr int OC = HD / 2;  // output columns of a thread
    const int quarter = warp & 3, half = (warp - 4) >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16), pair = pair0 + 8 * quarter;
    const float sc = fabsf(a.p.scale) * paged::LOG2E, sign = a.p.scale > 0.f ? 1.f : a.p.scale < 0.f ? -1.f : 0.f;
    int block = 0, trades = 0;
    bool ok = true;
    auto trade = [&](float mine) -> float {  // the partner's value
      xch[(2 * (trades & 1) + half) * MT + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      if (!wait_for(pair, trades & 1, err)) ok = false;
      __syncwarp();  // (TMEM is read and written by whole warps)
      const float other = xch[(2 * (trades & 1) + (half ^ 1)) * MT + row];
      ++trades;
      return other;
    };
    do {
      const int kv = p.u / p.nt, tile = p.u - kv * p.nt, nb = blocks_of<MT>(p, r.end);
      const Row mine = row_of(a, p, kv, tile * MT + row);
      {  // the unit's queries, 16 of the quarter's rows a warp, a row at a time; zeros for rows that take no part
        constexpr int DL = HD / 32;  // dimensions of a lane
        const int d0 = lane * DL;
        const uint32_t at = base + (d0 >> 6) * (MT * 128) + (d0 & 7) * 2;
        const long long q_row = mine.in ? mine.b * a.p.q_stride + mine.h * a.p.hd : -1;
        float x[4][DL], next[4][DL];
        auto fetch = [&](int i0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long off = __shfl_sync(0xffffffffu, q_row, half * 16 + i0 + i);
            const bool there = off >= 0 && d0 < a.p.hd;
            const float* q = (const float*)a.p.q + (there ? off + d0 : 0);
#pragma unroll
            for (int d = 0; d < DL; d += 2) {
              const float2 two = there ? *reinterpret_cast<const float2*>(q + d) : make_float2(0.f, 0.f);
              next[i][d] = two.x;
              next[i][d + 1] = two.y;
            }
          }
        };
        fetch(0);
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < DL; ++d) x[i][d] = next[i][d] * sign;
          if (i0 < 12) fetch(i0 + 4);  // (the next rows come while these are taken apart)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = quarter * 32 + half * 16 + i0 + i;
            float up = 1.f, down = 1.f;
            // a power of two that keeps the pieces normal: fp16 pieces with the row's largest at 2^10, whatever its size; bf16
            // pieces, whose range is fp32's own, with only small ones raised to 2^-50. The scores undo it.
            float top = 0.f;
#pragma unroll
            for (int d = 0; d < DL; ++d) top = fmaxf(top, fabsf(x[i][d]));
            top = warp_max(top);
            const int ex = (int)(__float_as_uint(top) >> 23) - 127;
            if (ex < 128) {  // (a row with an infinity passes as it is)
              const int shift = C::BF ? max(-50 - ex, 0) : min(10 - ex, 126);
              up = __uint_as_float((uint32_t)(127 + shift) << 23);
              down = __uint_as_float((uint32_t)(127 - shift) << 23);
            }
            if (lane == 0) undo[rr] = down;
            const uint32_t dst = at + rr * 128 + ((((d0 >> 3) & 7) ^ (rr & 7)) << 4);
            uint32_t w[DL / 2][NQ];
#pragma unroll
            for (int d = 0; d < DL; d += 2) split<T, NQ>(x[i][d] * up, x[i][d + 1] * up, w[d / 2]);
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
              if constexpr (DL == 4)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + k * MT * HD * 2), "r"(w[0][k]), "r"(w[1][k]) : "memory");
              else
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + k * MT * HD * 2), "r"(w[0][k]) : "memory");
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float o[OC];
#pragma unroll
      for (int i = 0; i < OC; ++i) o[i] = 0.f;
      float m = -INFINITY, l = 0.f, f_last = 1.f, c = 0.f;
      bool any = false;
      auto fold = [&](int j) {  // O of block j, whose probabilities moved the reference by f_last
        if (!wait_for(o_full0 + 8 * (j & 1), j >> 1 & 1, err)) {
          ok = false;
          return;
        }
        tc::tc_fence_after();
        if (__any_sync(0xffffffffu, f_last != 1.f)) {
#pragma unroll
          for (int i = 0; i < OC; ++i) o[i] *= f_last;
        }
        const uint32_t from = lanes + C::O_COL + (j & 1) * (C::NO - 1) * 128 + half * OC;
#pragma unroll
        for (int i = 0; i < OC; i += 32) {
          float x[32];
          tc::tmem_ld32(from + i, x);
#pragma unroll
          for (int d = 0; d < 32; ++d) o[i + d] += x[d];
        }
        tc::tc_fence_before();
      };
#pragma unroll 1
      for (int j = 0; j < nb; ++j, ++block) {
        const int b = block & 1;
        if (*s_abort || !wait_for(s_full0 + 8 * b, block >> 1 & 1, err)) ok = false;
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc::tc_fence_after();
        if (j == 0) c = fmaxf(sc * undo[row], 1e-38f);  // (not 0: masked scores stay -inf)
        uint32_t u[64];
        tc::tmem_ld32_nowait(lanes + b * 128 + 64 * half, u);
        tc::tmem_ld32_nowait(lanes + b * 128 + 64 * half + 32, u + 32);
        tc::tmem_wait_ld();
        const uint2 mask = *reinterpret_cast<const uint2*>(masks + (block % TC_MASKS) * 4 + 2 * half);
        const uint32_t* all = masks + (block % TC_MASKS) * 4;
        any |= (all[0] | all[1] | all[2] | all[3]) != 0;
        if ((mask.x & mask.y) != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!(mask.x >> i & 1)) u[i] = 0xff800000u;
            if (!(mask.y >> i & 1)) u[32 + i] = 0xff800000u;
          }
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = __uint_as_float(u[i]);
#pragma unroll
        for (int i = 4; i < 64; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(u[i]));
        const float own = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), other = trade(own);
        if (C::three && j > 0) fold(block - 1);  // (one O buffer: it is read before P is handed over)
        const float mn = fmaxf(m, fmaxf(own, other) * c), f = mn > m ? ex2(m - mn) : 1.f;
        l *= f;
        m = mn;
        const float ref = (mn == -INFINITY ? 0.f : mn) - PA_BIAS;
        const f32x2 c2 = pack2(c, c), r2 = pack2(-ref, -ref);
        f32x2 acc[2] = {0ull, 0ull};
#pragma unroll
        for (int i0 = 0; i0 < 32; i0 += 16) {
          uint32_t pp[NP][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = unpack2(fma2_to(pack2(__uint_as_float(u[2 * (i0 + i)]), __uint_as_float(u[2 * (i0 + i) + 1])), c2, r2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            acc[i & 1] = add2(acc[i & 1], pack2(p0, p1));
            uint32_t w[NP];
            split<T, NP>(p0, p1, w);
#pragma unroll
            for (int k = 0; k < NP; ++k) pp[k][i] = w[k];
          }
#pragma unroll
          for (int k = 0; k < NP; ++k) tmem_st16(lanes + (k < 2 ? b * 128 + 64 * k : C::P3 + b * 64) + 32 * half + i0, pp[k]);
        }
        const float2 s0 = unpack2(acc[0]), s1 = unpack2(acc[1]);
        l += (s0.x + s0.y) + (s1.x + s1.y);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full0 + 8 * b);
        if (!C::three && j > 0) fold(block - 1);
        f_last = f;
      }
      if (!ok) break;
      fold(block - 1);
      l += trade(l);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (mine.in) {
        const bool whole = nb == p.nb;
        float* dst = state_of<MT, HD>(a, r, p, whole, mine, row);
        const int width = whole ? a.p.hd : HD;
#pragma unroll
        for (int i = 0; i < OC; i += 4)
          if (half * OC + i < width)
            *reinterpret_cast<float4*>(dst + half * OC + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        if (half == 0) *reinterpret_cast<float2*>(dst + width) = make_float2(paged::state_max(m, any), l);
      }
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
  const cudaError_t e = cudaFuncSetAttribute(shared_tc_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<T, HD>::SMEM);
  return e ? e : launch_k(shared_tc_kernel<T, HD>, dim3(ctas), dim3(THREADS), Cfg<T, HD>::SMEM, s, true, m, a);
}

}  // namespace

cudaError_t launch_shared_tc(const qw_paged_kv& cache, int ctas, const SharedArgs& a, cudaStream_t s) {
  PageMaps m{};
  make_page_maps(cache, m);
  if (cache.dtype == QW_F16) return a.p.hd <= 64 ? run<f16, 64>(ctas, m, a, s) : run<f16, 128>(ctas, m, a, s);
  return a.p.hd <= 64 ? run<bf16, 64>(ctas, m, a, s) : run<bf16, 128>(ctas, m, a, s);
}

}  // namespace shared_attn
}  // namespace qw
