// Decode attention over a paged cache on the CUDA cores; attn_paged.cu has the entry point and the method.
#include "attn_paged.cuh"

namespace qw {
namespace paged {
namespace {

// ---- CUDA cores: fp32 caches, and heads of more than 128 dimensions -------------------------------------------
//
// A warp takes RW positions of a tile, LPR = 32 / RW lanes each. Scores: lane (position lane % RW, part
// lane / RW) sums every LPR-th group of 4 dimensions for all HB heads (q in shared memory), shuffles add the
// parts, and the lane then keeps HB / LPR heads of its position. Values: a lane owns groups of 4 dimensions
// (several lanes share one where the head is short, each taking every PG-th position); the HB probabilities
// of a position come from shared memory. Products are packed pairs (f32x2): two dimensions in the
// scores, two heads in the values. Two CTAs of 4 warps an SM: 200 sequences of up to 1500 positions, fp32, 3 heads a
// group of 32 dimensions, take 25.7 us against 28 us with one CTA of 8 warps, since one goes on while the
// other ends a unit. (On the tensor cores, whose units are larger and joined more often, it is the other
// way round: 16 ragged sequences 13.3 against 15.4 us, 256 of up to 8192 positions 326 against 337 us.)
template <typename T, int HD, int HB_>
struct SimtCfg {
  static constexpr int HB = HB_, RW = HD <= 32 ? 32 : HD <= 64 ? 16 : 8, NW = HD * sizeof(T) > 512 ? 2 : 4, NT = NW * 32;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4, QS = HB * HD * 4, PS = NW * (RW + 1) * HB * 4;
  static constexpr int NS_FIT = (113 * 1024 - COMB - QS - PS) / (NW * Ld::STAGE);
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

template <typename T, int HD, int HB, typename IO, typename A>
__global__ void __launch_bounds__(SimtCfg<T, HD, HB>::NT, 2) paged_simt_kernel(const A a) {
  using C = SimtCfg<T, HD, HB>;
  using Ld = typename C::Ld;
  using Fin = Finish<IO, HB, HD, C::NT, C::SMEM>;
  constexpr int NW = C::NW, NS = C::NS, RW = C::RW, CS = comb_stride(HD), TILE = Ld::TILE, V = Ld::V;
  constexpr int LPR = 32 / RW, HPL = HB / LPR;  // lanes of a position, heads a lane keeps
  constexpr int G4 = HD / 4;                    // groups of 4 dimensions
  constexpr int PG = G4 >= 32 ? 1 : 32 / G4;    // lanes that share a group, by position
  constexpr int GL = G4 >= 32 ? G4 / 32 : 1;    // groups a lane owns
  static_assert(NS >= 2, "ring");
  static_assert(TILE >= least_tile(sizeof(T) == 4, HD) && V <= PA_MAX_WEIGHT, "length of the list of tiles");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[NW][NS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * NW * Ld::STAGE);
  float* qs = comb + NW * HB * CS;                  // [HB][HD]
  float* ps = qs + HB * HD + warp * (RW + 1) * HB;  // [RW][HB] probabilities, then [HB] factors
  unsigned char* ring_p = pa_smem + warp * NS * Ld::STAGE;
  const uint32_t ring = smem_addr(ring_p);
  if constexpr (A::OWN) pdl_trigger();  // (the shared beginning's attention goes on beside this one)
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
    bool fresh = true, any = false;  // any: position so far
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
        any = true;
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
        for (int i = 0; i < HPL; ++i) {
          ps[pos * HB + HPL * part + i] = e[i];
          if (pos == 0) ps[RW * HB + HPL * part + i] = f[i];
        }
        moved = __any_sync(0xffffffffu, moved);
        __syncwarp();
        auto pairs = [&](int row, f32x2* w) {
#pragma unroll
          for (int h = 0; h < HB; h += 4) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(ps + row * HB + h);
            w[h / 2] = x.x;
            w[h / 2 + 1] = x.y;
          }
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
        cw[(part * HPL + i) * CS + HD] = state_max(m[i], any);
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

template <typename T, int HD, int HB, typename IO, typename A>
cudaError_t run(int ctas, const A& a, cudaStream_t s) {
  using C = SimtCfg<T, HD, HB>;
  return launch(paged_simt_kernel<T, HD, HB, IO, A>, C::NT, C::SMEM, ctas, a, s);
}
// groups of at most 4 heads take half the arithmetic
template <typename T, int HD, typename IO, typename A>
cudaError_t run(int ctas, const A& a, cudaStream_t s) {
  return a.nq / a.nkv <= 4 ? run<T, HD, 4, IO>(ctas, a, s) : run<T, HD, 8, IO>(ctas, a, s);
}

template <typename A>
cudaError_t run(int cache_dtype, int io_dtype, int ctas, const A& a, cudaStream_t s) {
  if (cache_dtype == QW_F16)
    return io_dtype == QW_F32 ? run<f16, 256, float>(ctas, a, s) : run<f16, 256, f16>(ctas, a, s);
  if (cache_dtype == QW_BF16)
    return io_dtype == QW_F32 ? run<bf16, 256, float>(ctas, a, s) : run<bf16, 256, bf16>(ctas, a, s);
  return a.hd <= 32    ? run<float, 32, float>(ctas, a, s)
         : a.hd <= 64  ? run<float, 64, float>(ctas, a, s)
         : a.hd <= 128 ? run<float, 128, float>(ctas, a, s) : run<float, 256, float>(ctas, a, s);
}

}  // namespace

cudaError_t launch_simt(int cache_dtype, int io_dtype, int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  return run(cache_dtype, io_dtype, ctas, a, s);
}
cudaError_t launch_simt(int cache_dtype, int io_dtype, int ctas, const OwnAttnArgs& a, cudaStream_t s) {
  return run(cache_dtype, io_dtype, ctas, a, s);
}

}  // namespace paged
}  // namespace qw
