// The own positions of attn_shared.cu for 16-bit caches and heads of at most 128 dimensions: what a sequence holds behind the
// shared part, mostly short.
//
// The tensor-core kernel of attn_paged.cu, but a warp works alone: tiles of 16 or 32 positions of all units form one list
// (sequence, unit, tile) that is cut into equal ranges, one a warp, and what a warp has of a unit goes to the workspace
// as a state, for the join that has to come anyway. There, eight warps share a unit's tiles and meet at its end, 2 to 4 us each
// time, which short sequences pay with little work between: 256 sequences of 1 to 256 positions, 28 and 4 heads of
// 128, bf16: 27 us there, 19 to 21 here (71 MB, 3.5 TB/s).
// What bounds it: latency. Lists of some ten tiles a warp: 5 us until the first tile has come (lengths, list, table, rows are
// loads in a chain), then HBM for 10, then the last states.
// Products, pieces and sums are those of attn_paged.cu.
#include "attn_shared.cuh"

namespace qw {
namespace shared_attn {
namespace {

using namespace paged;

constexpr int OWN_NT = OWN_WARPS * 32;

template <typename T, int HD, int HB, typename IO>
struct OwnCfg {
  static constexpr bool F32IO = std::is_same<IO, float>::value;
  static constexpr int R = own_rows(HD) / 16, RW = 16 * R;
  static constexpr bool three = F32IO && !std::is_same<T, f16>::value;
  static constexpr int NQ = !F32IO ? 1 : three ? 3 : 2, NP = three ? 3 : 2;
  using Ld = Loader<T, HD, RW, 1>;
  static constexpr int COMB = OWN_WARPS * HB * comb_stride(HD) * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB) / (OWN_WARPS * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;  // stages of a warp's ring
  static constexpr int SMEM = NS * OWN_WARPS * Ld::STAGE + COMB;
};

// The warps' cuts of the list, and each sequence's place in it for the join.
template <int RW, int HB>
__device__ __forceinline__ Range find_own(const SharedArgs& a, int n_units, Place& first) {
  __shared__ int w_sum[OWN_WARPS];
  __shared__ Place s_at[OWN_WARPS + 1];
  const OwnAttnArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n_seqs + OWN_NT - 1) / OWN_NT, b0 = min(p.n_seqs, tid * per), b1 = min(p.n_seqs, b0 + per);
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    bool bad;
    int from;
    const int len = seq_len(p, b, from, bad);
    if (len) mine += OWN_WEIGHT + (len + RW - 1) / RW;
    if (bad && blockIdx.x == 0) atomicOr(p.err, ERR_PAGE);
  }
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
  for (int w = 0; w < OWN_WARPS; ++w) {
    if (w < warp) base += w_sum[w];
    total += w_sum[w];
  }
  base *= n_units;
  mine *= n_units;
  total *= n_units;
  const int parts = min((int)gridDim.x * OWN_WARPS, total);
  Range r{0, 0, 0, 0};
  if (parts) {
    r.each = total / parts;
    r.rest = total - r.each * parts;
  }
  if (blockIdx.x == 0 && tid == 0) *a.own_head = SharedHead{0, r.each, r.rest, total};
  int at = base;
  if (mine || blockIdx.x == 0)
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      int from;
      const int len = seq_len(p, b, from), nt = (len + RW - 1) / RW, unit = nt ? OWN_WEIGHT + nt : 0;
      if (blockIdx.x == 0) a.own_at[b] = at;
#pragma unroll 1
      for (int k = 0; k <= OWN_WARPS; ++k) {
        const int c = blockIdx.x * OWN_WARPS + k, x = cut(r, c);
        if (c > parts || x < at || x >= at + unit * n_units) continue;
        const int u = (x - at) / unit, v = at + u * unit;
        s_at[k] = Place{b, u, nt <= OWN_WHOLE ? 0 : max(0, x - v - OWN_WEIGHT), nt, len, v, from};
      }
      at += unit * n_units;
    }
  __syncthreads();
  const int c = blockIdx.x * OWN_WARPS + warp;
  if (c < parts) {
    first = s_at[warp];
    r.begin = first.v + (first.t ? OWN_WEIGHT + first.t : 0);
    r.end = c + 1 == parts ? total : s_at[warp + 1].v + (s_at[warp + 1].t ? OWN_WEIGHT + s_at[warp + 1].t : 0);
  }
  return r;
}

template <typename T, int HD, int HB, typename IO>
__global__ void __launch_bounds__(OWN_NT, 1) own_kernel(const SharedArgs sa) {
  using C = OwnCfg<T, HD, HB, IO>;
  using Ld = typename C::Ld;
  const OwnAttnArgs& a = sa.p;
  constexpr int NS = C::NS, R = C::R, NQ = C::NQ, NP = C::NP, CS = comb_stride(HD), TILE = Ld::TILE, V = OWN_WEIGHT;
  using Raw = typename std::conditional<C::F32IO, float2, uint32_t>::type;  // two query elements
  constexpr int NKK = HD / 16, NA = HB == 8 ? (NQ + 1) / 2 : NQ, NPA = HB == 8 ? (NP + 1) / 2 : NP;  // products per step
  static_assert(NS >= 2, "ring");
  extern __shared__ __align__(128) unsigned char pa_smem[];
  __shared__ uint32_t s_mask[OWN_WARPS][NS];  // rows of a stage that exist
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int group = a.nq / a.nkv, n_hb = (group + HB - 1) / HB, n_units = a.nkv * n_hb;
  float* comb = reinterpret_cast<float*>(pa_smem + NS * OWN_WARPS * Ld::STAGE);
  const uint32_t ring = smem_addr(pa_smem) + warp * NS * Ld::STAGE;
  pdl_trigger();  // (the shared beginning's attention goes on beside this one)
  Place ld;
  const Range r = find_own<TILE, HB>(sa, n_units, ld);
  if (r.begin >= r.end) return;
  Place p = ld;
  bool more = true;  // tiles to request
  long long row_off = Ld::row(a, ld, n_hb, 0, lane);
  int ld_stage = 0;
  const bool col = lane % Ld::CH * Ld::CE < a.hd;
  const char *kl = (const char*)a.k + lane % Ld::CH * 16, *vl = (const char*)a.v + lane % Ld::CH * 16;
  auto load_next = [&]() {  // requests the tile at ld and looks up the rows of the one after it
    if (more) {
      const uint32_t mask = __ballot_sync(0xffffffffu, row_off >= 0);
      Ld::request(kl, vl, row_off, mask, ring + ld_stage * Ld::STAGE, lane, col, a.hd);
      if (lane == 0) s_mask[warp][ld_stage] = mask;
      more = advance<TILE, V>(a, n_units, r.end, ld);
      if (more) row_off = Ld::row(a, ld, n_hb, 0, lane);
    }
    cp_commit();
    if (++ld_stage == NS) ld_stage = 0;
  };
  int stage = 0, ahead = NS - 1;  // tiles still to be requested before the first is used
  const float sc = a.scale * LOG2E;
  // a unit's queries, columns 2 tig, 2 tig + 1 and 2 tig + 8, 2 tig + 9 of every 16: requested before the unit
  // ahead of it ends, used after its first tile has come
  Raw xq[HB / 8][NKK][2];
  auto fetch_q = [&](const Place& u) {
    const int g = u.u / n_hb, hb = u.u - g * n_hb;
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      const int h = hb * HB + gid + 8 * half;
      const IO* q = (const IO*)a.q + u.b * a.q_stride + (g * group + h) * a.hd + 2 * tig;
#pragma unroll
      for (int i = 0; i < 2 * NKK; ++i)
        xq[half][i / 2][i % 2] = h < group && i * 8 < a.hd ? *reinterpret_cast<const Raw*>(q + i * 8) : Raw{};
    }
  };
  fetch_q(p);
#pragma unroll 1
  for (bool left = true; left;) {
    const int t0 = p.t, t1 = min(p.nt, r.end - p.v - V);
    bool fresh = true;
    uint32_t qa[NA][NKK][4];  // A fragments: pieces of rows gid and gid + 8
    float undo[2];                // of the queries' power of two
    float o[HD / 8][4], m[HB / 8], l[HB / 8], m_there[HB / 8];
    bool any = false;    // position so far
    bool there = false;  // part of o is in comb already, relative to m_there
    int since = 0;
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
    for (int h = 0; h < HB / 8; ++h) {
      m[h] = m_there[h] = -INFINITY;
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
            // fp32 queries times a power of two that keeps the pieces normal: fp16 pieces with the row's largest at
            // 2^10, whatever its size; bf16 pieces, whose range is fp32's own, with only small ones raised to 2^-50, so
            // that no product overflows that would not in fp32. The scores undo it before they are scaled.
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NKK; ++i) top = fmaxf(top, fmaxf(fabsf(xq[half][i / 2][i % 2].x), fabsf(xq[half][i / 2][i % 2].y)));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = (int)(__float_as_uint(top) >> 23) - 127;
            if (ex < 128) {  // (a row with an infinity passes as it is)
              const int shift = std::is_same<T, f16>::value ? min(10 - ex, 126) : max(-50 - ex, 0);
              up = __uint_as_float((uint32_t)(127 + shift) << 23);
              down = __uint_as_float((uint32_t)(127 - shift) << 23);
            }
          }
          undo[half] = down;
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
        if (HB == 8) undo[1] = undo[0];
      }
      const uint32_t mask = s_mask[warp][stage];
      if (mask) {
        any = true;
        const uint32_t ks = ring + stage * Ld::STAGE, vs = ks + Ld::STAGE / 2;
        // lower pieces have sums of their own: the additions cut, and would do so twice as often at the top
        constexpr int NC = NA > 1 ? 2 : 1;
        float c[NC][2 * R][4];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < 2 * R; ++i) c[n][i][0] = c[n][i][1] = c[n][i][2] = c[n][i][3] = 0.f;
        const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
#pragma unroll
          for (int rr = 0; rr < R; ++rr) {
            uint32_t b[4];  // keys 0 - 7 and 8 - 15 of 16, dimensions kk * 16 .. + 15
            ldmatrix_x4(b, ks + Ld::at(rr * 16 + (mi >> 1) * 8 + r8, kk * 2 + (mi & 1)));
#pragma unroll
            for (int n = 0; n < NA; ++n) {
              mma_t(c[n ? NC - 1 : 0][2 * rr], qa[n][kk], b[0], b[1], T());
              mma_t(c[n ? NC - 1 : 0][2 * rr + 1], qa[n][kk], b[2], b[3], T());
            }
          }
        }
        if constexpr (NC > 1) {
#pragma unroll
          for (int i = 0; i < 2 * R; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[0][i][k] += c[NC - 1][i][k];
        }
        uint32_t pa[R][NPA][4];
#pragma unroll
        for (int half = 0; half < HB / 8; ++half) {
          float s[4 * R];  // positions 2 tig, 2 tig + 1, and + 8, + 16, ...
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4 * R; ++i) {
            const float x = HB == 8 ? c[0][i >> 1][i & 1] + c[0][i >> 1][2 + (i & 1)] : c[0][i >> 1][2 * half + (i & 1)];
            s[i] = (mask >> (2 * tig + (i & 1) + 8 * (i >> 1))) & 1 ? (C::F32IO ? x * undo[half] : x) * sc : -INFINITY;
            top = fmaxf(top, s[i]);
          }
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
#pragma unroll
          for (int rr = 0; rr < R; ++rr) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = ex2(s[4 * rr + i] - ref);
            l[half] += (e[0] + e[1]) + (e[2] + e[3]);
            uint32_t lo[4], hi[4];
            split<T, NP>(e[0], e[1], lo);
            split<T, NP>(e[2], e[3], hi);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const int n = HB == 8 ? i / 2 : i, rw = HB == 8 ? i & 1 : half;
              pa[rr][n][rw] = lo[i];
              pa[rr][n][2 + rw] = hi[i];
            }
            if (HB == 8 && NP & 1) pa[rr][NPA - 1][1] = pa[rr][NPA - 1][3] = 0u;
          }
        }
#pragma unroll
        for (int dd = 0; dd < NKK; ++dd) {
#pragma unroll
          for (int rr = 0; rr < R; ++rr) {
            uint32_t b[4];  // dimensions dd * 16 .. + 7 and + 8 .. + 15
            ldmatrix_x4_t(b, vs + Ld::at(rr * 16 + (mi & 1) * 8 + r8, dd * 2 + (mi >> 1)));
#pragma unroll
            for (int n = 0; n < NPA; ++n) {
              mma_t(o[2 * dd], pa[rr][n], b[0], b[1], T());
              mma_t(o[2 * dd + 1], pa[rr][n], b[2], b[3], T());
            }
          }
        }
      }
      __syncwarp();
      if (++stage == NS) stage = 0;
      if (t == t1 || (C::F32IO && ++since == PA_FLUSH / NPA)) {  // o to the warp's place in comb, added to what is there
        since = 0;
#pragma unroll
        for (int half = 0; half < HB / 8; ++half) {
          float* row = comb + ((size_t)warp * HB + gid + 8 * half) * CS + 2 * tig;
          const float f = m_there[half] == m[half] ? 1.f : ex2(m_there[half] - m[half]);
#pragma unroll
          for (int n = 0; n < HD / 8; ++n) {
            float2 v = HB == 8 ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]) : make_float2(o[n][2 * half], o[n][2 * half + 1]);
            if (C::F32IO && there) {
              const float2 w = *reinterpret_cast<const float2*>(row + n * 8);
              v.x = fmaf(w.x, f, v.x);
              v.y = fmaf(w.y, f, v.y);
            }
            *reinterpret_cast<float2*>(row + n * 8) = v;
            o[n][2 * half] = o[n][2 * half + 1] = 0.f;
            if (HB == 8) o[n][2] = o[n][3] = 0.f;
          }
          m_there[half] = m[half];
        }
        there = true;
      }
    }
    float* cw = comb + (size_t)warp * HB * CS;
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      float sum = l[half];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (tig == 0) *reinterpret_cast<float2*>(cw + (gid + 8 * half) * CS + HD) = make_float2(state_max(m[half], any), sum);
    }
    __syncwarp();
    {  // the warp's state of the unit: of all its tiles, or as a part
      const bool whole = t0 == 0 && t1 == p.nt;
      const int g = p.u / n_hb, hb = p.u - g * n_hb, c = blockIdx.x * OWN_WARPS + warp;
      float* part = a.part + (size_t)(2 * c + (cut(r, c) < p.v ? 1 : 0)) * HB * CS;
      const int width = whole ? a.hd : HD;
#pragma unroll 1
      for (int h = 0; h < HB && hb * HB + h < group; ++h) {
        float* dst = whole ? a.state + ((size_t)p.b * a.nq + g * group + hb * HB + h) * comb_stride(a.hd) : part + h * CS;
        if (4 * lane < width) *reinterpret_cast<float4*>(dst + 4 * lane) = *reinterpret_cast<const float4*>(cw + h * CS + 4 * lane);
        if (lane == 0) *reinterpret_cast<float2*>(dst + width) = *reinterpret_cast<const float2*>(cw + h * CS + HD);
      }
    }
    __syncwarp();
    p.t = t1 - 1;
    left = advance<TILE, V>(a, n_units, r.end, p);
    if (left) fetch_q(p);
  }
  cp_wait<0>();
}

template <typename T, int HD, int HB, typename IO>
cudaError_t run(int ctas, const SharedArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(own_kernel<T, HD, HB, IO>, cudaFuncAttributeMaxDynamicSharedMemorySize, OwnCfg<T, HD, HB, IO>::SMEM);
  return e ? e : launch_k(own_kernel<T, HD, HB, IO>, dim3(ctas), dim3(OWN_NT), OwnCfg<T, HD, HB, IO>::SMEM, s, false, a);
}
template <typename T, typename IO>
cudaError_t run(int ctas, const SharedArgs& a, cudaStream_t s) {
  if (a.p.nq / a.p.nkv <= 8)
    return a.p.hd <= 32 ? run<T, 32, 8, IO>(ctas, a, s) : a.p.hd <= 64 ? run<T, 64, 8, IO>(ctas, a, s) : run<T, 128, 8, IO>(ctas, a, s);
  return a.p.hd <= 64 ? run<T, 64, 16, IO>(ctas, a, s) : run<T, 128, 16, IO>(ctas, a, s);
}

}  // namespace

cudaError_t launch_own(int cache_dtype, int io_dtype, int ctas, const SharedArgs& a, cudaStream_t s) {
  if (cache_dtype == QW_F16) return io_dtype == QW_F32 ? run<f16, float>(ctas, a, s) : run<f16, f16>(ctas, a, s);
  return io_dtype == QW_F32 ? run<bf16, float>(ctas, a, s) : run<bf16, bf16>(ctas, a, s);
}

}  // namespace shared_attn
}  // namespace qw
