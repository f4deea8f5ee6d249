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
//   - One CTA of 8 warps per SM (two of 4 warps on the CUDA cores, see there). The tiles of all sequences
//     and KV heads form one list (sequence, unit, tile), cut into equal consecutive ranges, one per CTA,
//     from the lengths on the device: ragged batches and single long sequences load every SM alike, and
//     a captured graph follows the lengths.
//   - Each of the CTA's warps owns the same rows of every tile and copies them itself (cp.async, 16 bytes a
//     lane) into its own ring of stages, looking the rows' pages up one tile ahead. Warps meet only where
//     a unit ends; the ring runs on into the next unit meanwhile.
//   - A unit that one CTA covers is finished there. The parts of a split unit go to the workspace; the
//     CTAs that arrive last merge them, as a tree (one CTA reading every part of a long sequence would be
//     bound by latency). The order of every sum is fixed by the lengths, so results repeat bit by bit.
// Measured in a CUDA graph (a lone call costs the host about 3 us from C, 10 to 14 from Python; 12 query and 2 KV heads of 128,
// fp16 cache, fp32 queries, unless stated): 256 sequences of 1 to 8192 positions, 28 and 4 heads, bf16: 326 us, 6.5 TB/s; one sequence of 131071: 34 us, 3.9 TB/s, of which 5 us pass
// before the first tile and 8 us in the join's two levels; 16 sequences of 256 to 2048: 12.9 us (3.7 us of
// traffic); one of 178: 6.7 us (lengths, table and first rows are loads that wait for one another). Instructions
// matter off the main loop: with everything inlined and unrolled, 130 KB a kernel, their misses cost 8 us
// at every unit's end and 10 us in the join.
#include "attn_paged.cuh"

#include <cmath>
#include <type_traits>

namespace qw {
namespace paged {
namespace {

// ---- 16-bit caches on the tensor cores -----------------------------------------------------------------------
//
// A unit is a KV head with HB of its query heads. S = Q K^T and O += P V by mma.sync m16n8k16 with the
// query heads as the 16 rows: the bound is HBM (tcgen05's M = 64 rows would idle for groups of at most
// 16), and the products must not lose an fp32 caller's digits. Queries and probabilities are therefore
// fed as sums of pieces of the cache's type: with HB = 8, rows 0 - 7 hold the first piece and rows
// 8 - 15 the second, so two pieces cost what one does; bf16 caches of fp32 callers take a third piece
// (8 digits each) as a second product. Groups of more than 8 heads use HB = 16, one product per piece.
// What is rounded to fewer bits than fp32: an fp32 caller's queries and probabilities over fp16 caches to two pieces (22
// bits of the row's largest element, the smallest step 2^-34 of it), the probabilities of 16-bit callers to two
// pieces too (22 bits; bf16 16, for outputs of 8); exponentials are ex2's, good to 2^-22. The fp32 caller of a bf16
// cache with groups of more than 8 heads of 128 keeps three pieces of 16 rows: 210 bytes a thread spill (with at most 8
// heads 20 bytes).
template <typename T, int HD, int HB, typename IO>
struct MmaCfg {
  static constexpr bool F32IO = std::is_same<IO, float>::value;
  // 16 positions a product; two products a tile for short heads, whose tiles would else be all latency
  static constexpr int NW = 8, R = HD <= 64 ? 2 : 1, RW = 16 * R, NT = NW * 32;
  static constexpr bool three = F32IO && sizeof(T) == 2 && !std::is_same<T, f16>::value;
  static constexpr int NQ = !F32IO ? 1 : three ? 3 : 2, NP = three ? 3 : 2;
  using Ld = Loader<T, HD, RW, NW>;
  static constexpr int COMB = NW * HB * comb_stride(HD) * 4;
  static constexpr int NS_FIT = (226 * 1024 - COMB) / (NW * Ld::STAGE);
  static constexpr int NS = NS_FIT > 8 ? 8 : NS_FIT;  // stages of a warp's ring
  static constexpr int SMEM = NS * NW * Ld::STAGE + COMB;
};

template <typename T, int HD, int HB, typename IO>
__global__ void __launch_bounds__(MmaCfg<T, HD, HB, IO>::NT, 1) paged_mma_kernel(const PagedAttnArgs a) {
  using C = MmaCfg<T, HD, HB, IO>;
  using Ld = typename C::Ld;
  using Fin = Finish<IO, HB, HD, C::NT, C::SMEM>;
  constexpr int NW = C::NW, NS = C::NS, R = C::R, NQ = C::NQ, NP = C::NP, CS = comb_stride(HD), TILE = Ld::TILE, V = Ld::V;
  using Raw = typename std::conditional<C::F32IO, float2, uint32_t>::type;  // two query elements
  constexpr int NKK = HD / 16, NA = HB == 8 ? (NQ + 1) / 2 : NQ, NPA = HB == 8 ? (NP + 1) / 2 : NP;  // products per step
  static_assert(NS >= 2, "ring");
  static_assert(TILE >= least_tile(sizeof(T) == 4, HD) && V <= PA_MAX_WEIGHT, "length of the list of tiles");
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
    const Place done = p;
    p.t = t1 - 1;
    left = advance<TILE, V>(a, n_units, r.end, p);
    if (left) fetch_q(p);
    if (Fin::template unit<NW>(a, r, done, n_hb, comb, t0, t1)) {
      pend[n_pend] = done;
      ++n_pend;
    }
  }
  cp_wait<0>();
  if (n_pend) Fin::template join<V>(a, r, pend, n_pend, n_hb, reinterpret_cast<float*>(pa_smem));
}

// ---- host ------------------------------------------------------------------------------------------------------

template <typename T, int HD, int HB, typename IO>
cudaError_t launch_mma(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  using C = MmaCfg<T, HD, HB, IO>;
  return launch(paged_mma_kernel<T, HD, HB, IO>, C::NT, C::SMEM, ctas, a, s);
}
// Heads of sizes between the instances are padded with zeros in shared memory to the next one.
template <typename T, typename IO>
cudaError_t launch_16bit(int ctas, const PagedAttnArgs& a, cudaStream_t s) {
  if (a.nq / a.nkv <= 8)
    return a.hd <= 32   ? launch_mma<T, 32, 8, IO>(ctas, a, s)
           : a.hd <= 64 ? launch_mma<T, 64, 8, IO>(ctas, a, s) : launch_mma<T, 128, 8, IO>(ctas, a, s);
  return a.hd <= 64 ? launch_mma<T, 64, 16, IO>(ctas, a, s) : launch_mma<T, 128, 16, IO>(ctas, a, s);
}

// floats of one part: of the largest instance that the shape may take, whatever its types (launch_16bit's HB and HD; the
// CUDA cores' HB is at most 8, their HD at most this one)
size_t part_floats(int n_heads, int n_kv_heads, int head_dim) {
  const bool wide = n_heads / n_kv_heads > 8;
  const int hd = head_dim <= 32 && !wide ? 32 : head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  return (size_t)(wide ? 16 : 8) * comb_stride(hd);
}
static_assert(PA_LEVELS * 2 * PA_MAX_CTAS * sizeof(unsigned int) <= OP_COUNTER_BYTES, "counters");

}  // namespace
}  // namespace paged
}  // namespace qw

using namespace qw;
using namespace qw::paged;

extern "C" {

size_t qw_op_paged_attention_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 8 || head_dim % 8 || head_dim > PA_MAX_HD) return 0;
  return OP_COUNTER_BYTES + 2 * PA_MAX_CTAS * part_floats(n_heads, n_kv_heads, head_dim) * sizeof(float);
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
  // the tile list's numbers are 31-bit: a unit (at most one a head) has its tiles, the last one cut, and its weight
  const int64_t unit = (int64_t)max_blocks * c.page_size / least_tile(c.dtype == QW_F32, c.head_dim) + 1 + PA_MAX_WEIGHT;
  if ((int64_t)n_seqs * n_heads * unit > 0x7fffffffll)
    return op_fail(QW_ERR_UNSUPPORTED, "n_seqs * n_heads * max_blocks * page_size too large");
  // (the kernels take scale * log2(e), which must be finite too: else scores of 0 would be NaN)
  if (!(std::fabs(scale) <= 0x1p127f)) return op_fail(QW_ERR_INVALID_ARG, "scale not finite, or above 2^127");
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
                  (unsigned int*)workspace, (float*)((char*)workspace + OP_COUNTER_BYTES), err_dev};
  cudaStream_t s = (cudaStream_t)cuda_stream;
  const int ctas = nsm < PA_MAX_CTAS / 2 ? nsm : PA_MAX_CTAS / 2;
  if (c.dtype == QW_F32 || c.head_dim > 128) e = launch_simt(c.dtype, io_dtype, 2 * ctas, a, s);
  else if (c.dtype == QW_F16)
    e = io_dtype == QW_F32 ? launch_16bit<f16, float>(ctas, a, s) : launch_16bit<f16, f16>(ctas, a, s);
  else
    e = io_dtype == QW_F32 ? launch_16bit<bf16, float>(ctas, a, s) : launch_16bit<bf16, bf16>(ctas, a, s);
  if (e) return op_cuda_fail(e, "paged attention launch");
  return QW_OK;
}

}  // extern "C"
