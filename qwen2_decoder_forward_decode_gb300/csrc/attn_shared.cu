// Decode attention of groups of sequences that share a beginning, over a paged cache ("LLM Speedrun: Architecture":
// Attention, Grouped Query Attention): samples and beams of one prompt, or users of one system prompt.
//
// Mathematics: the state (m, l, o) of a set of positions is the maximum score m (base 2), l = sum 2^(s - m) and
// o = sum 2^(s - m) V. States of disjoint sets merge as M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i. So
// the shared positions are read once for all rows (sequence, head) of a group and KV head, and each sequence's own
// positions by themselves:
//   1. the own positions: a list of short tiles, a range a warp (attn_shared_own.cu; fp32 caches and longer heads by the
//      kernels of attn_paged_simt.cu with each sequence's first positions left out), their states kept in fp32;
//   2. the shared ones: matrix products of up to 256 rows with blocks of keys and values on the tensor cores
//      (attn_shared_pair.cu, for fp32 callers attn_shared_tc.cu; fp32 caches and longer heads on the CUDA cores,
//      attn_shared_simt.cu). All blocks of all groups form one list that is cut into
//      equal ranges, one a CTA;
//   3. the join: a warp a row, or a CTA a row where rows are few and their parts many.
// The second launch goes on beside the first (programmatic dependent launch: it waits for it at its end only), the third
// is in place when the second ends.
// Measured in a CUDA graph: 4 samples of a prompt of 178 (12 and 2 heads of 128, fp16 cache, fp32 queries) 15.4 us, three launches'
// chains of loads; 256 sequences of 1 to 256 own positions behind 16383 (28 and 4 heads, bf16) 101 us: own positions 20, shared
// ones 70, join 11 (7168 rows of 8 states each, 30 MB that L2 holds). The same without sharing reads 8.7 GB, 1.3 ms at the copy rate.
// When it pays, next to attn_paged.cu over tables that hold all pages (us, paged / shared; 28 and 4 heads, bf16, own positions 64):
// one prompt of 2048, 4 rows 11 / 16, 32 rows 27 / 26; of 8192, 4 rows 19 / 20, 8 rows 25 / 24; 64 prompts of 512, 2 rows 32 / 39,
// 4 rows 56 / 47; 8 prompts of 2048, 4 rows 27.0 / 27.5, 8 rows 44 / 30; 64 prompts of 2048 of one row 57 / 75. 12 and 2 heads,
// fp32 over fp16: 64 prompts of 512, 4 rows 34 / 33; of 2048, 2 rows 49 / 55. So from 100 to 150 MB on that need not be read again; which call
// to make is the caller's choice, who knows the lengths.
#include "attn_shared.cuh"

#include <algorithm>

namespace qw {
namespace shared_attn {
namespace {

constexpr int JN_THREADS = 256, JN_WARPS = JN_THREADS / 32;

struct JoinArgs {
  SharedArgs s;
  Geometry geo;
  int own_hb, own_hd;  // of attn_shared_own.cu's parts; own_hb 0: it has not run
};

// The sum of states, NV groups of 4 dimensions a lane.
template <int NV>
struct Sum {
  float m, l;
  float4 o[NV];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(float m2, float l2, const float4* x) {  // (its o is not looked at where m2 is -inf)
    if (m2 == -INFINITY) return;
    const float top = fmaxf(m, m2), f = m == -INFINITY ? 0.f : ex2(m - top), w = ex2(m2 - top);
    m = top;
    l = fmaf(w, l2, l * f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      o[i].x = fmaf(w, x[i].x, o[i].x * f);
      o[i].y = fmaf(w, x[i].y, o[i].y * f);
      o[i].z = fmaf(w, x[i].z, o[i].z * f);
      o[i].w = fmaf(w, x[i].w, o[i].w * f);
    }
  }
};

// The sum of the states of head h of sequence b (of WPR warps, the part `part`). What places them is loaded in three rounds, and
// the code is short: cold, it costs a cycle a byte. false: the call's groups are bad.
template <int NV, int WPR, int MT>
__device__ __forceinline__ bool join_row(const JoinArgs& ja, int b, int h, int part, Sum<NV>& sum) {
  const SharedArgs& a = ja.s;
  const OwnAttnArgs& p = a.p;
  const int lane = threadIdx.x & 31, grp = p.nq / p.nkv, kv = h / grp, hg = h - kv * grp;
  constexpr int BK = MT == 64 ? 64 : 128;
  sum.clear();
  const int mine = __ldg(p.skip + b), len = __ldg(p.lens + b);
  // the last group that begins at or before b: 32 of them at a time
  int lo = 0, hi = a.n_groups;
#pragma unroll 1
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned before = __ballot_sync(0xffffffffu, at < hi && __ldg(a.cu + min(at, hi - 1)) <= b);
    const int last = before ? 31 - __clz(before) : 0;
    lo += last * step;
    hi = min(hi, lo + step);
  }
  const int first = min(max(__ldg(a.cu + lo), 0), b), end = __ldg(a.cu + lo + 1), pre = __ldg(p.skip + first);  // (bad ones stay inside)
  pdl_wait();  // (what stands above are the call's inputs, that no kernel of it writes)
  const SharedHead head = *a.head, own = ja.own_hb ? *a.own_head : SharedHead{0, 1, 0, 0};
  const int own_at = ja.own_hb ? a.own_at[b] : 0, at = a.at[lo];
  if (head.bad) return false;
  int from;
  const int left = paged::seq_len(p, b, from), rw = ja.own_hb ? own_rows(ja.own_hd) : 1, nt_own = (left + rw - 1) / rw;
  const int hb_own = ja.own_hb == 16 ? hg >> 4 : hg >> 3, n_hb = ja.own_hb == 16 ? (grp + 15) >> 4 : (grp + 7) >> 3;
  const int v_own = own_at + (kv * n_hb + hb_own) * (OWN_WEIGHT + nt_own);
  const long long room = (long long)p.max_blocks * p.page;
  const bool in = pre > 0 && pre <= room && mine == pre && len >= pre;
  // a sequence that claims a shared part which its group's first sequence does not have misses positions
  if (!in && part == 0 && lane == 0 && h == 0 && mine != pre && mine > 0 && mine <= len) atomicOr(p.err, ERR_PAGE);
  const int rows = (end - first) * grp, nt = (rows + MT - 1) / MT, nb = (pre + BK - 1) / BK, i = (b - first) * grp + hg, tile = i / MT;
  const int cost = block_cost<MT>(rows, tile);
  const bool halves = MT == 256 && cost == 1;  // even and odd blocks have states of their own
  const int v = at + kv * head_numbers<MT>(rows, nt, nb) + tile * (unit_weight<MT>(block_cost<MT>(MT, 0)) + block_cost<MT>(MT, 0) * nb);
  // the first and the last range of each list that has a part: lanes 0, 1 own positions, 2, 3 shared ones
  const Range r = lane < 2 ? Range{max(own.each, 1), own.rest, 0, 0} : Range{max(head.each, 1), head.rest, 0, 0};
  const int x = lane == 0 ? v_own + OWN_WEIGHT : lane == 1 ? v_own + OWN_WEIGHT + nt_own - 1 : v + unit_weight<MT>(cost) + (lane == 2 ? 0 : cost * (nb - 1));
  const int c = cta_of(r, x);
  const int odd = cut(r, c) < (lane < 2 ? v_own : v);  // the slot's number, in the first range
  const int c0_own = __shfl_sync(0xffffffffu, c, 0), c1_own = __shfl_sync(0xffffffffu, c, 1), odd_own = __shfl_sync(0xffffffffu, odd, 0);
  const int c0 = __shfl_sync(0xffffffffu, c, 2), c1 = __shfl_sync(0xffffffffu, c, 3), odd_sh = __shfl_sync(0xffffffffu, odd, 2);
  const size_t row = (size_t)b * p.nq + h;
  const bool split_own = ja.own_hb && nt_own > OWN_WHOLE && c0_own != c1_own, split = in && c0 != c1;
  const int n_own = ja.own_hb && !nt_own ? 0 : split_own ? c1_own - c0_own + 1 : 1;
  const int n = n_own + (!in ? 0 : (c1 - c0 + 1) << halves);
  const int hd_own = split_own ? ja.own_hd : p.hd, hd_sh = split ? ja.geo.hd : p.hd;
  const float* s_own = split_own ? p.part + (hg - hb_own * ja.own_hb) * comb_stride(ja.own_hd) : p.state + row * comb_stride(p.hd);
  const float* s_sh = split ? a.parts + (i - tile * MT) * comb_stride(ja.geo.hd) : a.whole + row * comb_stride(p.hd);
  const long long slot_own = split_own ? ja.own_hb * comb_stride(ja.own_hd) : 0, slot_sh = split ? MT * comb_stride(ja.geo.hd) : 0;
  const long long second = split ? MT / 2 * comb_stride(ja.geo.hd) : (long long)p.n_seqs * p.nq * comb_stride(p.hd);
#pragma unroll 1
  for (int j0 = part; j0 < n; j0 += 4 * WPR) {
    float2 ml[4];
    float4 o[4][NV];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = j0 + q * WPR, js = j - n_own, k = j < n_own ? j : js >> halves;
      const bool is_own = j < n_own;
      const int slot = 2 * ((is_own ? c0_own : c0) + k) + (k == 0 ? (is_own ? odd_own : odd_sh) : 0), hd = is_own ? hd_own : hd_sh;
      const float* s = is_own ? s_own + slot * slot_own : s_sh + slot * slot_sh + (halves && (js & 1) ? second : 0);
      ml[q] = j < n ? *reinterpret_cast<const float2*>(s + hd) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int w = 0; w < NV; ++w)
        o[q][w] = j < n && 4 * lane + 128 * w < p.hd ? *reinterpret_cast<const float4*>(s + 4 * lane + 128 * w) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sum.add(ml[q].x, ml[q].y, o[q]);
  }
  return true;
}

template <int NV, typename IO>
__device__ __forceinline__ void write_row(const OwnAttnArgs& p, int b, int h, const Sum<NV>& s) {
  const int lane = threadIdx.x & 31;
  // l = 0: no position was left, and out is 0; or every score was -inf, and 0 / 0 is the formula's NaN
  const float inv = s.l == 0.f && s.m == -INFINITY ? 1.f : 1.f / s.l;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = 4 * lane + 128 * i;
    if (d < p.hd)
      paged::store4((IO*)p.out + b * p.out_stride + h * p.hd + d,
                    make_float4(s.o[i].x * inv, s.o[i].y * inv, s.o[i].z * inv, s.o[i].w * inv));
  }
  if (lane == 0 && p.lse) p.lse[(size_t)b * p.nq + h] = (s.m - PA_BIAS + log2f(s.l)) * paged::LN2;
}

// A row a warp, or a CTA where rows are few and their parts may be many.
template <int NV, int WPR, int MT, typename IO>
__global__ void __launch_bounds__(JN_THREADS, 4) join_kernel(const __grid_constant__ JoinArgs ja) {
  const OwnAttnArgs& p = ja.s.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = WPR == 1 ? blockIdx.x * JN_WARPS + warp : blockIdx.x, b = x / p.nq, h = x - b * p.nq;
  Sum<NV> sum;
  if constexpr (WPR == 1) {
    if (b >= p.n_seqs) return;
    join_row<NV, 1, MT>(ja, b, h, 0, sum);
    write_row<NV, IO>(p, b, h, sum);
  } else {
    static_assert(WPR == JN_WARPS, "a CTA a row");
    __shared__ float2 s_ml[JN_WARPS];
    __shared__ float4 s_o[JN_WARPS][NV * 32];
    join_row<NV, WPR, MT>(ja, b, h, warp, sum);
    if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
#pragma unroll
    for (int i = 0; i < NV; ++i) s_o[warp][32 * i + lane] = sum.o[i];
    __syncthreads();
    if (warp) return;
#pragma unroll 1
    for (int w = 1; w < JN_WARPS; ++w) {
      float4 x[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = s_o[w][32 * i + lane];
      sum.add(s_ml[w].x, s_ml[w].y, x);
    }
    write_row<NV, IO>(p, b, h, sum);
  }
}

template <int NV, int MT, typename IO>
cudaError_t launch_join(const JoinArgs& ja, int nsm, cudaStream_t s) {
  const int nq = ja.s.p.nq, n = ja.s.p.n_seqs;
  if (n * nq <= 8 * nsm) return launch_k(join_kernel<NV, JN_WARPS, MT, IO>, dim3(nq * n), dim3(JN_THREADS), 0, s, true, ja);
  return launch_k(join_kernel<NV, 1, MT, IO>, dim3((nq * n + JN_WARPS - 1) / JN_WARPS), dim3(JN_THREADS), 0, s, true, ja);
}
template <typename IO>
cudaError_t launch_join(const JoinArgs& ja, int nsm, cudaStream_t s) {
  if (ja.s.p.hd > 128) return launch_join<2, 64, IO>(ja, nsm, s);
  if (ja.geo.mt == 64) return launch_join<1, 64, IO>(ja, nsm, s);
  return launch_join<1, std::is_same<IO, float>::value ? 128 : 256, IO>(ja, nsm, s);
}

// The workspace: the counters and parts of attn_paged.cu, the head and the groups' places, states, parts.
struct Layout {
  size_t head, at, own_at, own, whole, parts, bytes;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
Layout layout(int n_seqs, int n_heads, int n_kv_heads, int head_dim) {
  Layout y;
  // (parts of the paged kernels' CTAs, or of attn_shared_own.cu's warps)
  static_assert(paged::PA_MAX_CTAS <= SH_MAX_CTAS * OWN_WARPS, "parts");
  y.head = up256(OP_COUNTER_BYTES + 2 * SH_MAX_CTAS * OWN_WARPS * paged::part_floats(n_heads, n_kv_heads, head_dim) * sizeof(float));
  y.at = y.head + 256;
  y.own_at = y.at + up256((size_t)n_seqs * sizeof(int));
  y.own = y.own_at + up256((size_t)n_seqs * sizeof(int));
  const size_t states = up256((size_t)n_seqs * n_heads * comb_stride(head_dim) * sizeof(float));
  y.whole = y.own + states;
  y.parts = y.whole + 2 * states;
  size_t most = 0;
  for (int io : {(int)QW_F32, (int)QW_F16}) {  // of the kernels that the shape may take: io is the cache's type or fp32
    const Geometry g = geometry(io == QW_F32 ? QW_F32 : QW_F16, io, head_dim, SH_MAX_CTAS);
    most = std::max(most, (size_t)2 * g.ctas * g.mt * comb_stride(g.hd) * sizeof(float));
  }
  y.bytes = y.parts + most;
  return y;
}

}  // namespace
}  // namespace shared_attn
}  // namespace qw

using namespace qw;
using namespace qw::shared_attn;

extern "C" {

size_t qw_op_shared_attention_workspace(int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_seqs < 0 || n_seqs > 65535 || n_heads > 4096 || !qw_op_paged_attention_workspace(n_heads, n_kv_heads, head_dim)) return 0;
  return layout(n_seqs < 1 ? 1 : n_seqs, n_heads, n_kv_heads, head_dim).bytes;
}

qw_status qw_op_shared_attention(const qw_paged_kv* cache, int32_t n_seqs, int32_t n_heads, const int32_t* block_table,
                                 int32_t max_blocks, const int32_t* lens, int32_t n_groups, const int32_t* cu_seqs,
                                 const int32_t* shared_lens, int32_t io_dtype, const void* q, int64_t q_stride, float scale,
                                 void* out, int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes,
                                 int32_t* err_dev, void* cuda_stream) {
  set_error_message("");
  qw_paged_kv c;
  qw_status st = paged::check_attention(cache, &c, n_seqs, n_heads, max_blocks, io_dtype, scale);
  if (st) return st;
  if (n_groups < 0 || n_groups > n_seqs) return op_fail(QW_ERR_INVALID_ARG, "n_groups must be at most n_seqs");
  if (n_seqs == 0) return QW_OK;
  if (n_groups == 0) return op_fail(QW_ERR_INVALID_ARG, "sequences without a group");
  const Geometry least = geometry(c.dtype, io_dtype, c.head_dim, 1);
  const int64_t tiles = ((int64_t)n_seqs * (n_heads / c.n_kv_heads) + least.mt - 1) / least.mt + n_groups;
  const int64_t own = (int64_t)max_blocks * c.page_size / own_rows(c.head_dim) + 1 + OWN_WEIGHT;
  if ((int64_t)n_seqs * n_heads * own > 0x7fffffffll) return op_fail(QW_ERR_UNSUPPORTED, "n_seqs * n_heads * max_blocks * page_size too large");
  if (tiles * c.n_kv_heads * (2 * ((int64_t)max_blocks * c.page_size / least.bk + 1) + unit_weight<256>(2)) > 0x7fffffffll)
    return op_fail(QW_ERR_UNSUPPORTED, "n_seqs * n_heads * max_blocks * page_size too large");
  if (!block_table || !lens || !cu_seqs || !shared_lens || !workspace || !err_dev) return op_fail(QW_ERR_INVALID_ARG, "null pointer");
  const int64_t width = (int64_t)n_heads * c.head_dim;
  if ((st = op_check_rows(q, q_stride, width, io_dtype, "q"))) return st;
  if ((st = op_check_rows(out, out_stride, width, io_dtype, "out"))) return st;
  if (out == q && out_stride != q_stride) return op_fail(QW_ERR_INVALID_ARG, "out may be q with the same stride only");
  if (!aligned16(workspace)) return op_fail(QW_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  const Layout y = layout(n_seqs, n_heads, c.n_kv_heads, c.head_dim);
  if (workspace_bytes < y.bytes) return op_fail(QW_ERR_INVALID_ARG, "workspace too small");
  if ((st = op_check_device({c.k, c.v, block_table, lens, cu_seqs, shared_lens, q, out, lse, workspace, err_dev}))) return st;
  int dev = 0, nsm = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) || (e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
    return op_cuda_fail(e, "device query");
  char* ws = (char*)workspace;
  JoinArgs ja;
  ja.s.p = OwnAttnArgs{{c.k, c.v, c.page_stride, c.head_stride, c.pos_stride, n_seqs, n_heads, c.n_kv_heads, c.head_dim,
                         c.page_size, c.n_pages, max_blocks, block_table, lens, q, out, q_stride, out_stride, scale, lse,
                         (unsigned int*)ws, (float*)(ws + OP_COUNTER_BYTES), err_dev}, shared_lens, (float*)(ws + y.own)};
  ja.s.n_groups = n_groups;
  ja.s.cu = cu_seqs;
  ja.s.head = (SharedHead*)(ws + y.head);
  ja.s.at = (int*)(ws + y.at);
  ja.s.own_head = ja.s.head + 1;
  ja.s.own_at = (int*)(ws + y.own_at);
  ja.s.whole = (float*)(ws + y.whole);
  ja.s.parts = (float*)(ws + y.parts);
  ja.geo = geometry(c.dtype, io_dtype, c.head_dim, nsm);
  cudaStream_t s = (cudaStream_t)cuda_stream;
  const bool tc = c.dtype != QW_F32 && c.head_dim <= 128;
  ja.own_hb = !tc ? 0 : n_heads / c.n_kv_heads <= 8 ? 8 : 16;
  ja.own_hd = c.head_dim <= 32 && ja.own_hb == 8 ? 32 : c.head_dim <= 64 ? 64 : 128;
  e = tc ? launch_own(c.dtype, io_dtype, ja.geo.ctas, ja.s, s)
         : paged::launch_simt(c.dtype, io_dtype, 2 * std::min(nsm, paged::PA_MAX_CTAS / 2), ja.s.p, s);
  if (e) return op_cuda_fail(e, "shared attention launch");
  e = !tc ? launch_shared_simt(c.dtype, io_dtype, ja.geo.ctas, ja.s, s)
      : io_dtype == QW_F32 ? launch_shared_tc(c, ja.geo.ctas, ja.s, s)
                           : launch_shared_pair(c, ja.geo.ctas, ja.s, s);
  if (e) return op_cuda_fail(e, "shared attention launch");
  e = io_dtype == QW_F32 ? launch_join<float>(ja, nsm, s) : io_dtype == QW_F16 ? launch_join<f16>(ja, nsm, s) : launch_join<bf16>(ja, nsm, s);
  if (e) return op_cuda_fail(e, "shared attention launch");
  return QW_OK;
}

}  // extern "C"
