// The shared positions of attn_shared.cu on the CUDA cores: fp32 caches, whose digits the tensor cores' types do not hold,
// and heads of more than 128 dimensions.
//
// A unit is 64 rows (sequence, head) of one group and KV head, blocks of 64 positions stream past them in shared memory as
// fp32. 256 threads as 16 x 16: thread (y, x) has the scores of rows y + 16 i and positions x + 16 j, i, j < 4, and then the
// outputs of the same rows at dimensions 4 x + 64 c; rows' statistics go across the 16 threads x, probabilities through
// shared memory within the warp. Products are packed pairs (f32x2).
// What bounds it: shared-memory loads, 16 bytes for every 4 packed products; two CTAs an SM up to 128 dimensions, so that
// one computes while the other waits for its block. 256 rows of 28 and 4 heads of 128 behind 8000 positions: 739 us
// (40 TFLOP/s; one CTA an SM 848), of 8 and 2 heads 225.
#include "attn_shared.cuh"

namespace qw {
namespace shared_attn {
namespace {

constexpr int MT = 64, BK = 64, THREADS = 256;

template <int HD>
struct Cfg {
  static constexpr int LD = HD + 4;   // floats of a row: 8 rows' same 16 bytes lie in distinct banks
  static constexpr int PS = BK + 4;
  static constexpr int SMEM = (MT + 2 * BK) * LD * 4;
  static_assert(SMEM <= 226 * 1024 && (HD > 128 || SMEM <= 112 * 1024), "shared memory: two CTAs an SM up to 128 dimensions");
  static_assert(MT * PS <= BK * LD, "probabilities take the keys' place");
};

// 4 elements at p as floats
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = paged::Pair<T>::unpack(u.x), b = paged::Pair<T>::unpack(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T, int HD, typename IO>
__global__ void __launch_bounds__(THREADS, HD <= 128 ? 2 : 1) shared_simt_kernel(const SharedArgs a) {
  using C = Cfg<HD>;
  constexpr int LD = C::LD, PS = C::PS, G4 = HD / 4, NC = HD / 64;  // groups of 4 dimensions; those of a thread
  extern __shared__ __align__(16) float sh_f[];
  __shared__ long long s_off[BK];
  float *qs = sh_f, *ks = qs + MT * LD, *vs = ks + BK * LD, *ps = ks;  // (probabilities take the place of used keys)
  const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
  pdl_trigger();
  Unit p;
  const Range r = find_groups<MT, BK, THREADS>(a, p, sh_f);
  if (r.begin >= r.end) {
    pdl_wait();  // (this grid ends after the one before it)
    return;
  }
  const float sc = a.p.scale * paged::LOG2E;
  do {
    const int kv = p.u / p.nt, tile = p.u - kv * p.nt, t1 = p.t + blocks_of<MT>(p, r.end);
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < MT * G4; i += THREADS) {
      const int rr = i / G4, d = (i - rr * G4) * 4;
      const Row row = row_of(a, p, kv, tile * MT + rr);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row.in && d < a.p.hd) v = load4((const IO*)a.p.q + row.b * a.p.q_stride + row.h * a.p.hd + d);
      *reinterpret_cast<float4*>(qs + rr * LD + d) = v;
    }
    float m[4], l[4];  // l: of this thread's positions
    bool any = false;
    f32x2 o[4][NC][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c][0] = o[i][c][1] = 0ull;
    }
#pragma unroll 1
    for (int t = p.t; t < t1; ++t) {
      __syncthreads();  // (the last block is used up)
      if (tid < BK) s_off[tid] = position_of<T>(a, p, kv, t * BK + tid);
      __syncthreads();
#pragma unroll 4
      for (int i = tid; i < BK * G4; i += THREADS) {
        const int j = i / G4, d = (i - j * G4) * 4;
        const long long off = s_off[j];
        const bool there = off >= 0 && d < a.p.hd;
        if constexpr (sizeof(T) == 4) {
          const long long at = there ? off + d * 4 : 0;
          paged::cp_async16_or_zero(smem_addr(ks + j * LD + d), (const char*)a.p.k + at, there);
          paged::cp_async16_or_zero(smem_addr(vs + j * LD + d), (const char*)a.p.v + at, there);
        } else {
          float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
          if (there) {
            kx = load4((const T*)((const char*)a.p.k + off) + d);
            vx = load4((const T*)((const char*)a.p.v + off) + d);
          }
          *reinterpret_cast<float4*>(ks + j * LD + d) = kx;
          *reinterpret_cast<float4*>(vs + j * LD + d) = vx;
        }
      }
      paged::cp_commit();
      paged::cp_wait<0>();
      __syncthreads();
      f32x2 dot[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dot[i][j] = 0ull;
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        ulonglong2 q4[4], k4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q4[i] = *reinterpret_cast<const ulonglong2*>(qs + (y + 16 * i) * LD + d);
          k4[i] = *reinterpret_cast<const ulonglong2*>(ks + (x + 16 * i) * LD + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fma2(dot[i][j], q4[i].x, k4[j].x);
            fma2(dot[i][j], q4[i].y, k4[j].y);
          }
      }
      bool there[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) there[j] = s_off[x + 16 * j] >= 0;
      any |= __syncthreads_or(there[0] | there[1] | there[2] | there[3]) != 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float s[4], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 two = unpack2(dot[i][j]);
          s[j] = there[j] ? (two.x + two.y) * sc : -INFINITY;
          top = fmaxf(top, s[j]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float mn = fmaxf(m[i], top), f = mn > m[i] ? ex2(m[i] - mn) : 1.f, ref = (mn == -INFINITY ? 0.f : mn) - PA_BIAS;
        m[i] = mn;
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = ex2(s[j] - ref);
          ps[(y + 16 * i) * PS + x + 16 * j] = e[j];
        }
        l[i] = fmaf(l[i], f, (e[0] + e[1]) + (e[2] + e[3]));
        const f32x2 f2 = pack2(f, f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          mul2(o[i][c][0], f2);
          mul2(o[i][c][1], f2);
        }
      }
      __syncwarp();  // (a row's probabilities come from and go to the 16 threads of one y)
#pragma unroll 2
      for (int j = 0; j < BK; j += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (y + 16 * i) * PS + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(vs + (j + jj) * LD + 4 * x + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float wi = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
              const f32x2 w2 = pack2(wi, wi);
              fma2(o[i][c][0], w2, v4.x);
              fma2(o[i][c][1], w2, v4.y);
            }
          }
      }
    }
    const bool whole = p.t == 0 && t1 == p.nb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = l[i];
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const int rr = y + 16 * i;
      const Row row = row_of(a, p, kv, tile * MT + rr);
      if (!row.in) continue;
      float* dst = state_of<MT, HD>(a, r, p, whole, row, rr);
      const int width = whole ? a.p.hd : HD;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float2 lo = unpack2(o[i][c][0]), hi = unpack2(o[i][c][1]);
        if (4 * x + 64 * c < width) *reinterpret_cast<float4*>(dst + 4 * x + 64 * c) = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
      if (x == 0) *reinterpret_cast<float2*>(dst + width) = make_float2(paged::state_max(m[i], any), sum);
    }
  } while (next_unit<MT, BK>(a, r.end, p));
  pdl_wait();  // (this grid ends after the one before it)
}

template <typename T, int HD, typename IO>
cudaError_t run(int ctas, const SharedArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(shared_simt_kernel<T, HD, IO>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::SMEM);
  return e ? e : launch_k(shared_simt_kernel<T, HD, IO>, dim3(ctas), dim3(THREADS), Cfg<HD>::SMEM, s, true, a);
}

}  // namespace

cudaError_t launch_shared_simt(int cache_dtype, int io_dtype, int ctas, const SharedArgs& a, cudaStream_t s) {
  if (cache_dtype == QW_F16) return io_dtype == QW_F32 ? run<f16, 256, float>(ctas, a, s) : run<f16, 256, f16>(ctas, a, s);
  if (cache_dtype == QW_BF16) return io_dtype == QW_F32 ? run<bf16, 256, float>(ctas, a, s) : run<bf16, 256, bf16>(ctas, a, s);
  return a.p.hd <= 64 ? run<float, 64, float>(ctas, a, s) : a.p.hd <= 128 ? run<float, 128, float>(ctas, a, s) : run<float, 256, float>(ctas, a, s);
}

}  // namespace shared_attn
}  // namespace qw
