// Products of a few fp32 rows (tokens) with fp32 weights, on the CUDA cores: the
// weights' bytes bound the time, so they are read once, as they lie, and not split
// into the tensor cores' terms first (which takes four times the traffic). One
// token through 4096 -> 4712 twice takes 29 us, 5.3 TB/s; eight take 46 to 50, with
// the FMA units half busy, and from some 24 on the terms are cheaper.
//
// Up to eight tokens share a read; more go in groups of eight, side by side, whose
// reads meet in L2. Either the weights' K is contiguous (a warp takes four outputs,
// its lanes go along K) or their outputs are (a lane takes four, the CTA's warps
// take K in turn). K is split into ranges until the GPU is full; every range writes
// a plane of sums, which nys_join.cu adds up in order.
#include <cuda_runtime.h>

#include "nys_gemm.h"

namespace nys {
namespace gemm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return reinterpret_cast<float2&>(d);
}

// blockIdx.x: group of T tokens, y: outputs, z: 2 split + i, with weights i.
// Weights [N][K]: a warp takes outputs n .. n + 3.
template <int T>
__global__ void __launch_bounds__(kThreads, 2)
few_k(const __grid_constant__ Few p) {
  constexpr int kChunk = 1024;  // of K, whose x stands in shared memory
  __shared__ __align__(16) float xs[T][kChunk];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.z & 1, split = blockIdx.z >> 1, t0 = blockIdx.x * T;
  const int n = ((int)blockIdx.y * kWarps + warp) * 4;
  const long long k0 = (long long)split * p.range, k1 = min((long long)p.K, k0 + p.range);
  const float* x = p.x[i];
  const float* w[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) w[r] = p.w[i] + (long long)min(n + r, p.N - 1) * p.w_stride;
  float2 acc[4][T];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = make_float2(0.f, 0.f);
  for (long long c = k0; c < k1; c += kChunk) {
    const int len = (int)min((long long)kChunk, k1 - c);  // a multiple of 8
    __syncthreads();
    for (int e = threadIdx.x * 4; e < T * kChunk; e += kThreads * 4) {
      const int t = e / kChunk, k = e % kChunk;
      const float4 v = t0 + t < p.T && k < len
                           ? *reinterpret_cast<const float4*>(x + (long long)(t0 + t) * p.x_stride + c + k)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(&xs[t][k]) = v;
    }
    __syncthreads();
#pragma unroll 2
    for (int k = lane * 4; k < len; k += 128) {
      float4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __ldcs(reinterpret_cast<const float4*>(w[r] + c + k));
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float4 a = *reinterpret_cast<const float4*>(&xs[t][k]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r][t] = fma2(make_float2(v[r].x, v[r].y), make_float2(a.x, a.y), acc[r][t]);
          acc[r][t] = fma2(make_float2(v[r].z, v[r].w), make_float2(a.z, a.w), acc[r][t]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[r] = acc[r][t].x + acc[r][t].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
    }
    if (lane == 0 && n < p.N && t0 + t < p.T)  // N is a multiple of 8
      *reinterpret_cast<float4*>(p.part + ((long long)blockIdx.z * p.T + t0 + t) * p.N + n) =
          make_float4(s[0], s[1], s[2], s[3]);
  }
}

// Weights [K][N]: a lane takes outputs n .. n + 3, warp j the k's j, j + 8, ...
template <int T>
__global__ void __launch_bounds__(kThreads, 2)
few_n(const __grid_constant__ Few p) {
  constexpr int kChunk = 512;
  // x, each value twice: the packed products take pairs; then the warps' sums
  __shared__ __align__(16) float2 xs[kChunk][T];
  static_assert(sizeof(xs) >= sizeof(float4) * T * 32 * kWarps / 2, "sums of the warps, in two goes");
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.z & 1, split = blockIdx.z >> 1, t0 = blockIdx.x * T;
  const int n = ((int)blockIdx.y * 32 + lane) * 4;
  const bool in = n < p.N;  // N is a multiple of 8
  const long long k0 = (long long)split * p.range, k1 = min((long long)p.K, k0 + p.range);
  const float* x = p.x[i];
  const float* w = p.w[i] + (in ? n : 0);
  float2 lo[T], hi[T];
#pragma unroll
  for (int t = 0; t < T; ++t) lo[t] = hi[t] = make_float2(0.f, 0.f);
  for (long long c = k0; c < k1; c += kChunk) {
    const int len = (int)min((long long)kChunk, k1 - c);
    __syncthreads();
    for (int e = threadIdx.x; e < T * kChunk; e += kThreads) {
      const int t = e / kChunk, k = e % kChunk;
      const float v = t0 + t < p.T && k < len ? x[(long long)(t0 + t) * p.x_stride + c + k] : 0.f;
      xs[k][t] = make_float2(v, v);
    }
    __syncthreads();
#pragma unroll 4
    for (int k = warp; k < len; k += kWarps) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(w + (c + k) * p.w_stride));
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float2 a = xs[k][t];
        lo[t] = fma2(make_float2(v.x, v.y), a, lo[t]);
        hi[t] = fma2(make_float2(v.z, v.w), a, hi[t]);
      }
    }
  }
  // warps 4 .. 7 hand their sums to 0 .. 3, those theirs to 0 and 1, 1 to 0
  float4* sums = reinterpret_cast<float4*>(&xs[0][0]);
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (warp >= half && warp < 2 * half)
#pragma unroll
      for (int t = 0; t < T; ++t)
        sums[((warp - half) * T + t) * 32 + lane] = make_float4(lo[t].x, lo[t].y, hi[t].x, hi[t].y);
    __syncthreads();
    if (warp < half)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float4 v = sums[(warp * T + t) * 32 + lane];
        lo[t].x += v.x, lo[t].y += v.y, hi[t].x += v.z, hi[t].y += v.w;
      }
  }
  if (warp || !in) return;
#pragma unroll
  for (int t = 0; t < T; ++t)
    if (t0 + t < p.T)
      *reinterpret_cast<float4*>(p.part + ((long long)blockIdx.z * p.T + t0 + t) * p.N + n) =
          make_float4(lo[t].x, lo[t].y, hi[t].x, hi[t].y);
}

int outputs_per_cta(bool k_contiguous) { return k_contiguous ? kWarps * 4 : 128; }

}  // namespace

int few_range(int T, int N, int K, bool k_contiguous) {
  const long long ctas = 2ll * ((N + outputs_per_cta(k_contiguous) - 1) / outputs_per_cta(k_contiguous)) *
                         ((T + 7) / 8);
  long long splits = (4ll * plan_sms() + ctas - 1) / ctas;
  if (splits > 16) splits = 16;
  if (splits > K / 256) splits = K / 256;  // of 256 at least
  if (splits < 1) splits = 1;
  return (int)(((K + splits - 1) / splits + 7) / 8 * 8);
}

int launch_few(const char* name, const Few& p, bool k_contiguous, cudaStream_t st) {
  const int per = outputs_per_cta(k_contiguous);
  auto go = [&](auto tokens) {
    constexpr int T = decltype(tokens)::value;
    const dim3 grid((p.T + T - 1) / T, (p.N + per - 1) / per, 2 * p.splits());
    return k_contiguous ? launch_behind(name, few_k<T>, grid, dim3(kThreads), 0, st, p)
                        : launch_behind(name, few_n<T>, grid, dim3(kThreads), 0, st, p);
  };
  using std::integral_constant;
  if (p.T == 1) return go(integral_constant<int, 1>{});
  if (p.T == 2) return go(integral_constant<int, 2>{});
  if (p.T <= 4) return go(integral_constant<int, 4>{});
  return go(integral_constant<int, 8>{});
}

}  // namespace gemm
}  // namespace nys
