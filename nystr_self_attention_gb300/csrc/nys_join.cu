// What follows a product whose K was split over CTAs (nys_gemm.h): the partial
// sums are added in the order of their ranges, so the same call gives the same
// bits, then rounded, or gated, and written. Bound by reading the partial sums,
// mostly from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nys_gemm.h"

namespace nys {
namespace gemm {
namespace {

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void add(float4& a, const float4& b) {
  a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

// Four columns per thread.
template <typename T>
__global__ void __launch_bounds__(256)
join_rows(const Join j, int parts) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int quads = j.N / 4;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = e / quads;  // of all parts
  if (row >= (long long)j.M * parts) return;
  const int part = row >= j.M, c = (int)(e - row * quads) * 4;
  const long long m = row - (long long)part * j.M, plane = (long long)j.M * j.N;
  const float* at = j.part + part * plane + m * j.N + c;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < j.splits; ++s) add(v, *reinterpret_cast<const float4*>(at + s * parts * plane));
  put4(static_cast<T*>(part ? j.out[1] : j.out[0]) + m * (part ? j.stride[1] : j.stride[0]) + c, v);
}

// Turned planes: a CTA takes 32 columns of the result x 32 rows.
template <typename T>
__global__ void __launch_bounds__(256)
join_turned(const Join j) {
  __shared__ float tile[32][33];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 32;
  const int n = n0 + threadIdx.x / 8, m = m0 + (threadIdx.x & 7) * 4;
  const long long plane = (long long)j.N * j.line.width;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n < j.N && m < j.M) {
    const float* at = j.part + (long long)n * j.line.width + m;
    const int planes = j.line.planes(0, n0);
#pragma unroll 8
    for (int s = 0; s < planes; ++s) add(v, *reinterpret_cast<const float4*>(at + s * plane));
  }
  const int q = (threadIdx.x & 7) * 4;
  tile[q][threadIdx.x / 8] = v.x, tile[q + 1][threadIdx.x / 8] = v.y;
  tile[q + 2][threadIdx.x / 8] = v.z, tile[q + 3][threadIdx.x / 8] = v.w;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x / 32; r < 32 && m0 + r < j.M; r += 8)
    if (n0 + lane < j.N) put(static_cast<T*>(j.out[0]) + (m0 + r) * j.stride[0] + n0 + lane, tile[r][lane]);
}

template <typename T>
__global__ void __launch_bounds__(256)
join_gated_rows(const JoinGated j, int act) {
  constexpr bool kFast = sizeof(T) == 2;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int quads = j.N / 4;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x, m = e / quads;
  if (m >= j.M) return;
  const int c = (int)(e - m * quads) * 4;
  const long long plane = (long long)j.M * j.N;
  const float* at = j.part + m * j.N + c;
  float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
  for (int s = 0; s < j.splits; ++s) {
    add(g, *reinterpret_cast<const float4*>(at + 2 * s * plane));
    add(u, *reinterpret_cast<const float4*>(at + (2 * s + 1) * plane));
  }
  if (j.gate) {
    put4(static_cast<T*>(j.gate) + m * j.gate_stride + c, g);
    put4(static_cast<T*>(j.up) + m * j.up_stride + c, u);
  }
  act::by_act(act, [&](auto a) {
    constexpr int A = decltype(a)::value;
    put4(static_cast<T*>(j.h) + m * j.h_stride + c,
         make_float4(act::value<A, kFast>(g.x) * u.x, act::value<A, kFast>(g.y) * u.y,
                     act::value<A, kFast>(g.z) * u.z, act::value<A, kFast>(g.w) * u.w));
  });
}

template <typename T>
__global__ void __launch_bounds__(256)
join_gated_turned(const JoinGated j, int act) {
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ float gs[32][33], us[32][33];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 32;
  const int n = n0 + threadIdx.x / 8, m = m0 + (threadIdx.x & 7) * 4;
  const long long plane = (long long)j.N * j.line.width;
  float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
  if (n < j.N && m < j.M) {
    const float* at = j.part + (long long)n * j.line.width + m;
    const int of_g = j.line.planes(0, n0), of_u = j.line.planes(1, n0);
#pragma unroll 4
    for (int s = 0; s < of_g; ++s) add(g, *reinterpret_cast<const float4*>(at + 2 * s * plane));
#pragma unroll 4
    for (int s = 0; s < of_u; ++s) add(u, *reinterpret_cast<const float4*>(at + (2 * s + 1) * plane));
  }
  const int q = (threadIdx.x & 7) * 4, f = threadIdx.x / 8;
  gs[q][f] = g.x, gs[q + 1][f] = g.y, gs[q + 2][f] = g.z, gs[q + 3][f] = g.w;
  us[q][f] = u.x, us[q + 1][f] = u.y, us[q + 2][f] = u.z, us[q + 3][f] = u.w;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  if (n0 + lane >= j.N) return;
  for (int r = threadIdx.x / 32; r < 32 && m0 + r < j.M; r += 8) {
    const float a = gs[r][lane], b = us[r][lane];
    const long long row = m0 + r;
    if (j.gate) {
      put(static_cast<T*>(j.gate) + row * j.gate_stride + n0 + lane, a);
      put(static_cast<T*>(j.up) + row * j.up_stride + n0 + lane, b);
    }
    const float h = act::by_act(act, [&](auto k) { return act::value<decltype(k)::value, kFast>(a); }) * b;
    put(static_cast<T*>(j.h) + row * j.h_stride + n0 + lane, h);
  }
}

template <typename K, typename... Args>
int start(const char* name, K kernel, dim3 grid, cudaStream_t st, Args... args) {
  return launch_behind(name, kernel, grid, dim3(256), 0, st, args...);
}

}  // namespace

int join(const Join& j, int parts, int dtype, cudaStream_t st) {
  const bool bf16 = dtype == NYS_BF16;
  if (j.line.width) {
    const dim3 grid((j.N + 31) / 32, (j.M + 31) / 32);
    return bf16 ? start("product_join", join_turned<__nv_bfloat16>, grid, st, j)
                : start("product_join", join_turned<float>, grid, st, j);
  }
  const long long ctas = ((long long)j.M * parts * (j.N / 4) + 255) / 256;
  if (ctas >= (1ll << 31)) return NYS_ERR_SHAPE;
  return bf16 ? start("product_join", join_rows<__nv_bfloat16>, dim3((unsigned)ctas), st, j, parts)
              : start("product_join", join_rows<float>, dim3((unsigned)ctas), st, j, parts);
}

int join_gated(const JoinGated& j, int act, int dtype, cudaStream_t st) {
  const bool bf16 = dtype == NYS_BF16;
  if (j.line.width) {
    const dim3 grid((j.N + 31) / 32, (j.M + 31) / 32);
    return bf16 ? start("gated_join", join_gated_turned<__nv_bfloat16>, grid, st, j, act)
                : start("gated_join", join_gated_turned<float>, grid, st, j, act);
  }
  const long long ctas = ((long long)j.M * (j.N / 4) + 255) / 256;
  if (ctas >= (1ll << 31)) return NYS_ERR_SHAPE;
  return bf16 ? start("gated_join", join_gated_rows<__nv_bfloat16>, dim3((unsigned)ctas), st, j, act)
              : start("gated_join", join_gated_rows<float>, dim3((unsigned)ctas), st, j, act);
}

}  // namespace gemm
}  // namespace nys
