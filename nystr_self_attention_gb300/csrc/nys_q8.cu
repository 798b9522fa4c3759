// Matrices in 8 bits: written (quantised) and read back (format and entry
// points: include/nystrom.h). Both are bound by HBM: an element of the wide
// type on one side, a byte and 1/128 on the other.
//
// A CTA of 256 threads quantises a tile of 128 rows x 128 channels. Where the
// channels are contiguous a thread takes eight of them of a row, 16 threads the
// block, and the block's largest magnitude takes four shuffles. Where the rows
// are contiguous (a weight kept as [K][rows]) a thread takes eight rows of a
// channel; the rows' magnitudes meet in shared memory, and so do the codes, so
// that they leave in whole vectors.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "nys_q8.h"

namespace nys {
namespace q8 {
namespace {

constexpr int kTile = 128, kThreads = 256;

struct WriteParams {
  uint8_t *codes, *scales;
  long long stride, step;  // bytes between rows of codes; elements between the input's runs
  int rows, K;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Largest of the CTA's 256 values, in every thread.
__device__ __forceinline__ uint32_t cta_max(uint32_t top, uint32_t* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, slots[w]);
  return top;
}

// Channels contiguous. SHARED: the tile's rows share a scale.
template <typename T, bool SHARED>
__global__ void __launch_bounds__(kThreads)
q8_write(const WriteParams p, const T* __restrict__ x) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  __shared__ uint32_t slots[kThreads / 32];
  const int blocks = (p.K + kBlock - 1) / kBlock;
  const int block = blockIdx.x % (unsigned)blocks, r0 = (int)(blockIdx.x / (unsigned)blocks) * kTile;
  const int c = block * kBlock + (threadIdx.x & 15) * 8;
  const bool in = c < p.K;  // K is a multiple of 16
  float v[8][8];
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + i * 16 + threadIdx.x / 16;
    top[i] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (in && row < p.rows) load8<T>(x + row * p.step + c, v[i]);
  }
  uint32_t all = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) top[i] = max(top[i], magnitude(v[i][j]));
    all = max(all, top[i]);
  }
  if (SHARED) all = cta_max(all, slots);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + i * 16 + threadIdx.x / 16;
    if (!SHARED) {
      if (r0 + i * 16 >= p.rows) break;  // CTA-uniform
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    }
    const uint32_t byte = scale_byte(SHARED ? all : top[i]);
    const float inv = inverse_scale(byte);
    if (row >= p.rows) continue;
    if (in)
      *reinterpret_cast<uint2*>(p.codes + row * p.stride + c) =
          make_uint2(encode4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                     encode4(v[i][4], v[i][5], v[i][6], v[i][7], inv));
    if ((threadIdx.x & 15) == 0) store_scale(p.scales, block, blocks, row, p.rows, byte);
  }
}

// Rows contiguous: eight rows of channels k0 + t / 16 + 16 i per thread.
template <typename T, bool SHARED>
__global__ void __launch_bounds__(kThreads)
q8_write_turned(const WriteParams p, const T* __restrict__ x) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  constexpr int kPitch = kTile + 16;
  __shared__ uint32_t slots[kThreads / 32];
  __shared__ __align__(16) uint32_t tops[16][kTile];
  __shared__ __align__(16) uint8_t image[kTile][kPitch];  // [row][channel]
  const int blocks = (p.K + kBlock - 1) / kBlock;
  const int block = blockIdx.x % (unsigned)blocks, r0 = (int)(blockIdx.x / (unsigned)blocks) * kTile;
  const int k0 = block * kBlock, unit = threadIdx.x & 15, kt = threadIdx.x >> 4;
  const int row = r0 + unit * 8;
  float v[8][8];
  uint32_t top[8] = {};
  uint32_t all = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + kt + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (k < p.K && row < p.rows) load8<T>(x + k * p.step + row, v[i]);  // rows are a multiple of 8
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top[j] = max(top[j], magnitude(v[i][j]));
  if (SHARED) {
#pragma unroll
    for (int j = 0; j < 8; ++j) all = max(all, top[j]);
    all = cta_max(all, slots);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) tops[kt][unit * 8 + j] = top[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top[j] = 0u;
#pragma unroll
      for (int k = 0; k < 16; ++k) top[j] = max(top[j], tops[k][unit * 8 + j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float inv = inverse_scale(scale_byte(SHARED ? all : top[j]));
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const uint32_t four = encode4(v[i][j], v[i + 1][j], v[i + 2][j], v[i + 3][j], inv);
#pragma unroll
      for (int b = 0; b < 4; ++b) image[unit * 8 + j][kt + 16 * (i + b)] = (uint8_t)(four >> (8 * b));
    }
    if (kt == 0 && row + j < p.rows)
      store_scale(p.scales, block, blocks, row + j, p.rows, scale_byte(SHARED ? all : top[j]));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kTile * 8; e += kThreads) {
    const int r = e >> 3, c = (e & 7) * 16;
    if (r0 + r < p.rows && k0 + c < p.K)
      *reinterpret_cast<uint4*>(p.codes + (r0 + r) * p.stride + k0 + c) =
          *reinterpret_cast<const uint4*>(&image[r][c]);
  }
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sixteen threads take the eight channels each of a block; four blocks apart in
// rows per thread, so that their loads overlap.
template <typename T>
__global__ void __launch_bounds__(kThreads)
q8_read(const WriteParams p, T* __restrict__ out) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  constexpr int kAhead = 4;
  const int blocks = (p.K + kBlock - 1) / kBlock;
  const int block = blockIdx.x % (unsigned)blocks, r0 = (int)(blockIdx.x / (unsigned)blocks) * (16 * kAhead);
  const int c = block * kBlock + (threadIdx.x & 15) * 8;
  if (c >= p.K) return;
  uint2 codes[kAhead];
  uint32_t byte[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int row = r0 + i * 16 + threadIdx.x / 16;
    if (row >= p.rows) continue;
    codes[i] = *reinterpret_cast<const uint2*>(p.codes + row * p.stride + c);
    byte[i] = p.scales[scale_at(block, row, p.rows)];
  }
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int row = r0 + i * 16 + threadIdx.x / 16;
    if (row >= p.rows) continue;
    const float s = scale_value(byte[i]);
    const float2 a = decode2(codes[i].x & 0xffffu), b = decode2(codes[i].x >> 16);
    const float2 e = decode2(codes[i].y & 0xffffu), f = decode2(codes[i].y >> 16);
    const float v[8] = {a.x * s, a.y * s, b.x * s, b.y * s, e.x * s, e.y * s, f.x * s, f.y * s};
    store8(out + row * p.step + c, v);
  }
}

// CTAs of tiles of `rows` rows x 128 channels, or 0 where they are too many.
unsigned tiles_of(const nys_q8_t& q, int rows) {
  const long long n = ((long long)q.rows + rows - 1) / rows * ((q.K + kBlock - 1) / kBlock);
  return n < (1ll << 31) ? (unsigned)n : 0u;
}

WriteParams params_of(const nys_q8_t& q, long long step) {
  return WriteParams{static_cast<uint8_t*>(q.codes), static_cast<uint8_t*>(q.scales), q.stride, step,
                     q.rows, q.K};
}

}  // namespace
}  // namespace q8
}  // namespace nys

using namespace nys;
using namespace nys::q8;

extern "C" {

size_t nystrom_q8_scales_bytes(int rows, int K) {
  alignas(16) static int some[8] = {};
  const nys_q8_t q{some, some + 4, rows, K, (K + 15ll) / 16 * 16};
  if (check_q8(&q, false) != NYS_OK) return 0;
  return (size_t)((K + 4 * kBlock - 1) / (4 * kBlock)) * rows * 4;
}

int nystrom_q8_write(const nys_q8_t* q, const void* x, long long row_stride, long long channel_stride,
                     int block_rows, int dtype, nys_stream_t stream) {
  int rc = check_q8(q, true);
  if (rc != NYS_OK) return rc;
  if (!x || (dtype != NYS_FP32 && dtype != NYS_BF16) || (block_rows != 1 && block_rows != kTile))
    return NYS_ERR_ARG;
  const bool turned = channel_stride != 1;
  if (turned && row_stride != 1) return NYS_ERR_ARG;
  if (turned && q->rows % 8) return NYS_ERR_SHAPE;
  const long long step = turned ? channel_stride : row_stride;
  rc = check_rows(x, step, turned ? q->K : q->rows, turned ? q->rows : q->K, dtype, false);
  if (rc != NYS_OK) return rc;
  if (x == q->codes || x == q->scales) return NYS_ERR_ARG;
  const unsigned grid = tiles_of(*q, kTile);
  if (!grid) return NYS_ERR_SHAPE;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  const WriteParams p = params_of(*q, step);
  auto go = [&](auto type) {
    using T = decltype(type);
    auto launch = [&](auto kernel) {
      return launch_behind("q8_write", kernel, dim3(grid), dim3(kThreads), 0, stream, p, static_cast<const T*>(x));
    };
    if (turned) return block_rows == 1 ? launch(q8_write_turned<T, false>) : launch(q8_write_turned<T, true>);
    return block_rows == 1 ? launch(q8::q8_write<T, false>) : launch(q8::q8_write<T, true>);
  };
  return dtype == NYS_BF16 ? go(__nv_bfloat16{}) : go(float{});
}

int nystrom_q8_read(const nys_q8_t* q, void* out, long long stride, int dtype, nys_stream_t stream) {
  int rc = check_q8(q, false);
  if (rc != NYS_OK) return rc;
  if (!out || (dtype != NYS_FP32 && dtype != NYS_BF16)) return NYS_ERR_ARG;
  rc = check_rows(out, stride, q->rows, q->K, dtype, true);
  if (rc != NYS_OK) return rc;
  if (out == q->codes || out == q->scales) return NYS_ERR_ARG;
  const unsigned grid = tiles_of(*q, 64);
  if (!grid) return NYS_ERR_SHAPE;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  const WriteParams p = params_of(*q, stride);
  if (dtype == NYS_BF16)
    return launch_behind("q8_read", q8::q8_read<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, stream, p,
                         static_cast<__nv_bfloat16*>(out));
  return launch_behind("q8_read", q8::q8_read<float>, dim3(grid), dim3(kThreads), 0, stream, p,
                       static_cast<float*>(out));
}

}  // extern "C"
