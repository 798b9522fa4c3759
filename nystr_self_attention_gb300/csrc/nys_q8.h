// Format and checks of matrices in 8 bits (include/nystrom.h), shared by the
// kernels that write, read and multiply them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nys_internal.h"

namespace nys {
namespace q8 {

constexpr int kBlock = 128;  // channels of one scale

// Scale byte of a block whose largest magnitude has these bits: adding 2^21 - 1
// carries into the exponent exactly where the mantissa is above 1.75 (448 = 1.75
// * 2^8). 255 for an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return 255u;
  const int e = (int)((top_bits + 0x1fffffu) >> 23) - 8;
  return (uint32_t)max(e, 0);
}
// 1 / scale, exactly: 2^(127 - byte).
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Codes of four values over their scale, channel i in byte i. Rounded to nearest
// even by the conversion; a NaN becomes the code for NaN.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %5, %4;\n\tcvt.u32.u16 %0, l;\n\tcvt.u32.u16 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "f"(a * inv), "f"(b * inv), "f"(c * inv), "f"(d * inv));
  return lo | hi << 16;
}
// Two codes (low half of w) as fp32.
__device__ __forceinline__ float2 decode2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(w));
  float2 v;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

// Byte of a row's block among the scale words.
__device__ __forceinline__ size_t scale_at(int block, int row, int rows) {
  return ((size_t)(block >> 2) * rows + row) * 4 + (block & 3);
}
// Stores a block's scale; the last block of a row clears the bytes behind it.
__device__ __forceinline__ void store_scale(uint8_t* scales, int block, int blocks, int row, int rows,
                                            uint32_t byte) {
  uint8_t* at = scales + scale_at(block, row, rows);
  at[0] = (uint8_t)byte;
  if (block == blocks - 1)
    for (int j = 1; j < 4 - (block & 3); ++j) at[j] = 0;
}

// Host checks of a matrix; NYS_OK or the code of include/nystrom.h. apart: its rows
// may not overlap (an output, or read by tensor maps).
inline int check_q8(const nys_q8_t* q, bool apart) {
  if (!q || !q->codes || !q->scales) return NYS_ERR_ARG;
  if (q->rows < 1 || q->rows >= 0x7fffffff - 1023 || q->K < 1 || q->K % 16 || q->K > (1 << 20))
    return NYS_ERR_SHAPE;
  if (q->rows > 1 && q->stride < 0) return NYS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q->codes) & 15u) || (reinterpret_cast<uintptr_t>(q->scales) & 3u) ||
      (q->rows > 1 && q->stride % 16))
    return NYS_ERR_ALIGN;
  return q->codes == q->scales || (apart && q->rows > 1 && q->stride < q->K) ? NYS_ERR_ARG : NYS_OK;
}

// Host checks of a matrix of rows x `width` in dtype.
inline int check_rows(const void* p, long long stride, int rows, int width, int dtype, bool apart) {
  const long long per = dtype == NYS_FP32 ? 4 : 8;  // elements in 16 bytes
  if (rows > 1 && stride < 0) return NYS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) || (rows > 1 && stride % per)) return NYS_ERR_ALIGN;
  return apart && rows > 1 && stride < width ? NYS_ERR_ARG : NYS_OK;
}

}  // namespace q8
}  // namespace nys
