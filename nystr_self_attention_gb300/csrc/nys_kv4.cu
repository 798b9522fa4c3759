// The 4-bit key/value cache: tokens quantised as they are written, and read
// back (declared, with the format, in include/nystrom.h). Both directions are
// bound by HBM: 2 d elements on one side, 9 d / 8 bytes on the other, per token
// and head.
//
// A warp handles the keys or the values of one block of 16 tokens of one head:
// d/8 lanes per row, each eight channels (16 bytes of bf16), so four lanes share
// a scale and agree on it by two shuffles. The 9 d bytes are put together (or
// taken apart) in shared memory and cross to or from HBM as whole 16-byte
// vectors; a block that gets only some of its tokens is written piece by piece,
// never read and rewritten, so its other tokens are not touched.
//
// Written and read back, 2 x 32765 tokens x 16 heads, d = 128, bf16 (1.2 GB):
// 180 to 205 us on several cards, 5.9 to 6.7 TB/s where a copy reaches 6.8. Short calls are one wave of CTAs and
// bound by its chain of loads: 8 x 1021 tokens x 8 heads, d = 64, fp32: 21 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nys_kv4.h"

namespace nys {
namespace kv4 {

int check_cache(const nys_kv4_cache_t* c) {
  if (!c || !c->data || !c->block_table) return NYS_ERR_ARG;
  if (c->num_pages < 1 || c->max_pages < 1 || c->Hk < 1 || c->Hk > 65535) return NYS_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 4096 || c->page_size % 16) return NYS_ERR_SHAPE;
  if (c->d != 32 && c->d != 64 && c->d != 128) return NYS_ERR_SHAPE;
  // tiles and windows of pages past the last one keep 32-bit key indexes
  if ((long long)c->max_pages * c->page_size > (1ll << 31) - 65536) return NYS_ERR_SHAPE;
  // the pool's size and the addresses in it stay far from 64 bits
  if ((long long)c->num_pages * c->Hk > (1ll << 47) / ((long long)(c->page_size / kBlock) * block_bytes(c->d)))
    return NYS_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(c->data) & 15u) return NYS_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(c->block_table) & 3u) return NYS_ERR_ALIGN;
  return NYS_OK;
}

namespace {

constexpr int kWarps = 4;

struct IoParams {
  View cache;
  nys_strides_t ks, vs;
  const int *starts, *counts;
  int* status;
  int n;
  unsigned items;  // of a sequence: blocks x heads x 2 (keys, values)
};

// Eight channels of a row as they lie in memory, as fp32, and their largest
// magnitude's bits (magnitudes compare as integers, NaN above infinity).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)),
               max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;  // two magnitudes per word
    const uint32_t t = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
    return max(t & 0xffff0000u, t << 16);
  }
};

// Eight 4-bit fields (code + 8) of x / s rounded to the nearest integer, ties
// to even; channel i in bits 4i. The integers come out of the mantissa of
// 1.5 * 2^23 + 8 + code, whose low four bits they are.
//
// bf16 values over a bf16 scale: x / s is a tie (k + 1/2) or at least
// (k + 1/2) * 2^-12 away from one, since both have 8 significant bits. x *
// (1/s) is off by less than 2^-19 here (the reciprocal by two steps); rounding it to multiples of 2^-16
// first (C = 192: 1.5 * 2^7) puts ties exactly on k + 1/2 and keeps the others
// on their side, so the product decides as the exact quotient would.
__device__ __forceinline__ uint32_t fields_bf16(const float (&x)[8], float inv) {
  constexpr float C = 192.f, M = 12582920.f;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // two at a time
    unsigned long long v;
    asm("{\n\t.reg .b64 x, i, c, n, m;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 i, {%3, %3};\n\t"
        "mov.b64 c, {%4, %4};\n\tmov.b64 n, {%5, %5};\n\tmov.b64 m, {%6, %6};\n\t"
        "fma.rn.f32x2 x, x, i, c;\n\tadd.rn.f32x2 x, x, n;\n\tadd.rn.f32x2 %0, x, m;\n\t}"
        : "=l"(v)
        : "f"(x[i]), "f"(x[i + 1]), "f"(inv), "f"(C), "f"(-C), "f"(M));
    const float2 two = reinterpret_cast<const float2&>(v);
    t[i] = two.x;
    t[i + 1] = two.y;
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) w = w * 16u + __float_as_uint(t[i]);
  // each term brought 0x4B400000 along: its sum over 16^i, modulo 2^32
  return w - 0x4B400000u * 0x11111111u;
}

// Any fp32 value: a first guess, then the exact remainder x - q s (one fused
// multiply-add; no rounding, as q s has at most 12 bits) decides.
__device__ __forceinline__ uint32_t fields_exact(const float (&x)[8], float s, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    float q = fminf(fmaxf(rintf(x[i] * inv), -8.f), 8.f);
    const float e = 2.f * fmaf(-q, s, x[i]);
    const bool odd = ((int)q & 1) != 0;
    if (e > s || (e == s && odd)) q += 1.f;
    else if (e < -s || (e == -s && odd)) q -= 1.f;
    q = fminf(fmaxf(q, -7.f), 7.f);
    w = w * 16u + (uint32_t)((int)q + 8);
  }
  return w;
}

// The first guesses alone, two at a time, where all of them are clear of a
// border: x * (1/s) is off by less than 2^-19, so a remainder of at most (1/2 -
// 2^-17) s says that the guess is right (one warp in 250 has another). s is not
// tiny here: |x / s| < 7.5. A chunk of 8 x 1021 tokens x 8 heads, d = 64: written
// in 12 us by fields_exact, 8 us this way.
__device__ __forceinline__ bool fields_clear(const float (&x)[8], float s, float inv, uint32_t& fields) {
  constexpr float M = 12582920.f;
  float t[8], worst = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    unsigned long long v, e;
    asm("{\n\t.reg .b64 x, i, s, n, m, q;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 i, {%4, %4};\n\t"
        "mov.b64 s, {%5, %5};\n\tmov.b64 m, {%6, %6};\n\tmov.b64 n, {%7, %7};\n\t"
        "fma.rn.f32x2 %0, x, i, m;\n\tsub.rn.f32x2 q, n, %0;\n\tfma.rn.f32x2 %1, q, s, x;\n\t}"
        : "=&l"(v), "=l"(e)
        : "f"(x[i]), "f"(x[i + 1]), "f"(inv), "f"(s), "f"(M), "f"(M));
    const float2 two = reinterpret_cast<const float2&>(v), rest = reinterpret_cast<const float2&>(e);
    t[i] = two.x;
    t[i + 1] = two.y;
    worst = fmaxf(worst, fmaxf(fabsf(rest.x), fabsf(rest.y)));
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) w = w * 16u + __float_as_uint(t[i]);
  fields = w - 0x4B400000u * 0x11111111u;
  return worst <= s * (0.5f - 0x1p-17f);
}

// 1/x to within a step or two of fp32, for normal x and 1/x.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scale of the 32 channels that this lane shares with three others, and its
// eight fields.
template <typename T>
__device__ __forceinline__ uint32_t quantise(const Raw8<T>& raw, uint16_t& scale_bits) {
  uint32_t top = raw.top();
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (top >= 0x7f800000u) {
    scale_bits = 0x7fc0;
    return 0x88888888u;
  }
  const uint32_t sb = __float_as_uint(__fmul_rn(__uint_as_float(top), 1.f / 7.f)) & 0xffff0000u;
  scale_bits = (uint16_t)(sb >> 16);
  if (sb == 0u) return 0x88888888u;
  float s = __uint_as_float(sb);
  float x[8];
  raw.widen(x);
  if (s >= 0x1p-100f) {
    const float inv = reciprocal(s);
    if (sizeof(T) == 2) return fields_bf16(x, inv);
    uint32_t fields;
    return fields_clear(x, s, inv, fields) ? fields : fields_exact(x, s, inv);
  }
  // tiny scales: 1/s may be out of range, a subnormal s may be short of bits
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
  s *= 0x1p64f;
  return fields_exact(x, s, reciprocal(s));
}

// What a warp works on: the rows of a sequence that fall into one of its
// blocks, keys or values. blockIdx.y is the sequence.
struct Rows {
  int b, h, lo, hi;    // rows [lo, hi) of the block
  int kind;            // 0: keys, 1: values
  long long pos, row;  // position of the block's row 0; i of row 0 (may be < 0)
};

__device__ __forceinline__ bool rows_of(const IoParams& p, Rows& r) {
  const unsigned item = blockIdx.x * kWarps + threadIdx.x / 32;
  if (item >= p.items) return false;
  r.b = blockIdx.y;
  r.kind = (int)(item & 1u);
  const unsigned blk = (item >> 1) / (unsigned)p.cache.Hk;
  r.h = (int)((item >> 1) - blk * (unsigned)p.cache.Hk);
  const long long start = p.starts ? p.starts[r.b] : 0;
  const long long count = p.counts ? min(max(p.counts[r.b], 0), p.n) : p.n;
  // arithmetic shift: rounds down for negative starts too
  r.pos = ((start >> 4) + blk) * kBlock;
  r.row = r.pos - start;
  r.lo = (int)max(0ll, -r.row);
  r.hi = (int)max(min((long long)kBlock, count - r.row), 0ll);
  return r.lo < r.hi;
}

// Where a row's eight channels (quarter t of group y) sit among the codes of
// the keys; of the values, whose second half is d/2 bytes further on.
template <int D>
__device__ __forceinline__ int key_at(int row, int t, int y) {
  return row * (D / 2) + t * (D / 8) + y * 4;
}
template <int D>
__device__ __forceinline__ int value_at(int row, int t, int y) {
  return (row >> 3) * 4 * D + (8 * t + ((row & 7) >> 1)) * (D / 8) + (row & 1) * (D / 16) + 2 * y;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
kv4_write(const __grid_constant__ IoParams p, const T* __restrict__ k, const T* __restrict__ v) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, ITER = kBlock / RPI, HALF = v_codes(D);
  __shared__ __align__(16) uint8_t image[kWarps][HALF];
  const int lane = threadIdx.x & 31;
  Rows r;
  if (!rows_of(p, r)) return;  // warp-uniform
  const int unit = lane % LPR, t = unit & 3, y = unit >> 2;
  const nys_strides_t& st = r.kind ? p.vs : p.ks;
  const T* src = (r.kind ? v : k) + r.b * st.batch + r.h * st.head + r.row * st.token + unit * 8;
  Raw8<T> x[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int row = i * RPI + lane / LPR;
    x[i].clear();
    if (row >= r.lo && row < r.hi) x[i].load(src + row * st.token);
  }
  uint8_t* dst = block_at(p.cache, r.b, r.h, r.pos, D);
  if (!dst) {
    if (lane == 0) report_index(p.status);
    return;
  }
  dst += r.kind * HALF;
  uint8_t* im = image[threadIdx.x >> 5];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int row = i * RPI + lane / LPR;
    uint16_t scale;
    const uint32_t w = quantise<T>(x[i], scale);
    if (r.kind == 0) {
      *reinterpret_cast<uint32_t*>(im + key_at<D>(row, t, y)) = w;
    } else {
      uint8_t* at = im + value_at<D>(row, t, y);
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(at + D / 2) = (uint16_t)(w >> 16);
    }
    if (t == 0) *reinterpret_cast<uint16_t*>(im + k_scales(D) + (y * kBlock + row) * 2) = scale;
  }
  __syncwarp();
  if (r.hi - r.lo == kBlock) {
    for (int e = lane; e < HALF / 16; e += 32)
      reinterpret_cast<uint4*>(dst)[e] = reinterpret_cast<const uint4*>(im)[e];
    return;
  }
  // some rows only: key codes are d/2 bytes in a row, value codes 2-byte
  // pieces, scales 2 bytes each
  const int rows = r.hi - r.lo;
  if (r.kind == 0) {
    for (int e = lane; e < rows * (D / 8); e += 32) {
      const int at = (r.lo + e / (D / 8)) * (D / 2) + (e % (D / 8)) * 4;
      *reinterpret_cast<uint32_t*>(dst + at) = *reinterpret_cast<const uint32_t*>(im + at);
    }
  } else {
    for (int e = lane; e < rows * (D / 4); e += 32) {
      const int row = r.lo + e / (D / 4), piece = e % (D / 4);  // four channels: 8 per group
      const int at = (row >> 3) * 4 * D + ((piece & 7) * 4 + ((row & 7) >> 1)) * (D / 8) +
                     (row & 1) * (D / 16) + 2 * (piece >> 3);
      *reinterpret_cast<uint16_t*>(dst + at) = *reinterpret_cast<const uint16_t*>(im + at);
    }
  }
  for (int e = lane; e < rows * (D / 32); e += 32) {
    const int at = k_scales(D) + ((e % (D / 32)) * kBlock + r.lo + e / (D / 32)) * 2;
    *reinterpret_cast<uint16_t*>(dst + at) = *reinterpret_cast<const uint16_t*>(im + at);
  }
}

// code * scale of the eight fields of w to eight channels in memory.
__device__ __forceinline__ void decode8(uint32_t w, uint16_t scale_bits, float* p) {
  const float s = __uint_as_float((uint32_t)scale_bits << 16);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)  // 2^23 + field, less 2^23 + 8
    x[i] = (__uint_as_float(((w >> (4 * i)) & 15u) | 0x4B000000u) - 8388616.f) * s;
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// Two fields at a time: 128 + field as bf16 by putting the field into the
// mantissa of 128, less 136 (exact), times the scale (one rounding).
__device__ __forceinline__ void decode8(uint32_t w, uint16_t scale_bits, __nv_bfloat16* p) {
  const uint32_t ss = scale_bits * 0x10001u, off = 0x43084308u;  // 136
  uint32_t x[4];  // fields (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hsub2(reinterpret_cast<const __nv_bfloat162&>(f),
                                             reinterpret_cast<const __nv_bfloat162&>(off)),
                                     reinterpret_cast<const __nv_bfloat162&>(ss));
    x[i] = reinterpret_cast<const uint32_t&>(v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                                            __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
kv4_read(const __grid_constant__ IoParams p, T* __restrict__ k, T* __restrict__ v) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, ITER = kBlock / RPI, HALF = v_codes(D);
  __shared__ __align__(16) uint8_t image[kWarps][HALF];
  const int lane = threadIdx.x & 31;
  Rows r;
  if (!rows_of(p, r)) return;  // warp-uniform
  const uint8_t* src = block_at(p.cache, r.b, r.h, r.pos, D);
  if (!src && lane == 0) report_index(p.status);
  uint8_t* im = image[threadIdx.x >> 5];
#pragma unroll
  for (int e = lane; e < HALF / 16; e += 32)  // no block: scales of zero
    reinterpret_cast<uint4*>(im)[e] =
        src ? reinterpret_cast<const uint4*>(src + r.kind * HALF)[e] : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t none = src ? 0u : 0x88888888u;  // and codes of zero
  __syncwarp();
  const int unit = lane % LPR, t = unit & 3, y = unit >> 2;
  const nys_strides_t& st = r.kind ? p.vs : p.ks;
  T* dst = (r.kind ? v : k) + r.b * st.batch + r.h * st.head + r.row * st.token + unit * 8;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int row = i * RPI + lane / LPR;
    if (row < r.lo || row >= r.hi) continue;
    const uint16_t scale = *reinterpret_cast<const uint16_t*>(im + k_scales(D) + (y * kBlock + row) * 2);
    uint32_t w;
    if (r.kind == 0) {
      w = *reinterpret_cast<const uint32_t*>(im + key_at<D>(row, t, y));
    } else {
      const uint8_t* at = im + value_at<D>(row, t, y);
      w = *reinterpret_cast<const uint16_t*>(at) | (uint32_t)*reinterpret_cast<const uint16_t*>(at + D / 2) << 16;
    }
    decode8(w | none, scale, dst + row * st.token);
  }
}

int check_io(const nys_kv4_cache_t* c, const void* k, const void* v, const nys_strides_t* ks,
             const nys_strides_t* vs, const int* starts, const int* counts, int B, int n, int dtype,
             bool out) {
  if (!k || !v || !ks || !vs) return NYS_ERR_ARG;
  if (dtype != NYS_FP32 && dtype != NYS_BF16) return NYS_ERR_ARG;
  const int rc = check_cache(c);
  if (rc != NYS_OK) return rc;
  if (B < 1 || B > 65535 || n < 1) return NYS_ERR_SHAPE;
  if (!strides_ok(*ks) || !strides_ok(*vs)) return NYS_ERR_ARG;
  if (out && (!rows_apart(*ks, B, c->Hk, n, c->d) || !rows_apart(*vs, B, c->Hk, n, c->d)))
    return NYS_ERR_ARG;
  if (!rows_aligned(k, *ks, dtype) || !rows_aligned(v, *vs, dtype)) return NYS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(counts)) & 3u)
    return NYS_ERR_ALIGN;
  return NYS_OK;
}

int io_params(const nys_kv4_cache_t& c, const nys_strides_t& ks, const nys_strides_t& vs,
              const int* starts, const int* counts, int B, int n, int dev, IoParams* p) {
  p->cache = view_of(c);
  p->ks = ks;
  p->vs = vs;
  p->starts = starts;
  p->counts = counts;
  p->n = n;
  // n tokens from any start touch at most this many blocks
  const long long items = (((long long)n + 14) / 16 + 1) * c.Hk * 2;
  if (items >= (1ll << 31)) return NYS_ERR_SHAPE;
  p->items = (unsigned)items;
  return operator_status(dev, &p->status);
}

template <typename F>
int by_type(int dtype, int d, F&& f) {
  auto by_d = [&](auto type) -> int {
    switch (d) {
      case 32: return f(type, std::integral_constant<int, 32>{});
      case 64: return f(type, std::integral_constant<int, 64>{});
      default: return f(type, std::integral_constant<int, 128>{});
    }
  };
  return dtype == NYS_BF16 ? by_d(__nv_bfloat16{}) : by_d(float{});
}

}  // namespace
}  // namespace kv4
}  // namespace nys

using namespace nys;
using namespace nys::kv4;

extern "C" {

size_t nystrom_kv4_cache_bytes(int num_pages, int page_size, int Hk, int d) {
  alignas(16) static const int some[4] = {};
  const nys_kv4_cache_t c{const_cast<int*>(some), some, num_pages, 1, page_size, Hk, d};
  if (check_cache(&c) != NYS_OK) return 0;
  return (size_t)num_pages * Hk * (page_size / kBlock) * block_bytes(d);
}

int nystrom_kv4_write(const nys_kv4_cache_t* cache, const void* k, const void* v,
                      const nys_strides_t* k_strides, const nys_strides_t* v_strides,
                      const int* starts, const int* counts, int B, int n, int dtype,
                      nys_stream_t stream) {
  int rc = check_io(cache, k, v, k_strides, v_strides, starts, counts, B, n, dtype, false);
  if (rc != NYS_OK) return rc;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  IoParams p{};
  rc = io_params(*cache, *k_strides, *v_strides, starts, counts, B, n, dev, &p);
  if (rc != NYS_OK) return rc;
  return by_type(dtype, cache->d, [&](auto type, auto d) {
    using T = decltype(type);
    KernelScope scope("kv4_write", stream);
    nys::kv4::kv4_write<T, decltype(d)::value>
        <<<dim3((p.items + kWarps - 1) / kWarps, B), kWarps * 32, 0, stream>>>(
            p, static_cast<const T*>(k), static_cast<const T*>(v));
    return launch_status();
  });
}

int nystrom_kv4_read(const nys_kv4_cache_t* cache, void* k, void* v, const nys_strides_t* k_strides,
                     const nys_strides_t* v_strides, const int* starts, const int* counts, int B,
                     int n, int dtype, nys_stream_t stream) {
  int rc = check_io(cache, k, v, k_strides, v_strides, starts, counts, B, n, dtype, true);
  if (rc != NYS_OK) return rc;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (k == v) return NYS_ERR_ARG;
  IoParams p{};
  rc = io_params(*cache, *k_strides, *v_strides, starts, counts, B, n, dev, &p);
  if (rc != NYS_OK) return rc;
  return by_type(dtype, cache->d, [&](auto type, auto d) {
    using T = decltype(type);
    KernelScope scope("kv4_read", stream);
    nys::kv4::kv4_read<T, decltype(d)::value>
        <<<dim3((p.items + kWarps - 1) / kWarps, B), kWarps * 32, 0, stream>>>(
            p, static_cast<T*>(k), static_cast<T*>(v));
    return launch_status();
  });
}

}  // extern "C"
