// Attention over the 4-bit key/value cache (declared in include/nystrom.h):
//   out = softmax(q K^T scale) V,  K = s_k c_k, V = s_v c_v per 32 channels.
// One CTA per query row: a thread scores one key of a 128-key tile, then sums
// one channel of V over the tile; the running maximum and sum of the softmax
// rescale what came before.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "nys_kv4.h"

namespace nys {
namespace kv4 {
namespace {

constexpr int kTile = 128;

struct AttnParams {
  View cache;
  nys_strides_t qs, os;
  const int *lengths, *q_counts;
  int* status;
  int nq, Hq, rep, max_length, causal;
  float scale_log2;  // scale * log2(e)
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float scale_at(const uint8_t* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

template <typename T, int D>
__global__ void __launch_bounds__(kTile)
kv4_attn_rows(const __grid_constant__ AttnParams p, const T* __restrict__ q, T* __restrict__ out) {
  __shared__ float qs[D], ps[kTile], red[kTile / 32];
  const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, h = hq / p.rep, tid = threadIdx.x;
  const int count = p.q_counts ? min(max(p.q_counts[b], 0), p.nq) : p.nq;
  if (i >= count) return;
  const int given = p.lengths[b];
  const int limit = (int)min((long long)p.max_length, (long long)p.cache.max_pages * p.cache.page);
  const int len = min(max(given, 0), limit);
  if (len != given && tid == 0) report_index(p.status);
  const int seen = p.causal ? max(0, len - count + 1 + i) : len;
  if (tid < D) qs[tid] = as_float(q[b * p.qs.batch + hq * p.qs.head + i * p.qs.token + tid]) * p.scale_log2;
  __syncthreads();
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < seen; t0 += kTile) {
    const int t = t0 + tid, r = t & 15;
    const uint8_t* blk = t < seen ? block_at(p.cache, b, h, t - r, D) : nullptr;
    float s = -INFINITY;
    if (blk) {
      s = 0.f;
      for (int c = 0; c < D; ++c) {
        const int w = c & 31, y = c >> 5;
        const int code = (blk[r * (D / 2) + (w >> 3) * (D / 8) + 4 * y + ((w & 7) >> 1)] >> (4 * (c & 1))) & 15;
        s = fmaf(qs[c], (float)(code - 8) * scale_at(blk + k_scales(D) + (y * kBlock + r) * 2), s);
      }
    } else if (t < seen) {
      report_index(p.status);
    }
    float m = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    m = fmaxf(m, top);
    const float base = m == -INFINITY ? 0.f : m;
    const float keep = exp2f(top - base);
    ps[tid] = blk ? exp2f(s - base) : 0.f;
    top = m;
    __syncthreads();
    sum *= keep;
    acc *= keep;
    for (int j = 0; j < min(kTile, seen - t0); ++j) {
      const float pj = ps[j];
      sum += pj;
      if (pj == 0.f || tid >= D) continue;
      const int row = (t0 + j) & 15, w = tid & 31, y = tid >> 5;
      const uint8_t* vb = block_at(p.cache, b, h, t0 + j - row, D);
      const int code = (vb[v_codes(D) + (row >> 3) * 4 * D + ((w >> 2) * 4 + ((row & 7) >> 1)) * (D / 8) +
                           (row & 1) * (D / 16) + 2 * y + ((w & 3) >> 1)] >> (4 * (tid & 1))) & 15;
      acc = fmaf(pj, (float)(code - 8) * scale_at(vb + v_scales(D) + (y * kBlock + row) * 2), acc);
    }
    __syncthreads();
  }
  if (tid < D)
    put(out + b * p.os.batch + hq * p.os.head + i * p.os.token + tid, sum == 0.f ? 0.f : acc / sum);
}

int check_attn(const nys_kv4_cache_t* c, int B, int nq, int Hq, int max_length, int dtype) {
  if (dtype != NYS_FP32 && dtype != NYS_BF16) return NYS_ERR_ARG;
  const int rc = check_cache(c);
  if (rc != NYS_OK) return rc;
  if (B < 1 || B > 65535 || nq < 1 || Hq < 1 || Hq > 65535 || Hq % c->Hk || max_length < 0)
    return NYS_ERR_SHAPE;
  if ((long long)nq * (Hq / c->Hk) >= (1ll << 30)) return NYS_ERR_SHAPE;
  return NYS_OK;
}

}  // namespace
}  // namespace kv4
}  // namespace nys

using namespace nys;
using namespace nys::kv4;

extern "C" {

size_t nystrom_kv4_attn_workspace_bytes(const nys_kv4_cache_t* cache, int B, int nq, int Hq,
                                        int max_length, int dtype) {
  if (check_attn(cache, B, nq, Hq, max_length, dtype) != NYS_OK) return 0;
  return 0;
}

int nystrom_kv4_attn_fwd(const nys_kv4_cache_t* cache, const void* q, void* out,
                         const nys_strides_t* q_strides, const nys_strides_t* out_strides,
                         const int* lengths, const int* q_counts, int B, int nq, int Hq,
                         int max_length, int causal, float scale, int dtype, void* workspace,
                         size_t ws_bytes, nys_stream_t stream) {
  if (!q || !out || !q_strides || !out_strides || !lengths) return NYS_ERR_ARG;
  if ((causal != 0 && causal != 1) || !std::isfinite(scale)) return NYS_ERR_ARG;
  int rc = check_attn(cache, B, nq, Hq, max_length, dtype);
  if (rc != NYS_OK) return rc;
  if (!strides_ok(*q_strides) || !strides_ok(*out_strides) ||
      !rows_apart(*out_strides, B, Hq, nq, cache->d))
    return NYS_ERR_ARG;
  if (!rows_aligned(q, *q_strides, dtype) || !rows_aligned(out, *out_strides, dtype)) return NYS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(q_counts)) & 3u)
    return NYS_ERR_ALIGN;
  if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return NYS_ERR_ALIGN;
  const size_t need = nystrom_kv4_attn_workspace_bytes(cache, B, nq, Hq, max_length, dtype);
  if (workspace && ws_bytes < need) return NYS_ERR_NOMEM;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (need && !workspace) {
    rc = operator_workspace(dev, need, stream, &workspace);
    if (rc != NYS_OK) return rc;
  }
  AttnParams p{};
  rc = operator_status(dev, &p.status);
  if (rc != NYS_OK) return rc;
  p.cache = view_of(*cache);
  p.qs = *q_strides;
  p.os = *out_strides;
  p.lengths = lengths;
  p.q_counts = q_counts;
  p.nq = nq;
  p.Hq = Hq;
  p.rep = Hq / cache->Hk;
  p.max_length = max_length;
  p.causal = causal;
  p.scale_log2 = (scale == 0.f ? 1.f / std::sqrt((float)cache->d) : scale) * 1.4426950408889634f;
  auto go = [&](auto type, auto d) {
    using T = decltype(type);
    KernelScope scope("kv4_attn_rows", stream);
    kv4_attn_rows<T, decltype(d)::value><<<dim3(nq, Hq, B), kTile, 0, stream>>>(
        p, static_cast<const T*>(q), static_cast<T*>(out));
    return launch_status();
  };
  auto by_d = [&](auto type) {
    switch (cache->d) {
      case 32: return go(type, std::integral_constant<int, 32>{});
      case 64: return go(type, std::integral_constant<int, 64>{});
      default: return go(type, std::integral_constant<int, 128>{});
    }
  };
  return dtype == NYS_BF16 ? by_d(__nv_bfloat16{}) : by_d(float{});
}

}  // extern "C"
