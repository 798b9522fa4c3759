// Attention over the 4-bit key/value cache (declared in include/nystrom.h):
//   out = softmax(q K^T scale) V,  K = s_k c_k, V = s_v c_v per 32 channels.
//
// kv4_attn_split: up to 16 query rows (queries x heads of one cache head) per
// item. The keys of all items, in tiles of 32, form one line that is cut into
// equal ranges, one per CTA (three CTAs per SM): a long sequence is shared by
// many CTAs, a ragged batch loads them evenly. Inside a CTA four warps take
// tiles in turn, each with its own running maximum, sum and output, and join
// at the item's end; where ranges cut an item, kv4_attn_join adds up the parts.
// Each warp streams its tiles through a ring of its own: a block of 16 tokens
// (codes and scales of K and V, 18 d bytes) is one bulk copy.
//
// The products run on the matrix units with the codes as they are, and the
// scales are applied outside:
//   S    = sum over groups y of s_k[y] (q_y . c_k),  A = queries, B = keys
//   out^T += c_v[y]^T (p s_v[y]),                    A = values^T, B = p^T
// so that the scores come out in the very registers that the second product
// takes p from. A 4-bit field u = code + 8 becomes fp16 by masking alone (as a
// subnormal it is u 2^-24, in the upper half of a byte u 2^-20; the queries
// carry the factors and are scaled to the top of fp16's range), its offset 8
// goes into the product's starting value. For V it becomes bf16 128 + u by one
// more shift, less 136. The bound is HBM; what comes next is unpacking, about
// 0.7 integer instructions per code of K and one per code of V.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "nys_kv4.h"
#include "nys_sm100.h"

namespace nys {
namespace kv4 {
namespace {

using namespace sm100;

constexpr int kTile = 32;    // keys per tile: two blocks
constexpr int kWarps = 4;
constexpr int kCtasPerSm = 3;
constexpr int kStages = 2;   // tiles per warp in flight or in use
constexpr int kMinTiles = 4; // a CTA's range: at least one tile per warp
constexpr float kRebase = 8.0f;  // move the running maximum when it grows by 2^8
constexpr uint64_t kWaitNs = 2000000000ull;

struct AttnParams {
  View cache;
  nys_strides_t qs, os;
  const int *lengths, *q_counts;
  int* status;
  float* part;      // [CTAs][2][rows][D]: unnormalised outputs of cut items
  float2* part_ml;  // [CTAs][2][16]: their (maximum in log2 units, sum)
  int2* item_ctas;  // [items]: first CTA (-1 - CTA: its part is in slot 1), last
  int B, nq, rep, row_tiles, max_length, causal;
  int ctas;
  float scale_log2;  // scale * log2(e)
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_bf16_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float round_half(float x) { return __half2float(__float2half_rn(x)); }

// Eight channels of a query row as fp32.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = low_bf16(w[i]);
    v[2 * i + 1] = high_bf16(w[i]);
  }
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// Tokens of sequence b that its queries may see, and its real queries.
__device__ __forceinline__ int length_of(const AttnParams& p, int b, bool* bad) {
  const int given = p.lengths[b];
  const int limit = (int)min((long long)p.max_length, (long long)p.cache.max_pages * p.cache.page);
  const int len = min(max(given, 0), limit);
  *bad = len != given;
  return len;
}
__device__ __forceinline__ int count_of(const AttnParams& p, int b) {
  return p.q_counts ? min(max(p.q_counts[b], 0), p.nq) : p.nq;
}
__device__ __forceinline__ int tiles_of(const AttnParams& p, int b) {
  bool bad;
  return (length_of(p, b, &bad) + kTile - 1) / kTile;
}

// Where the CTA's range of the line of tiles starts.
struct Start {
  long long total, per;
  long long base;  // first tile of sequence b
  int b;
};

// Block-wide: sums the sequences' tiles in thread chunks, and finds the
// sequence that tile blockIdx.x * per falls into.
__device__ __forceinline__ void find_start(const AttnParams& p, Start* s, long long* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (p.B + kWarps * 32 - 1) / (kWarps * 32);
  const int b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
  const long long per_item = (long long)p.cache.Hk * p.row_tiles;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    bool bad;
    sum += (length_of(p, b, &bad) + kTile - 1) / kTile * per_item;
    if (bad && blockIdx.x == 0) report_index(p.status);
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  long long per = (total + p.ctas - 1) / p.ctas;
  if (per < kMinTiles) per = kMinTiles;
  const long long r0 = blockIdx.x * per;
  long long at = before + incl - sum;
  if (r0 >= at && r0 < at + sum) {  // one thread, if any
    int b = b0;
    for (; b < b1; ++b) {
      const long long n = tiles_of(p, b) * per_item;
      if (r0 < at + n) break;
      at += n;
    }
    s->base = at;
    s->b = b;
  }
  if (tid == 0) {
    s->total = total;
    s->per = per;
  }
  __syncthreads();
}

template <int D>
constexpr int ring_bytes() { return kWarps * kStages * 2 * block_bytes(D); }
template <int D, int NT>
constexpr int split_smem() { return ring_bytes<D>() + 2 * NT * 8 * D * 4; }

// NT: 8-row groups of query rows (1 or 2). TERMS: fp16 terms of a query, and
// EXACT codes with three bf16 terms of a probability, for fp32.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 && NT == 1 ? kCtasPerSm : 2)
kv4_attn_split(const __grid_constant__ AttnParams p, const T* __restrict__ q, T* __restrict__ out) {
  constexpr int G = D / 32, BB = block_bytes(D);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int QT = EXACT ? 2 : 1, PT = EXACT ? 3 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ Start start;
  __shared__ long long warp_sums[kWarps];
  __shared__ float2 ml_s[kWarps][16];
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  float* merge = reinterpret_cast<float*>(smem + ring_bytes<D>());  // [2][NT * 8][D]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * 2 * BB;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(&bars[w][s], 2);
    abort_s = 0;
    fence_barrier_init();
  }
  cudaTriggerProgrammaticLaunchCompletion();  // the join may be set up meanwhile
  find_start(p, &start, warp_sums);  // two block syncs
  const long long r0 = blockIdx.x * start.per, r1 = min(start.total, r0 + start.per);
  long long pos = r0, base = start.base;
  int b = start.b;
  uint32_t used = 0;  // tiles this warp has put through its ring

  while (pos < r1) {
    // ------------------------------------------------- the next segment
    bool bad;
    const int len = length_of(p, b, &bad);
    const int T_b = (len + kTile - 1) / kTile;
    const int items = p.cache.Hk * p.row_tiles;
    if (pos >= base + (long long)T_b * items) {
      base += (long long)T_b * items;
      ++b;
      continue;
    }
    const long long off = pos - base;
    const int item = (int)(off / T_b), tile0 = (int)(off - (long long)item * T_b);
    const int ntile = (int)min((long long)(T_b - tile0), r1 - pos);
    const bool whole = ntile == T_b;
    const int h = item / p.row_tiles, rt = item - h * p.row_tiles;
    const long long gitem = (long long)b * items + item;
    // only a range's first and last segment can be cut: two slots per CTA
    const int slot = pos == r0 ? 0 : 1;
    if (tile0 == 0 && tid == 0)
      p.item_ctas[gitem] = make_int2(slot ? -1 - (int)blockIdx.x : (int)blockIdx.x,
                                     (int)((pos + T_b - 1) / start.per));
    pos += ntile;

    // ------------------------------------- this lane's rows g and g + 8
    const int count = count_of(p, b);
    const int rows = min(16, count * p.rep - rt * 16);  // may be <= 0
    uint32_t qa[QT][G][2][2 * NT];  // [step][row half + NT * channel half]
    float first[G][4];              // starting value of a group's product
    float rf[NT];                   // score units -> log2 units
    int seen[NT];
    int seen_min = 0x7fffffff, seen_max = 0;
#pragma unroll
    for (int hr = 0; hr < NT; ++hr) {
      const int r = hr * 8 + g, row = rt * 16 + r;
      const bool live = r < rows;
      const int qi = live ? row / p.rep : 0, hq = h * p.rep + (live ? row - qi * p.rep : 0);
      seen[hr] = !live ? 0 : (p.causal ? max(0, len - count + 1 + qi) : len);
      if (live) seen_min = min(seen_min, seen[hr]);
      seen_max = max(seen_max, seen[hr]);
      const T* src = q + b * p.qs.batch + hq * p.qs.head + qi * p.qs.token + 8 * t;
      float x[G][8], top = 0.f;
      bool finite = true;
#pragma unroll
      for (int y = 0; y < G; ++y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[y][j] = 0.f;
        if (live) load8(src + 32 * y, x[y]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top = fmaxf(top, fabsf(x[y][j]));
          finite = finite && fabsf(x[y][j]) < INFINITY;
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      finite = (__ballot_sync(0xffffffffu, finite) >> (lane & 28) & 15u) == 15u;
      // scale the row so that its largest magnitude lies in [2^13, 2^14)
      const bool tiny = top < 0x1p-60f;
      if (tiny) top *= 0x1p80f;
      const int e = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 : 13;
      const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23) * (p.scale_log2 < 0.f ? -1.f : 1.f);
      rf[hr] = !finite ? NAN : scalbnf(fabsf(p.scale_log2), e - 13 + 24 - (tiny ? 80 : 0));
#pragma unroll
      for (int y = 0; y < G; ++y) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // odd fields sit four bits higher
          float v = finite ? (tiny ? x[y][j] * 0x1p80f : x[y][j]) * up : 0.f;
          x[y][j] = (j & 1) ? v * 0.0625f : v;
          sum += round_half(x[y][j]) * ((j & 1) ? 16.f : 1.f);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        first[y][2 * hr] = first[y][2 * hr + 1] = EXACT ? 0.f : sum * (-8.f * 0x1p-24f);
        if (NT == 1) first[y][2] = first[y][3] = 0.f;
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const float lo = x[y][2 * st + ch], hi = x[y][2 * st + ch + 4];
            qa[0][y][st][hr + NT * ch] = half2_bits(lo, hi);
            if (EXACT) qa[QT - 1][y][st][hr + NT * ch] = half2_bits(lo - round_half(lo), hi - round_half(hi));
          }
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      seen_min = min(seen_min, __shfl_xor_sync(0xffffffffu, seen_min, o));
      seen_max = max(seen_max, __shfl_xor_sync(0xffffffffu, seen_max, o));
    }
    if (rows <= 0) seen_max = 0;

    float O[2 * G][NT][4];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[i][nt][e] = 0.f;
    }

    // -------------------------------------------------- stream the tiles
    // tiles with a key that some row sees; this warp's are tile0 + warp + 4 i
    const int live_tiles = min(tile0 + ntile, (seen_max + kTile - 1) / kTile) - tile0;
    int mine = live_tiles > warp ? (live_tiles - warp + kWarps - 1) / kWarps : 0;
    if (__any_sync(0xffffffffu, *abort_flag)) mine = 0;
    const uint8_t* src = nullptr;  // this lane's block of the window
    uint32_t there[2] = {0u, 0u};  // blocks that exist, of even and odd windows
    auto issue = [&](int i) {
      if ((i & 15) == 0) {  // window of 16 tiles: a block per lane
        const int wi = i + (lane >> 1);
        const int key = (tile0 + warp + kWarps * wi) * kTile + (lane & 1) * kBlock;
        src = nullptr;
        if (wi < mine && key < seen_max) {
          src = block_at(p.cache, b, h, key, D);
          if (!src) report_index(p.status);
        }
        there[(i >> 4) & 1] = __ballot_sync(0xffffffffu, src != nullptr);
      }
      const uint32_t st = (used + i) % kStages;
      if ((lane >> 1) == (i & 15)) {
        if (src) {
          mbar_arrive_expect_tx(&bars[warp][st], BB);
          bulk_load(ring + (st * 2 + (lane & 1)) * BB, src, BB, &bars[warp][st]);
        } else {
          mbar_arrive(&bars[warp][st]);
        }
      }
    };

    auto tile_step = [&](int i, auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      const uint32_t st = (used + i) % kStages;
      const uint8_t* blk = ring + st * 2 * BB;
      const int key0 = (tile0 + warp + kWarps * i) * kTile;
      // scores: n-tile 2 blk + half holds keys 16 blk + 8 half + (2t, 2t + 1)
      float S[4][2 * NT];
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) {
        const uint8_t* kb = blk + (n8 >> 1) * BB;
        const uint8_t* row = kb + ((n8 & 1) * 8 + g) * (D / 2) + t * (D / 8);
        uint32_t w[G];
        if (G == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(row);
          w[0] = u.x; w[1 % G] = u.y; w[2 % G] = u.z; w[3 % G] = u.w;
        } else if (G == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(row);
          w[0] = u.x; w[1 % G] = u.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(row);
        }
#pragma unroll
        for (int e = 0; e < 2 * NT; ++e) S[n8][e] = 0.f;
#pragma unroll
        for (int y = 0; y < G; ++y) {
          uint32_t f[4] = {w[y] & 0x000f000fu, w[y] & 0x00f000f0u, (w[y] >> 8) & 0x000f000fu,
                           (w[y] >> 8) & 0x00f000f0u};
          if (EXACT) {  // fields less 8, exact in subnormals too
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t eight = (j & 1) ? 0x00800080u : 0x00080008u;
              const __half2 v = __hsub2(reinterpret_cast<const __half2&>(f[j]),
                                        reinterpret_cast<const __half2&>(eight));
              f[j] = reinterpret_cast<const uint32_t&>(v);
            }
          }
          float acc[4];
#pragma unroll
          for (int qt = QT - 1; qt >= 0; --qt)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint32_t(&a)[2 * NT] = qa[qt][y][s];
              if (qt == QT - 1 && s == 0)
                mma_f16(acc, a[0], NT == 2 ? a[NT - 1] : 0u, a[NT], NT == 2 ? a[2 * NT - 1] : 0u, f[0], f[1],
                        first[y]);
              else
                mma_f16(acc, a[0], NT == 2 ? a[NT - 1] : 0u, a[NT], NT == 2 ? a[2 * NT - 1] : 0u, f[2 * s],
                        f[2 * s + 1], acc);
            }
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(kb + k_scales(D) + y * 32 + (n8 & 1) * 16 + t * 4);
          const float s0 = low_bf16(sc), s1 = high_bf16(sc);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            S[n8][2 * nt] = fmaf(s0, acc[2 * nt], S[n8][2 * nt]);
            S[n8][2 * nt + 1] = fmaf(s1, acc[2 * nt + 1], S[n8][2 * nt + 1]);
          }
        }
      }
      if (MASK) {
        const uint32_t have = there[(i >> 4) & 1] >> (2 * (i & 15));
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e) {
            const int key = key0 + 8 * n8 + 2 * t + (e & 1);
            if (key >= seen[e >> 1] || !(have >> (n8 >> 1) & 1u)) S[n8][e] = -INFINITY;
          }
      }
      // running maximum and sum per row; the sum stays split over the lanes
      float alpha[NT];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = fmaxf(S[0][2 * nt], S[0][2 * nt + 1]);
#pragma unroll
        for (int n8 = 1; n8 < 4; ++n8) top = fmaxf(top, fmaxf(S[n8][2 * nt], S[n8][2 * nt + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        alpha[nt] = 1.f;
        if (top > m[nt] && (m[nt] == -INFINITY || (top - m[nt]) * rf[nt] > kRebase)) {
          alpha[nt] = m[nt] == -INFINITY ? 0.f : fast_exp2(m[nt] * rf[nt] - top * rf[nt]);
          m[nt] = top;
          l[nt] *= alpha[nt];
          moved = true;
        }
        const float off = m[nt] == -INFINITY ? 0.f : m[nt] * rf[nt];
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
          for (int e = 2 * nt; e < 2 * nt + 2; ++e) {
            S[n8][e] = MASK && S[n8][e] == -INFINITY ? 0.f : fast_exp2(fmaf(S[n8][e], rf[nt], -off));
            l[nt] += S[n8][e];
          }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float a0 = __shfl_sync(0xffffffffu, alpha[nt], 8 * t);
          const float a1 = __shfl_sync(0xffffffffu, alpha[nt], 8 * t + 4);
#pragma unroll
          for (int j = 0; j < 2 * G; ++j) {
            O[j][nt][0] *= a0; O[j][nt][1] *= a1;
            O[j][nt][2] *= a0; O[j][nt][3] *= a1;
          }
        }
      }
      // out^T += V^T (p s): channel rows, query columns
#pragma unroll
      for (int bk = 0; bk < 2; ++bk) {
        const uint8_t* vb = blk + bk * BB;
        uint32_t wa[2][(G + 1) / 2], wb[2][(G + 1) / 2];  // [token half]: tokens 2t, 2t + 1
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* at = vb + v_codes(D) + hf * 4 * D + lane * (D / 8);
          if (G == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(at);
            wa[hf][0] = u.x; wa[hf][1 % ((G + 1) / 2)] = u.y; wb[hf][0] = u.z; wb[hf][1 % ((G + 1) / 2)] = u.w;
          } else if (G == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(at);
            wa[hf][0] = u.x; wb[hf][0] = u.y;
          } else {
            wa[hf][0] = *reinterpret_cast<const uint32_t*>(at);  // both tokens' halves
            wb[hf][0] = 0u;
          }
        }
#pragma unroll
        for (int y = 0; y < G; ++y) {
          uint32_t v[2][4];  // [token half][field]: bf16 codes of tokens (2t, 2t + 1)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t x = G == 1 ? wa[hf][0]
                                      : __byte_perm(wa[hf][y >> 1], wb[hf][y >> 1], (y & 1) ? 0x7632 : 0x5410);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t f = ((x >> (4 * j)) & 0x000f000fu) | 0x43004300u, o = 0x43084308u;
              const __nv_bfloat162 c = __hsub2(reinterpret_cast<const __nv_bfloat162&>(f),
                                               reinterpret_cast<const __nv_bfloat162&>(o));
              v[hf][j] = reinterpret_cast<const uint32_t&>(c);
            }
          }
          const uint32_t sc0 = *reinterpret_cast<const uint32_t*>(vb + v_scales(D) + y * 32 + t * 4);
          const uint32_t sc1 = *reinterpret_cast<const uint32_t*>(vb + v_scales(D) + y * 32 + 16 + t * 4);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float pr = S[2 * bk + (e >> 1)][2 * nt + (e & 1)];
              const float s = (e & 1) ? high_bf16(e < 2 ? sc0 : sc1) : low_bf16(e < 2 ? sc0 : sc1);
              w[e] = MASK && pr == 0.f ? 0.f : pr * s;  // what is not seen may be NaN
            }
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              const uint32_t b0 = pack_bf16x2(w[0], w[1]), b1 = pack_bf16x2(w[2], w[3]);
              mma_bf16_acc(O[2 * y][nt], v[0][0], v[0][1], v[1][0], v[1][1], b0, b1);
              mma_bf16_acc(O[2 * y + 1][nt], v[0][2], v[0][3], v[1][2], v[1][3], b0, b1);
              if (PT > 1) {
                w[0] -= low_bf16(b0); w[1] -= high_bf16(b0);
                w[2] -= low_bf16(b1); w[3] -= high_bf16(b1);
              }
            }
          }
        }
      }
    };

    for (int i = 0; i < min(kStages, mine); ++i) issue(i);
    for (int i = 0; i < mine; ++i) {
      const uint32_t at = used + i;
      bool ok = mbar_wait(&bars[warp][at % kStages], (at / kStages) & 1u, abort_flag, kWaitNs);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) {
          abort_s = 1;
          atomicExch(p.status, (int)NYS_ERR_TIMEOUT);
          for (int j = i; j < min(mine, i + kStages); ++j)  // copies still in flight
            mbar_wait(&bars[warp][(used + j) % kStages], ((used + j) / kStages) & 1u, nullptr, kWaitNs);
        }
        __syncwarp();
        break;
      }
      const int end = (tile0 + warp + kWarps * i + 1) * kTile;
      const bool all = end <= seen_min && (there[(i >> 4) & 1] >> (2 * (i & 15)) & 3u) == 3u;
      if (all)
        tile_step(i, std::integral_constant<bool, false>{});
      else
        tile_step(i, std::integral_constant<bool, true>{});
      __syncwarp();  // the stage has been read
      if (i + kStages < mine) issue(i + kStages);
    }
    used += mine;

    // --------------------------------------------------- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 1);
      l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 2);
      if (t == 0) ml_s[warp][nt * 8 + g] = make_float2(m[nt] == -INFINITY ? -INFINITY : m[nt] * rf[nt], l[nt]);
    }
    __syncthreads();
    float top[NT][2], sum[NT][2];  // of rows 2t, 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml_s[w][r].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s = fmaf(ml_s[w][r].y, fast_exp2(ml_s[w][r].x - ref), s);
        const float own = fast_exp2(ml_s[warp][r].x - ref);
#pragma unroll
        for (int j = 0; j < 2 * G; ++j) {
          O[j][nt][e] *= own;
          O[j][nt][2 + e] *= own;
        }
        top[nt][e] = mx;
        sum[nt][e] = s;
      }
    auto exchange = [&](int buf, bool put) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int y = 0; y < G; ++y) {
            float4* at = reinterpret_cast<float4*>(merge + ((buf * NT * 8) + nt * 8 + 2 * t + e) * D + 32 * y + 4 * g);
            if (put) {
              *at = make_float4(O[2 * y][nt][e], O[2 * y][nt][2 + e], O[2 * y + 1][nt][e], O[2 * y + 1][nt][2 + e]);
            } else {
              const float4 o = *at;
              O[2 * y][nt][e] += o.x;
              O[2 * y][nt][2 + e] += o.y;
              O[2 * y + 1][nt][e] += o.z;
              O[2 * y + 1][nt][2 + e] += o.w;
            }
          }
    };
    if (warp >= 2) exchange(warp - 2, true);
    __syncthreads();
    if (warp < 2) exchange(warp, false);
    __syncthreads();
    if (warp == 1) exchange(0, true);
    __syncthreads();
    if (warp == 0) {
      exchange(0, false);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * t + e, row = rt * 16 + r;
          if (r >= rows) continue;
          const float norm = sum[nt][e] == 0.f ? 0.f : 1.f / sum[nt][e];
          const int qi = row / p.rep, hq = h * p.rep + row - qi * p.rep;
          T* dst = out + b * p.os.batch + hq * p.os.head + qi * p.os.token;
          float* prt = p.part + (((size_t)blockIdx.x * 2 + slot) * (NT * 8) + r) * D;
#pragma unroll
          for (int y = 0; y < G; ++y) {
            float v[4] = {O[2 * y][nt][e], O[2 * y][nt][2 + e], O[2 * y + 1][nt][e], O[2 * y + 1][nt][2 + e]};
            if (whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] *= norm;
              store4(dst + 32 * y + 4 * g, v);
            } else {
              store4(prt + 32 * y + 4 * g, v);
            }
          }
          if (!whole && g == 0)
            p.part_ml[((size_t)blockIdx.x * 2 + slot) * 16 + r] = make_float2(top[nt][e], sum[nt][e]);
        }
    }
    __syncthreads();  // ml_s and the exchange buffer are free again
  }
}

// Adds up the parts of items that several CTAs shared, and writes the zeros
// of sequences without keys. A CTA per item, a warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
kv4_attn_join(const __grid_constant__ AttnParams p, T* __restrict__ out, int part_rows) {
  constexpr int V = D / 32;  // channels per lane
  const int items = p.cache.Hk * p.row_tiles, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / items, item = blockIdx.x - b * items;
  const int h = item / p.row_tiles, rt = item - h * p.row_tiles;
  const int rows = min(16, count_of(p, b) * p.rep - rt * 16);
  const int tiles = tiles_of(p, b);
  cudaGridDependencySynchronize();  // launched while the split kernel ran
  int c0 = 0, c1 = -1, slot0 = 0;
  if (tiles > 0) {
    const int2 ctas = p.item_ctas[blockIdx.x];
    slot0 = ctas.x < 0 ? 1 : 0;
    c0 = slot0 ? -1 - ctas.x : ctas.x;
    c1 = ctas.y;
    if (c0 == c1) return;  // written whole
  }
  for (int r = warp; r < rows; r += kWarps) {
    const int row = rt * 16 + r, qi = row / p.rep, hq = h * p.rep + row - qi * p.rep;
    float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32)
      top = fmaxf(top, p.part_ml[((size_t)c * 2 + (c == c0 ? slot0 : 0)) * 16 + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const size_t at = (size_t)c * 2 + (c == c0 ? slot0 : 0);
      const float2 ml = p.part_ml[at * 16 + r];
      const float w = fast_exp2(ml.x - ref);
      sum = fmaf(w, ml.y, sum);
      const float* src = p.part + (at * part_rows + r) * D + lane * V;
      if (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(w, x.x, acc[0]); acc[1 % V] = fmaf(w, x.y, acc[1 % V]);
        acc[2 % V] = fmaf(w, x.z, acc[2 % V]); acc[3 % V] = fmaf(w, x.w, acc[3 % V]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(w, src[j], acc[j]);
      }
    }
    const float norm = sum == 0.f ? 0.f : 1.f / sum;
    T* dst = out + b * p.os.batch + hq * p.os.head + qi * p.os.token + lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (sizeof(T) == 4) reinterpret_cast<float*>(dst)[j] = acc[j] * norm;
      else reinterpret_cast<__nv_bfloat16*>(dst)[j] = __float2bfloat16_rn(acc[j] * norm);
    }
  }
}

// --------------------------------------------------------------------- host

struct Plan {
  int nt, row_tiles, ctas;
  long long items;
  size_t ml, item_ctas, total;  // workspace offsets after the parts, bytes
};

Plan plan_of(const nys_kv4_cache_t& c, int B, int nq, int Hq, int dtype) {
  Plan pl{};
  const long long rows = (long long)nq * (Hq / c.Hk);
  pl.nt = rows <= 8 ? 1 : 2;
  pl.row_tiles = (int)((rows + 15) / 16);
  pl.items = (long long)B * c.Hk * pl.row_tiles;
  pl.ctas = plan_sms() * (dtype == NYS_BF16 && pl.nt == 1 ? kCtasPerSm : 2);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  pl.ml = up((size_t)pl.ctas * 2 * pl.nt * 8 * c.d * sizeof(float));
  pl.item_ctas = up(pl.ml + (size_t)pl.ctas * 2 * 16 * sizeof(float2));
  pl.total = up(pl.item_ctas + (size_t)pl.items * sizeof(int2));
  return pl;
}

int check_attn(const nys_kv4_cache_t* c, int B, int nq, int Hq, int max_length, int dtype) {
  if (dtype != NYS_FP32 && dtype != NYS_BF16) return NYS_ERR_ARG;
  const int rc = check_cache(c);
  if (rc != NYS_OK) return rc;
  if (B < 1 || B > 65535 || nq < 1 || Hq < 1 || Hq > 65535 || Hq % c->Hk || max_length < 0)
    return NYS_ERR_SHAPE;
  if ((long long)nq * (Hq / c->Hk) >= (1ll << 30)) return NYS_ERR_SHAPE;
  if (plan_of(*c, B, nq, Hq, dtype).items >= (1ll << 31)) return NYS_ERR_SHAPE;
  return NYS_OK;
}

template <typename T, int D, int NT>
int launch_split(const AttnParams& p, const Plan& pl, const void* q, void* out, int dev,
                 cudaStream_t st) {
  constexpr int smem = split_smem<D, NT>();
  static bool ready[64] = {};  // per device; setting it twice does no harm
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kv4_attn_split<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return set_cuda_error(cudaGetLastError());
    ready[dev] = true;
  }
  {
    KernelScope scope("kv4_attn_split", st);
    kv4_attn_split<T, D, NT><<<pl.ctas, kWarps * 32, smem, st>>>(p, static_cast<const T*>(q),
                                                                static_cast<T*>(out));
    const int rc = launch_status();
    if (rc != NYS_OK) return rc;
  }
  KernelScope scope("kv4_attn_join", st);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)pl.items);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kv4_attn_join<T, D>, p, static_cast<T*>(out), NT * 8);
  return launch_status();
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
  return plan_of(*cache, B, nq, Hq, dtype).total;
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
  const Plan pl = plan_of(*cache, B, nq, Hq, dtype);
  if (workspace && ws_bytes < pl.total) return NYS_ERR_NOMEM;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (!workspace) {
    rc = operator_workspace(dev, pl.total, stream, &workspace);
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
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
  p.item_ctas = reinterpret_cast<int2*>(ws + pl.item_ctas);
  p.B = B;
  p.nq = nq;
  p.rep = Hq / cache->Hk;
  p.row_tiles = pl.row_tiles;
  p.max_length = max_length;
  p.causal = causal;
  p.ctas = pl.ctas;
  p.scale_log2 = (scale == 0.f ? 1.f / std::sqrt((float)cache->d) : scale) * 1.4426950408889634f;
  auto go = [&](auto type, auto d) {
    using T = decltype(type);
    constexpr int D = decltype(d)::value;
    return pl.nt == 1 ? launch_split<T, D, 1>(p, pl, q, out, dev, stream)
                      : launch_split<T, D, 2>(p, pl, q, out, dev, stream);
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
