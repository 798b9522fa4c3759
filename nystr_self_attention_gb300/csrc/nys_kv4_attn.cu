// Attention over the 4-bit key/value cache (declared in include/nystrom.h):
//   out = softmax(q K^T scale) V,  K = s_k c_k, V = s_v c_v per 32 channels.
//
// kv4_attn_split: up to 16 query rows (queries x heads of one cache head) per
// item. The keys of all items, in tiles of 32, form one line that is cut into
// equal ranges, one per CTA (four CTAs per SM): a long sequence is shared by
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
// carry the factors and are scaled to the top of fp16's range), its offset 8 is
// the product's starting value. V's fields are masked out as bf16 subnormals
// and brought to (u - 8) 2^-6 by one fused multiply-add per pair. fp32: fields
// less 8, as normal numbers, times two fp16 terms of the query, and three bf16
// terms of a probability. (The fields are e4m3 numbers as they lie, too, but the
// e4m3 form of the instruction took 11 instructions more a product: 62 us
// against 57 on the case below.)
//
// One token over 8 ragged sequences of up to 32768, 32 + 8 heads, d = 128 (203
// MB): 61 us a call, 52 of them here, 3.3 TB/s; four times as long 190 us (4.3
// TB/s). No unit is full (issue 51 %, HBM 48 %, integer pipe 42 %): 16 warps per
// SM, as many as the registers allow, wait for the results of about 310
// instructions per 16 keys and head, most of them unpacking; short calls: the
// launch, the queries and the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "nys_kv4_attn.h"

namespace nys {
namespace kv4 {
namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kStages = 2;   // tiles per warp in flight or in use
// Tiles of two blocks, 16 query rows, at least a tile per warp. With the item's
// start and join counted as 6 tiles the last CTA's end came 3 us nearer to the
// median one (8 ragged sequences of up to 32768 tokens, 8 heads).
using SplitLine = Line<32, 16, 6, 4>;
constexpr int kTile = SplitLine::TILE;
constexpr float kRebase = 8.0f;  // move the running maximum when it grows by 2^8
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

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

// CTAs per SM, by the registers a variant needs (fp32 with 16 rows, d = 64: three
// would fit but measured 27 us against 23, 5 drafted tokens over 4095 keys).
template <typename T, int D, int NT>
constexpr int kCtas = sizeof(T) == 2 ? (NT == 1 ? 4 : D == 128 ? 2 : 3) : (D == 128 || NT == 2 ? 2 : 3);

template <int D>
constexpr int ring_bytes() { return kWarps * kStages * 2 * block_bytes(D); }
template <int D, int NT>
constexpr int merge_bytes() { return 2 * NT * 8 * D * 4; }
// per group: the queries' operands, and for bf16 the product's starting values
template <typename T, int NT>
constexpr int kTable = sizeof(T) == 4 ? 2 * NT : 3;
// fp32 scales of a warp's tile: [K, V][group][32 tokens]
template <int D>
constexpr int scales_bytes() { return 2 * D / 32 * kTile * 4; }
template <typename T, int D, int NT>
constexpr int split_smem() {
  return ring_bytes<D>() + merge_bytes<D, NT>() + D / 32 * kTable<T, NT> * 512 + kWarps * scales_bytes<D>();
}

// NT: 8-row groups of query rows (1 or 2). fp32: a query is the sum of two
// fp16 terms, the codes lose their offset before the product, a probability
// times its scale is the sum of three bf16 terms.
// The code is kept short (one copy of each step, masks as uniform branches):
// a decoding step finds none of it in the instruction caches.
// out may be q: an item's rows are read by its CTA before they are written, or,
// where CTAs share it, by all of them before the join writes.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtas<T, D, NT>)
kv4_attn_split(const __grid_constant__ AttnParams p, const T* q, T* out) {
  constexpr int G = D / 32, BB = block_bytes(D);
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int ENTRIES = kTable<T, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ Start start;
  __shared__ int warp_sums[kWarps];
  __shared__ float2 ml_s[kWarps][16];
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  float* merge = reinterpret_cast<float*>(smem + ring_bytes<D>());  // [2][NT * 8][D]
  // [G][kTable][lane]: operands of the segment's queries, shared by the warps
  uint4* table = reinterpret_cast<uint4*>(smem + ring_bytes<D>() + merge_bytes<D, NT>());

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  float* scales = reinterpret_cast<float*>(table + G * kTable<T, NT> * 32) + warp * (scales_bytes<D>() / 4);
  uint8_t* ring = smem + warp * kStages * 2 * BB;
  if (tid < kWarps * kStages) mbar_init(&bars[0][0] + tid, 2);
  if (tid == 0) abort_s = 0;
  fence_barrier_init();
  cudaTriggerProgrammaticLaunchCompletion();  // the join may be set up meanwhile
  int pos = 0, r1 = 0, base = 0, b = 0;
  if (p.whole) {
    __syncthreads();
  } else {
    find_start<SplitLine, kWarps * 32>(p, &start, warp_sums);  // two block syncs
    pos = (int)min((long long)blockIdx.x * start.per, (long long)start.total);
    r1 = min(start.total, pos + start.per);
    base = start.base;
    b = start.b;
  }
  uint32_t used = 0;  // tiles this warp has put through its ring

  Segment seg;
  int mine = 0;                  // this warp's tiles of seg: tile0 + warp + 4 i
  const uint8_t* src = nullptr;  // this lane's block of the window of 16 tiles
  uint32_t there = 0, there_before = 0;  // blocks that exist in this window, the last
  float O[2 * G][NT][4];
  float m[NT], l[NT], rf[NT];  // rf: score units -> log2 units

  auto issue = [&](const Segment& sg, int i) {
    if ((i & 15) == 0) {
      const int wi = i + (lane >> 1);
      const int key = (sg.tile0 + warp + kWarps * wi) * kTile + (lane & 1) * kBlock;
      src = nullptr;
      if (wi < mine && key < sg.seen_max) {
        src = block_at(p.cache, sg.b, sg.h, key, D);
        if (!src) report_index(p.status);
      }
      there_before = there;
      there = __ballot_sync(0xffffffffu, src != nullptr);
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

  for (bool any = false;; any = true) {
    // ------------------- the next segment, its first tiles on their way ...
    Segment next;
    bool more = !any;
    if (!p.whole) more = next_segment<SplitLine>(p, pos, r1, base, b, next);
    else if (more) whole_segment<SplitLine>(p, blockIdx.x, next);
    if (more) {
      // tiles with a key that some row sees
      const int live = min(next.tile0 + next.ntile, (next.seen_max + kTile - 1) / kTile) - next.tile0;
      mine = live > warp ? (live - warp + kWarps - 1) / kWarps : 0;
      if (__any_sync(0xffffffffu, *abort_flag)) mine = 0;
      {  // the queries towards L2 while the page table is read
        const int row = next.rt * 16 + (lane & 15), qi = row / p.rep;
        if ((lane & 15) < next.rows)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + next.b * p.qs.batch +
                                                       (next.h * p.rep + row - qi * p.rep) * p.qs.head +
                                                       qi * p.qs.token + (lane >> 4) * (D / 2)));
      }
#pragma unroll 1
      for (int i = 0; i < min(kStages, mine); ++i) issue(next, i);
    }

    // -------------------------- ... while the warps join the one just done
    if (any) {
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
          const float own = fast_exp2(ml_s[warp][r].x - ref) * 64.f;  // codes carry 2^-6
#pragma unroll
          for (int j = 0; j < 2 * G; ++j) {
            O[j][nt][e] *= own;
            O[j][nt][2 + e] *= own;
          }
          top[nt][e] = mx;
          sum[nt][e] = s;
        }
      // warps 2, 3 into 0, 1, then 1 into 0
#pragma unroll 1
      for (int half = 2; half > 0; half >>= 1) {
        float4* at = reinterpret_cast<float4*>(merge + ((warp & (half - 1)) * NT * 8 + 2 * t) * D + 4 * g);
        if (warp >= half && warp < 2 * half) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int y = 0; y < G; ++y)
                at[((nt * 8 + e) * D + 32 * y) / 4] = make_float4(O[2 * y][nt][e], O[2 * y][nt][2 + e],
                                                                  O[2 * y + 1][nt][e], O[2 * y + 1][nt][2 + e]);
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int y = 0; y < G; ++y) {
                const float4 o = at[((nt * 8 + e) * D + 32 * y) / 4];
                O[2 * y][nt][e] += o.x;
                O[2 * y][nt][2 + e] += o.y;
                O[2 * y + 1][nt][e] += o.z;
                O[2 * y + 1][nt][2 + e] += o.w;
              }
        }
        __syncthreads();
      }
      if (warp == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = nt * 8 + 2 * t + e, row = seg.rt * 16 + r;
            if (r >= seg.rows) continue;
            const bool whole = seg.whole(kTile);
            const float norm = !whole ? 1.f : sum[nt][e] == 0.f ? 0.f : 1.f / sum[nt][e];
            const int qi = row / p.rep, hq = seg.h * p.rep + row - qi * p.rep;
            T* dst = out + seg.b * p.os.batch + hq * p.os.head + qi * p.os.token + 4 * g;
            const size_t part = part_slot(seg);
            float* prt = p.part + (part * (NT * 8) + r) * D + 4 * g;
#pragma unroll
            for (int y = 0; y < G; ++y) {
              const float v[4] = {O[2 * y][nt][e] * norm, O[2 * y][nt][2 + e] * norm,
                                  O[2 * y + 1][nt][e] * norm, O[2 * y + 1][nt][2 + e] * norm};
              if (whole) store4(dst + 32 * y, v);
              else store4(prt + 32 * y, v);
            }
            if (!whole && g == 0) p.part_ml[part * (NT * 8) + r] = make_float2(top[nt][e], sum[nt][e]);
          }
      }
    }
    if (!more) break;
    seg = next;

    // -------------------------------- the queries: this lane's rows g, g + 8
    uint32_t qa[4][4];  // of group `warp`: the table's operands
    float first[4] = {0.f, 0.f, 0.f, 0.f};  // -8 x the group's sum of the row
#pragma unroll
    for (int i = 0; i < 16; ++i) qa[i / 4][i % 4] = 0u;
    int seen[NT];
#pragma unroll
    for (int hr = 0; hr < NT; ++hr) {
      const int r = hr * 8 + g, row = seg.rt * 16 + r;
      const bool live = r < seg.rows;
      const int qi = live ? row / p.rep : 0, hq = seg.h * p.rep + (live ? row - qi * p.rep : 0);
      seen[hr] = !live ? 0 : (p.causal ? max(0, seg.len - seg.count + 1 + qi) : seg.len);
      const T* at = q + seg.b * p.qs.batch + hq * p.qs.head + qi * p.qs.token + 8 * t;
      float x[8], top = 0.f;  // x: of the group this warp prepares
      bool finite = true;
#pragma unroll
      for (int y = 0; y < G; ++y) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (live) load8(at + 32 * y, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top = fmaxf(top, fabsf(v[j]));
          finite = finite && fabsf(v[j]) < INFINITY;
          x[j] = y == 0 || y == warp ? v[j] : x[j];
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      finite = (__ballot_sync(0xffffffffu, finite) >> (lane & 28) & 15u) == 15u;
      // scale the row so that its largest magnitude lies in [2^13, 2^14); its
      // scores come out in units of that and of the fields' 2^-24
      const bool tiny = top < 0x1p-60f;
      if (tiny) top *= 0x1p80f;
      const int e = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 : 13;
      const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23) * (p.scale_log2 < 0.f ? -1.f : 1.f);
      const float down = fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + max(e - 13, -100)) << 23);
      rf[hr] = !finite ? NAN : down * (EXACT ? 0x1p9f : 0x1p24f) * (tiny ? 0x1p-80f : 1.f);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // bf16: odd fields sit four bits higher
        const float v = finite ? (tiny ? x[j] * 0x1p80f : x[j]) * up : 0.f;
        x[j] = !EXACT && (j & 1) ? v * 0.0625f : v;
        sum += round_half(x[j]) * ((j & 1) ? 16.f : 1.f);
      }
      if (!EXACT) {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        first[2 * hr] = first[2 * hr + 1] = sum * (-8.f * 0x1p-24f);
      }
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const float lo = x[2 * st + ch], hi = x[2 * st + ch + 4];
          qa[st][hr + 2 * ch] = half2_bits(lo, hi);
          if (EXACT) {  // the second term: up to 8 rows leave the others free for it
            const uint32_t two = half2_bits(lo - round_half(lo), hi - round_half(hi));
            if (NT == 1) qa[st][1 + 2 * ch] = two;
            else qa[2 + st][hr + 2 * ch] = two;
          }
        }
    }
    if (warp < G) {
      uint4* to = table + warp * ENTRIES * 32 + lane;
#pragma unroll
      for (int k = 0; k < (EXACT ? 2 * NT : 2); ++k) to[k * 32] = make_uint4(qa[k][0], qa[k][1], qa[k][2], qa[k][3]);
      if (!EXACT)
        to[64] = make_uint4(__float_as_uint(first[0]), __float_as_uint(first[1]),
                                 __float_as_uint(first[2]), __float_as_uint(first[3]));
    }
    __syncthreads();

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[i][nt][e] = 0.f;
    }

    // ---------------------------------------------------- stream the tiles
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      const uint32_t at_tile = used + i, st = at_tile % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[warp][st], (at_tile / kStages) & 1u, abort_flag, kWaitNs))) {
        if (lane == 0) {
          abort_s = 1;
          atomicExch(p.status, (int)NYS_ERR_TIMEOUT);
#pragma unroll 1
          for (int j = i; j < min(mine, i + kStages); ++j)  // copies still in flight
            mbar_wait(&bars[warp][(used + j) % kStages], ((used + j) / kStages) & 1u, nullptr, kWaitNs);
        }
        __syncwarp();
        break;
      }
      const uint8_t* blk = ring + st * 2 * BB;
      const int key0 = (seg.tile0 + warp + kWarps * i) * kTile;
      // the window ahead of this tile's may have been opened already
      const uint32_t window = (min(i + kStages - 1, mine - 1) ^ i) & 16 ? there_before : there;
      const uint32_t have = window >> (2 * (i & 15)) & 3u;
      const bool masked = key0 + kTile > seg.seen_min || have != 3u;  // warp-uniform

      // The tile's scales to fp32, once for all lanes: a lane takes 8 tokens of
      // one group (a quarter-warp per kind and block for d = 128). Tokens that
      // no row sees get zeros, whatever their memory holds.
      bool odd = false;  // an infinity or a NaN among those that are seen
      __syncwarp();
      if (lane < 8 * G) {
        const int kind = lane / (4 * G), y = lane / 4 % G, part = lane & 3;  // part: 8 of 32 tokens
        const uint4 u = *reinterpret_cast<const uint4*>(blk + (part >> 1) * BB + (kind ? v_scales(D) : k_scales(D)) +
                                                        y * 32 + (part & 1) * 16);
        uint32_t x[8] = {u.x << 16, u.x & 0xffff0000u, u.y << 16, u.y & 0xffff0000u,
                         u.z << 16, u.z & 0xffff0000u, u.w << 16, u.w & 0xffff0000u};
        if (masked) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (key0 + part * 8 + j >= seg.seen_max || !(have >> (part >> 1) & 1u)) x[j] = 0u;
            odd = odd || (x[j] & 0x7f800000u) == 0x7f800000u;
          }
        }
        uint4* to = reinterpret_cast<uint4*>(scales + (kind * G + y) * kTile + part * 8);
        to[0] = make_uint4(x[0], x[1], x[2], x[3]);
        to[1] = make_uint4(x[4], x[5], x[6], x[7]);
      }
      odd = __any_sync(0xffffffffu, odd);
      __syncwarp();

      // scores: n-tile 2 blk + half holds keys 16 blk + 8 half + (2t, 2t + 1)
      float S[4][2 * NT];
      uint32_t w[4][G];
#pragma unroll
      for (int n8 = 0; n8 < 4; ++n8) {
        const uint8_t* row = blk + (n8 >> 1) * BB + ((n8 & 1) * 8 + g) * (D / 2) + t * (D / 8);
        if (G == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(row);
          w[n8][0] = u.x; w[n8][1 % G] = u.y; w[n8][2 % G] = u.z; w[n8][3 % G] = u.w;
        } else if (G == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(row);
          w[n8][0] = u.x; w[n8][1 % G] = u.y;
        } else {
          w[n8][0] = *reinterpret_cast<const uint32_t*>(row);
        }
#pragma unroll
        for (int e = 0; e < 2 * NT; ++e) S[n8][e] = 0.f;
      }
#pragma unroll
      for (int y = 0; y < G; ++y) {
        uint4 a[ENTRIES];
#pragma unroll
        for (int k = 0; k < ENTRIES; ++k) a[k] = table[(y * ENTRIES + k) * 32 + lane];
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8) {
          uint32_t f[4] = {w[n8][y] & 0x000f000fu, w[n8][y] & 0x00f000f0u, (w[n8][y] >> 8) & 0x000f000fu,
                           (w[n8][y] >> 8) & 0x00f000f0u};
          if (EXACT) {
            // To (u - 8) 2^-9, normal numbers: with subnormal operands the unit
            // keeps fewer bits of a sum. Relative error of 5 tokens over 4095
            // keys: 1.0e-6 that way, 1.5e-7 this way.
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t up = (j & 1) ? 0x68006800u : 0x78007800u, o = 0xa400a400u;  // 2^11, 2^15; -2^-6
              const __half2 v = __hfma2(reinterpret_cast<const __half2&>(f[j]), reinterpret_cast<const __half2&>(up),
                                        reinterpret_cast<const __half2&>(o));
              f[j] = reinterpret_cast<const uint32_t&>(v);
            }
          }
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          if (!EXACT) {
            const uint4 c = a[2];
            acc[0] = __uint_as_float(c.x); acc[1] = __uint_as_float(c.y);
            acc[2] = __uint_as_float(c.z); acc[3] = __uint_as_float(c.w);
          }
#pragma unroll
          for (int k = EXACT ? 2 * NT - 1 : 1; k >= 0; --k)  // the smaller terms first
            mma_f16(acc, a[k].x, a[k].y, a[k].z, a[k].w, f[2 * (k & 1)], f[2 * (k & 1) + 1], acc);
          if (EXACT && NT == 1) {
            acc[0] += acc[2];
            acc[1] += acc[3];
          }
          const float2 sc = *reinterpret_cast<const float2*>(scales + y * kTile + n8 * 8 + 2 * t);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            S[n8][2 * nt] = fmaf(sc.x, acc[2 * nt], S[n8][2 * nt]);
            S[n8][2 * nt + 1] = fmaf(sc.y, acc[2 * nt + 1], S[n8][2 * nt + 1]);
          }
        }
      }
      uint32_t hidden = 0;  // of this lane's scores
      if (masked) {
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e) {
            const int key = key0 + 8 * n8 + 2 * t + (e & 1);
            if (key >= seen[e >> 1] || !(have >> (n8 >> 1) & 1u)) {
              S[n8][e] = -INFINITY;
              hidden |= 1u << (n8 * 2 * NT + e);
            }
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
          for (int e = 2 * nt; e < 2 * nt + 2; ++e) S[n8][e] = fast_exp2(fmaf(S[n8][e], rf[nt], -off));
      }
      if (masked) {
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8)
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e)
            if (hidden >> (n8 * 2 * NT + e) & 1u) S[n8][e] = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8) l[nt] += S[n8][2 * nt] + S[n8][2 * nt + 1];
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
      // out^T += V^T (p s): channel rows, query columns. `careful`: rows that
      // do not see a token must not meet its infinite or NaN scale.
      auto add_values = [&](auto careful) {
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
                // u 2^-133 or, four bits up, u 2^-129; to (u - 8) 2^-6
                const uint32_t f = (j < 2 ? x : x >> 8) & ((j & 1) ? 0x00f000f0u : 0x000f000fu);
                const uint32_t up = (j & 1) ? 0x7d007d00u : 0x7f007f00u, o = 0xbe00be00u;  // 2^123, 2^127; -1/8
                const __nv_bfloat162 c = __hfma2(reinterpret_cast<const __nv_bfloat162&>(f),
                                                 reinterpret_cast<const __nv_bfloat162&>(up),
                                                 reinterpret_cast<const __nv_bfloat162&>(o));
                v[hf][j] = reinterpret_cast<const uint32_t&>(c);
              }
            }
            const float2 sc0 = *reinterpret_cast<const float2*>(scales + (G + y) * kTile + bk * 16 + 2 * t);
            const float2 sc1 = *reinterpret_cast<const float2*>(scales + (G + y) * kTile + bk * 16 + 8 + 2 * t);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float z[4] = {S[2 * bk][2 * nt] * sc0.x, S[2 * bk][2 * nt + 1] * sc0.y,
                            S[2 * bk + 1][2 * nt] * sc1.x, S[2 * bk + 1][2 * nt + 1] * sc1.y};
              if (decltype(careful)::value) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (hidden >> ((2 * bk + (e >> 1)) * 2 * NT + 2 * nt + (e & 1)) & 1u) z[e] = 0.f;
              }
              if constexpr (!EXACT) {
                const uint32_t b0 = pack_bf16x2(z[0], z[1]), b1 = pack_bf16x2(z[2], z[3]);
                mma_bf16_acc(O[2 * y][nt], v[0][0], v[0][1], v[1][0], v[1][1], b0, b1);
                mma_bf16_acc(O[2 * y + 1][nt], v[0][2], v[0][3], v[1][2], v[1][3], b0, b1);
              } else {
                // The matrix units cut their sums off towards zero, so a long
                // chain of them drifts (half a step of 2^-24 per product, all of
                // one sign): 16 keys, the smallest terms first, then an ordinary
                // sum.
                uint32_t b[3][2];
#pragma unroll
                for (int pt = 0; pt < 3; ++pt) {
                  b[pt][0] = pack_bf16x2(z[0], z[1]);
                  b[pt][1] = pack_bf16x2(z[2], z[3]);
                  z[0] -= low_bf16(b[pt][0]); z[1] -= high_bf16(b[pt][0]);
                  z[2] -= low_bf16(b[pt][1]); z[3] -= high_bf16(b[pt][1]);
                }
                float part[2][4] = {};
#pragma unroll
                for (int pt = 2; pt >= 0; --pt) {
                  mma_bf16_acc(part[0], v[0][0], v[0][1], v[1][0], v[1][1], b[pt][0], b[pt][1]);
                  mma_bf16_acc(part[1], v[0][2], v[0][3], v[1][2], v[1][3], b[pt][0], b[pt][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  O[2 * y][nt][e] += part[0][e];
                  O[2 * y + 1][nt][e] += part[1][e];
                }
              }
            }
          }
        }
      };
      if (odd) add_values(std::integral_constant<bool, true>{});
      else add_values(std::integral_constant<bool, false>{});
      __syncwarp();  // the stage has been read
      if (i + kStages < mine) issue(seg, i + kStages);
    }
    used += mine;
  }
}

// Warps of a joining CTA: one for every other row, or for four rows at once
// (16-row items, 5 fp32 tokens over 16 sequences of up to 4095: 4 warps 5 us, 8
// warps 3 us).
template <typename L>
constexpr int kJoinWarps = L::ROWS == 16 ? 8 : 4;

// Adds up the parts of items that several CTAs shared, and writes the zeros
// of sequences without keys. A CTA takes consecutive items, a warp a row. It
// is launched while the split kernel runs (which items were cut follows from
// the lengths alone) and waits for it before it reads a part. Its time is the
// chain of loads: 5 us behind 8 long sequences, 11 (40 MB of parts in L2) behind
// the chunk kernel's 128 items of 256 rows.
template <typename T, int D, typename L>
__global__ void __launch_bounds__(kJoinWarps<L> * 32)
kv4_attn_join(const __grid_constant__ AttnParams p, T* __restrict__ out, int part_rows,
              int items_per_cta, int n_items) {
  constexpr int SUB = L::ROWS / 16;  // a unit of work: 16 rows of an item
  // channels per lane; rows of a warp and their parts in flight: an item of few
  // rows has many parts, one of many rows a few
  constexpr int V = D / 32, AT_ONCE = SUB > 1 ? 4 : 1, AHEAD = SUB > 1 ? 2 : 8;
  __shared__ int warp_sums[2][kJoinWarps<L>];
  const int per_b = p.cache.Hk * p.row_tiles * SUB, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = blockIdx.x * items_per_cta, i1 = min(n_items, i0 + items_per_cta);
  int b = i0 / per_b;
  int before = 0, all = 0;
#pragma unroll 1
  for (int j = tid; j < p.B; j += kJoinWarps<L> * 32) {
    const int n = L::places(L::tiles(p, j));
    all += n;
    if (j < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    warp_sums[0][warp] = before;
    warp_sums[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps<L>; ++w) {
    before += warp_sums[0][w];
    all += warp_sums[1][w];
  }
  const int per = L::range(p, all * (per_b / SUB));
  int base = before * (per_b / SUB);  // first place of sequence b
  cudaGridDependencySynchronize();
  for (int i = i0; i < i1; ++i) {
    if (i >= (b + 1) * per_b) {
      base += L::places(L::tiles(p, b)) * (per_b / SUB);
      ++b;
    }
    const int tiles = L::tiles(p, b), item = (i - b * per_b) / SUB, sub = (i - b * per_b) % SUB;
    const int t0 = base + item * L::places(tiles) + L::COST;
    int c0 = 0, c1 = -1;
    if (tiles > 0) {
      c0 = t0 / per;
      c1 = (t0 + tiles - 1) / per;
      if (c0 == c1) continue;  // written whole
    }
    const int h = item / p.row_tiles, rt = item - h * p.row_tiles;
    const int rows = min(L::ROWS, count_of(p, b) * p.rep - rt * L::ROWS);
    const int end = min(rows, sub * 16 + 16);
#pragma unroll 1
    for (int r0 = sub * 16 + warp * AT_ONCE; r0 < end; r0 += kJoinWarps<L> * AT_ONCE) {
      float top[AT_ONCE], sum[AT_ONCE], acc[AT_ONCE][V];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        top[u] = -INFINITY;
        sum[u] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[u][j] = 0.f;
      }
#pragma unroll 1
      for (int c = c0; c <= c1; c += AHEAD) {
        float2 ml[AT_ONCE][AHEAD];
        float x[AT_ONCE][AHEAD][V];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            ml[u][k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int j = 0; j < V; ++j) x[u][k][j] = 0.f;
            if (c + k <= c1 && r0 + u < end) {
              const size_t at = ((size_t)(c + k) * 2 + (c + k == c0 ? 1 : 0)) * part_rows + r0 + u;
              ml[u][k] = p.part_ml[at];
              const float* src = p.part + at * D + lane * V;
              if (V == 4) {
                const float4 f = *reinterpret_cast<const float4*>(src);
                x[u][k][0] = f.x; x[u][k][1 % V] = f.y; x[u][k][2 % V] = f.z; x[u][k][3 % V] = f.w;
              } else {
#pragma unroll
                for (int j = 0; j < V; ++j) x[u][k][j] = src[j];
              }
            }
          }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          float now = top[u];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) now = fmaxf(now, ml[u][k].x);
          const float ref = now == -INFINITY ? 0.f : now, keep = fast_exp2(top[u] - ref);
          sum[u] *= keep;
#pragma unroll
          for (int j = 0; j < V; ++j) acc[u][j] *= keep;
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            const float w = fast_exp2(ml[u][k].x - ref);
            sum[u] = fmaf(w, ml[u][k].y, sum[u]);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[u][j] = fmaf(w, x[u][k][j], acc[u][j]);
          }
          top[u] = now;
        }
      }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        if (r0 + u >= end) continue;
        const int row = rt * L::ROWS + r0 + u, qi = row / p.rep, hq = h * p.rep + row - qi * p.rep;
        const float norm = sum[u] == 0.f ? 0.f : 1.f / sum[u];
        T* dst = out + b * p.os.batch + hq * p.os.head + qi * p.os.token + lane * V;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[u][j] *= norm;
        if constexpr (V == 4) {
          store4(dst, acc[u]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (sizeof(T) == 4) reinterpret_cast<float*>(dst)[j] = acc[u][j];
            else reinterpret_cast<__nv_bfloat16*>(dst)[j] = __float2bfloat16_rn(acc[u][j]);
          }
        }
      }
    }
  }
}

// --------------------------------------------------------------------- host

// bf16 calls with more query rows per cache head than this go to the tensor
// core kernel (d = 32 stays: its rows are half a swizzled operand row). 8 ragged
// sequences of up to 4096 / 32768 keys, 8 cache heads, d = 128, a call here
// against there (us): 32 rows 37 / 145 against 41 / 201, 48 rows 46 / 207 against
// 41 / 201, 64 rows 54 / 268 against 41 / 203, 128 rows 89 / 510 against 46 / 207.
constexpr int kChunkRows = 48;

// Contexts of up to kWholeTiles tiles (in a batch of kWholeItems items or more,
// of up to kWholeTilesBatch): a CTA per item and no join. Against ranges and a
// join, d = 128, 16 + 4 heads (us): 512 keys 13 / 19, 1024 keys 17 / 20, 2048
// keys 27 / 21; 64 sequences: 512 keys 15 / 29, 2048 keys 35 / 43.
constexpr int kWholeTiles = 32, kWholeTilesBatch = 64, kWholeItems = 64;

struct Plan {
  bool chunk, whole;
  int nt, row_tiles, ctas;
  long long items;
  size_t ml, total;  // workspace: offset behind the parts, bytes
};

Plan plan_of(const nys_kv4_cache_t& c, int B, int nq, int Hq, int max_length, int dtype) {
  Plan pl{};
  const long long rows = (long long)nq * (Hq / c.Hk);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  pl.chunk = dtype == NYS_BF16 && c.d >= 64 && rows > kChunkRows;
  if (pl.chunk) {
    pl.row_tiles = (int)((rows + ChunkLine::ROWS - 1) / ChunkLine::ROWS);
    pl.items = (long long)B * c.Hk * pl.row_tiles;
    pl.ctas = plan_sms();
    pl.ml = up((size_t)pl.ctas * 2 * ChunkLine::ROWS * c.d * sizeof(float));
    pl.total = up(pl.ml + (size_t)pl.ctas * 2 * ChunkLine::ROWS * sizeof(float2));
    return pl;
  }
  pl.nt = rows <= 8 ? 1 : 2;
  pl.row_tiles = (int)((rows + 15) / 16);
  pl.items = (long long)B * c.Hk * pl.row_tiles;
  const int ctas[2][2] = {{c.d == 128 ? kCtas<float, 128, 1> : kCtas<float, 64, 1>,
                           c.d == 128 ? kCtas<float, 128, 2> : kCtas<float, 64, 2>},
                          {c.d == 128 ? kCtas<__nv_bfloat16, 128, 1> : kCtas<__nv_bfloat16, 64, 1>,
                           c.d == 128 ? kCtas<__nv_bfloat16, 128, 2> : kCtas<__nv_bfloat16, 64, 2>}};
  pl.ctas = plan_sms() * ctas[dtype == NYS_BF16][pl.nt - 1];
  pl.whole = max_length <= (pl.items >= kWholeItems ? kWholeTilesBatch : kWholeTiles) * kTile;
  if (pl.whole) return pl;
  pl.ml = up((size_t)pl.ctas * 2 * pl.nt * 8 * c.d * sizeof(float));
  pl.total = up(pl.ml + (size_t)pl.ctas * 2 * pl.nt * 8 * sizeof(float2));
  return pl;
}

int check_attn(const nys_kv4_cache_t* c, int B, int nq, int Hq, int max_length, int dtype) {
  if (dtype != NYS_FP32 && dtype != NYS_BF16) return NYS_ERR_ARG;
  const int rc = check_cache(c);
  if (rc != NYS_OK) return rc;
  if (B < 1 || B > 65535 || nq < 1 || Hq < 1 || Hq > 65535 || Hq % c->Hk || max_length < 0)
    return NYS_ERR_SHAPE;
  if ((long long)nq * (Hq / c->Hk) >= (1ll << 30)) return NYS_ERR_SHAPE;
  // the line of tiles (and the items) of the longest sequences allowed
  const long long length = std::min((long long)max_length, (long long)c->max_pages * c->page_size);
  const Plan pl = plan_of(*c, B, nq, Hq, max_length, dtype);
  const long long places = pl.chunk ? ChunkLine::places((int)((length + ChunkLine::TILE - 1) / ChunkLine::TILE))
                                    : SplitLine::places((int)((length + kTile - 1) / kTile));
  const long long units = pl.chunk ? pl.items * (ChunkLine::ROWS / 16) : pl.items;
  if (units >= (1ll << 31) || pl.items * places >= (1ll << 31) - 65536) return NYS_ERR_SHAPE;
  return NYS_OK;
}

// units: items, or for items of more than 16 rows their 16-row pieces
template <typename T, int D, typename L>
int launch_join(const AttnParams& p, void* out, int part_rows, cudaStream_t st) {
  const long long units = (long long)p.B * p.cache.Hk * p.row_tiles * (L::ROWS / 16);
  KernelScope scope("kv4_attn_join", st);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const long long most = 8ll * plan_sms();
  const int per = (int)((units + most - 1) / most);
  cfg.gridDim = dim3((unsigned)((units + per - 1) / per));
  cfg.blockDim = dim3(kJoinWarps<L> * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kv4_attn_join<T, D, L>, p, static_cast<T*>(out), part_rows, per, (int)units);
  return launch_status();
}

template <typename T, int D, int NT>
int launch_split(const AttnParams& p, const Plan& pl, const void* q, void* out, int dev,
                 cudaStream_t st) {
  constexpr int smem = split_smem<T, D, NT>();
  static bool ready[64] = {};  // per device; setting it twice does no harm
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kv4_attn_split<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return set_cuda_error(cudaGetLastError());
    ready[dev] = true;
  }
  {
    KernelScope scope("kv4_attn_split", st);
    kv4_attn_split<T, D, NT><<<(unsigned)(pl.whole ? pl.items : pl.ctas), kWarps * 32, smem, st>>>(p, static_cast<const T*>(q),
                                                                static_cast<T*>(out));
    const int rc = launch_status();
    if (rc != NYS_OK || pl.whole) return rc;
  }
  return launch_join<T, D, SplitLine>(p, out, NT * 8, st);
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
  return plan_of(*cache, B, nq, Hq, max_length, dtype).total;
}

int nystrom_kv4_attn_fwd(const nys_kv4_cache_t* cache, const void* q, void* out,
                         const nys_strides_t* q_strides, const nys_strides_t* out_strides,
                         const int* lengths, const int* q_counts, int B, int nq, int Hq,
                         int max_length, int causal, float scale, int dtype, void* workspace,
                         size_t ws_bytes, nys_stream_t stream) {
  if (!q || !out || !q_strides || !out_strides || !lengths) return NYS_ERR_ARG;
  if ((causal != 0 && causal != 1) || !std::isfinite(scale * kLog2e)) return NYS_ERR_ARG;
  int rc = check_attn(cache, B, nq, Hq, max_length, dtype);
  if (rc != NYS_OK) return rc;
  if (!strides_ok(*q_strides) || !strides_ok(*out_strides) ||
      !rows_apart(*out_strides, B, Hq, nq, cache->d))
    return NYS_ERR_ARG;
  if (!rows_aligned(q, *q_strides, dtype) || !rows_aligned(out, *out_strides, dtype)) return NYS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(q_counts)) & 3u)
    return NYS_ERR_ALIGN;
  if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return NYS_ERR_ALIGN;
  const Plan pl = plan_of(*cache, B, nq, Hq, max_length, dtype);
  if (workspace && ws_bytes < pl.total) return NYS_ERR_NOMEM;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (!apart_or_same_rows(out, *out_strides, q, *q_strides, B, Hq, nq)) return NYS_ERR_ARG;
  OperatorWorkspace own;
  if (!workspace && pl.total > 0) {
    rc = own.take(dev, pl.total, stream, &workspace);
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
  p.B = B;
  p.nq = nq;
  p.rep = Hq / cache->Hk;
  p.row_tiles = pl.row_tiles;
  p.max_length = max_length;
  p.causal = causal;
  p.ctas = pl.ctas;
  p.whole = pl.whole ? 1 : 0;
  p.scale_log2 = (scale == 0.f ? 1.f / std::sqrt((float)cache->d) : scale) * kLog2e;
  if (pl.chunk) {
    rc = launch_kv4_chunk(p, cache->d, q, out, stream);
    if (rc != NYS_OK) return rc;
    return cache->d == 64 ? launch_join<__nv_bfloat16, 64, ChunkLine>(p, out, ChunkLine::ROWS, stream)
                          : launch_join<__nv_bfloat16, 128, ChunkLine>(p, out, ChunkLine::ROWS, stream);
  }
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
