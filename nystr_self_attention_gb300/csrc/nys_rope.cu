// Per-head RMS norm of queries and keys with the rotation of their positions
// in the same pass, and its gradients (declared in include/nystrom.h):
//   z = w x / sqrt(mean(x^2) + eps),  y = R(position) z
// Forward reads and writes each row once, backward reads x and g and writes
// dx once: HBM bounds both. A row (d channels, 16 bytes per lane and load in
// bf16) belongs to LP = 4, 8 or 16 consecutive lanes; a lane owns four rotated
// pairs, so the rotation needs no exchange and the norm is one shuffle
// reduction. A lane group keeps its token's angles in registers and walks the
// heads of the token, q's and then k's, several rows in flight: the sine and
// cosine are computed once per token, not once per row. Calls with few tokens
// split the heads over CTAs instead.
//
// Angles: a frequency is kept as the fraction of a turn it adds per position,
// in units of 2^-64. position * fraction modulo 2^64 is the exact remainder of
// the product, whatever the position, in one 64-bit integer multiplication;
// its top two bits pick the quadrant and what is left, at most an eighth of a
// turn, goes to the sine and cosine.
//
// Forward, 2 x 32768 tokens, 16 + 16 heads, d = 128, bf16 (1.07 GB): 165 us, 6.5
// TB/s where a copy reaches 6.8; fp32 pairs over three axes, 8 x 8190 tokens, 8 +
// 8 heads, d = 64 (537 MB): 88 us, 6.1 TB/s. Backward, 8 x 8192 tokens, 8 + 8
// heads, d = 64, bf16 (403 MB): 77 us with the weights' sums, 5.2 TB/s (fp32, 805
// MB: 122 us, 6.6 TB/s); with 128 registers a thread only 16 warps fit an SM, and between loads and stores they
// issue 2.4 instructions a cycle: latency and issue bound it together.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "nys_internal.h"

namespace nys {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;
constexpr int kMaxAxes = 4;

enum Mode : int {
  kHalves = 0,        // pair (i, i + rot/2), rot % 8 == 0: vector loads
  kPairs = 1,         // pair (2i, 2i + 1)
  kHalvesScalar = 2,  // pair (i, i + rot/2), any even rot
};

struct RopeParams {
  unsigned long long freq[kMaxPairs];  // turns per position, units of 2^-64
  const int* positions;                // [axes][B][n], or null: 0 .. n-1
  const float *qw, *kw;                // [d] or null
  int tokens;                          // B * n
  int n, Hq, Hk, d, half;              // half: rotated pairs
  int end[kMaxAxes];                   // first pair past each axis
  int heads_per_chunk;                 // heads of q and k a CTA walks
  int norm;
  float eps, inv_d;
  nys_strides_t qi, ki, qo, ko;  // x rows; y rows (backward: rows of g)
  nys_strides_t dq, dk;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store4(float* p, float2 u, float2 v) {
  *reinterpret_cast<float4*>(p) = make_float4(u.x, u.y, v.x, v.y);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float2 u, float2 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(u.x, u.y), pack2(v.x, v.y));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two fp32 values in one instruction.
__device__ __forceinline__ unsigned long long bits(const float2& v) {
  return reinterpret_cast<const unsigned long long&>(v);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The eight channels of one lane: a, b hold the members of its pairs 0, 1 and
// 2, 3.
struct Pairs {
  float2 a[2], b[2];
};

// Where a lane's channels sit in a row. Past the rotated channels a "pair" is
// two neighbours, turned by nothing.
struct Place {
  int lo, hi;  // first channel of a[0..3] and of b[0..3] (kPairs: of all eight)
  int unit, half;
};

template <int MODE>
__device__ __forceinline__ Place place_of(int unit, int half, int d) {
  if (8 * unit >= d) unit = 0;  // a lane without channels reads the first ones
  Place pl;
  pl.unit = unit;
  pl.half = half;
  const bool turned = MODE == kHalves && 4 * unit < half;
  pl.lo = turned ? 4 * unit : 8 * unit;
  pl.hi = turned ? 4 * unit + half : 8 * unit + 4;
  return pl;
}

// Channel of member a[j] (second: b[j]).
template <int MODE>
__device__ __forceinline__ int channel_of(const Place& pl, int j, bool second) {
  if (MODE == kHalves) return (second ? pl.hi : pl.lo) + j;
  const int i = 4 * pl.unit + j;
  if (MODE == kPairs || i >= pl.half) return 2 * i + (second ? 1 : 0);
  return i + (second ? pl.half : 0);
}

// A lane's channels of one row as they lie in memory: held while earlier rows
// are worked on, in half the registers (bf16) that their values take.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  uint4 lo, hi;
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 lo, hi;
};

template <int MODE>
__device__ __forceinline__ void load_raw(const float* row, const Place& pl, Raw<float>& r) {
  if (MODE != kHalvesScalar) {
    r.lo = *reinterpret_cast<const uint4*>(row + pl.lo);
    r.hi = *reinterpret_cast<const uint4*>(row + pl.hi);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
    r.lo = make_uint4(w[channel_of<MODE>(pl, 0, false)], w[channel_of<MODE>(pl, 1, false)],
                      w[channel_of<MODE>(pl, 2, false)], w[channel_of<MODE>(pl, 3, false)]);
    r.hi = make_uint4(w[channel_of<MODE>(pl, 0, true)], w[channel_of<MODE>(pl, 1, true)],
                      w[channel_of<MODE>(pl, 2, true)], w[channel_of<MODE>(pl, 3, true)]);
  }
}
template <int MODE>
__device__ __forceinline__ void load_raw(const __nv_bfloat16* row, const Place& pl,
                                         Raw<__nv_bfloat16>& r) {
  if (MODE == kPairs) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + pl.lo);
    r.lo = make_uint2(u.x, u.y);
    r.hi = make_uint2(u.z, u.w);
  } else if (MODE == kHalves) {
    r.lo = *reinterpret_cast<const uint2*>(row + pl.lo);
    r.hi = *reinterpret_cast<const uint2*>(row + pl.hi);
  } else {
    const uint16_t* w = reinterpret_cast<const uint16_t*>(row);
    auto two = [&](int j, bool second) {
      return (uint32_t)w[channel_of<MODE>(pl, j, second)] |
             (uint32_t)w[channel_of<MODE>(pl, j + 1, second)] << 16;
    };
    r.lo = make_uint2(two(0, false), two(2, false));
    r.hi = make_uint2(two(0, true), two(2, true));
  }
}

__device__ __forceinline__ void widen(const uint4& u, float2& v, float2& w) {
  v = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  w = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void widen(const uint2& u, float2& v, float2& w) {
  v = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  w = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <int MODE, typename T>
__device__ __forceinline__ Pairs pairs_of(const Raw<T>& r) {
  Pairs x;
  if (MODE == kPairs) {
    float2 u[4];
    widen(r.lo, u[0], u[1]);
    widen(r.hi, u[2], u[3]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x.a[j] = make_float2(u[2 * j].x, u[2 * j + 1].x);
      x.b[j] = make_float2(u[2 * j].y, u[2 * j + 1].y);
    }
  } else {
    widen(r.lo, x.a[0], x.a[1]);
    widen(r.hi, x.b[0], x.b[1]);
  }
  return x;
}

template <int MODE, typename T>
__device__ __forceinline__ void store_pairs(T* row, const Place& pl, const Pairs& x) {
  if (MODE == kHalves) {
    store4(row + pl.lo, x.a[0], x.a[1]);
    store4(row + pl.hi, x.b[0], x.b[1]);
  } else if (MODE == kPairs) {
    store4(row + pl.lo, make_float2(x.a[0].x, x.b[0].x), make_float2(x.a[0].y, x.b[0].y));
    store4(row + pl.hi, make_float2(x.a[1].x, x.b[1].x), make_float2(x.a[1].y, x.b[1].y));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      store1(row + channel_of<MODE>(pl, j, false), (j & 1) ? x.a[j / 2].y : x.a[j / 2].x);
      store1(row + channel_of<MODE>(pl, j, true), (j & 1) ? x.b[j / 2].y : x.b[j / 2].x);
    }
  }
}

// cos and sin of a 64-bit fraction of a turn. EXACT: to fp32 rounding; else
// with the special-function unit, off by less than 2^-20 on an eighth of a
// turn either way, far inside bf16's half step of 2^-9.
template <bool EXACT>
__device__ __forceinline__ void turn_cos_sin(unsigned long long phase, float& c, float& s) {
  const unsigned long long shifted = phase + (1ull << 61);
  const unsigned quadrant = (unsigned)(shifted >> 62);
  const long long rest = (long long)(phase - ((unsigned long long)quadrant << 62));
  const float half_turns = (float)(int)(rest >> 32) * 0x1p-31f;  // within +-1/4
  float cs, sn;
  if (EXACT) {
    sincospif(half_turns, &sn, &cs);
  } else {
    __sincosf(half_turns * 3.14159265358979f, &sn, &cs);
  }
  const float c1 = (quadrant & 1u) ? -sn : cs, s1 = (quadrant & 1u) ? cs : sn;
  c = (quadrant & 2u) ? -c1 : c1;
  s = (quadrant & 2u) ? -s1 : s1;
}

struct Turn {
  float2 c[2], s[2], ns[2];  // cos, sin, -sin
};

template <bool EXACT>
__device__ __forceinline__ Turn turn_of(const RopeParams& p, const unsigned long long* freq,
                                        int unit, int token, int t) {
  float c[4], s[4];
  int axis = -1;
  unsigned long long pos = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 4 * unit + j;
    c[j] = 1.f;
    s[j] = 0.f;
    if (i < p.half) {
      int ax = 0;
      while (i >= p.end[ax]) ++ax;  // sections sum to half, so ax stays below axes
      if (ax != axis) {
        axis = ax;
        pos = (unsigned long long)(long long)(p.positions ? p.positions[(size_t)ax * p.tokens + token] : t);
      }
      turn_cos_sin<EXACT>(freq[i] * pos, c[j], s[j]);
    }
  }
  return Turn{{make_float2(c[0], c[1]), make_float2(c[2], c[3])},
              {make_float2(s[0], s[1]), make_float2(s[2], s[3])},
              {make_float2(-s[0], -s[1]), make_float2(-s[2], -s[3])}};
}

// Sum over the LP lanes of a row, in every one of them.
template <int LP>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of x y over the lane's channels.
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  const float2 s = fma2(x.a[0], y.a[0], mul2(x.a[1], y.a[1])), t = fma2(x.b[0], y.b[0], mul2(x.b[1], y.b[1]));
  return (s.x + s.y) + (t.x + t.y);
}

template <int MODE>
__device__ __forceinline__ void load_weights(const float* w, const Place& pl, Pairs& x) {
  // 4-byte aligned: scalar loads, once per walk
  auto at = [&](int j, bool second) { return w ? w[channel_of<MODE>(pl, j, second)] : 1.f; };
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    x.a[j] = make_float2(at(2 * j, false), at(2 * j + 1, false));
    x.b[j] = make_float2(at(2 * j, true), at(2 * j + 1, true));
  }
}

// Heads [h0, h1) of one tensor for one token: UNROLL rows at a time, the next
// ones' loads in flight while these are worked on. Lanes without channels and
// groups without a token (`live` false) read some row's first channels and
// write none.
template <typename T, int LP, int MODE, int UNROLL>
__device__ __forceinline__ void walk_forward(const T* x, T* y, long long xs, long long ys, int h0,
                                             int h1, const float* w, const Turn& turn,
                                             const Place& pl, bool live, const RopeParams& p) {
  Raw<T> next[UNROLL];
  Pairs wt;
  if (p.norm) load_weights<MODE>(w, pl, wt);
  x += h0 * xs;
  y += h0 * ys;
  int left = h1 - h0;
  auto fetch = [&](int count) {
#pragma unroll
    for (int k = 0; k < UNROLL; ++k)
      if (k < count) load_raw<MODE>(x + k * xs, pl, next[k]);
    x += count * xs;
  };
  auto turn_rows = [&](const Raw<T>(&now)[UNROLL], int count) {
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (k >= count) break;
      Pairs v = pairs_of<MODE, T>(now[k]);
      if (p.norm) {
        const float ss = row_sum<LP>(live ? dot(v, v) : 0.f);
        const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v.a[j] = mul2(v.a[j], mul2(both(r), wt.a[j]));
          v.b[j] = mul2(v.b[j], mul2(both(r), wt.b[j]));
        }
      }
      Pairs o;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        o.a[j] = fma2(v.a[j], turn.c[j], mul2(v.b[j], turn.ns[j]));
        o.b[j] = fma2(v.b[j], turn.c[j], mul2(v.a[j], turn.s[j]));
      }
      if (live) store_pairs<MODE>(y + k * ys, pl, o);
    }
    y += count * ys;
  };
  if (left >= UNROLL) fetch(UNROLL);
#pragma unroll 1
  while (left >= UNROLL) {
    Raw<T> now[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) now[k] = next[k];
    left -= UNROLL;
    if (left >= UNROLL) fetch(UNROLL);
    turn_rows(now, UNROLL);
  }
#pragma unroll 1
  for (; left > 0; --left) {
    fetch(1);
    turn_rows(next, 1);
  }
}

// Rows in flight per lane: 64 bytes' worth.
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;

// Four CTAs per SM: 8 x 8190 tokens, 8 + 8 heads, d = 64, fp32 / bf16 86 / 47.5 us;
// with the registers of three 88 / 49.6, though a few are spilled around the loop.
template <typename T, int LP, int MODE>
__global__ void __launch_bounds__(kThreads, 4)
qk_norm_rope(const __grid_constant__ RopeParams p, const T* q, const T* k, T* qo, T* ko) {
  __shared__ unsigned long long freq[kMaxPairs];
  if (threadIdx.x < p.half) freq[threadIdx.x] = p.freq[threadIdx.x];
  __syncthreads();
  const int unit = threadIdx.x % LP;
  const unsigned token = blockIdx.x * (unsigned)(kThreads / LP) + threadIdx.x / LP;  // below 2^31 + 64
  const bool live = token < (unsigned)p.tokens && 8 * unit < p.d;
  const int bi = live ? (int)(token / (unsigned)p.n) : 0;
  const long long b = bi, t = live ? (int)token - bi * p.n : 0;
  const Place pl = place_of<MODE>(unit, p.half, p.d);
  Turn turn{};
  if (live) turn = turn_of<sizeof(T) == 4>(p, freq, unit, (int)token, (int)t);
  const int h0 = blockIdx.y * p.heads_per_chunk;
  const int h1 = min(p.Hq + p.Hk, h0 + p.heads_per_chunk);
  if (h0 < p.Hq)
    walk_forward<T, LP, MODE, kAhead<T>>(q + b * p.qi.batch + t * p.qi.token, qo + b * p.qo.batch + t * p.qo.token,
                                 p.qi.head, p.qo.head, h0, min(h1, p.Hq), p.qw, turn, pl, live, p);
  if (h1 > p.Hq)
    walk_forward<T, LP, MODE, kAhead<T>>(k + b * p.ki.batch + t * p.ki.token, ko + b * p.ko.batch + t * p.ko.token,
                                 p.ki.head, p.ko.head, max(h0 - p.Hq, 0), h1 - p.Hq, p.kw, turn, pl,
                                 live, p);
}

// Gradients of one tensor's heads in chunks: CTAs y < q_chunks take q's, the
// others k's, so that a thread keeps one set of weight sums. part: [CTAs][d]
// sums of g h over a CTA's rows (q's CTAs first), or null.
template <typename T, int LP, int MODE>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_rope_back(const __grid_constant__ RopeParams p, const T* q, const T* k, const T* gq,
                  const T* gk, T* dq, T* dk, float* part, int q_chunks) {
  __shared__ unsigned long long freq[kMaxPairs];
  __shared__ float sums[kThreads / 32][LP][9];
  if (threadIdx.x < p.half) freq[threadIdx.x] = p.freq[threadIdx.x];
  __syncthreads();
  cudaTriggerProgrammaticLaunchCompletion();
  constexpr int UNROLL = kAhead<T>;
  const bool keys = (int)blockIdx.y >= q_chunks;  // CTA-uniform
  const nys_strides_t &xs = keys ? p.ki : p.qi, &gs = keys ? p.ko : p.qo, &ds = keys ? p.dk : p.dq;
  const int unit = threadIdx.x % LP;
  const Place pl = place_of<MODE>(unit, p.half, p.d);
  const int h0 = ((int)blockIdx.y - (keys ? q_chunks : 0)) * p.heads_per_chunk;
  const int h1 = min(keys ? p.Hk : p.Hq, h0 + p.heads_per_chunk);
  constexpr int kRows = kThreads / LP;
  const int tiles = (int)(((long long)p.tokens + kRows - 1) / kRows);
  Pairs acc{}, wt;
  if (p.norm) load_weights<MODE>(keys ? p.kw : p.qw, pl, wt);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const unsigned token = tile * (unsigned)kRows + threadIdx.x / LP;
    const bool live = token < (unsigned)p.tokens && 8 * unit < p.d;
    const int bi = live ? (int)(token / (unsigned)p.n) : 0;
    const long long b = bi, t = live ? (int)token - bi * p.n : 0;
    const T* x = (keys ? k : q) + b * xs.batch + t * xs.token + h0 * xs.head;
    const T* gy = (keys ? gk : gq) + b * gs.batch + t * gs.token + h0 * gs.head;
    T* dx = (keys ? dk : dq) + b * ds.batch + t * ds.token + h0 * ds.head;
    Raw<T> next_x[UNROLL], next_g[UNROLL];
    int left = h1 - h0;
    auto fetch = [&](int count) {
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        if (i >= count) break;
        load_raw<MODE>(gy, pl, next_g[i]);
        if (p.norm) load_raw<MODE>(x, pl, next_x[i]);
        gy += gs.head;
        x += xs.head;
      }
    };
    auto turn_back = [&](const Raw<T>(&now_x)[UNROLL], const Raw<T>(&now_g)[UNROLL], const Turn& turn, int count) {
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        if (i >= count) break;
        const Pairs g = pairs_of<MODE, T>(now_g[i]);
        Pairs o;  // the rotation undone
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          o.a[j] = fma2(g.a[j], turn.c[j], mul2(g.b[j], turn.s[j]));
          o.b[j] = fma2(g.b[j], turn.c[j], mul2(g.a[j], turn.ns[j]));
        }
        if (p.norm) {
          const Pairs v = pairs_of<MODE, T>(now_x[i]);
          Pairs wo, ov;  // w g, g x
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            wo.a[j] = mul2(wt.a[j], o.a[j]);
            wo.b[j] = mul2(wt.b[j], o.b[j]);
            ov.a[j] = mul2(v.a[j], o.a[j]);
            ov.b[j] = mul2(v.b[j], o.b[j]);
          }
          const float ss = row_sum<LP>(live ? dot(v, v) : 0.f);
          const float gh = row_sum<LP>(live ? dot(wt, ov) : 0.f);
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          // dx = r (w g - h mean(w g h)) with h = r x, mean = r gh / d
          const float2 m = both(-r * gh * p.inv_d), rr = both(r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (live) {
              acc.a[j] = fma2(ov.a[j], rr, acc.a[j]);
              acc.b[j] = fma2(ov.b[j], rr, acc.b[j]);
            }
            o.a[j] = mul2(rr, fma2(mul2(v.a[j], rr), m, wo.a[j]));
            o.b[j] = mul2(rr, fma2(mul2(v.b[j], rr), m, wo.b[j]));
          }
        }
        if (live) store_pairs<MODE>(dx, pl, o);
        dx += ds.head;
      }
    };
    if (left >= UNROLL) fetch(UNROLL);
    Turn turn{};
    if (live) turn = turn_of<sizeof(T) == 4>(p, freq, unit, (int)token, (int)t);
#pragma unroll 1
    while (left >= UNROLL) {
      Raw<T> now_x[UNROLL], now_g[UNROLL];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        now_x[i] = next_x[i];
        now_g[i] = next_g[i];
      }
      left -= UNROLL;
      if (left >= UNROLL) fetch(UNROLL);
      turn_back(now_x, now_g, turn, UNROLL);
    }
#pragma unroll 1
    for (; left > 0; --left) {
      fetch(1);
      turn_back(next_x, next_g, turn, 1);
    }
  }
  if (!part) return;
  // lanes of one unit: over the warp by shuffles, over the warps in order
  const float v[8] = {acc.a[0].x, acc.a[0].y, acc.a[1].x, acc.a[1].y,
                      acc.b[0].x, acc.b[0].y, acc.b[1].x, acc.b[1].y};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float s = v[j];
#pragma unroll
    for (int o = 16; o >= LP; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane < LP) sums[warp][lane][j] = s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < LP * 8; e += kThreads) {
    const int u = e / 8, j = e % 8;
    if (8 * u >= p.d) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += sums[w][u][j];
    const int c = channel_of<MODE>(place_of<MODE>(u, p.half, p.d), j & 3, (j & 4) != 0);
    part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d + c] = s;
  }
}

// dw[c] = sum over CTAs of part, 32 channels per CTA in 32 row slices: fixed
// order. CTAs y = 0: q's rows [0, q_ctas) of part, y = 1: k's behind them.
// Set up while the kernel that writes part still runs.
__global__ void __launch_bounds__(1024)
qk_weight_grad(const float* part, float* dqw, float* dkw, int d, int q_ctas, int k_ctas) {
  __shared__ float s[32][33];
  cudaGridDependencySynchronize();
  float* dst = blockIdx.y ? dkw : dqw;
  if (!dst) return;
  const float* rows = part + (blockIdx.y ? (size_t)q_ctas * d : 0);
  const int ctas = blockIdx.y ? k_ctas : q_ctas;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int r = slice; r < ctas; r += 32) v += rows[(size_t)r * d + c];
  }
  s[slice][threadIdx.x & 31] = v;
  __syncthreads();
  // warp `slice` sums channel `slice` of this CTA's 32
  float x = s[threadIdx.x & 31][slice];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + slice < d) dst[blockIdx.x * 32 + slice] = x;
}

int lanes_per_row(int d) { return d <= 32 ? 4 : (d <= 64 ? 8 : 16); }

Mode mode_of(const nys_qk_rope_t& a) {
  if (a.pairing == NYS_ROPE_PAIRS) return kPairs;
  return a.rot % 8 == 0 ? kHalves : kHalvesScalar;
}

struct Grid {
  int x, y, heads_per_chunk;
  int q_chunks;  // backward: of y
};

// One CTA per (tile of 256 / LP tokens, chunk of heads). All heads in one
// chunk when the tiles alone give four CTAs per SM; else as many chunks as
// that takes, so that a single token's heads run side by side. Backward CTAs
// walk several tiles (one partial of the weight sums each) and take heads of
// q or of k; there are two per SM, as many as fit, so that all run at once (8 x
// 8192 tokens, 8 + 8 heads, d = 64, bf16: 72 us, with four 74; 1 x 8192: 17
// against 23).
Grid grid_of(const nys_qk_rope_t& a, bool back) {
  const int rows = kThreads / lanes_per_row(a.d);
  const long long tiles = ((long long)a.B * a.n + rows - 1) / rows;
  const int heads = a.Hq + a.Hk;
  const long long want = (back ? 2ll : 4ll) * plan_sms();
  long long chunks = (want + tiles - 1) / tiles;
  if (chunks < 1) chunks = 1;
  if (chunks > heads) chunks = heads;
  Grid g;
  g.heads_per_chunk = (int)((heads + chunks - 1) / chunks);
  g.x = (int)tiles;
  g.y = (heads + g.heads_per_chunk - 1) / g.heads_per_chunk;
  g.q_chunks = 0;
  if (back) {
    g.q_chunks = (a.Hq + g.heads_per_chunk - 1) / g.heads_per_chunk;
    g.y = g.q_chunks + (a.Hk + g.heads_per_chunk - 1) / g.heads_per_chunk;
    const long long most = want / g.y > 0 ? want / g.y : 1;
    if (g.x > most) g.x = (int)most;
  }
  return g;
}

bool strides_ok(const nys_strides_t& s) { return s.batch >= 0 && s.head >= 0 && s.token >= 0; }

bool rows_aligned(const void* p, const nys_strides_t& s, int dtype) {
  const long long per = dtype == NYS_FP32 ? 4 : 8;  // elements in 16 bytes
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.batch % per == 0 && s.head % per == 0 &&
         s.token % per == 0;
}

int check_common(const nys_qk_rope_t* a, const double* inv_freq) {
  if (!a) return NYS_ERR_ARG;
  if (a->dtype != NYS_FP32 && a->dtype != NYS_BF16) return NYS_ERR_ARG;
  if (a->pairing != NYS_ROPE_HALVES && a->pairing != NYS_ROPE_PAIRS) return NYS_ERR_ARG;
  if (a->norm != 0 && a->norm != 1) return NYS_ERR_ARG;
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return NYS_ERR_ARG;
  if (a->B < 1 || a->n < 1 || a->Hq < 1 || a->Hk < 0 || a->d < 8 || a->d > 128 || a->d % 8)
    return NYS_ERR_SHAPE;
  if (a->rot < 0 || a->rot > a->d || a->rot % 2) return NYS_ERR_SHAPE;
  if (a->axes < 1 || a->axes > kMaxAxes) return NYS_ERR_SHAPE;
  if ((long long)a->B * a->n >= (1ll << 31) || (long long)a->Hq + a->Hk > 65535) return NYS_ERR_SHAPE;
  long long sum = 0;
  for (int i = 0; i < a->axes; ++i) {
    if (a->section[i] < 0) return NYS_ERR_SHAPE;
    sum += a->section[i];
  }
  if (sum != a->rot / 2) return NYS_ERR_SHAPE;
  if (a->rot > 0) {
    if (!inv_freq) return NYS_ERR_ARG;
    for (int i = 0; i < a->rot / 2; ++i)
      if (!std::isfinite(inv_freq[i])) return NYS_ERR_ARG;
  }
  return NYS_OK;
}

// Output rows must not share memory: a stride shorter than a row along an
// axis with more than one entry is refused.
bool rows_apart(const nys_strides_t& s, int B, int H, int n, int d) {
  return (B == 1 || s.batch >= d) && (H == 1 || s.head >= d) && (n == 1 || s.token >= d);
}

RopeParams params_of(const nys_qk_rope_t& a, const float* qw, const float* kw, const int* positions,
                     const double* inv_freq, int heads_per_chunk) {
  RopeParams p{};
  p.half = a.rot / 2;
  for (int i = 0; i < p.half; ++i) {
    // turns per position, modulo one (positions are whole numbers)
    double turns = inv_freq[i] * 0.15915494309189533577;
    turns -= std::floor(turns);
    const double units = std::ldexp(turns, 64);
    p.freq[i] = units >= 18446744073709551616.0 ? 0ull : (unsigned long long)units;
  }
  p.positions = positions;
  p.qw = qw;
  p.kw = kw;
  p.tokens = a.B * a.n;
  p.n = a.n;
  p.Hq = a.Hq;
  p.Hk = a.Hk;
  p.d = a.d;
  int at = 0;
  for (int i = 0; i < kMaxAxes; ++i) {
    if (i < a.axes) at += a.section[i];
    p.end[i] = at;
  }
  p.heads_per_chunk = heads_per_chunk;
  p.norm = a.norm;
  p.eps = a.eps;
  p.inv_d = 1.0f / (float)a.d;
  p.qi = a.q;
  p.ki = a.k;
  p.qo = a.q_out;
  p.ko = a.k_out;
  p.dq = a.dq;
  p.dk = a.dk;
  return p;
}

template <typename T, int LP, int MODE>
int launch_fwd(const RopeParams& p, const Grid& g, const void* q, const void* k, void* qo, void* ko,
               cudaStream_t st) {
  KernelScope scope("qk_norm_rope", st);
  qk_norm_rope<T, LP, MODE><<<dim3(g.x, g.y), kThreads, 0, st>>>(
      p, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<T*>(qo), static_cast<T*>(ko));
  return launch_status();
}

template <typename T, int LP, int MODE>
int launch_bwd(const RopeParams& p, const Grid& g, const void* q, const void* k, const void* gq,
               const void* gk, void* dq, void* dk, float* part, cudaStream_t st) {
  KernelScope scope("qk_norm_rope_back", st);
  qk_norm_rope_back<T, LP, MODE><<<dim3(g.x, g.y), kThreads, 0, st>>>(
      p, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(gq),
      static_cast<const T*>(gk), static_cast<T*>(dq), static_cast<T*>(dk), part, g.q_chunks);
  return launch_status();
}

// f.template operator()<T, LP, MODE>() for the call's type and sizes.
template <typename F>
int dispatch(const nys_qk_rope_t& a, F&& f) {
  auto by_mode = [&](auto type, auto lp) -> int {
    using T = decltype(type);
    constexpr int LP = decltype(lp)::value;
    switch (mode_of(a)) {
      case kHalves: return f(T{}, lp, std::integral_constant<int, kHalves>{});
      case kPairs: return f(T{}, lp, std::integral_constant<int, kPairs>{});
      default: return f(T{}, std::integral_constant<int, LP>{}, std::integral_constant<int, kHalvesScalar>{});
    }
  };
  auto by_lanes = [&](auto type) -> int {
    switch (lanes_per_row(a.d)) {
      case 4: return by_mode(type, std::integral_constant<int, 4>{});
      case 8: return by_mode(type, std::integral_constant<int, 8>{});
      default: return by_mode(type, std::integral_constant<int, 16>{});
    }
  };
  return a.dtype == NYS_BF16 ? by_lanes(__nv_bfloat16{}) : by_lanes(float{});
}

size_t weight_part_bytes(const nys_qk_rope_t& a) {
  const Grid g = grid_of(a, true);
  return ((size_t)g.x * g.y * a.d * sizeof(float) + 255) & ~size_t(255);
}

}  // namespace
}  // namespace nys

using namespace nys;

extern "C" {

int nystrom_qk_norm_rope_fwd(const nys_qk_rope_t* a, const void* q, const void* k,
                             const float* q_weight, const float* k_weight, const int* positions,
                             const double* inv_freq_host, void* q_out, void* k_out,
                             nys_stream_t stream) {
  int rc = check_common(a, inv_freq_host);
  if (rc != NYS_OK) return rc;
  if (!q || !q_out || (a->Hk > 0 && (!k || !k_out))) return NYS_ERR_ARG;
  if (!strides_ok(a->q) || !strides_ok(a->q_out) || !rows_apart(a->q_out, a->B, a->Hq, a->n, a->d))
    return NYS_ERR_ARG;
  if (!rows_aligned(q, a->q, a->dtype) || !rows_aligned(q_out, a->q_out, a->dtype)) return NYS_ERR_ALIGN;
  if (a->Hk > 0) {
    if (!strides_ok(a->k) || !strides_ok(a->k_out) || !rows_apart(a->k_out, a->B, a->Hk, a->n, a->d))
      return NYS_ERR_ARG;
    if (!rows_aligned(k, a->k, a->dtype) || !rows_aligned(k_out, a->k_out, a->dtype)) return NYS_ERR_ALIGN;
  }
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight) |
       reinterpret_cast<uintptr_t>(positions)) & 3u)
    return NYS_ERR_ALIGN;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (!apart_or_same_rows(q_out, a->q_out, q, a->q, a->B, a->Hq, a->n)) return NYS_ERR_ARG;
  if (a->Hk > 0 && (!apart_or_same_rows(k_out, a->k_out, k, a->k, a->B, a->Hk, a->n) || q_out == k_out ||
                    q_out == k || k_out == q))
    return NYS_ERR_ARG;
  const Grid g = grid_of(*a, false);
  const RopeParams p = params_of(*a, q_weight, k_weight, positions, inv_freq_host, g.heads_per_chunk);
  return dispatch(*a, [&](auto type, auto lp, auto mode) {
    return launch_fwd<decltype(type), decltype(lp)::value, decltype(mode)::value>(p, g, q, k, q_out,
                                                                                 k_out, stream);
  });
}

size_t nystrom_qk_norm_rope_workspace_bytes(const nys_qk_rope_t* a) {
  static const double ones[kMaxPairs] = {};
  if (check_common(a, ones) != NYS_OK || !a->norm) return 0;
  return weight_part_bytes(*a);
}

int nystrom_qk_norm_rope_bwd(const nys_qk_rope_t* a, const void* q, const void* k, const void* gq,
                             const void* gk, const float* q_weight, const float* k_weight,
                             const int* positions, const double* inv_freq_host, void* dq, void* dk,
                             float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes,
                             nys_stream_t stream) {
  int rc = check_common(a, inv_freq_host);
  if (rc != NYS_OK) return rc;
  if (!gq || !dq || (a->norm && !q)) return NYS_ERR_ARG;
  if (!strides_ok(a->q) || !strides_ok(a->q_out) || !strides_ok(a->dq) ||
      !rows_apart(a->dq, a->B, a->Hq, a->n, a->d))
    return NYS_ERR_ARG;
  if ((a->norm && !rows_aligned(q, a->q, a->dtype)) || !rows_aligned(gq, a->q_out, a->dtype) ||
      !rows_aligned(dq, a->dq, a->dtype))
    return NYS_ERR_ALIGN;
  if (a->Hk > 0) {
    if (!gk || !dk || (a->norm && !k)) return NYS_ERR_ARG;
    if (!strides_ok(a->k) || !strides_ok(a->k_out) || !strides_ok(a->dk) ||
        !rows_apart(a->dk, a->B, a->Hk, a->n, a->d))
      return NYS_ERR_ARG;
    if ((a->norm && !rows_aligned(k, a->k, a->dtype)) || !rows_aligned(gk, a->k_out, a->dtype) ||
        !rows_aligned(dk, a->dk, a->dtype))
      return NYS_ERR_ALIGN;
  }
  // without the norm there are no weights, with no keys none of theirs
  if ((!a->norm && (dq_weight || dk_weight)) || (a->Hk == 0 && dk_weight)) return NYS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight) |
       reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight) |
       reinterpret_cast<uintptr_t>(positions)) & 3u)
    return NYS_ERR_ALIGN;
  const bool sums = dq_weight || dk_weight;
  const size_t need = sums ? weight_part_bytes(*a) : 0;
  if (sums && workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return NYS_ERR_ALIGN;
    if (ws_bytes < need) return NYS_ERR_NOMEM;
  }
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  if (!apart_or_same_rows(dq, a->dq, gq, a->q_out, a->B, a->Hq, a->n)) return NYS_ERR_ARG;
  if (a->Hk > 0 && (!apart_or_same_rows(dk, a->dk, gk, a->k_out, a->B, a->Hk, a->n) || dq == dk || dq == gk ||
                    dk == gq))
    return NYS_ERR_ARG;
  if (dq_weight && dq_weight == dk_weight) return NYS_ERR_ARG;
  std::unique_lock<std::mutex> held;
  if (sums && !workspace) {
    rc = operator_workspace(dev, need, stream, &workspace, &held);
    if (rc != NYS_OK) return rc;
  }
  const Grid g = grid_of(*a, true);
  const RopeParams p = params_of(*a, q_weight, k_weight, positions, inv_freq_host, g.heads_per_chunk);
  float* part = sums ? static_cast<float*>(workspace) : nullptr;
  rc = dispatch(*a, [&](auto type, auto lp, auto mode) {
    return launch_bwd<decltype(type), decltype(lp)::value, decltype(mode)::value>(p, g, q, k, gq, gk, dq,
                                                                                 dk, part, stream);
  });
  if (rc != NYS_OK || !sums) return rc;
  KernelScope scope("qk_weight_grad", stream);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a->d + 31) / 32, a->Hk > 0 ? 2 : 1);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, qk_weight_grad, static_cast<const float*>(part), dq_weight, dk_weight, a->d,
                     g.x * g.q_chunks, g.x * (g.y - g.q_chunks));
  return launch_status();
}

}  // extern "C"
