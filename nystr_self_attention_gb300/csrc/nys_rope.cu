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
  long long tokens;                    // B * n
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
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The eight channels of one lane: a[j], b[j] are the members of its pair j.
struct Pairs {
  float a[4], b[4];
};

// Where a lane's channels sit in a row. Past the rotated channels a "pair" is
// two neighbours, turned by nothing.
struct Place {
  int lo, hi;  // first channel of a[0..3] and of b[0..3] (kPairs: of all eight)
  int unit, half;
};

template <int MODE>
__device__ __forceinline__ Place place_of(int unit, int half) {
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

__device__ __forceinline__ void widen(const uint4& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(const uint2& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}

template <int MODE, typename T>
__device__ __forceinline__ Pairs pairs_of(const Raw<T>& r) {
  Pairs x;
  if (MODE == kPairs) {
    float u[4], v[4];
    widen(r.lo, u);
    widen(r.hi, v);
    x.a[0] = u[0]; x.b[0] = u[1]; x.a[1] = u[2]; x.b[1] = u[3];
    x.a[2] = v[0]; x.b[2] = v[1]; x.a[3] = v[2]; x.b[3] = v[3];
  } else {
    widen(r.lo, x.a);
    widen(r.hi, x.b);
  }
  return x;
}

template <int MODE, typename T>
__device__ __forceinline__ void store_pairs(T* row, const Place& pl, const Pairs& x) {
  if (MODE == kHalves) {
    store4(row + pl.lo, x.a);
    store4(row + pl.hi, x.b);
  } else if (MODE == kPairs) {
    const float u[4] = {x.a[0], x.b[0], x.a[1], x.b[1]}, v[4] = {x.a[2], x.b[2], x.a[3], x.b[3]};
    store4(row + pl.lo, u);
    store4(row + pl.hi, v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      store1(row + channel_of<MODE>(pl, j, false), x.a[j]);
      store1(row + channel_of<MODE>(pl, j, true), x.b[j]);
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
  float c[4], s[4];
};

template <bool EXACT>
__device__ __forceinline__ Turn turn_of(const RopeParams& p, const unsigned long long* freq,
                                        int unit, long long token, int t) {
  Turn r;
  int axis = -1;
  unsigned long long pos = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 4 * unit + j;
    r.c[j] = 1.f;
    r.s[j] = 0.f;
    if (i < p.half) {
      int ax = 0;
      while (i >= p.end[ax]) ++ax;  // sections sum to half, so ax stays below axes
      if (ax != axis) {
        axis = ax;
        pos = (unsigned long long)(long long)(p.positions ? p.positions[ax * p.tokens + token] : t);
      }
      turn_cos_sin<EXACT>(freq[i] * pos, r.c[j], r.s[j]);
    }
  }
  return r;
}

// Sum over the LP lanes of a row, in every one of them.
template <int LP>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float square_sum(const Pairs& x) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fmaf(x.a[j], x.a[j], fmaf(x.b[j], x.b[j], s));
  return s;
}

template <int MODE>
__device__ __forceinline__ void load_weights(const float* w, const Place& pl, bool live, Pairs& x) {
  const bool given = w && live;  // 4-byte aligned: scalar loads, once per walk
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x.a[j] = given ? w[channel_of<MODE>(pl, j, false)] : 1.f;
    x.b[j] = given ? w[channel_of<MODE>(pl, j, true)] : 1.f;
  }
}

// Heads [h0, h1) of one tensor for one token: UNROLL rows at a time, the next
// ones' loads in flight while these are worked on.
template <typename T, int LP, int MODE, int UNROLL>
__device__ __forceinline__ void walk_forward(const T* x, T* y, long long xs, long long ys, int h0,
                                             int h1, const float* w, const Turn& turn,
                                             const Place& pl, bool live, const RopeParams& p) {
  Raw<T> next[UNROLL];
  auto fetch = [&](int h) {
#pragma unroll
    for (int k = 0; k < UNROLL; ++k)
      if (live && h + k < h1) load_raw<MODE>(x + (h + k) * xs, pl, next[k]);
  };
  fetch(h0);
  Pairs wt;
  if (p.norm) load_weights<MODE>(w, pl, live, wt);
  for (int h = h0; h < h1; h += UNROLL) {
    Raw<T> now[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) now[k] = next[k];
    fetch(h + UNROLL);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const bool on = live && h + k < h1;
      Pairs v = pairs_of<MODE, T>(now[k]);
      if (p.norm) {
        const float ss = row_sum<LP>(on ? square_sum(v) : 0.f);
        const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v.a[j] *= r * wt.a[j];
          v.b[j] *= r * wt.b[j];
        }
      }
      Pairs o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o.a[j] = fmaf(v.a[j], turn.c[j], -v.b[j] * turn.s[j]);
        o.b[j] = fmaf(v.b[j], turn.c[j], v.a[j] * turn.s[j]);
      }
      if (on) store_pairs<MODE>(y + (h + k) * ys, pl, o);
    }
  }
}

// Rows in flight per lane: 64 bytes' worth.
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;

template <typename T, int LP, int MODE>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope(const __grid_constant__ RopeParams p, const T* q, const T* k, T* qo, T* ko) {
  __shared__ unsigned long long freq[kMaxPairs];
  if (threadIdx.x < p.half) freq[threadIdx.x] = p.freq[threadIdx.x];
  __syncthreads();
  const int unit = threadIdx.x % LP;
  const long long token = (long long)blockIdx.x * (kThreads / LP) + threadIdx.x / LP;
  const bool live = token < p.tokens && 8 * unit < p.d;
  const long long b = live ? token / p.n : 0, t = live ? token - b * p.n : 0;
  const Place pl = place_of<MODE>(unit, p.half);
  Turn turn{};
  if (live) turn = turn_of<sizeof(T) == 4>(p, freq, unit, token, (int)t);
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
  constexpr int UNROLL = kAhead<T>;
  const bool keys = (int)blockIdx.y >= q_chunks;  // CTA-uniform
  const nys_strides_t &xs = keys ? p.ki : p.qi, &gs = keys ? p.ko : p.qo, &ds = keys ? p.dk : p.dq;
  const int unit = threadIdx.x % LP;
  const Place pl = place_of<MODE>(unit, p.half);
  const int h0 = ((int)blockIdx.y - (keys ? q_chunks : 0)) * p.heads_per_chunk;
  const int h1 = min(keys ? p.Hk : p.Hq, h0 + p.heads_per_chunk);
  constexpr int kRows = kThreads / LP;
  const long long tiles = (p.tokens + kRows - 1) / kRows;
  Pairs acc{}, wt;
  if (p.norm) load_weights<MODE>(keys ? p.kw : p.qw, pl, 8 * unit < p.d, wt);
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long token = tile * kRows + threadIdx.x / LP;
    const bool live = token < p.tokens && 8 * unit < p.d;
    const long long b = live ? token / p.n : 0, t = live ? token - b * p.n : 0;
    const T* x = (keys ? k : q) + b * xs.batch + t * xs.token;
    const T* gy = (keys ? gk : gq) + b * gs.batch + t * gs.token;
    T* dx = (keys ? dk : dq) + b * ds.batch + t * ds.token;
    Raw<T> next_x[UNROLL], next_g[UNROLL];
    auto fetch = [&](int h) {
#pragma unroll
      for (int i = 0; i < UNROLL; ++i)
        if (live && h + i < h1) {
          load_raw<MODE>(gy + (h + i) * gs.head, pl, next_g[i]);
          if (p.norm) load_raw<MODE>(x + (h + i) * xs.head, pl, next_x[i]);
        }
    };
    fetch(h0);
    Turn turn{};
    if (live) turn = turn_of<sizeof(T) == 4>(p, freq, unit, token, (int)t);
    for (int h = h0; h < h1; h += UNROLL) {
      Raw<T> now_x[UNROLL], now_g[UNROLL];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        now_x[i] = next_x[i];
        now_g[i] = next_g[i];
      }
      fetch(h + UNROLL);
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        const bool on = live && h + i < h1;
        const Pairs g = pairs_of<MODE, T>(now_g[i]);
        Pairs o;  // the rotation undone
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o.a[j] = fmaf(g.a[j], turn.c[j], g.b[j] * turn.s[j]);
          o.b[j] = fmaf(g.b[j], turn.c[j], -g.a[j] * turn.s[j]);
        }
        if (p.norm) {
          const Pairs v = pairs_of<MODE, T>(now_x[i]);
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dot = fmaf(wt.a[j] * o.a[j], v.a[j], fmaf(wt.b[j] * o.b[j], v.b[j], dot));
          const float ss = row_sum<LP>(on ? square_sum(v) : 0.f);
          dot = row_sum<LP>(on ? dot : 0.f);
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          const float m = r * dot * p.inv_d;  // mean(w g h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ha = v.a[j] * r, hb = v.b[j] * r;
            if (on) {
              acc.a[j] = fmaf(o.a[j], ha, acc.a[j]);
              acc.b[j] = fmaf(o.b[j], hb, acc.b[j]);
            }
            o.a[j] = r * fmaf(wt.a[j], o.a[j], -ha * m);
            o.b[j] = r * fmaf(wt.b[j], o.b[j], -hb * m);
          }
        }
        if (on) store_pairs<MODE>(dx + (h + i) * ds.head, pl, o);
      }
    }
  }
  if (!part) return;
  // lanes of one unit: over the warp by shuffles, over the warps in order
  const float v[8] = {acc.a[0], acc.a[1], acc.a[2], acc.a[3], acc.b[0], acc.b[1], acc.b[2], acc.b[3]};
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
    const int c = channel_of<MODE>(place_of<MODE>(u, p.half), j & 3, (j & 4) != 0);
    part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d + c] = s;
  }
}

// dw[c] = sum over CTAs of part, 32 channels per CTA in 32 row slices: fixed
// order. CTAs y = 0: q's rows [0, q_ctas) of part, y = 1: k's behind them.
__global__ void __launch_bounds__(1024)
qk_weight_grad(const float* __restrict__ part, float* dqw, float* dkw, int d, int q_ctas, int k_ctas) {
  __shared__ float s[32][33];
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
// q or of k.
Grid grid_of(const nys_qk_rope_t& a, bool back) {
  const int rows = kThreads / lanes_per_row(a.d);
  const long long tiles = ((long long)a.B * a.n + rows - 1) / rows;
  const int heads = a.Hq + a.Hk;
  const long long want = 4ll * plan_sms();
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
  p.tokens = (long long)a.B * a.n;
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
  if (sums && !workspace) {
    rc = operator_workspace(dev, need, stream, &workspace);
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
  qk_weight_grad<<<dim3((a->d + 31) / 32, a->Hk > 0 ? 2 : 1), 1024, 0, stream>>>(
      part, dq_weight, dk_weight, a->d, g.x * g.q_chunks, g.x * (g.y - g.q_chunks));
  return launch_status();
}

}  // extern "C"
