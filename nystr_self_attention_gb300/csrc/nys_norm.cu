// The residual's addition with the root-mean-square norm of the sum, output in
// the input's type or in 8 bits, and its gradients (declared in
// include/nystrom.h). All are bound by HBM: each element is read and written
// once, with the row held in registers between its sum of squares and its
// output.
//
// TPR threads share a row (or as many as it needs, where it has a CTA to itself), V
// vectors of eight channels each; vector i of thread t is channels 8 (i TPR + t), so
// 16 neighbouring threads hold the 128 channels of one 8-bit block. A CTA holds several short rows or one long one and walks
// rows with the grid's step; the weight stays in registers, and the next row's
// loads are in flight while this one is summed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "nys_q8.h"
#include "nys_sm100.h"

namespace nys {
namespace {

using q8::kBlock;
constexpr int kMaxD = 16384;

struct NormParams {
  long long x, r, s, y, gs, dx;  // row strides
  int rows, d;
  float eps, inv_d;
  uint8_t *codes, *scales;
  int ring;     // backward: rows of shared memory
  int* status;  // and where a wait that runs out is reported
};
// 16384 x 4096 in bf16: 86 us with three rows, 92 with four, 90 from registers; in
// fp32 4096 x 8192 87 us with two, 125 from registers.
constexpr int kMostRing = 3;

// Eight channels as they lie in memory.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
};

// Two fp32 operations at a time.
__device__ __forceinline__ unsigned long long bits(float2 a) { return reinterpret_cast<unsigned long long&>(a); }
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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2& pair_of(float (&v)[8], int i) { return reinterpret_cast<float2&>(v[2 * i]); }

// Sum of v over the TPR threads of a row, the same bits in each: shuffles, then
// one slot per warp. The slots alternate between two sets, so one barrier per
// sum is enough.
// A group that has its CTA to itself (TPR >= 256) may have fewer threads than TPR.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*slots)[N], int& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  if (TPR == 32) return;
  const int W = TPR >= 256 ? blockDim.x / 32 : TPR / 32;
  const int warp = threadIdx.x >> 5, group = TPR >= 256 ? 0 : threadIdx.x / TPR;
  float(*set)[N] = slots + phase * (blockDim.x / 32);
  phase ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int j = 0; j < N; ++j) set[warp][j] = v[j];
  if (TPR >= 256)
    __syncthreads();  // the CTA is the group
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w)
      if (TPR < 256 || w < W) s += set[group * W + w][j];
    v[j] = s;
  }
}

// r + low = 1 / sqrt((total + rest) / d + eps), to 1e-14 of it: a step of
// Newton's on the special-function unit's result, with the remainders of the
// division, the sum and the product kept (fused multiply-adds have no rounding
// between their product and their sum).
__device__ __forceinline__ float2 inverse_root(float total, float rest, float d, float inv_d, float eps) {
  const float q = total * inv_d, ql = (fmaf(-q, d, total) + rest) * inv_d;
  const float v = q + eps, b = v - q, vl = (q - (v - b)) + (eps - b) + ql;
  const float r = rsqrtf(v), h = v * r, hl = fmaf(v, r, -h);
  const float e = fmaf(-h, r, 1.f) - fmaf(hl, r, vl * r * r);
  return make_float2(r, 0.5f * r * e);
}

// The root of a row's mean square to 1e-14 or so of the fp32 sums of its warps: the
// group's first warp adds those, with what the additions round away, and hands the
// root on. (Each thread adding them for itself took 7 instructions per element.)
template <int TPR>
__device__ __forceinline__ float2 exact_root(float v, float (*slots)[1], float2* roots, int& phase, float d, float inv_d,
                                             float eps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR == 32) return inverse_root(v, 0.f, d, inv_d, eps);
  const int W = TPR >= 256 ? blockDim.x / 32 : TPR / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = TPR >= 256 ? 0 : threadIdx.x / TPR;
  auto barrier = [&] {
    if (TPR >= 256)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
  };
  float(*set)[1] = slots + phase * (blockDim.x / 32);
  float2* root = roots + phase * 8 + group;
  phase ^= 1;
  if (lane == 0) set[warp][0] = v;
  barrier();
  if (warp == group * W) {
    float x = lane < W ? set[group * W + lane][0] : 0.f, low = 0.f;
#pragma unroll
    for (int o = TPR / 64; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o), rest = __shfl_xor_sync(0xffffffffu, low, o);
      const float sum = x + y, b = sum - x;
      low = low + rest + ((x - (sum - b)) + (y - b));
      x = sum;
    }
    if (lane == 0) *root = inverse_root(x, low, d, inv_d, eps);
  }
  barrier();
  return *root;
}

constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }
// Threads per SM that the registers are cut for.
template <typename T, int TPR, bool RES>
constexpr int fwd_threads() {
  return TPR == 1024 ? 1024 : sizeof(T) == 4 && RES ? 1024 : 1536;
}
constexpr int kBwdThreads = 512;
constexpr int bwd_ctas(int threads) { return threads < kBwdThreads ? kBwdThreads / threads : 1; }  // per SM

template <typename T, int TPR, int V, bool EIGHT, bool RES>
__global__ void __launch_bounds__(threads_of(TPR), fwd_threads<T, TPR, RES>() / threads_of(TPR))
add_rms_norm(const NormParams p, const T* x, const T* res, const float* __restrict__ weight, T* sum, T* y) {
  constexpr int THREADS = threads_of(TPR), GROUPS = THREADS / TPR;
  __shared__ float slots[2 * THREADS / 32][1];
  __shared__ float2 roots[2 * 8];
  int phase = 0;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int across = GROUPS == 1 ? blockDim.x : TPR, t = threadIdx.x % TPR;  // threads of a row
  const int step = gridDim.x * GROUPS;
  int row = blockIdx.x * GROUPS + threadIdx.x / TPR;
  Vec<T> nx[V], nr[V];
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (i * across + t);
      nx[i].clear();
      if (RES) nr[i].clear();
      if (r < p.rows && c < p.d) {
        nx[i].load(x + r * p.x + c);
        if (RES) nr[i].load(res + r * p.r + c);
      }
    }
  };
  fetch(row);
  float w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = 8 * (i * across + t);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = c < p.d ? (weight ? weight[c + j] : 1.f) : 0.f;
  }
  // the threads of a row leave together: `row` is the group's
  for (; row < p.rows; row += step) {
    float s[V][8], total[1];
    float2 squares = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      nx[i].widen(s[i]);
      if (RES) {
        float r[8];
        nr[i].widen(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) pair_of(s[i], j) = add2(pair_of(s[i], j), pair_of(r, j));
        Vec<T> out;  // s is what is kept: rounded
        out.narrow(s[i]);
        out.widen(s[i]);
        const int c = 8 * (i * across + t);
        if (sum && c < p.d) out.store(sum + row * p.s + c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) squares = fma2(pair_of(s[i], j), pair_of(s[i], j), squares);
    }
    total[0] = squares.x + squares.y;
    fetch(row < p.rows - step ? row + step : p.rows);
    // To 8 bits, y carries half the error of the fp32 sum of squares (a thread's and
    // a warp's share of it: 10 or 14 roundings in a row; the sums across warps keep
    // theirs) and one rounding of its own. A code next to a border may then differ
    // from the exact one's; in the form below the product and the root add to that.
    float2 root;
    if (EIGHT) {
      root = exact_root<TPR>(total[0], slots, roots, phase, (float)p.d, p.inv_d, p.eps);
    } else {
      row_sums<TPR, 1>(total, slots, phase);
      root = make_float2(rsqrtf(fmaf(total[0], p.inv_d, p.eps)), 0.f);
    }
    const float low = root.y - root.y == 0.f ? root.y : 0.f;  // none where the sum of squares is infinite
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (i * across + t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2& v = pair_of(s[i], j);
        const float2 wj = pair_of(w[i], j);
        const float2 h = mul2(v, both(root.x));
        if (EIGHT) {
          const float2 hl = fma2(v, both(low), fma2(v, both(root.x), make_float2(-h.x, -h.y)));
          v = fma2(h, wj, mul2(hl, wj));
        } else {
          v = mul2(h, wj);
        }
      }
      if (!EIGHT) {
        Vec<T> out;
        out.narrow(s[i]);
        if (c < p.d) out.store(y + row * p.y + c);
      } else {
        uint32_t top = 0u;  // magnitudes compare as integers, NaN above infinity
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, c < p.d ? __float_as_uint(s[i][j]) & 0x7fffffffu : 0u);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t byte = q8::scale_byte(top);
        const float inv = q8::inverse_scale(byte);
        if (c < p.d) {
          const uint2 codes = make_uint2(q8::encode4(s[i][0], s[i][1], s[i][2], s[i][3], inv),
                                         q8::encode4(s[i][4], s[i][5], s[i][6], s[i][7], inv));
          *reinterpret_cast<uint2*>(p.codes + row * p.y + c) = codes;
          if ((t & 15) == 0)
            q8::store_scale(p.scales, c / kBlock, (p.d + kBlock - 1) / kBlock, row, p.rows, byte);
        }
      }
    }
    if (row >= p.rows - step) break;  // the next index may pass 2^31
  }
}

// A row of memory to shared memory, reported to a barrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sm100::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}

// part: [CTAs][d] sums of gy h over a CTA's rows, or null. Rows that a CTA has to
// itself come through p.ring rows of shared memory, filled by bulk copies that far
// ahead; the others are loaded into registers one row ahead.
template <typename T, int TPR, int V>
__global__ void __launch_bounds__(threads_of(TPR), bwd_ctas(threads_of(TPR)))
add_rms_norm_back(const NormParams p, const T* s, const T* gy, const T* gs, const float* __restrict__ weight,
                  T* dx, float* part) {
  constexpr bool RING = TPR >= 256;
  constexpr int THREADS = threads_of(TPR), GROUPS = THREADS / TPR;
  // the weight in registers, and the next row in flight, as long as both fit
  constexpr bool ROOMY = RING || V * sizeof(T) <= 4;
  // the longest rows: read from the ring twice instead of held
  constexpr bool TWICE = RING && TPR == 1024;
  __shared__ float slots[2 * THREADS / 32][2];
  extern __shared__ __align__(16) float sums[];  // [GROUPS][d] where a CTA holds several rows; the ring
  __shared__ uint64_t full[kMostRing];
  __shared__ int abort_flag;
  uint8_t* ring = reinterpret_cast<uint8_t*>(sums);
  const uint32_t row_bytes = p.d * sizeof(T), slot_bytes = (gs ? 3 : 2) * row_bytes;
  int phase = 0;
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int across = GROUPS == 1 ? blockDim.x : TPR, t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int step = gridDim.x * GROUPS;
  int row = blockIdx.x * GROUPS + group;
  Vec<T> ns[V], ng[V], na[V];
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (i * across + t);
      ns[i].clear();
      ng[i].clear();
      na[i].clear();
      if (r < p.rows && c < p.d) {
        ns[i].load(s + r * p.s + c);
        ng[i].load(gy + r * p.y + c);
        if (gs) na[i].load(gs + r * p.gs + c);
      }
    }
  };
  auto load_weight = [&](int i, float (&w)[8]) {
    const int c = 8 * (i * across + t);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c < p.d ? (weight ? weight[c + j] : 1.f) : 0.f;
  };
  // one thread: row r's three parts to the slot of the CTA's n-th row
  auto fill = [&](int r, int n) {
    uint8_t* to = ring + n % p.ring * slot_bytes;
    uint64_t* bar = &full[n % p.ring];
    sm100::mbar_arrive_expect_tx(bar, slot_bytes);
    bulk_load(to, s + r * p.s, row_bytes, bar);
    bulk_load(to + row_bytes, gy + r * p.y, row_bytes, bar);
    if (gs) bulk_load(to + 2 * row_bytes, gs + r * p.gs, row_bytes, bar);
  };
  int nth = 0, filled = 0;  // of the CTA's rows; slots filled (the thread that fills them)
  if (RING) {
    if (threadIdx.x == 0) {
      abort_flag = 0;
      for (int i = 0; i < p.ring; ++i) sm100::mbar_init(&full[i], 1);
      sm100::fence_barrier_init();
      for (int r = row; filled < p.ring && r < p.rows; ++filled) {
        fill(r, filled);
        r = r < p.rows - step ? r + step : p.rows;
      }
    }
    __syncthreads();
  } else {
    fetch(row);
  }
  float kept[ROOMY ? V : 1][8], acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (ROOMY) load_weight(i, kept[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  for (; row < p.rows; row += step) {
    Vec<T> xs[V], xg[V], xa[V];
    if (RING) {
      if (!sm100::mbar_wait(&full[nth % p.ring], nth / p.ring & 1, const_cast<volatile int*>(&abort_flag),
                            2000000000ull)) {
        abort_flag = 1;
        atomicExch(p.status, (int)NYS_ERR_TIMEOUT);
      }
    }
    // the row's parts of vector i, from its slot
    const uint8_t* from = ring + nth % (RING ? p.ring : 1) * slot_bytes;
    auto read = [&](int i, Vec<T>& a, Vec<T>& g, Vec<T>& e) {
      const int c = 8 * (i * across + t);
      a.clear();
      g.clear();
      e.clear();
      if (c >= p.d) return;
      a.load(reinterpret_cast<const T*>(from) + c);
      g.load(reinterpret_cast<const T*>(from + row_bytes) + c);
      if (gs) e.load(reinterpret_cast<const T*>(from + 2 * row_bytes) + c);
    };
    float2 ss = both(0.f), gs2 = both(0.f);  // s^2, weight gy s
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (RING) {
        read(i, xs[i], xg[i], xa[i]);
      } else {
        xs[i] = ns[i];
        xg[i] = ng[i];
        xa[i] = na[i];
      }
      float a[8], g[8], w[8];
      xs[i].widen(a);
      xg[i].widen(g);
      if (!ROOMY) load_weight(i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss = fma2(pair_of(a, j), pair_of(a, j), ss);
        gs2 = fma2(mul2(ROOMY ? pair_of(kept[ROOMY ? i : 0], j) : pair_of(w, j), pair_of(g, j)), pair_of(a, j), gs2);
      }
    }
    float total[2] = {ss.x + ss.y, gs2.x + gs2.y};
    const int next = row < p.rows - step ? row + step : p.rows;
    if (ROOMY && !RING) fetch(next);
    row_sums<TPR, 2>(total, slots, phase);
    auto refill = [&] {  // behind a barrier: every thread has read the slot
      const long long later = row + (long long)p.ring * step;
      if (threadIdx.x == 0 && later < p.rows && !abort_flag) fill((int)later, filled++);
      ++nth;
    };
    if (RING && !TWICE) refill();
    const float r = rsqrtf(fmaf(total[0], p.inv_d, p.eps));
    const float m = -r * r * total[1] * p.inv_d;  // -mean(weight gy h) r
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float a[8], g[8], e[8], w[8];
      if (TWICE) read(i, xs[i], xg[i], xa[i]);
      xs[i].widen(a);
      xg[i].widen(g);
      xa[i].widen(e);
      if (!ROOMY) load_weight(i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 h = mul2(pair_of(a, j), both(r)), gj = pair_of(g, j);
        const float2 wg = mul2(ROOMY ? pair_of(kept[ROOMY ? i : 0], j) : pair_of(w, j), gj);
        pair_of(acc[i], j) = fma2(gj, h, pair_of(acc[i], j));
        pair_of(e, j) = fma2(both(r), wg, fma2(h, both(m), pair_of(e, j)));
      }
      const int c = 8 * (i * across + t);
      Vec<T> out;
      out.narrow(e);
      if (c < p.d) out.store(dx + row * p.dx + c);
    }
    if (!ROOMY) fetch(next);
    if (TWICE) {
      __syncthreads();
      refill();
    }
    if (next == p.rows) break;  // row + step may pass 2^31
  }
  // where a wait ran out: nothing may land in shared memory behind the kernel's end
  if (RING && threadIdx.x == 0 && abort_flag)
    for (int i = filled > p.ring ? filled - p.ring : 0; i < filled; ++i)
      sm100::mbar_wait(&full[i % p.ring], i / p.ring & 1, nullptr, 2000000000ull);
  if (!part) return;
  float* dst = part + (size_t)blockIdx.x * p.d;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (i * across + t);
      if (c < p.d)
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[c + j] = acc[i][j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = 8 * (i * across + t);
      if (c < p.d)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[group * p.d + c + j] = acc[i][j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) v += sums[g * p.d + c];
      dst[c] = v;
    }
  }
}

// dw[c] = sum over the CTAs of part, 32 channels per CTA in 32 row slices: a
// fixed order. Set up while the kernel that writes part still runs.
__global__ void __launch_bounds__(1024)
norm_weight_grad(const float* part, float* dw, int d, int ctas) {
  __shared__ float s[32][33];
  cudaGridDependencySynchronize();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int r = slice; r < ctas; r += 32) v += part[(size_t)r * d + c];
  }
  s[slice][lane] = v;
  __syncthreads();
  float x = s[lane][slice];  // warp `slice` sums channel `slice` of this CTA's 32
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0 && blockIdx.x * 32 + slice < d) dw[blockIdx.x * 32 + slice] = x;
}

int check_common(const nys_add_rms_norm_t* p) {
  if (!p) return NYS_ERR_ARG;
  if (p->dtype != NYS_FP32 && p->dtype != NYS_BF16) return NYS_ERR_ARG;
  if (!(p->eps >= 0.f) || std::isinf(p->eps)) return NYS_ERR_ARG;
  if (p->rows < 1 || p->d < 8 || p->d % 8 || p->d > kMaxD) return NYS_ERR_SHAPE;
  return NYS_OK;
}

// f(TPR, V) for a row of d channels: one vector per thread until a row has 1024
// threads; backward (MORE), whose threads also carry the weight's sums, two, and one
// where a warp then holds a row. Forward to 8 bits, 65536 x 2048: 160 us with two,
// 149 with one; backward, 16384 x 4096: 91 us with two, 95 with one.
template <bool MORE, typename F>
auto by_width(int d, F&& f) {
  using std::integral_constant;
  constexpr int V = MORE ? 2 : 1;
  const int units = (d + 8 * V - 1) / (8 * V);
  if (MORE && d <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (units <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, V>{});
  if (units <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, V>{});
  if (units <= 128) return f(integral_constant<int, 128>{}, integral_constant<int, V>{});
  if (units <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, V>{});
  if (units <= 512) return f(integral_constant<int, 512>{}, integral_constant<int, V>{});
  return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}
// CTAs: one per group of rows until the GPU is full.
int grid_of(int rows, int groups, int ctas_per_sm) {
  const long long want = ((long long)rows + groups - 1) / groups, most = (long long)plan_sms() * ctas_per_sm;
  return (int)(want < most ? want : most);
}

// Threads of a CTA: as many warps as a row has vectors for, where it has one row.
template <int TPR, int V>
int cta_threads(int d) {
  return TPR < 256 ? 256 : ((d + 8 * V - 1) / (8 * V) + 31) / 32 * 32;
}
template <int TPR, int V>
int back_grid(const nys_add_rms_norm_t& a) {
  return grid_of(a.rows, threads_of(TPR) / TPR, bwd_ctas(cta_threads<TPR, V>(a.d)));
}

int back_ctas(const nys_add_rms_norm_t& a) {
  return by_width<true>(a.d, [&](auto tpr, auto v) { return back_grid<decltype(tpr)::value, decltype(v)::value>(a); });
}

NormParams params_of(const nys_add_rms_norm_t& a) {
  NormParams p{};
  p.x = a.x;
  p.r = a.residual;
  p.s = a.sum;
  p.y = a.y;
  p.gs = a.gs;
  p.dx = a.dx;
  p.rows = a.rows;
  p.d = a.d;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)a.d;
  return p;
}

template <typename T>
int launch_fwd(const nys_add_rms_norm_t& a, const void* x, const void* res, const float* weight, void* sum,
               void* y, const nys_q8_t* y8, cudaStream_t st) {
  NormParams p = params_of(a);
  if (y8) {
    p.codes = static_cast<uint8_t*>(y8->codes);
    p.scales = static_cast<uint8_t*>(y8->scales);
    p.y = y8->stride;
  }
  return by_width<false>(a.d, [&](auto tpr, auto v) {
    constexpr int TPR = decltype(tpr)::value, V = decltype(v)::value, THREADS = threads_of(TPR);
    const int threads = cta_threads<TPR, V>(a.d);
    auto go = [&](auto kernel, int per_sm) {
      const int grid = grid_of(a.rows, THREADS / TPR, per_sm / threads);
      return launch_behind("add_rms_norm", kernel, dim3(grid), dim3(threads), 0, st, p, static_cast<const T*>(x),
                           static_cast<const T*>(res), weight, static_cast<T*>(sum), static_cast<T*>(y));
    };
    constexpr int with = fwd_threads<T, TPR, true>(), without = fwd_threads<T, TPR, false>();
    if (res)
      return y8 ? go(add_rms_norm<T, TPR, V, true, true>, with) : go(add_rms_norm<T, TPR, V, false, true>, with);
    return y8 ? go(add_rms_norm<T, TPR, V, true, false>, without) : go(add_rms_norm<T, TPR, V, false, false>, without);
  });
}

template <typename T>
int launch_bwd(const nys_add_rms_norm_t& a, const void* s, const void* gy, const void* gs, const float* weight,
               void* dx, float* part, int* status, cudaStream_t st) {
  NormParams p = params_of(a);
  p.status = status;
  return by_width<true>(a.d, [&](auto tpr, auto v) {
    constexpr int TPR = decltype(tpr)::value, V = decltype(v)::value, THREADS = threads_of(TPR);
    constexpr int GROUPS = THREADS / TPR;
    const int threads = cta_threads<TPR, V>(a.d);
    auto go = [&](auto kernel, size_t smem) {
      if (smem > 32 * 1024) {  // 48 KB with what is static
        const int rc = allow_shared(reinterpret_cast<const void*>(kernel), smem);
        if (rc != NYS_OK) return rc;
      }
      return launch_behind("add_rms_norm_back", kernel, dim3(back_grid<TPR, V>(a)), dim3(threads), smem, st, p,
                           static_cast<const T*>(s), static_cast<const T*>(gy), static_cast<const T*>(gs), weight,
                           static_cast<T*>(dx), part);
    };
    if (TPR >= 256) {  // as many rows as the CTAs of an SM have room for: one of 16384 in fp32
      const size_t slot = (size_t)(gs ? 3 : 2) * a.d * sizeof(T), room = 220 * 1024 / bwd_ctas(threads);
      p.ring = (int)(room / slot < kMostRing ? room / slot : kMostRing);
      return go(add_rms_norm_back<T, TPR, V>, p.ring * slot);
    }
    // at most 16 KB
    return go(add_rms_norm_back<T, TPR, V>, GROUPS > 1 && part ? (size_t)GROUPS * a.d * sizeof(float) : 0);
  });
}

// The same address means the same rows: one stride, or one row.
bool apart_or_same(const void* out, long long os, const void* in, long long is, int rows) {
  return out != in || rows == 1 || os == is;
}

}  // namespace
}  // namespace nys

using namespace nys;

extern "C" {

int nystrom_add_rms_norm_fwd(const nys_add_rms_norm_t* p, const void* x, const void* residual,
                             const float* weight, void* sum, void* y, const nys_q8_t* y8,
                             nys_stream_t stream) {
  int rc = check_common(p);
  if (rc != NYS_OK) return rc;
  if (!x || (y == nullptr) == (y8 == nullptr) || (sum && !residual)) return NYS_ERR_ARG;
  auto rows = [&](const void* at, long long stride, bool out) {
    return at ? q8::check_rows(at, stride, p->rows, p->d, p->dtype, out) : NYS_OK;
  };
  if ((rc = rows(x, p->x, false)) != NYS_OK || (rc = rows(residual, p->residual, false)) != NYS_OK ||
      (rc = rows(sum, p->sum, true)) != NYS_OK || (rc = rows(y, p->y, true)) != NYS_OK)
    return rc;
  if (y8) {
    if ((rc = q8::check_q8(y8, true)) != NYS_OK) return rc;
    if (y8->rows != p->rows || y8->K != p->d) return NYS_ERR_SHAPE;
    for (const void* other : {x, residual, static_cast<const void*>(sum), static_cast<const void*>(weight)})
      if (other && (y8->codes == other || y8->scales == other)) return NYS_ERR_ARG;
  }
  if (reinterpret_cast<uintptr_t>(weight) & 3u) return NYS_ERR_ALIGN;
  if (sum && sum == y) return NYS_ERR_ARG;
  if (weight && (sum == weight || y == weight)) return NYS_ERR_ARG;
  if ((sum && (!apart_or_same(sum, p->sum, x, p->x, p->rows) ||
               !apart_or_same(sum, p->sum, residual, p->residual, p->rows))) ||
      (y && (!apart_or_same(y, p->y, x, p->x, p->rows) ||
             (residual && !apart_or_same(y, p->y, residual, p->residual, p->rows)))))
    return NYS_ERR_ARG;
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  return p->dtype == NYS_BF16 ? launch_fwd<__nv_bfloat16>(*p, x, residual, weight, sum, y, y8, stream)
                              : launch_fwd<float>(*p, x, residual, weight, sum, y, y8, stream);
}

size_t nystrom_add_rms_norm_workspace_bytes(const nys_add_rms_norm_t* p) {
  if (check_common(p) != NYS_OK) return 0;
  return ((size_t)back_ctas(*p) * p->d * sizeof(float) + 255) & ~size_t(255);
}

int nystrom_add_rms_norm_bwd(const nys_add_rms_norm_t* p, const void* s, const void* gy, const void* gs,
                             const float* weight, void* dx, float* dweight, void* workspace,
                             size_t ws_bytes, nys_stream_t stream) {
  int rc = check_common(p);
  if (rc != NYS_OK) return rc;
  if (!s || !gy || !dx) return NYS_ERR_ARG;
  auto rows = [&](const void* at, long long stride, bool out) {
    return at ? q8::check_rows(at, stride, p->rows, p->d, p->dtype, out) : NYS_OK;
  };
  if ((rc = rows(s, p->sum, false)) != NYS_OK || (rc = rows(gy, p->y, false)) != NYS_OK ||
      (rc = rows(gs, p->gs, false)) != NYS_OK || (rc = rows(dx, p->dx, true)) != NYS_OK)
    return rc;
  if ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(dweight)) & 3u) return NYS_ERR_ALIGN;
  if (dx == s || !apart_or_same(dx, p->dx, gy, p->y, p->rows) ||
      (gs && !apart_or_same(dx, p->dx, gs, p->gs, p->rows)))
    return NYS_ERR_ARG;
  if (dweight && (dweight == weight || dweight == dx || dweight == s || dweight == gy || dweight == gs))
    return NYS_ERR_ARG;
  const size_t need = dweight ? nystrom_add_rms_norm_workspace_bytes(p) : 0;
  if (dweight && workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return NYS_ERR_ALIGN;
    if (ws_bytes < need) return NYS_ERR_NOMEM;
  }
  int dev = 0;
  rc = check_device(&dev);
  if (rc != NYS_OK) return rc;
  OperatorWorkspace own;
  if (dweight && !workspace) {
    rc = own.take(dev, need, stream, &workspace);
    if (rc != NYS_OK) return rc;
  }
  float* part = dweight ? static_cast<float*>(workspace) : nullptr;
  int* status = nullptr;
  if ((rc = operator_status(dev, &status)) != NYS_OK) return rc;
  rc = p->dtype == NYS_BF16 ? launch_bwd<__nv_bfloat16>(*p, s, gy, gs, weight, dx, part, status, stream)
                            : launch_bwd<float>(*p, s, gy, gs, weight, dx, part, status, stream);
  if (rc != NYS_OK || !dweight) return rc;
  return launch_behind("norm_weight_grad", norm_weight_grad, dim3((p->d + 31) / 32), dim3(1024), 0, stream,
                       static_cast<const float*>(part), dweight, p->d, back_ctas(*p));
}

}  // extern "C"
