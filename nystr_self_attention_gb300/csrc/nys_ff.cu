// The gated feed-forward product and its gradients (declared in
// include/nystrom.h):
//   g = x W_gate, u = x W_up, h = act(g) u
//   dg = gh u act'(g), du = gh act(g)
//   dx = dg W_gate^T + du W_up^T, dW_gate = x^T dg, dW_up = x^T du
// The products run in nys_gemm.h's kernel. Forward, a tile's 256 columns are 128
// of the gate and the same 128 of the other projection, so the lane that holds
// g holds u, and neither is written unless it is kept. Backward, one pass over
// g, u and gh makes dg and du; dx is one product whose K runs over both, and both
// weight gradients are one launch. Every operand is read as it lies: the weights
// in either order, x and dg turned.
//
// Up to 128 tokens the weights are the 128-row operand and the tokens the short
// one, with K split over the SMs and the partial sums joined (and gated there):
// the weights then stream at HBM's pace.
//
// fp32, up to 24 tokens: on the CUDA cores (nys_few.cu), but for the gradients of
// the weights. More: an operand is split into three bf16 terms, 24 bits in all, in a
// pass of its own, and the product sums the six pairs that matter at 2^-24. bf16: dg
// and du enter the products rounded to bf16, an error as large as the results' own
// rounding; of few tokens, where nothing averages it and the weights' bytes bound
// the time, as two terms (16 bits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>


#include "nys_gemm.h"
#include "nys_q8.h"

namespace nys {
namespace {

using namespace nys::gemm;

// ------------------------------------------------- terms of fp32 operands

__device__ __forceinline__ void three_terms(float x, float (&t)[3]) {
  t[0] = __bfloat162float(__float2bfloat16_rn(x));
  const float r = x - t[0];
  t[1] = __bfloat162float(__float2bfloat16_rn(r));
  t[2] = r - t[1];
}
__device__ __forceinline__ void store_terms(__nv_bfloat16* to, long long plane, const float (&v)[8]) {
  float t[8][3];
#pragma unroll
  for (int i = 0; i < 8; ++i) three_terms(v[i], t[i]);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<uint4*>(to + k * plane) =
        make_uint4(pack_bf16x2(t[0][k], t[1][k]), pack_bf16x2(t[2][k], t[3][k]), pack_bf16x2(t[4][k], t[5][k]),
                   pack_bf16x2(t[6][k], t[7][k]));
}

__device__ __forceinline__ void store8(float* to, const float (&v)[8]) {
  reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_bf16(__nv_bfloat16* to, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(to) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// What rounding to bf16 left (nothing of an infinity or a NaN).
__device__ __forceinline__ void rest_of(float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = v[i] - __bfloat162float(__float2bfloat16_rn(v[i]));
    v[i] = r - r == 0.f ? r : 0.f;
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Matrices to split: x [rows][cols] -> terms [3][rows][cols], eight elements per
// thread, each matrix by a range of a launch's CTAs.
struct Splits {
  struct One {
    const float* x;
    __nv_bfloat16* terms;
    long long stride, rows;
    int cols;
    unsigned end;  // CTAs up to and with this matrix's
  } one[3];
  int count;
  void add(const void* x, long long stride, void* terms, long long rows, int cols) {
    const unsigned start = ctas();
    one[count++] = One{static_cast<const float*>(x), static_cast<__nv_bfloat16*>(terms), stride, rows, cols,
                       start + (unsigned)((rows * (cols / 8) + 255) / 256)};
  }
  unsigned ctas() const { return count ? one[count - 1].end : 0u; }
};
__device__ __forceinline__ void split_matrix(const Splits& p, unsigned cta) {
  int i = 0;
  while (cta >= p.one[i].end) ++i;
  const Splits::One& m = p.one[i];
  const int units = m.cols / 8;
  const long long e = (long long)(cta - (i ? p.one[i - 1].end : 0u)) * 256 + threadIdx.x, r = e / units;
  if (r >= m.rows) return;
  const int c = (int)(e - r * units) * 8;
  float v[8];
  load8(m.x + r * m.stride + c, v);
  store_terms(m.terms + r * m.cols + c, m.rows * m.cols, v);
}
__global__ void __launch_bounds__(256) split_terms(const __grid_constant__ Splits p) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  split_matrix(p, blockIdx.x);
}

// ------------------------------------------------------- dg and du

struct GradParams {
  long long g, u, h;  // row strides
  long long T;
  int f;
  unsigned ctas;  // those behind split the matrices of `more`
  int two;        // bf16: two terms
  float *dg32, *du32;  // fp32: as they are, too, or null
};

// dg, du as terms [1, 2 or (fp32) 3][T][f]. Eight elements per thread.
template <typename T, int ACT>
__global__ void __launch_bounds__(256)
gated_ff_back(const __grid_constant__ GradParams p, const __grid_constant__ Splits more, const T* __restrict__ gate,
              const T* __restrict__ up, const T* __restrict__ gh, __nv_bfloat16* __restrict__ dg,
              __nv_bfloat16* __restrict__ du) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  if (sizeof(T) == 4 && blockIdx.x >= p.ctas) {
    split_matrix(more, blockIdx.x - p.ctas);
    return;
  }
  const int units = p.f / 8;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x, r = e / units;
  if (r >= p.T) return;
  const int c = (int)(e - r * units) * 8;
  float g[8], u[8], h[8];
  load8(gate + r * p.g + c, g);
  load8(up + r * p.u + c, u);
  load8(gh + r * p.h + c, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, slope;
    act::with_slope<ACT, sizeof(T) == 2>(g[i], a, slope);
    g[i] = h[i] * u[i] * slope;
    u[i] = h[i] * a;
  }
  const long long at = r * p.f + c;
  if (sizeof(T) == 4) {
    store_terms(dg + at, p.T * p.f, g);
    store_terms(du + at, p.T * p.f, u);
    if (p.dg32) {
      store8(p.dg32 + at, g);
      store8(p.du32 + at, u);
    }
  } else {
    store_bf16(dg + at, g);
    store_bf16(du + at, u);
    if (p.two) {
      rest_of(g);
      rest_of(u);
      store_bf16(dg + p.T * p.f + at, g);
      store_bf16(du + p.T * p.f + at, u);
    }
  }
}

// ------------------------------------------------------------------ plans

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// One launch of the products: `parts` results [M][N], K = k_parts x k.
struct Product {
  bool turned;  // D is the result's transpose: its N are the 128-row operand's rows
  int range;    // on the CUDA cores (nys_few.cu): K's range; 0: on the tensor cores
  int bn, splits, its, its_per_split, k_blocks, m_tiles, n_tiles;
  Line line;     // turned
  size_t bytes;  // of partial sums
};

Product product_of(long long M, long long N, long long k, int k_parts, int parts, int pairs, bool gated,
                   bool may_turn) {
  Product q{};
  q.turned = may_turn && M <= kMostTokens;
  q.k_blocks = (int)((k + 63) / 64);
  const int steps = q.k_blocks * k_parts;
  q.its = steps * pairs;
  if (q.turned) {
    q.bn = columns_of((int)M);
    q.line = line_of(N, q.its, parts, pairs > 2 ? pairs : 2, q.bn);
    q.splits = most_planes(q.line);
    q.m_tiles = q.line.m_tiles;
    q.n_tiles = 1;
    q.bytes = align256((size_t)q.splits * parts * N * q.bn * 4);
    return q;
  }
  const Cut cut = cut_pair(M, N, steps, 1, pairs, parts, 256, gated ? 64 : 32, gated, pairs > 2 ? 1 : 4);
  q.bn = cut.bn;
  q.splits = cut.splits;
  q.its_per_split = range_of(steps, q.splits, 1) * pairs;  // all pairs of a block
  const int width = gated && q.splits == 1 ? q.bn / 2 : q.bn;  // of each part
  q.m_tiles = (int)((M + 255) / 256);
  q.n_tiles = (int)((N + width - 1) / width);
  if (q.splits > 1) q.bytes = align256((size_t)q.splits * parts * M * N * 4);
  return q;
}

// Few tokens in fp32, on the CUDA cores.
Product few_of(long long T, long long N, long long K, bool k_contiguous) {
  Product q{};
  q.range = few_range((int)T, (int)N, (int)K, k_contiguous);
  q.splits = (int)((K + q.range - 1) / q.range);
  q.bytes = align256((size_t)q.splits * 2 * T * N * 4);
  return q;
}

struct Plan {
  bool f32, few;
  int pairs;       // of the forward product
  int grad_terms;  // of dg and du: 1, 2 (few tokens), or fp32's 3
  int grad_pairs;  // products summed for a gradient
  Product fwd, dx, dw;
  // byte offsets in the workspace
  size_t x, wg, wu, dg, du, dg32, du32, part, total;
};

Plan plan_of(const nys_gated_ff_t& a, bool back, bool want_dx, bool want_dw) {
  Plan pl{};
  pl.f32 = a.dtype == NYS_FP32;
  pl.pairs = pl.f32 ? 6 : 1;
  pl.few = pl.f32 && a.T <= kMostFew;
  pl.grad_terms = pl.f32 ? 3 : a.T <= kMostTokens ? 2 : 1;
  pl.grad_pairs = pl.f32 ? 6 : pl.grad_terms;
  const size_t T = a.T, d = a.d, f = a.f;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align256(bytes); return o; };
  const bool io = a.layout == NYS_FF_IN_OUT;
  size_t part = 0;
  if (pl.f32 && (back ? want_dw : !pl.few)) pl.x = take(3 * T * d * 2);
  if (pl.f32 && !pl.few && (!back || want_dx)) {
    pl.wg = take(3 * d * f * 2);
    pl.wu = take(3 * d * f * 2);
  }
  if (!back) {
    pl.fwd = pl.few ? few_of(a.T, a.f, a.d, !io) : product_of(a.T, a.f, a.d, 1, 2, pl.pairs, true, true);
    part = pl.fwd.bytes;
  } else {
    pl.dg = take(pl.grad_terms * T * f * 2);
    pl.du = take(pl.grad_terms * T * f * 2);
    if (want_dx) {
      pl.dx = pl.few ? few_of(a.T, a.d, a.f, io) : product_of(a.T, a.d, a.f, 2, 1, pl.grad_pairs, false, true);
      if (pl.few) {
        pl.dg32 = take(T * f * 4);
        pl.du32 = take(T * f * 4);
      }
      part = pl.dx.bytes;
    }
    if (want_dw) {
      pl.dw = product_of(io ? a.d : a.f, io ? a.f : a.d, a.T, 1, 2, pl.grad_pairs, false, false);
      if (pl.dw.bytes > part) part = pl.dw.bytes;
    }
  }
  pl.part = take(part);
  pl.total = off;
  return pl;
}

int check_common(const nys_gated_ff_t* p) {
  if (!p) return NYS_ERR_ARG;
  if (p->dtype != NYS_FP32 && p->dtype != NYS_BF16) return NYS_ERR_ARG;
  if (p->act < NYS_ACT_SILU || p->act > NYS_ACT_RELU) return NYS_ERR_ARG;
  if (p->layout != NYS_FF_IN_OUT && p->layout != NYS_FF_OUT_IN) return NYS_ERR_ARG;
  if (p->T < 1 || p->T > (1 << 30) || p->d < 8 || p->f < 8 || p->d % 8 || p->f % 8 || p->d > (1 << 20) ||
      p->f > (1 << 20))
    return NYS_ERR_SHAPE;
  // sizes of the launches stay in 32 bits, those of arrays far from 64
  const long long T = p->T, d = p->d, f = p->f, most = 1ll << 44;
  if (T * d >= most || T * f >= most || (T / 128 + 1) * (f / 128 + 1) >= (1ll << 26) ||
      (T / 128 + 1) * (d / 128 + 1) >= (1ll << 26) || (d / 128 + 1) * (f / 128 + 1) >= (1ll << 25) ||
      (T / 8) * f >= (1ll << 37) || (T / 8) * d >= (1ll << 37))
    return NYS_ERR_SHAPE;
  return NYS_OK;
}

// ----------------------------------------------------------------- launches

// a_terms, b_terms: how many each operand has.
Params params_of(const Product& q, int parts, int a_terms, int b_terms, int a_by, int b_by, int* status) {
  Params p{};
  const int pairs = a_terms == 3 ? 6 : a_terms > b_terms ? a_terms : b_terms;
  if (pairs == 6) p.a_terms = kTermsA, p.b_terms = kTermsB;
  if (pairs == 2) (a_terms == 2 ? p.a_terms : p.b_terms) = 0x01;  // the small one first

  p.m_tiles = q.m_tiles;
  p.n_tiles = q.n_tiles;
  p.parts = parts;
  p.splits = q.splits;
  p.k_blocks = q.k_blocks;
  p.its = q.its;
  p.its_per_split = q.its_per_split;
  p.pairs = pairs;
  p.bn = q.bn;
  p.unit = pairs > 2 ? pairs : 2;
  p.units = q.line.units;
  p.chunk = pairs > 2 ? pairs : kLongest;  // fp32: the six products of a K block
  p.a_by = a_by;
  p.b_by = b_by;
  p.group = 16;
  p.status = status;
  return p;
}

// The turned form: weights (k contiguous, or turned themselves) x tokens.
int launch_turned(const char* name, bool amn, const Product& q, const Maps& maps, const Params& p, cudaStream_t st) {
  return amn ? launch_tokens<kBf16, true>(name, q.bn, q.line.ctas, maps, p, st)
             : launch_tokens<kBf16, false>(name, q.bn, q.line.ctas, maps, p, st);
}

// Results, or (wide) fp32 results or partial sums, in rows.
template <bool AMN, bool BMN>
int launch_plain(const char* name, bool wide, const Maps& maps, const Params& p, cudaStream_t st) {
  return wide ? launch_pair<kBf16, AMN, BMN, kPlain, float>(name, maps, p, st)
              : launch_pair<kBf16, AMN, BMN, kPlain, __nv_bfloat16>(name, maps, p, st);
}

// Operand of `rows` lines of `k`, or stored [k][rows] (mn): as it lies, or in terms.
Matrix operand(const void* at, long long rows, long long cols, long long stride, int terms) {
  return terms > 1 ? Matrix{at, rows, cols, cols, 2, terms, rows * cols} : Matrix{at, rows, cols, stride, 2};
}

int forward(const nys_gated_ff_t& a, const Plan& pl, const void* x, const void* wg, const void* wu, void* h,
            void* gate, void* up, char* ws, int* status, cudaStream_t st) {
  const bool io = a.layout == NYS_FF_IN_OUT;
  int rc;
  if (pl.few) {
    Few w{};
    w.x[0] = w.x[1] = static_cast<const float*>(x);
    w.w[0] = static_cast<const float*>(wg);
    w.w[1] = static_cast<const float*>(wu);
    w.x_stride = a.x;
    w.w_stride = a.w;
    w.part = reinterpret_cast<float*>(ws + pl.part);
    w.T = a.T;
    w.N = a.f;
    w.K = a.d;
    w.range = pl.fwd.range;
    if ((rc = launch_few("gated_ff_few", w, !io, st)) != NYS_OK) return rc;
    const JoinGated j{w.part, pl.fwd.splits, a.T, a.f, Line{}, h, gate, up, a.h, a.gate, a.up};
    return join_gated(j, a.act, a.dtype, st);
  }
  if (pl.f32) {
    const int wr = io ? a.d : a.f, wc = io ? a.f : a.d;
    Splits m{};
    m.add(x, a.x, ws + pl.x, a.T, a.d);
    m.add(wg, a.w, ws + pl.wg, wr, wc);
    m.add(wu, a.w, ws + pl.wu, wr, wc);
    if ((rc = launch_behind("split_terms", split_terms, dim3(m.ctas()), dim3(256), 0, st, m)) != NYS_OK) return rc;
    x = ws + pl.x;
    wg = ws + pl.wg;
    wu = ws + pl.wu;
  }
  const Product& q = pl.fwd;
  const bool direct = !q.turned && q.splits == 1;
  const int terms = pl.f32 ? 3 : 1;
  Params p = params_of(q, direct ? 1 : 2, terms, terms, q.turned ? kByPart : kOnly, q.turned ? kOnly : kByPart, status);
  p.act = a.act;
  p.keep = gate != nullptr;
  Maps maps{};
  const Matrix xm = operand(x, a.T, a.d, a.x, terms);
  const Matrix w[2] = {operand(wg, io ? a.d : a.f, io ? a.f : a.d, a.w, terms),
                       operand(wu, io ? a.d : a.f, io ? a.f : a.d, a.w, terms)};
  bool ok = true;
  if (q.turned) {
    for (int i = 0; i < 2; ++i) ok = ok && (io ? map_mn(&maps.a[i], w[i]) : map_k(&maps.a[i], w[i], 128));
    ok = ok && map_k(&maps.b[0], xm, q.bn) &&
         map_out(&maps.c[0], Matrix{ws + pl.part, a.f, q.bn, q.bn, 4, 2 * q.splits, (long long)a.f * q.bn},
                 q.bn == 16 ? 16 : 32);
  } else {
    ok = map_k(&maps.a[0], xm, 128);
    for (int i = 0; i < 2; ++i)
      ok = ok && (io ? map_mn(&maps.b[i], w[i]) : map_k(&maps.b[i], w[i], q.bn / 2));
    if (direct) {
      const int e = pl.f32 ? 4 : 2;
      ok = ok && map_out(&maps.c[0], Matrix{h, a.T, a.f, a.h, e});
      if (gate)
        ok = ok && map_out(&maps.c[1], Matrix{gate, a.T, a.f, a.gate, e}) &&
             map_out(&maps.c[2], Matrix{up, a.T, a.f, a.up, e});
    } else {
      ok = ok && map_out(&maps.c[0], Matrix{ws + pl.part, a.T, a.f, a.f, 4, 2 * q.splits, (long long)a.T * a.f});
    }
  }
  if (!ok) return tensor_map_error(__FILE__, __LINE__);
  if (q.turned) {
    rc = launch_turned("gated_ff_tokens", io, q, maps, p, st);
  } else if (!direct) {
    rc = io ? launch_plain<false, true>("gated_ff_split", true, maps, p, st)
            : launch_plain<false, false>("gated_ff_split", true, maps, p, st);
  } else if (pl.f32) {
    rc = io ? launch_pair<kBf16, false, true, kGated, float>("gated_ff", maps, p, st)
            : launch_pair<kBf16, false, false, kGated, float>("gated_ff", maps, p, st);
  } else {
    rc = io ? launch_pair<kBf16, false, true, kGated, __nv_bfloat16>("gated_ff", maps, p, st)
            : launch_pair<kBf16, false, false, kGated, __nv_bfloat16>("gated_ff", maps, p, st);
  }
  if (rc != NYS_OK || direct) return rc;
  const JoinGated j{reinterpret_cast<const float*>(ws + pl.part), q.splits, a.T, a.f, q.line, h, gate, up, a.h, a.gate,
                    a.up};
  return join_gated(j, a.act, a.dtype, st);
}

// dx = dg W_gate^T + du W_up^T: K runs over the features of both.
int input_gradient(const nys_gated_ff_t& a, const Plan& pl, const void* wg, const void* wu, void* dx, char* ws,
                   int* status, cudaStream_t st) {
  const bool io = a.layout == NYS_FF_IN_OUT;
  const Product& q = pl.dx;
  if (q.range) {
    Few w{};
    w.x[0] = reinterpret_cast<const float*>(ws + pl.dg32);
    w.x[1] = reinterpret_cast<const float*>(ws + pl.du32);
    w.w[0] = static_cast<const float*>(wg);
    w.w[1] = static_cast<const float*>(wu);
    w.x_stride = a.f;
    w.w_stride = a.w;
    w.part = reinterpret_cast<float*>(ws + pl.part);
    w.T = a.T;
    w.N = a.d;
    w.K = a.f;
    w.range = q.range;
    const int rc = launch_few("gated_ff_few", w, io, st);
    if (rc != NYS_OK) return rc;
    const Join j{w.part, 2 * q.splits, a.T, a.d, Line{}, {dx, nullptr}, {a.dx, 0}};
    return join(j, 1, a.dtype, st);
  }
  const bool direct = !q.turned && q.splits == 1;
  const int terms = pl.f32 ? 3 : 1;  // of the weights
  const Params p = params_of(q, 1, q.turned ? terms : pl.grad_terms, q.turned ? pl.grad_terms : terms, kByKPart, kByKPart,
                             status);
  Maps maps{};
  const Matrix g[2] = {operand(ws + pl.dg, a.T, a.f, a.f, pl.grad_terms),
                       operand(ws + pl.du, a.T, a.f, a.f, pl.grad_terms)};
  const Matrix w[2] = {operand(wg, io ? a.d : a.f, io ? a.f : a.d, a.w, terms),
                       operand(wu, io ? a.d : a.f, io ? a.f : a.d, a.w, terms)};
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    CUtensorMap &wm = q.turned ? maps.a[i] : maps.b[i], &gm = q.turned ? maps.b[i] : maps.a[i];
    ok = ok && (io ? map_k(&wm, w[i], q.turned ? 128 : q.bn / 2) : map_mn(&wm, w[i])) &&
         map_k(&gm, g[i], q.turned ? q.bn : 128);
  }
  char* part = ws + pl.part;
  if (direct)
    ok = ok && map_out(&maps.c[0], Matrix{dx, a.T, a.d, a.dx, pl.f32 ? 4 : 2});
  else if (q.turned)
    ok = ok && map_out(&maps.c[0], Matrix{part, a.d, q.bn, q.bn, 4, q.splits, (long long)a.d * q.bn}, q.bn == 16 ? 16 : 32);
  else
    ok = ok && map_out(&maps.c[0], Matrix{part, a.T, a.d, a.d, 4, q.splits, (long long)a.T * a.d});
  if (!ok) return tensor_map_error(__FILE__, __LINE__);
  int rc;
  const char* name = "gated_ff_dx";
  if (q.turned)
    rc = launch_turned(name, !io, q, maps, p, st);
  else
    rc = io ? launch_plain<false, false>(name, pl.f32 || !direct, maps, p, st)
            : launch_plain<false, true>(name, pl.f32 || !direct, maps, p, st);
  if (rc != NYS_OK || direct) return rc;
  const Join j{reinterpret_cast<const float*>(part), q.splits, a.T, a.d, q.line, {dx, nullptr}, {a.dx, 0}};
  return join(j, 1, a.dtype, st);
}

// x^T dg and x^T du, or (weights [f][d]) their transposes.
int weight_gradients(const nys_gated_ff_t& a, const Plan& pl, const void* x, void* dwg, void* dwu, char* ws,
                     int* status, cudaStream_t st) {
  const bool io = a.layout == NYS_FF_IN_OUT;
  const Product& q = pl.dw;
  const bool direct = q.splits == 1;
  const int M = io ? a.d : a.f, N = io ? a.f : a.d;
  const int terms = pl.f32 ? 3 : 1;  // of x
  Params p = params_of(q, 2, io ? terms : pl.grad_terms, io ? pl.grad_terms : terms, io ? kOnly : kByPart,
                       io ? kByPart : kOnly, status);
  p.c_by_part = direct;
  Maps maps{};
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    CUtensorMap &xm = io ? maps.a[i] : maps.b[i], &gm = io ? maps.b[i] : maps.a[i];
    ok = ok && map_mn(&xm, operand(x, a.T, a.d, a.x, terms)) &&
         map_mn(&gm, operand(ws + (i ? pl.du : pl.dg), a.T, a.f, a.f, pl.grad_terms));
    if (direct) ok = ok && map_out(&maps.c[i], Matrix{i ? dwu : dwg, M, N, a.dw, pl.f32 ? 4 : 2});
  }
  char* part = ws + pl.part;
  if (!direct) ok = ok && map_out(&maps.c[0], Matrix{part, M, N, N, 4, 2 * q.splits, (long long)M * N});
  if (!ok) return tensor_map_error(__FILE__, __LINE__);
  const char* name = "gated_ff_dw";
  const int rc = launch_plain<true, true>(name, pl.f32 || !direct, maps, p, st);
  if (rc != NYS_OK || direct) return rc;
  const Join j{reinterpret_cast<const float*>(part), q.splits, M, N, q.line, {dwg, dwu}, {a.dw, a.dw}};
  return join(j, 2, a.dtype, st);
}

template <typename T>
int launch_grads(const nys_gated_ff_t& a, const Plan& pl, const void* gate, const void* up, const void* gh,
                 const Splits& more, char* ws, cudaStream_t st) {
  const GradParams p{a.gate, a.up, a.h, a.T, a.f, (unsigned)(((long long)a.T * (a.f / 8) + 255) / 256),
                     pl.grad_terms == 2, pl.dx.range ? reinterpret_cast<float*>(ws + pl.dg32) : nullptr,
                     pl.dx.range ? reinterpret_cast<float*>(ws + pl.du32) : nullptr};
  return act::by_act(a.act, [&](auto k) {
    return launch_behind("gated_ff_back", gated_ff_back<T, decltype(k)::value>, dim3(p.ctas + more.ctas()), dim3(256),
                         0, st, p, more, static_cast<const T*>(gate), static_cast<const T*>(up),
                         static_cast<const T*>(gh), reinterpret_cast<__nv_bfloat16*>(ws + pl.dg),
                         reinterpret_cast<__nv_bfloat16*>(ws + pl.du));
  });
}

// Whether an address is any of the others.
template <typename... P>
bool among(const void* p, P... others) {
  return p && ((p == others) || ...);
}

}  // namespace
}  // namespace nys

using namespace nys;

extern "C" {

size_t nystrom_gated_ff_workspace_bytes(const nys_gated_ff_t* p, int back) {
  if (check_common(p) != NYS_OK || (back != 0 && back != 1)) return 0;
  return plan_of(*p, back != 0, true, true).total;
}

int nystrom_gated_ff_fwd(const nys_gated_ff_t* p, const void* x, const void* w_gate, const void* w_up, void* h,
                         void* gate, void* up, void* workspace, size_t ws_bytes, nys_stream_t stream) {
  int rc = check_common(p);
  if (rc != NYS_OK) return rc;
  if (!x || !w_gate || !w_up || !h || (gate == nullptr) != (up == nullptr)) return NYS_ERR_ARG;
  const bool io = p->layout == NYS_FF_IN_OUT;
  const int wr = io ? p->d : p->f, wc = io ? p->f : p->d;
  auto rows = [&](const void* at, long long stride, int n, int width, bool apart) {
    return at ? q8::check_rows(at, stride, n, width, p->dtype, apart) : NYS_OK;
  };
  if ((rc = rows(x, p->x, p->T, p->d, true)) != NYS_OK || (rc = rows(w_gate, p->w, wr, wc, true)) != NYS_OK ||
      (rc = rows(w_up, p->w, wr, wc, true)) != NYS_OK || (rc = rows(h, p->h, p->T, p->f, true)) != NYS_OK ||
      (rc = rows(gate, p->gate, p->T, p->f, true)) != NYS_OK || (rc = rows(up, p->up, p->T, p->f, true)) != NYS_OK)
    return rc;
  if (among(h, x, w_gate, w_up, gate, up) || among(gate, x, w_gate, w_up, up) || among(up, x, w_gate, w_up))
    return NYS_ERR_ARG;
  const Plan pl = plan_of(*p, false, true, true);
  if (pl.total && workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return NYS_ERR_ALIGN;
    if (ws_bytes < pl.total) return NYS_ERR_NOMEM;
  }
  int dev = 0;
  if ((rc = check_device(&dev)) != NYS_OK || (rc = have_context(dev)) != NYS_OK) return rc;
  OperatorWorkspace own;
  if (pl.total && !workspace) {
    rc = own.take(dev, pl.total, stream, &workspace);
    if (rc != NYS_OK) return rc;
  }
  int* status = nullptr;
  if ((rc = operator_status(dev, &status)) != NYS_OK) return rc;
  return forward(*p, pl, x, w_gate, w_up, h, gate, up, static_cast<char*>(workspace), status, stream);
}

int nystrom_gated_ff_bwd(const nys_gated_ff_t* p, const void* x, const void* w_gate, const void* w_up,
                         const void* gate, const void* up, const void* gh, void* dx, void* dw_gate, void* dw_up,
                         void* workspace, size_t ws_bytes, nys_stream_t stream) {
  int rc = check_common(p);
  if (rc != NYS_OK) return rc;
  const bool want_dw = dw_gate != nullptr;
  if (!gate || !up || !gh || want_dw != (dw_up != nullptr) || (!dx && !want_dw) || (want_dw && !x) ||
      (dx && (!w_gate || !w_up)))
    return NYS_ERR_ARG;
  const bool io = p->layout == NYS_FF_IN_OUT;
  const int wr = io ? p->d : p->f, wc = io ? p->f : p->d;
  auto rows = [&](const void* at, long long stride, int n, int width, bool apart) {
    return at ? q8::check_rows(at, stride, n, width, p->dtype, apart) : NYS_OK;
  };
  if ((want_dw && (rc = rows(x, p->x, p->T, p->d, true)) != NYS_OK) ||
      (dx && ((rc = rows(w_gate, p->w, wr, wc, true)) != NYS_OK || (rc = rows(w_up, p->w, wr, wc, true)) != NYS_OK)) ||
      (rc = rows(gate, p->gate, p->T, p->f, false)) != NYS_OK || (rc = rows(up, p->up, p->T, p->f, false)) != NYS_OK ||
      (rc = rows(gh, p->h, p->T, p->f, false)) != NYS_OK || (rc = rows(dx, p->dx, p->T, p->d, true)) != NYS_OK ||
      (rc = rows(dw_gate, p->dw, wr, wc, true)) != NYS_OK || (rc = rows(dw_up, p->dw, wr, wc, true)) != NYS_OK)
    return rc;
  if (among(dx, x, w_gate, w_up, gate, up, gh, dw_gate, dw_up) ||
      among(dw_gate, x, w_gate, w_up, gate, up, gh, dw_up) || among(dw_up, x, w_gate, w_up, gate, up, gh))
    return NYS_ERR_ARG;
  const Plan pl = plan_of(*p, true, dx != nullptr, want_dw);
  if (workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return NYS_ERR_ALIGN;
    if (ws_bytes < pl.total) return NYS_ERR_NOMEM;
  }
  int dev = 0;
  if ((rc = check_device(&dev)) != NYS_OK || (rc = have_context(dev)) != NYS_OK) return rc;
  OperatorWorkspace own;
  if (!workspace) {
    rc = own.take(dev, pl.total, stream, &workspace);
    if (rc != NYS_OK) return rc;
  }
  int* status = nullptr;
  if ((rc = operator_status(dev, &status)) != NYS_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  const void *xs = x, *wg = w_gate, *wu = w_up;
  Splits more{};
  if (pl.f32 && want_dw) {
    more.add(x, p->x, ws + pl.x, p->T, p->d);
    xs = ws + pl.x;
  }
  if (pl.f32 && dx && !pl.few) {
    more.add(w_gate, p->w, ws + pl.wg, wr, wc);
    more.add(w_up, p->w, ws + pl.wu, wr, wc);
    wg = ws + pl.wg;
    wu = ws + pl.wu;
  }
  rc = pl.f32 ? launch_grads<float>(*p, pl, gate, up, gh, more, ws, stream)
              : launch_grads<__nv_bfloat16>(*p, pl, gate, up, gh, more, ws, stream);
  if (rc != NYS_OK) return rc;
  if (dx && (rc = input_gradient(*p, pl, wg, wu, dx, ws, status, stream)) != NYS_OK) return rc;
  return want_dw ? weight_gradients(*p, pl, xs, dw_gate, dw_up, ws, status, stream) : NYS_OK;
}

}  // extern "C"
