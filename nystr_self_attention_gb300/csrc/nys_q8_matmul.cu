// The product of two matrices in 8 bits (declared in include/nystrom.h):
// out[t][n] = sum over k of A[t][k] W[n][k]. The scales are powers of two, so the
// tensor cores' block-scaled form applies them exactly: one scale for four
// instructions of 32 channels, its byte named by the instruction, words of four
// blocks copied into TMEM as they are needed.
//
// Up to 128 tokens the weights are the 128-row operand and the tokens the short
// one (nothing is padded to 128 rows, so the weights stream at HBM's pace), K
// split so that every SM has an equal share; the partial sums are joined. More
// tokens are the rows themselves, in tiles of 256 x up to 224 by two CTAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>


#include "nys_gemm.h"
#include "nys_q8.h"

namespace nys {
namespace {

using namespace nys::gemm;

struct Q8Plan {
  bool turned;
  int bn, splits, its_per_split;
  Line line;
  size_t bytes;  // of partial sums
};

Q8Plan plan_of(int T, int N, int K) {
  Q8Plan q{};
  const int its = (K + 127) / 128;
  q.turned = T <= kMostTokens;
  if (q.turned) {
    q.bn = columns_of(T);
    q.line = line_of(N, its, 1, 2, q.bn);
    q.splits = most_planes(q.line);
    q.bytes = (size_t)q.splits * N * q.bn * 4;
  } else {
    const Cut cut = cut_pair(T, N, its, 4, 1, 1, 224, 32, false, 4);
    q.bn = cut.bn;
    q.splits = cut.splits;
    q.its_per_split = range_of(its, q.splits, 4);
    if (q.splits > 1) q.bytes = (size_t)q.splits * T * N * 4;
  }
  q.bytes = (q.bytes + 255) & ~size_t(255);
  return q;
}

int check_sizes(int T, int N, int K) {
  if (T < 1 || N < 1 || N % 8 || K < 1) return NYS_ERR_SHAPE;
  if ((long long)((T + 127) / 128) * ((N + 127) / 128) >= (1ll << 26)) return NYS_ERR_SHAPE;
  return NYS_OK;
}

Matrix codes_of(const nys_q8_t& q) { return Matrix{q.codes, q.rows, q.K, q.stride, 1}; }

}  // namespace
}  // namespace nys

using namespace nys;

extern "C" {

size_t nystrom_q8_matmul_workspace_bytes(int T, int N, int K, int dtype) {
  if ((dtype != NYS_FP32 && dtype != NYS_BF16) || check_sizes(T, N, K) != NYS_OK || K % 16 || K > (1 << 20))
    return 0;
  return plan_of(T, N, K).bytes;
}

int nystrom_q8_matmul(const nys_q8_t* a, const nys_q8_t* w, void* out, long long out_stride, int dtype,
                      void* workspace, size_t ws_bytes, nys_stream_t stream) {
  int rc;
  if ((rc = q8::check_q8(a, true)) != NYS_OK || (rc = q8::check_q8(w, true)) != NYS_OK) return rc;
  if (!out || (dtype != NYS_FP32 && dtype != NYS_BF16)) return NYS_ERR_ARG;
  if (a->K != w->K) return NYS_ERR_SHAPE;
  const int T = a->rows, N = w->rows, K = a->K;
  if ((rc = check_sizes(T, N, K)) != NYS_OK) return rc;
  if ((rc = q8::check_rows(out, out_stride, T, N, dtype, true)) != NYS_OK) return rc;
  if (out == a->codes || out == w->codes || out == a->scales || out == w->scales) return NYS_ERR_ARG;
  const Q8Plan plan = plan_of(T, N, K);
  if (plan.bytes && workspace) {
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return NYS_ERR_ALIGN;
    if (ws_bytes < plan.bytes) return NYS_ERR_NOMEM;
  }
  int dev = 0;
  if ((rc = check_device(&dev)) != NYS_OK || (rc = have_context(dev)) != NYS_OK) return rc;
  OperatorWorkspace own;
  if (plan.bytes && !workspace) {
    rc = own.take(dev, plan.bytes, stream, &workspace);
    if (rc != NYS_OK) return rc;
  }
  const nys_q8_t &rows = plan.turned ? *w : *a, &cols = plan.turned ? *a : *w;
  Params p{};
  if ((rc = operator_status(dev, &p.status)) != NYS_OK) return rc;
  p.m_tiles = plan.turned ? (rows.rows + 127) / 128 : (rows.rows + 255) / 256;
  p.n_tiles = plan.turned ? 1 : (cols.rows + plan.bn - 1) / plan.bn;
  p.parts = p.pairs = 1;
  p.splits = plan.splits;
  p.unit = 2;
  p.units = plan.line.units;
  p.k_blocks = p.its = (K + 127) / 128;
  p.its_per_split = plan.its_per_split;
  p.bn = plan.bn;
  p.group = 16;
  p.a_scales = static_cast<const uint32_t*>(rows.scales);
  p.b_scales = static_cast<const uint32_t*>(cols.scales);
  p.a_rows = rows.rows;
  p.b_rows = cols.rows;
  Maps maps{};
  bool ok = map_k(&maps.a[0], codes_of(rows), 128) && map_k(&maps.b[0], codes_of(cols), plan.turned ? plan.bn : plan.bn / 2);
  const bool direct = !plan.turned && plan.splits == 1;
  p.chunk = direct && dtype == NYS_BF16 ? kLongest : 8;
  if (direct)
    ok = ok && map_out(&maps.c[0], Matrix{out, T, N, out_stride, dtype == NYS_FP32 ? 4 : 2});
  else if (plan.turned)
    ok = ok && map_out(&maps.c[0], Matrix{workspace, N, plan.bn, plan.bn, 4, plan.splits, (long long)N * plan.bn},
                       plan.bn == 16 ? 16 : 32);
  else
    ok = ok && map_out(&maps.c[0], Matrix{workspace, T, N, N, 4, plan.splits, (long long)T * N});
  if (!ok) return tensor_map_error(__FILE__, __LINE__);
  const char* name = "q8_matmul";
  if (plan.turned)
    rc = launch_tokens<kMx8, false>(name, plan.bn, plan.line.ctas, maps, p, stream);
  else if (!direct || dtype == NYS_FP32)
    rc = launch_pair<kMx8, false, false, kPlain, float>(name, maps, p, stream);
  else
    rc = launch_pair<kMx8, false, false, kPlain, __nv_bfloat16>(name, maps, p, stream);
  if (rc != NYS_OK || direct) return rc;
  const Join j{static_cast<const float*>(workspace), plan.splits, T, N, plan.line, {out, nullptr},
               {out_stride, 0}};
  return join(j, 1, dtype, stream);
}

}  // extern "C"
