// Matrix products on the tensor cores for the operators around the attention
// module: D[m][n] = sum over k of A[m][k] B[n][k], accumulated in fp32 in TMEM.
//
// Two kernels, both persistent: a warp issues the TMA copies, one the products,
// and others carry finished tiles out while the next ones run. A step of K is 128
// bytes, 64 bf16 or 128 e4m3, four instructions. A stage of gemm_pair is one step of
// bf16 (a gradient of the input: 670,000 cycles; with two, 700,000) or two steps of 8
// bits, whose products are issued with their scales (65536 x 4096 x 2048: 620,000
// cycles; with one, 690,000).
//   gemm_pair: tiles of 256 x 256 by a cluster of two CTAs. Each holds half of A's
//     rows and half of B's in shared memory and the instruction reads both CTAs'
//     halves of B, so a CTA fetches 32 KB per step where a tile of its own would
//     take 48 (and 96 bytes a cycle instead of 64 out of shared memory).
//   gemm_tokens: tiles of 128 rows x up to 128 columns by one CTA, for products
//     with few columns (tokens) whose other operand (weights) has to stream: the
//     CTAs divide its K steps evenly, whatever the number of tiles.
//
// Either operand may lie with its k contiguous (rows of 128 bytes, 128-byte
// swizzle) or with its m or n contiguous ("MN-major": boxes of 64 elements x 64
// k), so a weight and the transposed factors of its gradient are read as they
// lie. Coordinates past a matrix's end read zeros and are not stored.
//
// The matrix units cut sums off towards zero: 120 instructions in a row leave
// 2e-6 of a result (of values of both signs; of one sign each takes up to 1e-7 of
// the sum), too much for fp32. Kernels with fp32 results therefore sum a few K
// blocks at a time in TMEM and add those sums in registers, rounding to nearest
// (relative error 1e-7). So do those with bf16 results whose K takes more than
// kLongest steps: 2^20 tokens of one sign left 0.6 % of a weight's gradient, always
// towards zero, and leave 0.01 % so.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "nys_act.h"
#include "nys_internal.h"
#include "nys_sm100.h"
#include "nys_tma_host.h"

namespace nys {
namespace gemm {

using namespace nys::sm100;

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kLongest = 256;  // steps, of four instructions, summed in TMEM for bf16 results

enum Kind { kBf16, kMx8 };
enum Epilogue { kPlain, kGated };
enum By { kOnly = 0, kByPart = 1, kByKPart = 2 };

struct Maps {
  CUtensorMap a[2], b[2], c[3];
};

struct Params {
  int m_tiles, n_tiles;  // of one part
  int parts;             // products side by side in one launch (a[part], b[part], plane of c)
  int splits;            // ranges of its; each writes a plane of fp32 partial sums (gemm_pair)
  int unit, units;       // gemm_tokens: steps that stay together, and how many of them a tile has
  int k_blocks;          // 128-byte blocks of one K part
  int its, its_per_split;  // K parts x k_blocks x pairs
  int bn;                // columns of a tile (gemm_pair)
  int chunk;             // steps (even) summed in TMEM before the sum moves to registers
  int pairs;             // products of the operands' terms that are summed: 1, 2 or 6
  uint32_t a_terms, b_terms;  // the terms of pair i in nibble i
  int a_by, b_by;        // By
  int c_by_part;         // results of part i to c[i]; else to plane split * parts + part of c[0]
  int group;             // row tiles that neighbouring CTAs share: 16 (8: 486 us for the
                         // feed-forward of 16384 tokens, 16: 471, 32: 474, 64: 508)
  int act, keep;         // kGated
  int* status;
  // 8-bit operands: scale words, groups of four K blocks x rows
  const uint32_t *a_scales, *b_scales;
  int a_rows, b_rows;
};

// One output tile of a CTA's walk.
struct Tile {
  int split, part, m, n, it0, it1;
};
__device__ __forceinline__ Tile tile_of(const Params& p, int t) {
  Tile r;
  const int per = p.m_tiles * p.n_tiles, z = t / per;
  t -= z * per;
  r.split = z / p.parts;
  r.part = z - r.split * p.parts;
  // groups of row tiles, column by column: the tiles in flight share operands
  const int g = t / (p.group * p.n_tiles), first = g * p.group;
  const int rows = min(p.group, p.m_tiles - first);
  t -= g * p.group * p.n_tiles;
  r.n = t / rows;
  r.m = first + t - r.n * rows;
  r.it0 = r.split * p.its_per_split;
  r.it1 = min(p.its, r.it0 + p.its_per_split);
  return r;
}

// gemm_pair's walk: every so-manyth tile.
struct GridWalk {
  Tile tile;
  int t, step, tiles;
  bool more;
  __device__ __forceinline__ explicit GridWalk(const Params& p)
      : t(blockIdx.x / 2), step(gridDim.x / 2), tiles(p.m_tiles * p.n_tiles * p.parts * p.splits) {
    enter(p);
  }
  __device__ __forceinline__ void enter(const Params& p) {
    more = t < tiles;
    if (more) tile = tile_of(p, t);
  }
  __device__ __forceinline__ void next(const Params& p) {
    t += step;
    enter(p);
  }
};

// gemm_tokens' walk: the units of all tiles form one line, which the CTAs divide
// evenly, so a CTA has the end of a tile, whole ones and the start of another. A
// tile's n-th CTA writes plane n of the partial sums.
__host__ __device__ __forceinline__ long long line_start(long long line, int ctas, int cta) {
  return line * cta / ctas;
}
__host__ __device__ __forceinline__ int line_cta(long long line, int ctas, long long unit) {
  return (int)(((unit + 1) * ctas - 1) / line);
}
struct LineWalk {
  Tile tile;
  long long u, end, line;
  bool more;
  __device__ __forceinline__ explicit LineWalk(const Params& p) : line((long long)p.m_tiles * p.parts * p.units) {
    u = line_start(line, gridDim.x, blockIdx.x);
    end = line_start(line, gridDim.x, blockIdx.x + 1);
    enter(p);
  }
  __device__ __forceinline__ void enter(const Params& p) {
    more = u < end;
    if (!more) return;
    const int t = (int)(u / p.units), r = (int)(u - (long long)t * p.units);
    const int n = (int)min((long long)(p.units - r), end - u);
    tile.part = t / p.m_tiles;
    tile.m = t - tile.part * p.m_tiles;
    tile.n = 0;
    tile.split = (int)blockIdx.x - line_cta(line, gridDim.x, (long long)t * p.units);
    tile.it0 = r * p.unit;
    tile.it1 = min(p.its, (r + n) * p.unit);
    u += n;
  }
  __device__ __forceinline__ void next(const Params& p) { enter(p); }
};

__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, int* status,
                                             volatile int* abort_flag) {
  if (mbar_wait(bar, parity, abort_flag, kWaitNs)) return true;
  *abort_flag = 1;
  atomicExch(status, (int)NYS_ERR_TIMEOUT);
  return false;
}

// The same for a whole warp, whose lanes go on together. A phase that is over
// takes one test.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_fail(bar, parity, status, abort_flag));
}
// True in one lane of a converged warp. The warps that issue copies and products
// run their loops whole and elect a lane around the instructions: in a branch on
// the lane's number the compiler has to move every operand of such an instruction
// to the uniform registers one lane at a time, and a stage's four products took
// longer to issue than to run.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p)::"memory");
  return p != 0;
}

// The scales of 128 rows of an operand, 512 bytes in shared memory, to four
// columns of TMEM (repeated for each quarter of the lanes).
__device__ __forceinline__ void copy_scales(uint32_t tmem, const uint8_t* smem) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem),
               "l"(smem_desc(smem_u32(smem), 0, 128, SW_NONE))
               : "memory");
}
// D (+)= A B with e4m3 operands whose K step of 32 has one scale per row.
__device__ __forceinline__ void mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: e4m3 operands, K-major, scales in E8M0; `id` names the
// byte of a scale word (of both operands).
__device__ __forceinline__ uint32_t idesc_mx8(int M, int N, uint32_t id) {
  return (id << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (id << 29);
}

// Barriers and the like at the end of a kernel's shared memory.
struct Bars {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2], sf_full[4], sf_empty[4], fin;
  uint32_t tmem;
  int abort;
};
constexpr int kBarBytes = 512;
static_assert(sizeof(Bars) <= kBarBytes, "barriers");
constexpr int kSmem = 232448;  // of a CTA
constexpr int kSlots = 4;      // scale words of four K blocks each on their way

// 32 columns of a lane's row to a box in shared memory: rows of 128 bytes (fp32)
// or 64 (bf16), 16-byte pieces in the swizzle of that width.
__device__ __forceinline__ void stage32(uint8_t* box, int lane, const float (&v)[32], float) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(box + sw128_offset(lane, c * 16)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void stage32(uint8_t* box, int lane, const float (&v)[32], __nv_bfloat16) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(box + sw64_offset(lane, c * 16)) =
        make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                   pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
}
// 32 or 16 columns of a lane's row; the values hold after tmem_ld_wait().
__device__ __forceinline__ void start_columns(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void start_columns(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }

// A warp's boxes (one or two) in turn, each to memory by one TMA store.
template <int BYTES, int BOXES>
struct Staging {
  uint8_t* base;
  int lane, turn;
  __device__ __forceinline__ uint8_t* take() {  // the box of BOXES stores ago has left
    if (lane == 0) {
      if (BOXES == 1) bulk_wait_read0();
      else bulk_wait_read1();
    }
    __syncwarp();
    uint8_t* box = base + (BOXES == 1 ? 0 : (turn & 1) * BYTES);
    ++turn;
    return box;
  }
  __device__ __forceinline__ void send(const CUtensorMap* map, uint8_t* box, int x, int y, int z) {
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, box, x, y, z);
      bulk_commit();
    }
  }
};

// The terms of an operand that a pair multiplies: nibbles of a table.
__device__ __forceinline__ int term_of(uint32_t table, int pair) { return (table >> (4 * pair)) & 15; }
// Where a tile's first step lies.
struct Step {
  int pair, kb, kpart;
  __device__ __forceinline__ Step(const Params& p, int it) {
    pair = it % p.pairs;
    kb = it / p.pairs;
    kpart = kb / p.k_blocks;
    kb -= kpart * p.k_blocks;
  }
  __device__ __forceinline__ void next(const Params& p) {
    if (++pair == p.pairs) {
      pair = 0;
      if (++kb == p.k_blocks) kb = 0, ++kpart;
    }
  }
};
__device__ __forceinline__ int map_of(int by, const Tile& tile, const Step& s) {
  return by == kByPart ? tile.part : by == kByKPart ? s.kpart : 0;
}

// Scale words (four K blocks) of 128 rows from r0 on, as the copy to TMEM takes
// them: rows lane, lane + 32, + 64, + 96 side by side. Rows past the end get zeros.
__device__ __forceinline__ uint4 scale_words(const uint32_t* words, int rows, int group, int r0, int lane) {
  const uint32_t* at = words + (size_t)group * rows;
  auto one = [&](int r) { return r < rows ? at[r] : 0u; };
  return make_uint4(one(r0 + lane), one(r0 + lane + 32), one(r0 + lane + 64), one(r0 + lane + 96));
}

// The groups of four K blocks of a CTA's tiles, in order.
template <typename Walk>
struct ScaleWalk {
  Walk walk;
  int group;
  __device__ __forceinline__ explicit ScaleWalk(const Params& p) : walk(p), group(walk.more ? walk.tile.it0 >> 2 : 0) {}
  __device__ __forceinline__ void next(const Params& p) {
    if (++group <= (walk.tile.it1 - 1) >> 2) return;
    walk.next(p);
    if (walk.more) group = walk.tile.it0 >> 2;
  }
};

// The scale warp's loop: load(walk, w) reads a group's words, hand_over(slot)
// says that they are in shared memory. A group is loaded right behind the hand-over
// of the one before it and not sooner: the fence waits for every load that is on
// its way (2000 cycles, where four steps of products take 1800).
template <int N, typename Walk, typename Load, typename Hand>
__device__ __forceinline__ void scale_loop(const Params& p, Bars& bars, uint8_t* scales, Load load, Hand hand_over) {
  const int lane = threadIdx.x & 31;
  ScaleWalk<Walk> at(p);
  uint4 w[N];
  if (at.walk.more) load(at.walk.tile, at.group, w);
#pragma unroll 1
  for (uint32_t ns = 0; at.walk.more; ++ns) {
    const uint32_t slot = ns % kSlots;
    if (ns >= kSlots && !warp_wait(&bars.sf_empty[slot], (ns / kSlots - 1) & 1, p.status, &bars.abort)) return;
    uint4* to = reinterpret_cast<uint4*>(scales + slot * N * 512);
#pragma unroll
    for (int i = 0; i < N; ++i) to[32 * i + lane] = w[i];
    fence_async_smem();
    __syncwarp();
    if (lane == 0) hand_over(slot);
    at.next(p);
    if (at.walk.more) load(at.walk.tile, at.group, w);
  }
}

// ------------------------------------------------------ two CTAs per tile

template <int KIND, typename OutT>
struct PairLayout {
  // 8-bit tiles leave TMEM columns for the scales beside two accumulators
  static constexpr int kCols = KIND == kMx8 ? 224 : 256;  // most columns of a tile
  static constexpr int kA = 128 * 128;                    // a CTA's half of A, a step
  static constexpr int kSteps = KIND == kMx8 ? 2 : 1;     // of a stage
  static constexpr int kBox = 32 * 32 * sizeof(OutT), kBoxes = sizeof(OutT) == 4 ? 1 : 2;
  static constexpr int kStaging = 8 * kBoxes * kBox;
  static constexpr int kScaleSlot = 512 + 1024, kScales = KIND == kMx8 ? kSlots * kScaleSlot : 0;
  static constexpr int kRing = (kSmem - 1024 - kStaging - kScales - kBarBytes) / 1024 * 1024;  // of the stages
  static constexpr int kBytes = 1024 + kRing + kStaging + kScales + kBarBytes;
  static constexpr int kScaleCol = 2 * kCols, kScaleCols = 12;  // TMEM columns of the scales, of a slot
  static_assert(KIND != kMx8 || kScaleCol + kSlots * kScaleCols <= 512, "TMEM columns");
  static constexpr int kFirst = KIND == kMx8 ? 4 : 3;  // warps that carry out
  static constexpr int kThreads = (kFirst + 8) * 32;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of the first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
// What the arrival orders are this CTA's own accesses (its TMEM has been read, its
// scales stand in its shared memory, both fenced), so the release is of CTA scope:
// one of cluster scope takes 1500 cycles.
__device__ __forceinline__ void arrive_in_first(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
}
// Copy to this CTA's shared memory that reports to the first CTA's barrier.
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t more) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(more)
      : "memory");
}
__device__ __forceinline__ void pair_mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t a_scale,
                                             uint32_t b_scale, uint32_t more) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(more)
      : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t tmem, const uint8_t* smem) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem),
               "l"(smem_desc(smem_u32(smem), 0, 128, SW_NONE))
               : "memory");
}
// Arrives on both CTAs' copies of bar when the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Tiles of 256 rows x p.bn columns, a multiple of 32; EPI kGated: half of them are
// the gate's (B of the first CTA), half the same columns of the other projection
// (B of the second), bn is a multiple of 64, and the result has bn / 2. SUM: sums
// move to registers every p.chunk steps; else K is a single chunk.
template <int KIND, bool AMN, bool BMN, int EPI, typename OutT, bool SUM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairLayout<KIND, OutT>::kThreads, 1)
gemm_pair(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using L = PairLayout<KIND, OutT>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = align1024(raw);
  uint8_t* staging = sm + L::kRing;
  uint8_t* scales = staging + L::kStaging;
  Bars& bars = *reinterpret_cast<Bars*>(scales + L::kScales);
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  // B's lines per CTA, in whole boxes where they are MN-major; as many stages as fit
  const int lines = p.bn / 2, held = BMN ? (lines + 63) / 64 * 64 : lines;
  const uint32_t step_bytes = L::kA + held * 128, stage_bytes = L::kSteps * step_bytes;
  const uint32_t S = min(12u, L::kRing / stage_bytes);

  if (warp == 0 && lane < 7) {
    const CUtensorMap* maps_of[7] = {&maps.a[0], &maps.a[1], &maps.b[0], &maps.b[1], &maps.c[0], &maps.c[1], &maps.c[2]};
    tma_prefetch(maps_of[lane]);
  }

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < S; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 16);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars.sf_full[i], 2);
      mbar_init(&bars.sf_empty[i], 1);
    }
    mbar_init(&bars.fin, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  // All CTAs of the grid run at once, so what follows may be set up beside them. A
  // kernel set up so waits for the one before it here, before it takes TMEM that
  // the other may still need.
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and TMEM are there
  tc_fence_after_sync();
  const uint32_t tmem = bars.tmem;

  if (warp == 0 || warp == 2) {
    // -------------------------------------------------------------- copies
    // A's by one warp, B's by another: up to four copies a step take one as long
    // to issue as the products take to run (16384 tokens, 2048 -> 5632: forward
    // 761,000 cycles, gradients of the weights 779,000; with two 726,000, 747,000).
    const bool first = warp == 0;
    uint32_t st = 0, round = 0, n = 0;  // stage, times round the stages, stages filled
    const bool second = first || held > 64;  // a second box of 64 (MN-major)
    bool ok = true;
    for (GridWalk walk(p); ok && walk.more; walk.next(p)) {
      const Tile& tile = walk.tile;
      // rows of A, or of B (columns of the result)
      const int r0 = first            ? tile.m * 256 + rank * 128
                     : EPI == kGated ? tile.n * lines
                                     : tile.n * p.bn + rank * lines;
      Step s(p, tile.it0);
      for (int it = tile.it0; it < tile.it1; it += L::kSteps, ++n) {
        if (round > 0 && !warp_wait(&bars.empty[st], (round - 1) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        const int count = min(L::kSteps, tile.it1 - it);
        if (elect_one()) {
          if (first && rank == 0) mbar_arrive_expect_tx(&bars.full[st], count * 2 * step_bytes);
          const uint32_t bar = in_first(&bars.full[st]);
          Step at = s;
          for (int j = 0; j < count; ++j, at.next(p)) {
            uint8_t* to = sm + st * stage_bytes + j * step_bytes + (first ? 0 : L::kA);
            const int k = at.kb * (KIND == kMx8 ? 128 : 64), z = term_of(first ? p.a_terms : p.b_terms, at.pair);
            const CUtensorMap* map = first ? &maps.a[map_of(p.a_by, tile, at)]
                                           : &maps.b[EPI == kGated ? rank : map_of(p.b_by, tile, at)];
            if (first ? AMN : BMN) {
              pair_load_3d(to, map, bar, r0, k, z);
              if (second) pair_load_3d(to + 8192, map, bar, r0 + 64, k, z);
            } else {
              pair_load_3d(to, map, bar, k, r0, z);
            }
          }
        }
        __syncwarp();
        for (int j = 0; j < L::kSteps; ++j) s.next(p);
        if (++st == S) st = 0, ++round;
      }
    }
    // nothing may land in shared memory behind the kernel's end (the first
    // CTA's barriers count both CTAs' copies)
    if (rank == 0)
      for (uint32_t i = n > S ? n - S : 0; i < n; ++i) mbar_wait(&bars.full[i % S], (i / S) & 1, nullptr, kWaitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16(256, p.bn, AMN, BMN);
      const uint32_t first_stage = smem_u32(sm);
      const uint64_t a0 = AMN ? smem_desc(first_stage, 8192, 1024, SW_128B) : smem_desc(first_stage, 16, 1024, SW_128B);
      const uint64_t b0 = BMN ? smem_desc(first_stage + L::kA, 8192, 1024, SW_128B)
                              : smem_desc(first_stage + L::kA, 16, 1024, SW_128B);
      uint32_t st = 0, phase = 0, nc = 0, ns = 0;
      bool ok = true;
      for (GridWalk walk(p); ok && walk.more; walk.next(p)) {
        const Tile& tile = walk.tile;
        uint32_t d = 0;
        int left = 0;  // steps of this accumulator
        for (int it = tile.it0; it < tile.it1; it += L::kSteps) {
          const bool first = left == 0;
          if (first) {
            left = SUM ? min(p.chunk, tile.it1 - it) : tile.it1 - it;
            d = tmem + (nc & 1) * L::kCols;
            if (nc >= 2 && !warp_wait(&bars.acc_empty[nc & 1], (nc / 2 - 1) & 1, p.status, abort_flag)) {
              ok = false;
              break;
            }
          }
          const uint32_t slot = ns % kSlots, sf = tmem + L::kScaleCol + slot * L::kScaleCols;
          const bool new_scales = KIND == kMx8 && (it & 3) == 0;
          if (new_scales && !warp_wait(&bars.sf_full[slot], (ns / kSlots) & 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          if (!warp_wait(&bars.full[st], phase, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const int count = min(L::kSteps, tile.it1 - it);
          const bool last_scales = KIND == kMx8 && (it + L::kSteps >= tile.it1 || ((it + L::kSteps) & 3) == 0);
          left -= count;
          if (elect_one()) {
            if (new_scales) {
              const uint8_t* from = scales + slot * L::kScaleSlot;
#pragma unroll
              for (int i = 0; i < 3; ++i) pair_copy_scales(sf + 4 * i, from + 512 * i);
            }
            uint64_t ad = a0 + st * (stage_bytes / 16), bd = b0 + st * (stage_bytes / 16);
            for (int j = 0; j < count; ++j, ad += step_bytes / 16, bd += step_bytes / 16) {
              const uint32_t id = KIND == kMx8 ? idesc_mx8(256, p.bn, (it + j) & 3) : idesc;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint64_t ak = ad + (AMN ? kk * 128 : kk * 2), bk = bd + (BMN ? kk * 128 : kk * 2);
                const uint32_t more = !first || j > 0 || kk > 0;
                if (KIND == kMx8)
                  pair_mma_mx8(d, ak, bk, id, sf, sf + 4, more);
                else
                  pair_mma_bf16(d, ak, bk, id, more);
              }
            }
            pair_commit(&bars.empty[st]);
            if (last_scales) pair_commit(&bars.sf_empty[slot]);
            if (left == 0) pair_commit(&bars.acc_full[nc & 1]);
          }
          __syncwarp();
          if (last_scales) ++ns;
          if (left == 0) ++nc;
          if (++st == S) st = 0, phase ^= 1;
        }
      }
      // no product may be in flight when TMEM is freed
      if (elect_one())
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(&bars.fin))
                     : "memory");
      __syncwarp();
      mbar_wait(&bars.fin, 0, nullptr, kWaitNs);
    }
  } else if (warp >= L::kFirst) {
    // ------------------------------------------------------- finished tiles
    // Two warps for each quarter of the lanes, which take 32 columns of the
    // result in turn: the plain form up to four times, the gated one twice.
    const int quarter = warp & 3, half = (warp - L::kFirst) / 4;
    const int width = EPI == kGated ? p.bn / 2 : p.bn;  // columns of the result
    constexpr int kTurns = EPI == kGated ? 2 : 4;
    Staging<L::kBox, L::kBoxes> out{staging + (warp - L::kFirst) * L::kBoxes * L::kBox, lane, 0};
    uint32_t nc = 0;  // accumulators taken
    bool ok = true;
    for (GridWalk walk(p); ok && walk.more; walk.next(p)) {
      const Tile& tile = walk.tile;
      float f[4][32];  // a lane's row: columns of the result, or of g (0, 1) and u (2, 3)
      if (SUM) {
#pragma unroll
        for (int i = 0; i < 128; ++i) f[i / 32][i % 32] = 0.f;
      }
#pragma unroll 1
      for (int it = tile.it0; it < tile.it1;) {
        if (!warp_wait(&bars.acc_full[nc & 1], (nc / 2) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + (nc & 1) * L::kCols + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = (2 * (i % kTurns) + half) * 32;  // of the result
          if (c >= width) continue;
          const uint32_t at = d + c + (i >= kTurns ? width : 0);
          if constexpr (!SUM) {
            tmem_ld32(at, reinterpret_cast<uint32_t(&)[4][32]>(f)[i]);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[16];
              tmem_ld16(at + 16 * h, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) f[i][16 * h + j] += __uint_as_float(r[j]);
            }
          }
        }
        if (!SUM) tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_in_first(&bars.acc_empty[nc & 1]);
        ++nc;
        it += SUM ? min(p.chunk, tile.it1 - it) : tile.it1 - it;
      }
      if (!ok) break;
      const int y = tile.m * 256 + rank * 128 + quarter * 32, x = tile.n * width;
      const int z = EPI == kGated || p.c_by_part ? 0 : tile.split * p.parts + tile.part;
      auto send = [&](const CUtensorMap* map, int first) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const int c = (2 * i + half) * 32;
          if (c >= width) break;
          uint8_t* box = out.take();
          stage32(box, lane, f[first + i], OutT{});
          out.send(map, box, x + c, y, z);
        }
      };
      if constexpr (EPI == kPlain) {
        send(&maps.c[p.c_by_part ? tile.part : 0], 0);
      } else {
        if (p.keep) {
          send(&maps.c[1], 0);
          send(&maps.c[2], 2);
        }
        act::by_act(p.act, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              f[i][j] = act::value<decltype(a)::value, sizeof(OutT) == 2>(f[i][j]) * f[i + 2][j];
        });
        send(&maps.c[0], 0);
      }
    }
    if (lane == 0) bulk_wait_read0();  // shared memory stays until it has been read
  } else if (KIND == kMx8) {
    // -------------------------------------------------------------- scales
    // Of this CTA's rows of A and of all columns, which both CTAs need.
    scale_loop<3, GridWalk>(
        p, bars, scales,
        [&](const Tile& tile, int group, uint4(&w)[3]) {
          w[0] = scale_words(p.a_scales, p.a_rows, group, tile.m * 256 + rank * 128, lane);
          w[1] = scale_words(p.b_scales, p.b_rows, group, tile.n * p.bn, lane);
          w[2] = scale_words(p.b_scales, p.b_rows, group, tile.n * p.bn + 128, lane);
        },
        [&](uint32_t slot) { arrive_in_first(&bars.sf_full[slot]); });
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // neither CTA's products read the other's memory any more
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------- one CTA per tile

template <int KIND, int BN>
struct TokensLayout {
  static constexpr int kA = 128 * 128, kB = BN * 128, kStep = kA + kB, kSteps = 2, kStage = kSteps * kStep;
  static constexpr int kStaging = 4 * 2 * 4096;  // two boxes per warp that carries out
  static constexpr int kScaleSlot = 512 + 512, kScales = KIND == kMx8 ? kSlots * kScaleSlot : 0;
  static constexpr int kFree = kSmem - 1024 - kStaging - kScales - kBarBytes;
  static constexpr int kStages = kFree / kStage < 12 ? kFree / kStage : 12;
  static constexpr int kBytes = 1024 + kStages * kStage + kStaging + kScales + kBarBytes;
  static constexpr int kScaleCol = 2 * BN, kScaleCols = 8;  // TMEM columns of a slot's scales
  static constexpr int kCols = 2 * BN + (KIND == kMx8 ? kSlots * kScaleCols : 0);
  static constexpr int kAlloc = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kThreads = KIND == kMx8 ? 224 : 192;
};

// Tiles of 128 rows (weights) x BN columns (tokens), fp32 partial sums.
template <int KIND, bool AMN, int BN>
__global__ void __launch_bounds__(TokensLayout<KIND, BN>::kThreads, 1)
gemm_tokens(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using L = TokensLayout<KIND, BN>;
  constexpr int S = L::kStages;
  constexpr int kW = BN < 32 ? BN : 32;  // columns read from TMEM at a time
  extern __shared__ uint8_t raw[];
  uint8_t* sm = align1024(raw);
  uint8_t* staging = sm + S * L::kStage;
  uint8_t* scales = staging + L::kStaging;
  Bars& bars = *reinterpret_cast<Bars*>(scales + L::kScales);
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0 && lane < 5) {
    const CUtensorMap* maps_of[5] = {&maps.a[0], &maps.a[1], &maps.b[0], &maps.b[1], &maps.c[0]};
    tma_prefetch(maps_of[lane]);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 4);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars.sf_full[i], 1);
      mbar_init(&bars.sf_empty[i], 1);
    }
    mbar_init(&bars.fin, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  cudaTriggerProgrammaticLaunchCompletion();  // as above
  cudaGridDependencySynchronize();
  if (warp == 1) tmem_alloc(&bars.tmem, L::kAlloc);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars.tmem;

  if (warp == 0) {
    // -------------------------------------------------------------- copies
    uint32_t st = 0, round = 0, n = 0;  // stage, times round the stages, copies issued
    bool ok = true;
    for (LineWalk walk(p); ok && walk.more; walk.next(p)) {
      const Tile& tile = walk.tile;
      Step s(p, tile.it0);
      for (int it = tile.it0; it < tile.it1; it += L::kSteps, ++n) {
        if (round > 0 && !warp_wait(&bars.empty[st], (round - 1) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        const int count = min(L::kSteps, tile.it1 - it);
        if (elect_one()) {
          uint64_t* bar = &bars.full[st];
          mbar_arrive_expect_tx(bar, count * L::kStep);
          Step at = s;
          for (int j = 0; j < count; ++j, at.next(p)) {
            uint8_t* a = sm + st * L::kStage + j * L::kStep;
            const int k = at.kb * (KIND == kMx8 ? 128 : 64), pa = term_of(p.a_terms, at.pair);
            const CUtensorMap* am = &maps.a[map_of(p.a_by, tile, at)];
            if (AMN) {
              tma_load_3d(a, am, bar, tile.m * 128, k, pa);
              tma_load_3d(a + 8192, am, bar, tile.m * 128 + 64, k, pa);
            } else {
              tma_load_3d(a, am, bar, k, tile.m * 128, pa);
            }
            tma_load_3d(a + L::kA, &maps.b[map_of(p.b_by, tile, at)], bar, k, 0, term_of(p.b_terms, at.pair));
          }
        }
        __syncwarp();
        for (int j = 0; j < L::kSteps; ++j) s.next(p);
        if (++st == S) st = 0, ++round;
      }
    }
    // nothing may land in shared memory behind the kernel's end
    for (uint32_t i = n > S ? n - S : 0; i < n; ++i) mbar_wait(&bars.full[i % S], (i / S) & 1, nullptr, kWaitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    const uint32_t idesc = idesc_bf16(128, BN, AMN, false);
    const uint32_t first_stage = smem_u32(sm);
    const uint64_t a0 = AMN ? smem_desc(first_stage, 8192, 1024, SW_128B) : smem_desc(first_stage, 16, 1024, SW_128B);
    const uint64_t b0 = smem_desc(first_stage + L::kA, 16, 1024, SW_128B);
    uint32_t st = 0, phase = 0, nc = 0, ns = 0;
    bool ok = true;
    for (LineWalk walk(p); ok && walk.more; walk.next(p)) {
      const Tile& tile = walk.tile;
      uint32_t d = 0;
      int left = 0;  // steps of this accumulator
      for (int it = tile.it0; it < tile.it1; it += L::kSteps) {
        const bool first = left == 0;
        if (first) {
          left = min(p.chunk, tile.it1 - it);
          d = tmem + (nc & 1) * BN;
          if (nc >= 2 && !warp_wait(&bars.acc_empty[nc & 1], (nc / 2 - 1) & 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
        }
        const uint32_t slot = ns % kSlots, sf = tmem + L::kScaleCol + slot * L::kScaleCols;
        const bool new_scales = KIND == kMx8 && (it == tile.it0 || (it & 3) == 0);
        if (new_scales && !warp_wait(&bars.sf_full[slot], (ns / kSlots) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        if (!warp_wait(&bars.full[st], phase, p.status, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int count = min(L::kSteps, tile.it1 - it);
        const bool last_scales = KIND == kMx8 && (it + L::kSteps >= tile.it1 || ((it + L::kSteps) & 3) == 0);
        left -= count;
        if (elect_one()) {
          if (new_scales) {
            const uint8_t* from = scales + slot * L::kScaleSlot;
            copy_scales(sf, from);
            copy_scales(sf + 4, from + 512);
          }
          uint64_t ad = a0 + st * (L::kStage / 16), bd = b0 + st * (L::kStage / 16);
          for (int j = 0; j < count; ++j, ad += L::kStep / 16, bd += L::kStep / 16) {
            const uint32_t id = KIND == kMx8 ? idesc_mx8(128, BN, (it + j) & 3) : idesc;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ak = ad + (AMN ? kk * 128 : kk * 2), bk = bd + kk * 2;
              const uint32_t more = !first || j > 0 || kk > 0;
              if (KIND == kMx8)
                mma_mx8(d, ak, bk, id, sf, sf + 4, more);
              else
                mma_bf16(d, ak, bk, id, more);
            }
          }
          mma_commit(&bars.empty[st]);
          if (last_scales) mma_commit(&bars.sf_empty[slot]);
          if (left == 0) mma_commit(&bars.acc_full[nc & 1]);
        }
        __syncwarp();
        if (last_scales) ++ns;
        if (left == 0) ++nc;
        if (++st == S) st = 0, phase ^= 1;
      }
    }
    // no product may be in flight when TMEM is freed
    if (elect_one()) mma_commit(&bars.fin);
    __syncwarp();
    mbar_wait(&bars.fin, 0, nullptr, kWaitNs);
  } else if (warp < 6) {
    // ------------------------------------------------------- finished tiles
    const int quarter = warp & 3;
    Staging<4096, 2> out{staging + (warp - 2) * 8192, lane, 0};
    uint32_t nc = 0;  // accumulators taken
    bool ok = true;
    for (LineWalk walk(p); ok && walk.more; walk.next(p)) {
      const Tile& tile = walk.tile;
      float sum[BN / kW][kW];  // a lane's row
#pragma unroll
      for (int i = 0; i < BN; ++i) sum[i / kW][i % kW] = 0.f;
#pragma unroll 1
      for (int it = tile.it0; it < tile.it1; it += min(p.chunk, tile.it1 - it)) {
        if (!__all_sync(0xffffffffu, wait_or_fail(&bars.acc_full[nc & 1], (nc / 2) & 1, p.status, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (nc & 1) * BN;
#pragma unroll
        for (int c = 0; c < BN / kW; ++c) {
          uint32_t r[kW];
          start_columns(d + c * kW, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kW; ++i) sum[c][i] += __uint_as_float(r[i]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.acc_empty[nc & 1]);
        ++nc;
      }
      if (!ok) break;
      const int y = tile.m * 128 + quarter * 32, z = tile.split * p.parts + tile.part;
      if constexpr (BN < 32) {
        uint8_t* box = out.take();  // rows of 64 bytes
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<float4*>(box + sw64_offset(lane, c * 16)) =
              make_float4(sum[0][4 * c], sum[0][4 * c + 1], sum[0][4 * c + 2], sum[0][4 * c + 3]);
        out.send(&maps.c[0], box, 0, y, z);
      } else {
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          uint8_t* box = out.take();
          stage32(box, lane, sum[c], 0.f);
          out.send(&maps.c[0], box, 32 * c, y, z);
        }
      }
    }
    if (lane == 0) bulk_wait_read0();  // shared memory stays until it has been read
  } else if (KIND == kMx8) {
    // -------------------------------------------------------------- scales
    scale_loop<2, LineWalk>(
        p, bars, scales,
        [&](const Tile& tile, int group, uint4(&w)[2]) {
          w[0] = scale_words(p.a_scales, p.a_rows, group, tile.m * 128, lane);
          w[1] = scale_words(p.b_scales, p.b_rows, group, 0, lane);
        },
        [&](uint32_t slot) { mbar_arrive(&bars.sf_full[slot]); });
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, L::kAlloc);
}

// ------------------------------------------------------------------- host

// Tensor maps are encoded by the driver, which wants a context that is current in
// the calling thread; a thread whose first CUDA call this is has none yet.
inline int have_context(int dev) {
  static thread_local int bound = -1;
  if (bound == dev) return NYS_OK;
  const cudaError_t e = cudaSetDevice(dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  bound = dev;
  return NYS_OK;
}

// A matrix of `rows` rows of `cols` elements, `stride` elements apart, in
// `planes` copies `plane` elements apart.
struct Matrix {
  const void* at;
  long long rows, cols, stride;
  int esize;
  int planes = 1;
  long long plane = 0;
};

inline bool make_map(CUtensorMap* map, const Matrix& x, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  const CUtensorMapDataType dt = x.esize == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : x.esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t dims[3] = {(uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.planes};
  // one row, one plane: the distance to the next is never used
  const uint64_t own = ((uint64_t)x.cols * x.esize + 15) / 16 * 16;
  const uint64_t row = x.rows > 1 ? (uint64_t)x.stride * x.esize : own, all = row * (uint64_t)x.rows;
  const uint64_t strides[2] = {row, x.planes > 1 ? (uint64_t)x.plane * x.esize : all < (1ull << 40) ? all : own};
  const uint32_t box[3] = {(uint32_t)box_cols, (uint32_t)box_rows, 1};
  return make_tensor_map(map, dt, 3, x.at, dims, strides, box, swizzle);
}
// An operand read with its k contiguous (`lines` rows per box) ...
inline bool map_k(CUtensorMap* map, const Matrix& x, int lines) {
  return make_map(map, x, 128 / x.esize, lines, CU_TENSOR_MAP_SWIZZLE_128B);
}
// ... or stored [k][m or n].
inline bool map_mn(CUtensorMap* map, const Matrix& x) { return make_map(map, x, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B); }
// Results in boxes of 32 rows x 32 columns, or x 16 of fp32.
inline bool map_out(CUtensorMap* map, const Matrix& x, int columns = 32) {
  return make_map(map, x, columns, 32,
                  columns * x.esize == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// gemm_tokens' division: a tile of 128 columns has the planes of its CTAs.
struct Line {
  int width;  // 0: not turned
  int m_tiles, units, ctas;
  long long line;
  __host__ __device__ __forceinline__ int planes(int part, int column) const {
    const long long u = ((long long)part * m_tiles + column / 128) * units;
    return line_cta(line, ctas, u + units - 1) - line_cta(line, ctas, u) + 1;
  }
};
// Sums of the partial planes of a split product (nys_join.cu): part holds
// planes of fp32, plane split * parts + part, each [M][N] (rows of a result) or,
// of gemm_tokens, [N][width] (a result's columns, its rows side by side).
// Results in dtype; set up while the product still runs.
struct Join {
  const float* part;
  int splits, M, N;
  Line line;
  void* out[2];  // [M][N] of part 0, 1
  long long stride[2];
};
int join(const Join& j, int parts, int dtype, cudaStream_t st);
// part 0: g, part 1: u; h = act(g) u, and g, u where gate, up are set.
struct JoinGated {
  const float* part;
  int splits, M, N;
  Line line;
  void *h, *gate, *up;
  long long h_stride, gate_stride, up_stride;
};
int join_gated(const JoinGated& j, int act, int dtype, cudaStream_t st);

// Products of a few fp32 rows with fp32 weights on the CUDA cores (nys_few.cu):
// plane 2 split + i of part [T][N] is x[i] times w[i] over K's range `split`.
struct Few {
  const float *x[2], *w[2];
  long long x_stride, w_stride;  // w: [N][K] (k_contiguous) or [K][N]
  float* part;
  int T, N, K, range;
  int splits() const { return (K + range - 1) / range; }
};
// Tokens; 24 of them through 4096 -> 4712 twice take 88 to 115 us on the CUDA cores,
// 112 to 117 in terms on the tensor cores; one takes 29 against 110.
constexpr int kMostFew = 24;
int few_range(int T, int N, int K, bool k_contiguous);
int launch_few(const char* name, const Few& p, bool k_contiguous, cudaStream_t st);

// Every map is fetched ahead, used or not: those that a call leaves out are copies.
inline Maps filled(Maps m) {
  for (CUtensorMap* x : {&m.a[1], &m.b[0], &m.b[1], &m.c[0], &m.c[1], &m.c[2]}) {
    bool none = true;
    for (auto word : x->opaque) none = none && word == 0;
    if (none) *x = m.a[0];
  }
  return m;
}

// KERNEL with its dynamic shared memory.
template <auto KERNEL>
int start(const char* name, int grid, int threads, int bytes, const Maps& maps, const Params& p, cudaStream_t st) {
  const int rc = allow_shared(reinterpret_cast<const void*>(KERNEL), bytes);
  if (rc != NYS_OK) return rc;
  return launch_behind(name, KERNEL, dim3(grid), dim3(threads), bytes, st, filled(maps), p);
}
template <int KIND, bool AMN, bool BMN, int EPI, typename OutT>
int launch_pair(const char* name, const Maps& maps, const Params& p, cudaStream_t st) {
  using L = PairLayout<KIND, OutT>;
  const long long tiles = (long long)p.m_tiles * p.n_tiles * p.parts * p.splits;
  if (tiles >= (1ll << 31) - 1024) return NYS_ERR_SHAPE;
  const int most = plan_sms() / 2;
  const int grid = 2 * (tiles < most ? (int)tiles : most);
  if constexpr (sizeof(OutT) == 2)
    if (p.its_per_split <= p.chunk)
      return start<gemm_pair<KIND, AMN, BMN, EPI, OutT, false>>(name, grid, L::kThreads, L::kBytes, maps, p, st);
  return start<gemm_pair<KIND, AMN, BMN, EPI, OutT, true>>(name, grid, L::kThreads, L::kBytes, maps, p, st);
}
template <int KIND, bool AMN>
int launch_tokens(const char* name, int bn, int ctas, const Maps& maps, const Params& p, cudaStream_t st) {
  auto go = [&](auto n) {
    constexpr int BN = decltype(n)::value;
    using L = TokensLayout<KIND, BN>;
    return start<gemm_tokens<KIND, AMN, BN>>(name, ctas, L::kThreads, L::kBytes, maps, p, st);
  };
  using std::integral_constant;
  switch (bn) {
    case 16: return go(integral_constant<int, 16>{});
    case 32: return go(integral_constant<int, 32>{});
    case 64: return go(integral_constant<int, 64>{});
    default: return go(integral_constant<int, 128>{});
  }
}
constexpr int kMostTokens = 128;  // of gemm_tokens
inline int columns_of(int tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128; }

// Three terms of both operands, all pairs that matter at 2^-24, small products
// first: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0).
constexpr uint32_t kTermsA = 0x001102, kTermsB = 0x010120;

// How gemm_pair's product is cut: columns of a tile and ranges of K, whose partial
// sums are joined. The time of a choice is counted in steps of a full tile (0.3 us;
// `pairs` of them for a K block of fp32): rounds of tiles over the CTAs times a
// tile's steps, two more for its start and end, and for more than one range the join
// (ten steps' time to begin, then its bytes, write and read, at 5 TB/s).
struct Cut {
  int bn, splits;
};
// Steps of each of s ranges, a multiple of `unit` (8-bit operands: four, whose
// scales come in one word).
inline int range_of(int steps, int s, int unit) { return ((steps + s - 1) / s + unit - 1) / unit * unit; }

// gemm_tokens: the line of `parts` x N / 128 tiles in units of two steps (fp32: the
// six products of a K block) over the SMs; a CTA has three units at least, so that
// its partial sums stay few beside its weights.
inline Line line_of(long long N, int its, int parts, int unit, int width) {
  Line l{};
  l.width = width;
  l.m_tiles = (int)((N + 127) / 128);
  l.units = (its + unit - 1) / unit;
  l.line = (long long)l.m_tiles * parts * l.units;
  const long long most = l.line / 3 > 0 ? l.line / 3 : 1;
  l.ctas = (int)(most < plan_sms() ? most : plan_sms());
  return l;
}
// Planes that a tile may have: as many CTAs as its units can touch.
inline int most_planes(const Line& l) {
  const long long least = l.line / l.ctas;  // units of a CTA
  const long long n = (l.units + least - 2) / least + 1;
  return (int)(n < l.ctas ? n : l.ctas);
}
inline Cut cut_pair(long long M, long long N, int steps, int unit, int pairs, int parts, int most_bn, int bn_step,
                    bool gated, int least) {
  const int clusters = plan_sms() / 2;
  Cut best{most_bn, 1};
  double best_time = 1e30;
  for (int bn = most_bn; bn >= 128; bn -= bn_step) {
    for (int s = 1; s <= 16 && (s == 1 || steps / s >= least); ++s) {
      const int per = range_of(steps, s, unit);
      if ((steps + per - 1) / per != s) continue;
      // the gated form computes both parts in one tile, unless K is split
      const int columns = gated && s == 1 ? bn / 2 : bn, of = gated && s == 1 ? 1 : parts;
      const long long tiles = ((M + 255) / 256) * ((N + columns - 1) / columns) * of * s;
      const double rounds = (double)((tiles + clusters - 1) / clusters);
      double time = rounds * (per * (double)pairs * (bn + 8.0) / 264.0 + 2.0);
      if (s > 1) time += 10.0 + (double)s * parts * M * N * 8.0 / 1.5e6;
      if (time < best_time * 0.999) best_time = time, best = Cut{bn, s};
    }
  }
  return best;
}

}  // namespace gemm
}  // namespace nys
