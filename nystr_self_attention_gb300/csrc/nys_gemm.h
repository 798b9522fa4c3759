// Matrix products on the tensor cores for the operators around the attention
// module: D[m][n] = sum over k of A[m][k] B[n][k], accumulated in fp32 in TMEM.
//
// A persistent CTA works through output tiles of 128 x BN with one warp that
// issues the TMA copies, one that issues the products, four that carry finished
// tiles out, and (8-bit operands) one that lays the scales out. K advances 128
// bytes per stage: 64 bf16 or 128 e4m3, four instructions. Two accumulators in
// TMEM let a tile's products run while the previous one is carried out.
//
// The matrix units cut sums off towards zero: 120 instructions in a row leave
// 2e-6 of a result, too much for fp32. Kernels with fp32 results of up to 128
// columns therefore sum a few K blocks at a time in TMEM and add those sums in
// registers, rounding to nearest.
//
// Either operand may lie with its k contiguous (rows of 128 bytes, 128-byte
// swizzle) or with its m or n contiguous ("MN-major": boxes of 64 elements x 64
// k), so a weight and the transposed factors of its gradient are read as they
// lie. Coordinates past a matrix's end read zeros and are not stored.
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

enum Kind { kBf16, kMx8 };
enum Epilogue { kPlain, kGated };
enum By { kOnly = 0, kByPart = 1, kByKPart = 2 };

struct Maps {
  CUtensorMap a[2], b[2], c[3];
};

struct Params {
  int m_tiles, n_tiles;  // of one part
  int parts;             // products side by side in one launch (a[part], b[part], plane of c)
  int splits;            // ranges of its; each writes a plane of fp32 partial sums
  int k_blocks;          // 128-byte blocks of one K part
  int its, its_per_split;  // K parts x k_blocks x pairs
  int chunk;             // steps summed in TMEM before the sum moves to registers (fp32 results)
  int pairs;             // 1, or 6 pairs of the three terms of fp32 operands
  int a_by, b_by;        // By
  int c_by_part;         // results of part i to c[i]; else to plane split * parts + part of c[0]
  int group;             // row tiles that neighbouring CTAs share
  int act, keep;         // kGated
  int* status;
  // 8-bit operands: scale words [groups][rows]
  const uint32_t *a_scales, *b_scales;
  int a_rows, b_rows, groups;
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

__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, int* status,
                                             volatile int* abort_flag) {
  if (mbar_wait(bar, parity, abort_flag, kWaitNs)) return true;
  *abort_flag = 1;
  atomicExch(status, (int)NYS_ERR_TIMEOUT);
  return false;
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

// Places of a kernel's shared memory.
template <int KIND, int BN>
struct Layout {
  static constexpr int kA = 128 * 128, kB = BN * 128, kStage = kA + kB;
  static constexpr int kStaging = 4 * 2 * 4096;  // two boxes per warp that carries out
  static constexpr int kScales = KIND == kMx8 ? 2 * (512 + (BN + 127) / 128 * 512) : 0;
  static constexpr int kBars = 512;
  static constexpr int kFree = 232448 - 1024 - kStaging - kScales - kBars;
  static constexpr int kStages = kFree / kStage < 12 ? kFree / kStage : 12;
  static constexpr int kBytes = 1024 + kStages * kStage + kStaging + kScales + kBars;
  static constexpr int kScaleCol = 2 * BN;  // TMEM column of the scales: two slots of 4 + 8
  static constexpr int kCols = 2 * BN + (KIND == kMx8 ? 32 : 0);
  static constexpr int kAlloc = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM columns");
  static constexpr int kThreads = KIND == kMx8 ? 224 : 192;
};

struct Bars {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2], sf_full[2], sf_empty[2], fin;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// 32 columns of a lane's row as fp32 to a box in shared memory whose rows are
// 128 bytes, 16-byte pieces in the 128-byte swizzle; `half`: of bf16, which 64
// bytes.
__device__ __forceinline__ void stage32(uint8_t* box, int lane, int, const float (&v)[32], float) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void stage32(uint8_t* box, int lane, int half, const float (&v)[32], __nv_bfloat16) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(box + lane * 128 + (((c + 4 * half) ^ (lane & 7)) << 4)) =
        make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                   pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
}
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// A warp's two boxes in turn, each to memory by one TMA store.
struct Staging {
  uint8_t* base;
  int lane, turn;
  __device__ __forceinline__ uint8_t* take() {  // the box of two stores ago has left
    if (lane == 0) bulk_wait_read1();
    __syncwarp();
    uint8_t* box = base + (turn & 1) * 4096;
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

template <int KIND, bool AMN, bool BMN, int BN, int EPI, typename OutT>
__global__ void __launch_bounds__(Layout<KIND, BN>::kThreads, 1)
gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using L = Layout<KIND, BN>;
  constexpr int S = L::kStages;
  constexpr int kHalfN = EPI == kGated ? BN / 2 : BN;  // columns of the output per tile
  constexpr bool kSum = sizeof(OutT) == 4 && BN <= 128;  // sums move to registers
  constexpr int kW = BN < 32 ? BN : 32;                  // columns read from TMEM at a time
  constexpr int kBox = 128 / sizeof(OutT);               // columns stored at a time
  static_assert(BN >= 32 || (kSum && EPI == kPlain), "16 columns are partial sums");
  extern __shared__ uint8_t raw[];
  uint8_t* sm = align1024(raw);
  uint8_t* staging = sm + S * L::kStage;
  uint8_t* scales = staging + L::kStaging;
  Bars& bars = *reinterpret_cast<Bars*>(scales + L::kScales);
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = p.m_tiles * p.n_tiles * p.parts * p.splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 4);
      mbar_init(&bars.sf_full[i], 1);
      mbar_init(&bars.sf_empty[i], 1);
    }
    mbar_init(&bars.fin, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem, L::kAlloc);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // all CTAs of the grid run at once: a join behind it may take its place
  cudaTriggerProgrammaticLaunchCompletion();
  const uint32_t tmem = bars.tmem;

  if (warp == 0) {
    // -------------------------------------------------------------- copies
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        tma_prefetch(&maps.a[i]);
        tma_prefetch(&maps.b[i]);
      }
      uint32_t n = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tile = tile_of(p, t);
        int pair = tile.it0 % p.pairs, kb = tile.it0 / p.pairs, kpart = 0;
        while (kb >= p.k_blocks) kb -= p.k_blocks, ++kpart;
        for (int it = tile.it0; it < tile.it1; ++it, ++n) {
          const int st = n % S;
          if (n >= S && !wait_or_fail(&bars.empty[st], (n / S - 1) & 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* a = sm + st * L::kStage;
          uint8_t* b = a + L::kA;
          uint64_t* bar = &bars.full[st];
          mbar_arrive_expect_tx(bar, L::kStage);
          // the terms of pair 0 .. 5, small products first: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
          const int pa = p.pairs == 1 ? 0 : (0x001102 >> (4 * pair)) & 15;
          const int pb = p.pairs == 1 ? 0 : (0x010120 >> (4 * pair)) & 15;
          const int k = kb * (KIND == kMx8 ? 128 : 64);
          const CUtensorMap* am = &maps.a[p.a_by == kByPart ? tile.part : p.a_by == kByKPart ? kpart : 0];
          const CUtensorMap* bm = &maps.b[p.b_by == kByPart ? tile.part : p.b_by == kByKPart ? kpart : 0];
          if (AMN) {
            tma_load_3d(a, am, bar, tile.m * 128, k, pa);
            tma_load_3d(a + 8192, am, bar, tile.m * 128 + 64, k, pa);
          } else {
            tma_load_3d(a, am, bar, k, tile.m * 128, pa);
          }
          if (EPI == kGated) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint8_t* bh = b + h * (BN / 2) * 128;
              if (BMN) {
                for (int i = 0; i < BN / 128; ++i)
                  tma_load_3d(bh + i * 8192, &maps.b[h], bar, tile.n * kHalfN + 64 * i, k, pb);
              } else {
                tma_load_3d(bh, &maps.b[h], bar, k, tile.n * kHalfN, pb);
              }
            }
          } else if (BMN) {
            for (int i = 0; i < BN / 64; ++i)
              tma_load_3d(b + i * 8192, bm, bar, tile.n * BN + 64 * i, k, pb);
          } else {
            tma_load_3d(b, bm, bar, k, tile.n * BN, pb);
          }
          if (++pair == p.pairs) {
            pair = 0;
            if (++kb == p.k_blocks) kb = 0, ++kpart;
          }
        }
      }
      // nothing may land in shared memory behind the kernel's end
      for (uint32_t i = n > S ? n - S : 0; i < n; ++i)
        mbar_wait(&bars.full[i % S], (i / S) & 1, nullptr, kWaitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, BN, AMN, BMN);
      uint32_t n = 0, nc = 0, ns = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tile = tile_of(p, t);
        uint32_t d = 0;
        int left = 0;  // steps of this accumulator
        for (int it = tile.it0; it < tile.it1; ++it, ++n) {
          const int st = n % S;
          const bool first = left == 0;
          if (first) {
            left = kSum ? min(p.chunk, tile.it1 - it) : tile.it1 - it;
            d = tmem + (nc & 1) * BN;
            if (nc >= 2 && !wait_or_fail(&bars.acc_empty[nc & 1], (nc / 2 - 1) & 1, p.status, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
          }
          uint32_t sf = 0;
          if (KIND == kMx8) {
            const uint32_t slot = ns & 1;
            sf = tmem + L::kScaleCol + slot * 16;
            if (it == tile.it0 || (it & 3) == 0) {
              if (!wait_or_fail(&bars.sf_full[slot], (ns / 2) & 1, p.status, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
              const uint8_t* from = scales + slot * (L::kScales / 2);
              copy_scales(sf, from);
#pragma unroll
              for (int i = 0; i < (BN + 127) / 128; ++i) copy_scales(sf + 4 + 4 * i, from + 512 + 512 * i);
            }
          }
          if (!wait_or_fail(&bars.full[st], (n / S) & 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a = smem_u32(sm + st * L::kStage), b = a + L::kA;
          const uint64_t ad = AMN ? smem_desc(a, 8192, 1024, SW_128B) : smem_desc(a, 16, 1024, SW_128B);
          const uint64_t bd = BMN ? smem_desc(b, 8192, 1024, SW_128B) : smem_desc(b, 16, 1024, SW_128B);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ak = ad + (AMN ? kk * 128 : kk * 2), bk = bd + (BMN ? kk * 128 : kk * 2);
            const uint32_t more = !first || kk > 0;
            if (KIND == kMx8)
              mma_mx8(d, ak, bk, idesc_mx8(128, BN, it & 3), sf, sf + 4, more);
            else
              mma_bf16(d, ak, bk, idesc, more);
          }
          mma_commit(&bars.empty[st]);
          if (KIND == kMx8 && (it + 1 == tile.it1 || (it & 3) == 3)) {
            mma_commit(&bars.sf_empty[ns & 1]);
            ++ns;
          }
          if (--left == 0) {
            mma_commit(&bars.acc_full[nc & 1]);
            ++nc;
          }
        }
      }
      // no product may be in flight when TMEM is freed
      mma_commit(&bars.fin);
      mbar_wait(&bars.fin, 0, nullptr, kWaitNs);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------- finished tiles
    const int quarter = warp & 3;
    Staging out{staging + (warp - 2) * 8192, lane, 0};
    uint32_t nc = 0;  // accumulators taken
    auto ready = [&] {
      if (!__all_sync(0xffffffffu, wait_or_fail(&bars.acc_full[nc & 1], (nc / 2) & 1, p.status, abort_flag)))
        return false;
      tc_fence_after_sync();
      return true;
    };
    auto release = [&] {  // the accumulator has been read
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.acc_empty[nc & 1]);
      ++nc;
    };
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile tile = tile_of(p, t);
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const int y = tile.m * 128 + quarter * 32, z = p.c_by_part ? 0 : tile.split * p.parts + tile.part;
      const CUtensorMap* cm = &maps.c[p.c_by_part ? tile.part : 0];
      float sum[kSum ? BN / kW : 1][kW];  // a lane's row
      if constexpr (kSum) {
        for (int it = tile.it0; it < tile.it1; it += min(p.chunk, tile.it1 - it)) {
          if (!ready()) {
            ok = false;
            break;
          }
          const uint32_t d = lanes + (nc & 1) * BN;
#pragma unroll
          for (int c = 0; c < BN / kW; ++c) {
            float v[kW];
            load_columns(d + c * kW, v);
#pragma unroll
            for (int i = 0; i < kW; ++i) sum[c][i] = it == tile.it0 ? v[i] : sum[c][i] + v[i];
          }
          release();
        }
        if (!ok) break;
      } else if (!ready()) {
        break;
      }
      const uint32_t d = lanes + (nc & 1) * BN;
      // 32 columns c .. of the tile
      auto columns = [&](int c, float(&v)[kW]) {
        if constexpr (kSum) {
#pragma unroll
          for (int i = 0; i < kW; ++i) v[i] = sum[c / kW][i];
        } else {
          load_columns(d + c, v);
        }
      };
      if constexpr (BN < 32) {
        uint8_t* box = out.take();  // rows of 64 bytes
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<float4*>(box + sw64_offset(lane, c * 16)) =
              make_float4(sum[0][4 * c], sum[0][4 * c + 1], sum[0][4 * c + 2], sum[0][4 * c + 3]);
        out.send(cm, box, tile.n * BN, y, z);
      } else if constexpr (EPI == kPlain) {
#pragma unroll kSum ? BN / kBox : 1
        for (int c = 0; c < BN; c += kBox) {
          uint8_t* box = out.take();
#pragma unroll
          for (int h = 0; h < kBox / 32; ++h) {
            float v[32];
            columns(c + 32 * h, v);
            stage32(box, lane, h, v, OutT{});
          }
          if (!kSum && c + kBox == BN) release();
          out.send(cm, box, tile.n * BN + c, y, z);
        }
      } else {
        constexpr int kH = kBox / 32;
        constexpr bool kFast = sizeof(OutT) == 2;
#pragma unroll kSum ? kHalfN / kBox : 1
        for (int c = 0; c < kHalfN; c += kBox) {
          float g[kH][32], u[kH][32];
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            columns(c + 32 * h, g[h]);
            columns(kHalfN + c + 32 * h, u[h]);
          }
          if (!kSum && c + kBox == kHalfN) release();
          const int x = tile.n * kHalfN + c;
          if (p.keep) {
            uint8_t* box = out.take();
#pragma unroll
            for (int h = 0; h < kH; ++h) stage32(box, lane, h, g[h], OutT{});
            out.send(&maps.c[1], box, x, y, 0);
            box = out.take();
#pragma unroll
            for (int h = 0; h < kH; ++h) stage32(box, lane, h, u[h], OutT{});
            out.send(&maps.c[2], box, x, y, 0);
          }
          act::by_act(p.act, [&](auto a) {
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
              for (int i = 0; i < 32; ++i) g[h][i] = act::value<decltype(a)::value, kFast>(g[h][i]) * u[h][i];
          });
          uint8_t* box = out.take();
#pragma unroll
          for (int h = 0; h < kH; ++h) stage32(box, lane, h, g[h], OutT{});
          out.send(&maps.c[0], box, x, y, 0);
        }
      }
    }
    if (lane == 0) bulk_wait0();
  } else if (KIND == kMx8) {
    // -------------------------------------------------------------- scales
    // Words of four K blocks: rows lane, lane + 32, + 64, + 96 side by side.
    uint32_t ns = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile tile = tile_of(p, t);
      for (int g = tile.it0 >> 2; g <= (tile.it1 - 1) >> 2; ++g, ++ns) {
        const uint32_t slot = ns & 1;
        uint4 w[1 + (BN + 127) / 128];
        auto four = [&](const uint32_t* s, int rows, int r0) {
          const uint32_t* at = s + (size_t)g * rows;
          auto one = [&](int r) { return r < rows ? at[r] : 0u; };
          return make_uint4(one(r0 + lane), one(r0 + lane + 32), one(r0 + lane + 64), one(r0 + lane + 96));
        };
        w[0] = four(p.a_scales, p.a_rows, tile.m * 128);
#pragma unroll
        for (int i = 0; i < (BN + 127) / 128; ++i)
          w[1 + i] = four(p.b_scales, p.b_rows, tile.n * BN + 128 * i);
        if (ns >= 2) {
          const bool free = wait_or_fail(&bars.sf_empty[slot], (ns / 2 - 1) & 1, p.status, abort_flag);
          if (!__all_sync(0xffffffffu, free)) {
            ok = false;
            break;
          }
        }
        uint4* to = reinterpret_cast<uint4*>(scales + slot * (L::kScales / 2));
#pragma unroll
        for (int i = 0; i < 1 + (BN + 127) / 128; ++i) to[32 * i + lane] = w[i];
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sf_full[slot]);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, L::kAlloc);
}

// ------------------------------------------------------------------- host

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
// Results in boxes of 32 rows x 128 bytes, or x 64 where a row has no more.
inline bool map_out(CUtensorMap* map, const Matrix& x, bool narrow = false) {
  return make_map(map, x, (narrow ? 64 : 128) / x.esize, 32,
                  narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Sums of the partial planes of a split product (nys_join.cu): part holds
// `splits` x `parts` planes of fp32, plane split * parts + part, each [M][N]
// (rows of a result) or, turned, [N][width] (a result's columns, its rows
// side by side). Results in dtype; set up while the product still runs.
struct Join {
  const float* part;
  int splits, M, N, width;  // width: 0, or of turned planes
  void* out[2];             // [M][N] of part 0, 1
  long long stride[2];
};
int join(const Join& j, int parts, int dtype, cudaStream_t st);
// part 0: g, part 1: u; h = act(g) u, and g, u where gate, up are set.
struct JoinGated {
  const float* part;
  int splits, M, N, width;
  void *h, *gate, *up;
  long long h_stride, gate_stride, up_stride;
};
int join_gated(const JoinGated& j, int act, int dtype, cudaStream_t st);

template <int KIND, bool AMN, bool BMN, int BN, int EPI, typename OutT>
int launch(const char* name, const Maps& maps, const Params& p, cudaStream_t st) {
  using L = Layout<KIND, BN>;
  auto kernel = gemm_kernel<KIND, AMN, BMN, BN, EPI, OutT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
    return set_cuda_error(cudaGetLastError());
  const long long tiles = (long long)p.m_tiles * p.n_tiles * p.parts * p.splits;
  if (tiles >= (1ll << 31) - 1024) return NYS_ERR_SHAPE;
  const int sms = plan_sms();
  if (p.chunk < 1) return NYS_ERR_ARG;
  KernelScope scope(name, st);
  kernel<<<tiles < sms ? (int)tiles : sms, L::kThreads, L::kBytes, st>>>(maps, p);
  return launch_status();
}

// Ranges of K that fill the SMs: as many as leave the last round of tiles
// fullest, each at least `least` steps long, one where the tiles alone give
// whole rounds. More ranges cost partial sums, taken as `cost` steps each.
inline int splits_of(long long tiles, int its, int least, int most, double cost) {
  const int sms = plan_sms();
  int best = 1;
  double best_time = 1e30;
  for (int s = 1; s <= most && (s == 1 || its / s >= least); ++s) {
    const int per = (its + s - 1) / s;
    if ((its + per - 1) / per != s) continue;  // no empty range
    const double rounds = (double)((tiles * s + sms - 1) / sms);
    const double time = rounds * (per + (s > 1 ? cost : 0.0)) + (s > 1 ? 2 * cost : 0.0);
    if (time < best_time * 0.999) best_time = time, best = s;
  }
  return best;
}

}  // namespace gemm
}  // namespace nys
