// Chunks of queries over the 4-bit cache on the fifth-generation tensor cores
// (bf16, d in {64, 128}; the operator: include/nystrom.h):
//   out = softmax(q K^T scale) V,  K = s_k c_k, V = s_v c_v per 32 channels.
//
// One CTA per SM takes a range of the line of 128-key tiles (nys_kv4_attn.h)
// for items of 256 query rows: two groups of 128 rows that share every tile,
// so that a tile is unpacked once for 256 rows, and whose softmax and products
// alternate. Per tile and group g:
//   S_g = Q_g K^T           tcgen05, both operands in shared memory
//   p = 2^(S f - M)         thread = query row, S from tensor memory; P (fp16)
//                           overwrites S; the running maximum moves when it
//                           grows by more than 2^4 (O_g is rescaled then)
//   O_g += P V              tcgen05, P from tensor memory, V channels innermost
// Warps 0-3, 4-7: the groups' softmax; one thread of a group issues its products
// (P V of a tile, then S of the next), so that nobody else has to be woken.
// Warps 8-11 (K) and 12-15 (V): unpack 32 keys each of every tile into swizzled
// fp16 operands.
//
// fp16 operands: code * scale has 11 bits, as fp16 does (bf16 would keep 8, which
// alone would cost as much as rounding the result does). fp16's range is met by
// powers of two: a query row is scaled to 2^13 .. 2^14, the keys and the values
// of each 32 tokens by their largest scale; the factors come back in the exponent
// of p (keys: f, values: added to it, and taken out of the sum again), so each 32
// tokens and each row have their own. Keys and values use all of fp16's range, so
// that those of scales up to 2^29 below the largest of their 32 tokens are exact:
// a score is as if its operands were fp32 ones, and what is rounded is p. Where
// the value scales of 32 tokens span more than that, those keys' p and V are bf16
// (the instruction's types are chosen per 16 keys). The unpacking keeps the order
// of the 4-bit fields: the queries' channels are permuted to match, and the
// output's columns are put right when they are written.
//
// 1000 queries x 16 + 4 heads over 8192 tokens of 2 sequences, d = 128: 174 us
// here, 187 with the join, 672 TFLOP/s (over 16384 tokens 322 here, 335, 775).
// Tensor cores 33 % busy, HBM 1 %. Clock stamps: a tile of a group is a chain of 5900
// cycles - softmax 2600 (about 900 instructions of a warp), the products 1700
// (100 per issued instruction, the pipe's own time is 68), their handshakes and
// the last one's end 1300 -, of which the other group's softmax and products
// fill the gaps. Not kept: halves of 64 keys with the next scores under way (a
// shorter chain, twice the handshakes: 244 us against 196 then); two threads per
// row in 24 warps (191 against 176: exponentials and conversions share pipes).
//
// Every wait is bounded; one that runs out sets the status word, all roles wind
// down, and tensor memory is freed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "nys_kv4_attn.h"

namespace nys {
namespace kv4 {
namespace {

using namespace sm100;
using L = ChunkLine;

constexpr int kThreads = 16 * 32;
constexpr int kSlots = 2;  // K tiles and V tiles in shared memory
constexpr int kInfo = 4;   // tiles whose facts are kept
// p is at most 2^(kLift + kRebase), close to fp16's largest number: full 11 bits
// for keys down to 2^-25 of the row's largest p, 2^-36 of that the least that is
// seen. (The running maximum moves when it grows by more than 2^kRebase.)
constexpr float kRebase = 4.0f, kLift = 11.0f;
constexpr int kNarrow = 29;  // value scales of 32 tokens within 2^29: fp16
constexpr int kLeast = -68;  // the least power of two of 32 tokens' scales: keeps 1 / factor, times p, in range
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kSpins = 1 << 20;  // waits of up to 20 us each

// What a tile's softmax has to know, per 32 tokens: the powers of two of keys
// and values, and the tokens that must not enter a sum as they are.
struct TileInfo {
  float k2e[4];       // keys' factor, times 2^12
  float ev[4];        // log2 of the values' factor
  float vinv[4];      // its inverse
  alignas(16) uint32_t wide[4];  // p and V of these keys are bf16
  uint32_t have[4];   // which of the 32 tokens exist
  uint32_t odd[4];    // some value scale is infinite or NaN:
  uint32_t odd_of[4][4];  // [32 tokens][group]: which ones
};

struct Shared {
  uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
  uint64_t s_full[2], pv_done[2], fin;
  TileInfo info[kInfo];
  Start start;
  int warp_sums[kThreads / 32];
  uint32_t tmem;
  int abort;
  int turn;  // whether a group has the tensor cores
};

// The code is kept short where it can be (plain bounded spins, loops over
// pairs of 32 keys): the roles' loops share the SM's instruction caches.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, int* status,
                                             volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kSpins; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  atomicExch(status, (int)NYS_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_or_fail(bar, parity, status, abort_flag));
}

// A group's products, those of a tile's values and of the next tile's keys, run
// in one go: with both groups' interleaved, both would wait for all of them and
// then share the issue slots for their softmax. This orders time, not data: a
// thread that has waited long goes ahead.
__device__ __forceinline__ void take_turn(int* turn) {
#pragma unroll 1
  for (int i = 0; i < 4096 && atomicCAS(turn, 0, 1) != 0; ++i) {
  }
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b),
                            reinterpret_cast<const __half2&>(c));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight fields u of w to (u - 8) a, exactly: 1024 + u or, four bits up, 1024 +
// 16 u by putting the field into the mantissa of 1024, brought to u - 8, times a.
// A code of up to 7 times an 8-bit scale has 11 bits, as many as fp16.
__device__ __forceinline__ uint4 unpack8(uint32_t w, uint32_t a) {
  auto one = [&](uint32_t u_less_8) { return half2_mul(u_less_8, a); };
  const uint32_t k = 0x64006400u, sixteenth = 0x2c002c00u;  // 1024, 1/16
  return make_uint4(one(half2_fma((w & 0x000f000fu) | k, 0x3c003c00u, 0xe408e408u)),  // less 1032
                    one(half2_fma((w & 0x00f000f0u) | k, sixteenth, 0xd480d480u)),    // less 72
                    one(half2_fma(((w >> 8) & 0x000f000fu) | k, 0x3c003c00u, 0xe408e408u)),
                    one(half2_fma(((w >> 8) & 0x00f000f0u) | k, sixteenth, 0xd480d480u)));
}

// The same as bf16 (u - 8) a, a in bf16: u 2^-133 or u 2^-129 to (u - 8) 2^-6,
// times a (the one rounding), times 2^6.
__device__ __forceinline__ uint4 unpack8_wide(uint32_t w, uint32_t a) {
  auto one = [&](uint32_t f, uint32_t up) {
    const uint32_t eighth = 0xbe00be00u, six = 0x42804280u;  // -1/8, 2^6
    const __nv_bfloat162 c = __hfma2(reinterpret_cast<const __nv_bfloat162&>(f),
                                     reinterpret_cast<const __nv_bfloat162&>(up),
                                     reinterpret_cast<const __nv_bfloat162&>(eighth));
    const __nv_bfloat162 v = __hmul2(__hmul2(c, reinterpret_cast<const __nv_bfloat162&>(a)),
                                     reinterpret_cast<const __nv_bfloat162&>(six));
    return reinterpret_cast<const uint32_t&>(v);
  };
  return make_uint4(one(w & 0x000f000fu, 0x7f007f00u), one(w & 0x00f000f0u, 0x7d007d00u),
                    one((w >> 8) & 0x000f000fu, 0x7f007f00u), one((w >> 8) & 0x00f000f0u, 0x7d007d00u));
}

// a * b + c on two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return reinterpret_cast<float2&>(d);
}

// Tiles of a segment that some row sees, and the groups of rows it has.
__device__ __forceinline__ int tiles_seen(const Segment& sg) {
  return min(sg.tile0 + sg.ntile, (sg.seen_max + L::TILE - 1) / L::TILE) - sg.tile0;
}
__device__ __forceinline__ int groups_of(const Segment& sg) { return sg.rows > 128 ? 2 : 1; }

template <int D>
constexpr uint32_t tile_bytes() { return D / 64 * 16384; }
template <int D>
constexpr int stage_bytes() { return 32 * (D / 32) * 2; }  // a warp's scales as fp16
template <int D>
constexpr int chunk_smem() { return (2 + 2 * kSlots) * tile_bytes<D>() + 8 * stage_bytes<D>() + 1024; }

// One of the eight unpacking warps: 32 keys (KEYS) or values of every tile.
template <int D, bool KEYS>
__device__ __forceinline__ void unpack_tiles(const AttnParams& p, Shared& sh, uint8_t* slots, __half* stage,
                                             int part, int pos, int r1, int base, int b) {
  constexpr int G = D / 32, BB = block_bytes(D);
  volatile int* abort_flag = &sh.abort;
  const int lane = threadIdx.x & 31;
  uint64_t* full = KEYS ? sh.k_full : sh.v_full;
  uint64_t* empty = KEYS ? sh.k_empty : sh.v_empty;
  uint32_t n = 0;  // tiles done by this CTA
  Segment sg;
  while (next_segment<L>(p, pos, r1, base, b, sg)) {
    const int tiles = tiles_seen(sg);
    const uint8_t* src = nullptr;  // lane: block (lane & 1) of tile (lane >> 1) of the window
    uint4 raw[4];                  // codes of the next tile (d = 64: two words of each)
    uint2 raw_s;                   // its scales
    uint32_t have = 0;             // tokens of it that exist
    auto fetch = [&](int i) {
      if ((i & 15) == 0) {
        const int key = (sg.tile0 + i + (lane >> 1)) * L::TILE + part * 32 + (lane & 1) * kBlock;
        src = nullptr;
        if (i + (lane >> 1) < tiles && key < sg.seen_max) {
          src = block_at(p.cache, sg.b, sg.h, key, D);
          if (!src && KEYS) report_index(p.status);
        }
      }
      const uint8_t* blk[2];
      have = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        blk[h] = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), (i & 15) * 2 + h));
        if (blk[h]) have |= 0xffffu << (16 * h);
      }
      const int first = (sg.tile0 + i) * L::TILE + part * 32;
      if (first + 32 > sg.seen_max) have &= sg.seen_max > first ? (1u << (sg.seen_max - first)) - 1u : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* at = blk[k >> 1];
        raw[k] = make_uint4(0u, 0u, 0u, 0u);
        if (at) {
          // keys: row (k & 1) 8 + lane % 8, its quarter lane / 8; values: the
          // lane's place in the half block
          at += KEYS ? ((k & 1) * 8 + (lane & 7)) * (D / 2) + (lane >> 3) * (D / 8)
                     : v_codes(D) + (k & 1) * 4 * D + lane * (D / 8);
          if (D == 128) {
            raw[k] = *reinterpret_cast<const uint4*>(at);
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(at);
            raw[k].x = u.x;
            raw[k].y = u.y;
          }
        }
      }
      raw_s = make_uint2(0u, 0u);
      const uint8_t* at = blk[lane >> 4];
      if (at) {  // 16 lanes per block: four (d = 64: two) tokens of one group each
        at += (KEYS ? k_scales(D) : v_scales(D)) + (lane & 15) * (D / 16);
        if (D == 128) raw_s = *reinterpret_cast<const uint2*>(at);
        else raw_s.x = *reinterpret_cast<const uint32_t*>(at);
      }
    };
#pragma unroll 1
    for (int i = -1; i < tiles; ++i) {
      uint4 now[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) now[k] = raw[k];
      const uint2 now_s = raw_s;
      const uint32_t now_have = have;
      if (i + 1 < tiles) fetch(i + 1);
      if (i < 0) continue;
      const int slot = n % kSlots;
      TileInfo& info = sh.info[n % kInfo];
      // ---- scales: the largest one's exponent, then fp16 in [token][group]
      constexpr int N = D / 32;  // tokens per lane (= groups, by chance of the layout)
      const int y = (lane & 15) / (16 / G), tok = (lane >> 4) * 16 + (lane & 15) % (16 / G) * N;
      uint32_t bits[N];
      int top = 0, low = 255;
      bool odd = false;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t w = j < 2 ? now_s.x : now_s.y;
        bits[j] = (j & 1) ? w & 0xffff0000u : w << 16;
        if (!(now_have >> (tok + j) & 1u)) bits[j] = 0u;
        const int e = (int)(bits[j] >> 23 & 255u);
        odd = odd || e == 255;
        top = max(top, e == 255 ? 0 : e);
        if (bits[j] != 0u) low = min(low, e);
      }
      const int biased = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
      const bool wide = !KEYS && biased > (int)__reduce_min_sync(0xffffffffu, (unsigned)low) + kNarrow;
      top = max(biased - 127, kLeast);
      const bool any_odd = __any_sync(0xffffffffu, odd);
      const float factor = __uint_as_float((uint32_t)(127 + 12 - top) << 23);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const bool drop = !KEYS && (bits[j] >> 23 & 255u) == 255u;  // told to the softmax below
        const float a = drop ? 0.f : __uint_as_float(bits[j]) * factor;
        stage[(tok + j) * G + y] = wide ? __ushort_as_half(__float_as_uint(a) >> 16) : __float2half_rn(a);
      }
      // the facts of tile n - kInfo are no longer needed: the products that
      // freed this slot came after its softmax
      if (n >= (uint32_t)kSlots &&
          !warp_wait(&empty[slot], (n / kSlots - 1) & 1u, p.status, abort_flag))
        return;
      if (lane == 0) {
        if (KEYS) {
          info.k2e[part] = __uint_as_float((uint32_t)(127 + top) << 23);
          info.have[part] = now_have;
        } else {
          info.ev[part] = (float)(top - 12);
          info.vinv[part] = exp2f((float)(12 - top));
          info.wide[part] = wide ? 1u : 0u;
          info.odd[part] = any_odd ? 1u : 0u;
        }
      }
      if (!KEYS && any_odd) {
        if (lane < 4) info.odd_of[part][lane] = 0u;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < N; ++j)
          if ((bits[j] >> 23 & 255u) == 255u) atomicOr(&info.odd_of[part][y], 1u << (tok + j));
      }
      __syncwarp();
      // ---- codes, a vector at a time (rolled: the registers move up)
      uint8_t* dst = slots + slot * tile_bytes<D>();
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint32_t w[4] = {now[0].x, now[0].y, now[0].z, now[0].w};
        now[0] = now[1];
        now[1] = now[2];
        now[2] = now[3];
        if (KEYS) {
          const int token = k * 8 + (lane & 7), row = part * 32 + token;
          const uint16_t* a = reinterpret_cast<const uint16_t*>(stage) + token * G;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t chunk = (uint32_t)((g & 1) * 4 + (lane >> 3)) ^ (row & 7u);
            *reinterpret_cast<uint4*>(dst + (g >> 1) * 16384 + row * 128 + (chunk << 4)) =
                unpack8(w[g], a[g] * 0x10001u);
          }
        } else {
          // tokens 2t, 2t + 1 of the half block, pairs of groups
          auto values = [&](auto&& unpack) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int token = k * 8 + 2 * (lane & 3) + e, row = part * 32 + token;
              const uint32_t* a = reinterpret_cast<const uint32_t*>(stage) + token * (G / 2);
              const uint32_t chunk = (uint32_t)(lane >> 2) ^ (row & 7u);
#pragma unroll
              for (int pr = 0; pr < G / 2; ++pr)
                *reinterpret_cast<uint4*>(dst + pr * 16384 + row * 128 + (chunk << 4)) =
                    unpack(w[e * (G / 2) + pr], a[pr]);
            }
          };
          if (wide) values([](uint32_t f, uint32_t a) { return unpack8_wide(f, a); });
          else values([](uint32_t f, uint32_t a) { return unpack8(f, a); });
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[slot]);
      ++n;
    }
  }
}

// The 128 threads of a group meet (named barriers 1 and 2); true for all of
// them if any gave up at a wait, so that they leave together.
__device__ __forceinline__ bool group_failed(int g, bool failed) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(failed ? 1u : 0u), "r"(g + 1)
      : "memory");
  return any != 0;
}

// A softmax group: 128 query rows, one per thread.
template <int D>
__device__ __forceinline__ void softmax_rows(const AttnParams& p, Shared& sh, uint8_t* q_s, const uint8_t* k_s,
                                             const uint8_t* v_s, uint32_t tmem, int g,
                                             const __nv_bfloat16* q, __nv_bfloat16* out, int pos, int r1,
                                             int base, int b) {
  constexpr int G = D / 32;
  volatile int* abort_flag = &sh.abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lr = (warp & 3) * 32 + lane;  // tensor memory lane = row of the group
  const uint32_t lo = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t scol = tmem + lo + 128 * g, ocol = tmem + lo + 256 + g * D;
  uint8_t* qs = q_s + g * tile_bytes<D>();
  const uint32_t id_s = idesc_f16(128, 128), id_v = idesc_f16(128, D, true);
  const uint32_t id_w = idesc_bf16(128, D, false, true);
  uint32_t n = 0, n_s = 0;  // tiles of the CTA; of this group
  // One thread of the group: S of tile t, once its keys are there; P V of tile
  // t; and a slot of it that the group is done with. Both groups pass every tile
  // of the CTA in order, one without rows in the segment too: a slot is filled
  // anew only behind both, so nobody is ever more than one use of a slot away
  // from anybody else, which is as far as the barriers' one bit of phase tells.
  auto keys_there = [&](uint32_t t) {
    return wait_or_fail(&sh.k_full[t % kSlots], (t / kSlots) & 1u, p.status, abort_flag);
  };
  auto release = [&](uint64_t* empty, uint32_t t) { mbar_arrive(&empty[t % kSlots]); };
  auto issue_scores = [&](uint32_t t) {
    const int slot = t % kSlots;
    tc_fence_after_sync();
    const uint64_t a0 = smem_desc(smem_u32(qs), 16, 1024, SW_128B);
    const uint64_t b0 = smem_desc(smem_u32(k_s + slot * tile_bytes<D>()), 16, 1024, SW_128B);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);  // 16 KB chunk, 32 B step
      mma_bf16(tmem + 128 * g, a0 + off, b0 + off, id_s, kk > 0);
    }
    mma_commit(&sh.s_full[g]);
  };
  auto issue_values = [&](uint32_t t, bool first) {
    const int slot = t % kSlots;
    const uint64_t v0 = smem_desc(smem_u32(v_s + slot * tile_bytes<D>()), 16384, 1024, SW_128B);
    const uint4 wide = *reinterpret_cast<const uint4*>(sh.info[t % kInfo].wide);
    const uint32_t id[4] = {wide.x ? id_w : id_v, wide.y ? id_w : id_v, wide.z ? id_w : id_v, wide.w ? id_w : id_v};
    tc_fence_after_sync();
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)  // 16 keys: 2 KB of V, 8 columns of P
      mma_bf16_tA(tmem + 256 + g * D, tmem + 128 * g + kk * 8, v0 + (uint64_t)(kk * 128),
                  id[kk >> 1], (!first || kk > 0) ? 1u : 0u);
    mma_commit(&sh.pv_done[g]);
  };
  const bool leader = lr == 0;
  bool ok = true;
  Segment sg;
  while (next_segment<L>(p, pos, r1, base, b, sg)) {
    const int tiles = max(0, tiles_seen(sg));
    if (g >= groups_of(sg)) {  // no rows here: pass the tiles
      if (leader) {
#pragma unroll 1
        for (uint32_t t = n; ok && t < n + tiles; ++t) {
          ok = keys_there(t);
          if (!ok) break;
          release(sh.k_empty, t);
          ok = wait_or_fail(&sh.v_full[t % kSlots], (t / kSlots) & 1u, p.status, abort_flag);
          if (ok) release(sh.v_empty, t);
        }
      }
      __syncwarp();
      n += tiles;
      continue;
    }
    const int r = g * 128 + lr, row = sg.rt * L::ROWS + r;
    const bool live = r < sg.rows;
    const int qi = live ? row / p.rep : 0, hq = sg.h * p.rep + (live ? row - qi * p.rep : 0);
    const int seen = live && p.causal ? max(0, sg.len - sg.count + 1 + qi) : sg.len;
    const int warp_seen = __reduce_min_sync(0xffffffffu, seen);
    float m = -INFINITY, l = 0.f;
    uint32_t poison = 0;  // groups of channels that met a NaN
    if (tiles > 0) {
      // ---- the row's operand: scaled, fp16, fields' order (read twice rather
      // than held)
      float top = 0.f;
      bool finite = true;
      const uint4* src = reinterpret_cast<const uint4*>(q + sg.b * p.qs.batch + hq * p.qs.head + qi * p.qs.token);
#pragma unroll 8
      for (int k = 0; k < D / 8; ++k) {
        const uint4 x = live ? src[k] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = fabsf(__uint_as_float(w[j] << 16)), c = fabsf(__uint_as_float(w[j] & 0xffff0000u));
          top = fmaxf(top, fmaxf(a, c));
          finite = finite && a < INFINITY && c < INFINITY;
        }
      }
      const bool tiny = top < 0x1p-60f;
      if (tiny) top *= 0x1p80f;
      const int e = top > 0.f ? (int)(__float_as_uint(top) >> 23) - 127 : 13;
      float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
      const float pre = !finite ? 0.f : tiny ? 0x1p80f : 1.f;
      if (p.scale_log2 < 0.f) up = -up;
      // units of a score, less the keys' power of two
      float rf = fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + max(e - 13, -100)) << 23);
      rf = !finite ? NAN : rf * 0x1p-12f * (tiny ? 0x1p-80f : 1.f);
#pragma unroll 1
      for (int k0 = 0; k0 < D / 8; k0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = live ? src[k0 + j] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // k0 + c: group k / 4, quarter k % 4
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[2 * j] = finite ? __uint_as_float(w[j] << 16) * pre * up : 0.f;
            v[2 * j + 1] = finite ? __uint_as_float(w[j] & 0xffff0000u) * pre * up : 0.f;
          }
          *reinterpret_cast<uint4*>(qs + (k0 >> 3) * 16384 + lr * 128 + ((c ^ (lr & 7)) << 4)) =
              make_uint4(pack_half2(v[0], v[4]), pack_half2(v[1], v[5]), pack_half2(v[2], v[6]),
                         pack_half2(v[3], v[7]));
        }
      }
      fence_async_smem();
      tc_fence_before_sync();  // the previous segment's output has been read
      if (group_failed(g, !ok)) return;
      if (leader && keys_there(n)) issue_scores(n);
      __syncwarp();

#pragma unroll 1
      for (int i = 0; i < tiles; ++i, ++n, ++n_s) {
        const int key0 = (sg.tile0 + i) * L::TILE;
        ok = warp_wait(&sh.v_full[n % kSlots], (n / kSlots) & 1u, p.status, abort_flag) &&
             warp_wait(&sh.s_full[g], n_s & 1u, p.status, abort_flag);
        if (!ok) {
          group_failed(g, true);
          return;
        }
        tc_fence_after_sync();
        if (leader) release(sh.k_empty, n);
        const TileInfo& info = sh.info[n % kInfo];
        // tokens of 32-key chunk c that this row sees
        auto visible = [&](int c) {
          const int v = seen - key0 - 32 * c;
          return (v >= 32 ? 0xffffffffu : v <= 0 ? 0u : (1u << v) - 1u) & info.have[c];
        };
        const bool all = key0 + L::TILE <= warp_seen &&
                         (info.have[0] & info.have[1] & info.have[2] & info.have[3]) == 0xffffffffu;
        float alpha = 1.f;
        // `masked` in a copy of its own: the common tiles run without its code
        auto weigh = [&](auto masked) {
          float cand = -INFINITY;
          uint32_t x[2][32];
          // two passes over pairs of 32 keys; the second starts on the pair that
          // the first left in registers
#pragma unroll 1
          for (int pr = 1; pr >= 0; --pr) {
            tmem_ld32(scol + 64 * pr, x[0]);
            tmem_ld32(scol + 64 * pr + 32, x[1]);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 2 * pr + h;
              if (decltype(masked)::value) {
                const uint32_t vis = visible(c);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!(vis >> k & 1u)) x[h][k] = 0xff800000u;
              }
              float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int k = 0; k < 32; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(x[h][k]));
              const float mx = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
              if (mx > -INFINITY) cand = fmaxf(cand, fmaf(mx, rf * info.k2e[c], info.ev[c]));
            }
          }
          if (cand > m && (m == -INFINITY || cand - m > kRebase)) {
            alpha = m == -INFINITY ? 0.f : fast_exp2(m - cand);
            l *= alpha;
            m = cand;
          }
          const float ref = m == -INFINITY ? 0.f : m - kLift;
#pragma unroll 1
          for (int pr = 0; pr < 2; ++pr) {
            if (pr) {
              tmem_ld32(scol + 64, x[0]);
              tmem_ld32(scol + 96, x[1]);
              tmem_ld_wait();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 2 * pr + h;
              const float f = rf * info.k2e[c], off = info.ev[c] - ref;
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float2 e2 = fma2(make_float2(__uint_as_float(x[h][2 * k]), __uint_as_float(x[h][2 * k + 1])),
                                 make_float2(f, f), make_float2(off, off));
                x[h][2 * k] = __float_as_uint(fast_exp2(e2.x));
                x[h][2 * k + 1] = __float_as_uint(fast_exp2(e2.y));
              }
              if (decltype(masked)::value) {
                const uint32_t vis = visible(c);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!(vis >> k & 1u)) x[h][k] = 0u;
              }
#pragma unroll
              for (int k = 0; k < 16; ++k)
                sum[k & 1] = fma2(make_float2(__uint_as_float(x[h][2 * k]), __uint_as_float(x[h][2 * k + 1])),
                                  make_float2(1.f, 1.f), sum[k & 1]);
              if (info.wide[c]) {  // packed in place
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  x[h][k] = pack_bf16x2(__uint_as_float(x[h][2 * k]), __uint_as_float(x[h][2 * k + 1]));
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  x[h][k] = pack_half2(__uint_as_float(x[h][2 * k]), __uint_as_float(x[h][2 * k + 1]));
              }
              tmem_st16(scol + 16 * c, reinterpret_cast<const uint32_t(&)[16]>(x[h]));
              l = fmaf((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), info.vinv[c], l);
            }
          }
        };
        if (all) weigh(std::integral_constant<bool, false>{});
        else weigh(std::integral_constant<bool, true>{});
        if (info.odd[0] | info.odd[1] | info.odd[2] | info.odd[3]) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
            if (info.odd[c])
              for (int y = 0; y < G; ++y)
                if (info.odd_of[c][y] & visible(c)) poison |= 1u << y;
          __syncwarp();
        }
        if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // the group's earlier products are done: S of this tile waited for them
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(ocol + c0, o);
            tmem_ld_wait();
#pragma unroll
            for (int e2 = 0; e2 < 32; ++e2) o[e2] = __float_as_uint(__uint_as_float(o[e2]) * alpha);
            tmem_st32(ocol + c0, o);
          }
        }
        tmem_st_wait();
        tc_fence_before_sync();
        if (group_failed(g, false)) return;
        if (leader) {
          take_turn(&sh.turn);
          issue_values(n, i == 0);
          if (i + 1 < tiles) {
            bool there = mbar_test(&sh.k_full[(n + 1) % kSlots], ((n + 1) / kSlots) & 1u);
            // S is this tile's P until its product is done
            if (wait_or_fail(&sh.pv_done[g], n_s & 1u, p.status, abort_flag)) {
              if (!there) {  // their slot may be waiting for the other group
                atomicExch(&sh.turn, 0);
                there = keys_there(n + 1);
                take_turn(&sh.turn);
              }
              if (there) issue_scores(n + 1);
              release(sh.v_empty, n);
            }
          }
          atomicExch(&sh.turn, 0);
        }
        __syncwarp();
      }
      ok = warp_wait(&sh.pv_done[g], (n_s - 1) & 1u, p.status, abort_flag);
      if (!ok) continue;  // to where the group meets next
      tc_fence_after_sync();
      if (leader) release(sh.v_empty, n - 1);
    }
    // ---- the row's output: columns back in channels' order
    const bool whole = sg.whole(L::TILE);
    const float norm = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* dst = out + sg.b * p.os.batch + hq * p.os.head + qi * p.os.token;
    const size_t part = part_slot(sg) * L::ROWS + r;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      __syncwarp();
      if (tiles > 0) {
        tmem_ld32(ocol + c0, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
      }
      // columns 8 j + 2 i + x: group 2 (c0 / 64) + x, its channels 4 (j0 + j) + i
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int y = c0 / 64 * 2 + x, ch = 32 * y + (c0 % 64) / 2;
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          v[k] = __uint_as_float(o[8 * (k / 4) + 2 * (k % 4) + x]) * norm;
          if (poison >> y & 1u) v[k] = NAN;
        }
        if (!live) continue;
        if (whole) {
          uint4* to = reinterpret_cast<uint4*>(dst + ch);
          to[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
          to[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                             pack_bf16x2(v[14], v[15]));
        } else {
          // whole sectors: 32 bytes a lane
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p.part + part * D + ch + k),
                         "f"(v[k]), "f"(v[k + 1]), "f"(v[k + 2]), "f"(v[k + 3]), "f"(v[k + 4]), "f"(v[k + 5]),
                         "f"(v[k + 6]), "f"(v[k + 7])
                         : "memory");
        }
      }
    }
    if (live && !whole) p.part_ml[part] = make_float2(m, l);
  }
}

// out may be q: a row is read by its thread before it is written, or, where CTAs
// share the item, by all of them before the join writes.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kv4_attn_chunk(const __grid_constant__ AttnParams p, const __nv_bfloat16* q, __nv_bfloat16* out) {
  constexpr uint32_t TILE = tile_bytes<D>();
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* sm = align1024(smem_raw);
  uint8_t *q_s = sm, *k_s = sm + 2 * TILE, *v_s = k_s + kSlots * TILE;
  __half* stage = reinterpret_cast<__half*>(v_s + kSlots * TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.k_empty[i], 2);
      mbar_init(&sh.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.fin, 2);
    sh.abort = 0;
    sh.turn = 0;
    fence_barrier_init();
  }
  cudaTriggerProgrammaticLaunchCompletion();
  if (warp == 8) tmem_alloc(&sh.tmem, 512);
  tc_fence_before_sync();
  find_start<L, kThreads>(p, &sh.start, sh.warp_sums);  // two block syncs
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  int pos = (int)min((long long)blockIdx.x * sh.start.per, (long long)sh.start.total);
  const int r1 = min(sh.start.total, pos + sh.start.per);
  int base = sh.start.base, b = sh.start.b;

  if (warp < 8) {
    softmax_rows<D>(p, sh, q_s, k_s, v_s, tmem, warp >> 2, q, out, pos, r1, base, b);
    if ((warp & 3) == 0 && lane == 0) mma_commit(&sh.fin);  // behind all this thread issued
  } else if (warp < 12) {
    unpack_tiles<D, true>(p, sh, k_s, stage + (warp - 8) * 32 * (D / 32), warp - 8, pos, r1, base, b);
  } else {
    unpack_tiles<D, false>(p, sh, v_s, stage + (warp - 8) * 32 * (D / 32), warp - 12, pos, r1, base, b);
  }
  if (warp == 8) {  // no product is in flight when tensor memory is freed
    if (lane == 0) mbar_wait(&sh.fin, 0, nullptr, kWaitNs);
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D>
int launch(const AttnParams& p, const void* q, void* out, cudaStream_t st) {
  constexpr int smem = chunk_smem<D>();
  if (cudaFuncSetAttribute(kv4_attn_chunk<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return set_cuda_error(cudaGetLastError());
  KernelScope scope("kv4_attn_chunk", st);
  kv4_attn_chunk<D><<<p.ctas, kThreads, smem, st>>>(p, static_cast<const __nv_bfloat16*>(q),
                                                  static_cast<__nv_bfloat16*>(out));
  return launch_status();
}

}  // namespace

int launch_kv4_chunk(const AttnParams& p, int d, const void* q, void* out, cudaStream_t stream) {
  return d == 64 ? launch<64>(p, q, out, stream) : launch<128>(p, q, out, stream);
}

}  // namespace kv4
}  // namespace nys
