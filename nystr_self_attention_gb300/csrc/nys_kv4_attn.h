// What the kernels of attention over the 4-bit cache share: the call's
// parameters and the line of key tiles that its CTAs divide.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nys_kv4.h"
#include "nys_sm100.h"

namespace nys {
namespace kv4 {

struct AttnParams {
  View cache;
  nys_strides_t qs, os;
  const int *lengths, *q_counts;
  int* status;
  float* part;      // [CTAs][2][item rows][D]: unnormalised outputs of cut items
  float2* part_ml;  // [CTAs][2][item rows]: their (maximum in log2 units, sum)
  int B, nq, rep, row_tiles, max_length, causal;
  int ctas;
  int whole;          // an item per CTA, nothing is cut
  float scale_log2;  // scale * log2(e)
};

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

// An item is one cache head of one sequence and ROWS of its query rows
// (queries x heads of the group, queries first). The items' key tiles of TILE
// keys form a line, sequence by sequence, that is cut into equal ranges, one
// per CTA. COST: what starting on an item and finishing it costs a CTA, in
// tiles: each item is that much longer on the line, so that a CTA whose range
// crosses into one gets fewer tiles. MIN: the least tiles of a range.
template <int TILE_, int ROWS_, int COST_, int MIN_>
struct Line {
  static constexpr int TILE = TILE_, ROWS = ROWS_, COST = COST_, MIN = MIN_;

  static __device__ __forceinline__ int tiles(const AttnParams& p, int b) {
    bool bad;
    return (length_of(p, b, &bad) + TILE - 1) / TILE;
  }
  // Places that an item takes.
  static __host__ __device__ __forceinline__ int places(int tiles) { return tiles > 0 ? tiles + COST : 0; }
  // Places per CTA of a line of `total` (the host keeps lines below 2^31).
  static __device__ __forceinline__ int range(const AttnParams& p, int total) {
    return max((total + p.ctas - 1) / p.ctas, MIN);
  }
};

// Where a CTA's range starts.
struct Start {
  int total, per;
  int base;  // first place of sequence b
  int b;
};

// Block-wide, THREADS threads: sums the sequences' places in thread chunks
// and finds the sequence that place blockIdx.x * per falls into.
template <typename L, int THREADS>
__device__ __forceinline__ void find_start(const AttnParams& p, Start* s, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
  const int per_item = p.cache.Hk * p.row_tiles;
  int sum = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    bool bad;
    sum += L::places((length_of(p, b, &bad) + L::TILE - 1) / L::TILE) * per_item;
    if (bad && blockIdx.x == 0) report_index(p.status);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  const int per = L::range(p, total);
  const int r0 = min((long long)blockIdx.x * per, (long long)total);
  int at = before + incl - sum;
  if (r0 >= at && r0 < at + sum) {  // one thread, if any
    int b = b0;
#pragma unroll 1
    for (; b < b1; ++b) {
      const int n = L::places(L::tiles(p, b)) * per_item;
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

// The part of a CTA's range that lies in one item, and what its rows see.
struct Segment {
  int b, h, rt, tile0, ntile, len, count, rows, seen_min, seen_max;
  __device__ __forceinline__ bool whole(int tile) const { return ntile == (len + tile - 1) / tile; }
};

// The rows of a segment of the sequence's item, from b and len.
template <typename L>
__device__ __forceinline__ void rows_of_segment(const AttnParams& p, int item, Segment& sg) {
  sg.h = item / p.row_tiles;
  sg.rt = item - sg.h * p.row_tiles;
  sg.count = count_of(p, sg.b);
  sg.rows = min(L::ROWS, sg.count * p.rep - sg.rt * L::ROWS);  // may be <= 0
  sg.seen_min = sg.seen_max = sg.len;
  if (p.causal) {
    const int first = sg.len - sg.count + 1;  // keys the first query sees
    sg.seen_min = max(0, first + sg.rt * L::ROWS / p.rep);
    sg.seen_max = max(0, first + (sg.rt * L::ROWS + sg.rows - 1) / p.rep);
  }
  if (sg.rows <= 0) sg.seen_max = 0;
}

// Walks the segments of the range [pos, r1); base, b: as in Start.
template <typename L>
__device__ __forceinline__ bool next_segment(const AttnParams& p, int& pos, int r1, int& base, int& b,
                                             Segment& sg) {
  const int items = p.cache.Hk * p.row_tiles;
#pragma unroll 1
  while (pos < r1) {
    bool bad;
    sg.len = length_of(p, b, &bad);
    const int T_b = (sg.len + L::TILE - 1) / L::TILE, line = L::places(T_b);
    if (pos >= base + line * items) {
      base += line * items;
      ++b;
      continue;
    }
    const int item = (pos - base) / line;
    sg.b = b;
    sg.tile0 = pos - base - item * line - L::COST;
    if (sg.tile0 < 0) {  // to the item's first tile
      pos -= sg.tile0;
      sg.tile0 = 0;
      if (pos >= r1) break;
    }
    sg.ntile = min(T_b - sg.tile0, r1 - pos);
    rows_of_segment<L>(p, item, sg);
    pos += sg.ntile;
    return true;
  }
  return false;
}

// All of item `at` of the batch.
template <typename L>
__device__ __forceinline__ void whole_segment(const AttnParams& p, int at, Segment& sg) {
  const int items = p.cache.Hk * p.row_tiles;
  sg.b = at / items;
  bool bad;
  sg.len = length_of(p, sg.b, &bad);
  sg.tile0 = 0;
  sg.ntile = (sg.len + L::TILE - 1) / L::TILE;
  rows_of_segment<L>(p, at - sg.b * items, sg);
  if (bad && threadIdx.x == 0) report_index(p.status);
}

// Slot of a segment's part in its CTA: a range holds at most one item cut in
// front (0) and one that starts in it and is cut behind (1).
__device__ __forceinline__ size_t part_slot(const Segment& sg) {
  return (size_t)blockIdx.x * 2 + (sg.tile0 > 0 ? 0 : 1);
}

// Chunks of queries over the cache on the fifth-generation tensor cores
// (nys_kv4_chunk.cu): bf16, d in {64, 128}.
using ChunkLine = Line<128, 256, 2, 1>;
int launch_kv4_chunk(const AttnParams& p, int d, const void* q, void* out, cudaStream_t stream);

}  // namespace kv4
}  // namespace nys
