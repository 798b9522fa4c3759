// Layout and checks of the 4-bit key/value cache (include/nystrom.h), shared
// by the kernels that write, read and attend it.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nys_internal.h"

namespace nys {
namespace kv4 {

constexpr int kBlock = 16;  // tokens of one block

// Byte offsets inside a block of 16 tokens of one head.
__host__ __device__ constexpr int block_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int k_scales(int d) { return 8 * d; }
__host__ __device__ constexpr int v_codes(int d) { return 9 * d; }
__host__ __device__ constexpr int v_scales(int d) { return 17 * d; }

// What the kernels know of a cache.
struct View {
  uint8_t* data;
  const int* table;  // [B][max_pages]
  int num_pages, max_pages, page, Hk;
};

inline View view_of(const nys_kv4_cache_t& c) {
  return View{static_cast<uint8_t*>(c.data), c.block_table, c.num_pages, c.max_pages, c.page_size, c.Hk};
}

// The block of tokens pos .. pos+15 (pos a multiple of 16) of a sequence and
// head, or null where the page table has no such page or names one outside
// the pool.
__device__ __forceinline__ uint8_t* block_at(const View& c, int b, int h, long long pos, int d) {
  if (pos < 0 || pos >= (long long)c.max_pages * c.page) return nullptr;
  const int slot = (int)pos / c.page;
  const int page = c.table[(size_t)b * c.max_pages + slot];
  if (page < 0 || page >= c.num_pages) return nullptr;
  const int blocks = c.page / kBlock;
  const size_t at = ((size_t)page * c.Hk + h) * blocks + ((int)pos - slot * c.page) / kBlock;
  return c.data + at * block_bytes(d);
}

__device__ __forceinline__ void report_index(int* status) { atomicExch(status, (int)NYS_ERR_INDEX); }

// Host checks of a cache; NYS_OK or the code of include/nystrom.h.
int check_cache(const nys_kv4_cache_t* c);

inline bool rows_aligned(const void* p, const nys_strides_t& s, int dtype) {
  const long long per = dtype == NYS_FP32 ? 4 : 8;  // elements in 16 bytes
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.batch % per == 0 && s.head % per == 0 &&
         s.token % per == 0;
}
inline bool strides_ok(const nys_strides_t& s) { return s.batch >= 0 && s.head >= 0 && s.token >= 0; }
// Output rows must not share memory: a stride shorter than a row along an
// axis with more than one entry is refused.
inline bool rows_apart(const nys_strides_t& s, int B, int H, int n, int d) {
  return (B == 1 || s.batch >= d) && (H == 1 || s.head >= d) && (n == 1 || s.token >= d);
}

}  // namespace kv4
}  // namespace nys
