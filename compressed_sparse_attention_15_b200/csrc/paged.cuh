// The paged cache of compressed entries, as the kernels see it.
//
// Entry e of sequence b lies in page table[b, e / page] at row e % page. A row
// holds D elements of the cache's type, or, in the 4-bit form, D / 8 words of
// 32 bits and one E4M3 scale per 16 dims. A word's low half holds dims 0, 2,
// 4, 6 of its 8 dims in its nibbles, its high half dims 1, 3, 5, 7; nibble c
// under scale s stands for (c - 8) s. Even and odd dims sit 16 bits apart, so
// that one AND leaves a pair of neighbouring dims in the two halves of a
// register, where a packed bf16 instruction wants them.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

// The page of a sequence's entry, and its row there.
__device__ __forceinline__ uint2 page_and_row(const PagedCache &c, uint32_t e) {
  const uint32_t pg = c.shift >= 0 ? e >> c.shift : e / (uint32_t)c.page;
  return make_uint2(pg, e - pg * (uint32_t)c.page);
}

// Row of the flattened pages that holds entry e of sequence b; -1 with a
// status bit where the entry or its page does not exist.
__device__ __forceinline__ long long paged_slot(const PagedCache &c, int b, long long e, uint32_t *status) {
  if (e < 0 || e >= c.capacity()) {
    raise_status(status, CSA_STATUS_BAD_INDEX);
    return -1;
  }
  const uint2 at = page_and_row(c, (uint32_t)e);
  const int p = c.table[(size_t)b * c.per + at.x];
  if (p < 0 || p >= c.num_pages) {
    raise_status(status, CSA_STATUS_BAD_PAGE);
    return -1;
  }
  return (long long)p * c.page + at.y;
}

__device__ __forceinline__ float e4m3_value(uint8_t u) {
  __nv_fp8_e4m3 t;
  t.__x = u;
  return float(t);
}

// The 8 dims of a word under scale s.
__device__ __forceinline__ void unpack8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * s;
    v[2 * i + 1] = (float)((int)((w >> (4 * i + 16)) & 15u) - 8) * s;
  }
}

}  // namespace csa
