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

__device__ __forceinline__ uint32_t bf16x2_dup(float x) {
  const __nv_bfloat162 t = __float2bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t *>(&t);
}

// The 8 dims of a word as 4 pairs of bf16, exactly: a nibble c placed in the
// mantissa of 128 is 128 + c, and one packed fused multiply-add makes
// (128 + c) s - 136 s = (c - 8) s of it. sc and off hold s and -136 s (17 times
// 8 to 15 eighths: 8 significant bits), twice each.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t sc, uint32_t off, uint32_t (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[k]) : "r"(((w >> (4 * k)) & 0x000f000fu) | 0x43004300u), "r"(sc), "r"(off));
}

// The same in fp32.
__device__ __forceinline__ void unpack8(uint32_t w, float s, float (&v)[8]) {
  uint32_t t[4];
  widen8(w, bf16x2_dup(s), bf16x2_dup(-136.f * s), t);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(t[i] << 16);
    v[2 * i + 1] = __uint_as_float(t[i] & 0xffff0000u);
  }
}

}  // namespace csa
