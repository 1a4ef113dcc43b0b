// csa_paged_append / csa_paged_read: rows into and out of a paged cache.
//
// append: v = kv[b, i], its last rope_dims dims rotated in adjacent pairs by
//   (pos0[b] + i pos_stride) theta^(-2 j / rope_dims), rounded to its type;
//   stored as it is, or per 16 dims as s = E4M3(amax |v| / 7) and
//   c = 8 + clamp(rint(v / s), -7, 7)  (c = 8 under a zero or NaN scale).
// read: the rows' values, (c - 8) s (exact in bf16: 3 bits times 4).
//
// Bytes bound both: a row of D dims moves 2 D (bf16) and D / 2 + D / 16 bytes.
// A thread takes one group of 16 dims, so that a group's maximum needs no
// other thread. The rotation's angles need double precision (positions beyond
// 2^20); a block turns the rope dims of all its rows first, a thread per pair,
// each taking the sine and cosine of its first row's angle and of the step
// between its rows, and four products per row from there on.
#include "kernels.h"
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 32;       // rows per block
constexpr int kRopeElems = 4096;   // rotated elements a block holds

// 16 elements from 16-byte aligned memory.
__device__ __forceinline__ void load16v(const bf16 *p, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 u = reinterpret_cast<const uint4 *>(p)[h];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load16v(const float *p, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 u = reinterpret_cast<const float4 *>(p)[h];
    v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
  }
}
__device__ __forceinline__ void store16v(bf16 *p, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    reinterpret_cast<uint4 *>(p)[h] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void store16v(float *p, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
    reinterpret_cast<float4 *>(p)[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
}
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16], int n, bool vec) {
  if (vec) return load16v(p, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store16(T *p, const float (&v)[16], int n, bool vec) {
  if (vec) return store16v(p, v);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) p[i] = from_f<T>(v[i]);
}

// Slots of the block's rows [r0, r0 + rb) of sequence b (-1: nothing there).
__device__ __forceinline__ void block_slots(const PagedRowsArgs &a, int b, int r0, int rb, long long *slot) {
  for (int i = threadIdx.x; i < rb; i += blockDim.x) {
    uint32_t *st = r0 == 0 && i == 0 ? a.status : nullptr;
    const int n = a.n_new ? clamp_count(a.n_new[b], a.n, st) : a.n;
    slot[i] = r0 + i < n ? paged_slot(a.cache, b, (long long)a.entry0[b] + r0 + i, a.status) : -1;
  }
}

// The block's rope dims, rotated and rounded to T, into rot[rb][rope_dims].
template <typename T>
__device__ __forceinline__ void rotate_rows(const PagedRowsArgs &a, int b, int r0, int rb, const long long *slot, T *rot) {
  const int R = a.rope_dims, P = R / 2;
  const int at_once = max(1, (int)blockDim.x / P);  // rows turned at once
  for (int t = threadIdx.x; t < at_once * P; t += blockDim.x) {
    const int j = t % P;
    const double f = pow(a.rope_theta, -2.0 * j / R);
    double cs, sn, dc = 1.0, ds = 0.0;
    int i = t / P;
    if (i >= rb) continue;
    const double p = (double)((a.pos0 ? a.pos0[b] : 0) + (long long)(r0 + i) * a.pos_stride);
    sincos(p * f, &sn, &cs);
    if (i + at_once < rb) sincos((double)at_once * a.pos_stride * f, &ds, &dc);
    const T *x = static_cast<const T *>(a.rows) + b * a.seq_stride + (long long)(r0 + i) * a.row_stride + a.cache.D - R + 2 * j;
    for (; i < rb; i += at_once, x += (long long)at_once * a.row_stride) {
      if (slot[i] >= 0) {
        const double x0 = to_f(x[0]), x1 = to_f(x[1]);
        rot[i * R + 2 * j] = from_f<T>((float)(x0 * cs - x1 * sn));
        rot[i * R + 2 * j + 1] = from_f<T>((float)(x0 * sn + x1 * cs));
      }
      const double c = cs * dc - sn * ds;
      sn = sn * dc + cs * ds;
      cs = c;
    }
  }
}

// 16 values as nibbles and their scale.
__device__ __forceinline__ uint2 pack16(const float (&v)[16], uint8_t &scale) {
  uint32_t m = 0;  // largest magnitude as bits: a NaN is above every number
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  scale = __nv_cvt_float_to_fp8(__uint_as_float(m) / 7.f, __NV_SATFINITE, __NV_E4M3);
  const float s = e4m3_value(scale);
  uint32_t w[2] = {0x88888888u, 0x88888888u};
  if (s > 0.f) {
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = (int)fminf(fmaxf(rintf(v[i] / s), -7.f), 7.f) + 8;
      w[i >> 3] |= (uint32_t)c << (4 * ((i & 7) >> 1) + 16 * (i & 1));
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, bool kInt4>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(PagedRowsArgs a, int rb, int chunks, bool vec) {
  __shared__ long long slot[kMaxRows];
  __shared__ T rot[kRopeElems];
  pdl_wait();
  pdl_release();
  const int b = blockIdx.x / chunks, r0 = (blockIdx.x - b * chunks) * rb, D = a.cache.D, d_rot = D - a.rope_dims;
  block_slots(a, b, r0, rb, slot);
  __syncthreads();
  if (a.rope_dims) {
    rotate_rows<T>(a, b, r0, rb, slot, rot);
    __syncthreads();
  }
  const int G = (D + 15) / 16;
  const T *rows = static_cast<const T *>(a.rows) + b * a.seq_stride + (long long)r0 * a.row_stride;
  uint8_t *pages = const_cast<uint8_t *>(a.cache.pages);
  for (int t = threadIdx.x; t < rb * G; t += blockDim.x) {
    const int i = t / G, g = t - i * G, d = 16 * g;
    if (slot[i] < 0) continue;
    float v[16];
    const int n = min(16, D - d);
    if (d < d_rot) load16(rows + i * a.row_stride + d, v, n, vec);
    if (d + n > d_rot) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (d + e >= d_rot && e < n) v[e] = to_f(rot[i * a.rope_dims + d + e - d_rot]);
    }
    if constexpr (kInt4) {
      uint8_t s;
      const uint2 w = pack16(v, s);
      *reinterpret_cast<uint2 *>(pages + (size_t)slot[i] * a.cache.row_bytes + 8 * g) = w;
      const_cast<uint8_t *>(a.cache.scales)[(size_t)slot[i] * G + g] = s;
    } else {
      store16(reinterpret_cast<T *>(pages) + (size_t)slot[i] * D + d, v, n, vec);
    }
  }
}

template <typename T, bool kInt4>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(PagedRowsArgs a, int rb, int chunks, bool vec) {
  __shared__ long long slot[kMaxRows];
  pdl_wait();
  pdl_release();
  const int b = blockIdx.x / chunks, r0 = (blockIdx.x - b * chunks) * rb, D = a.cache.D;
  block_slots(a, b, r0, rb, slot);
  __syncthreads();
  const int G = (D + 15) / 16;
  T *out = static_cast<T *>(const_cast<void *>(a.rows)) + b * a.seq_stride + (long long)r0 * a.row_stride;
  for (int t = threadIdx.x; t < rb * G; t += blockDim.x) {
    const int i = t / G, g = t - i * G, d = 16 * g;
    if (slot[i] < 0) continue;
    float v[16];
    const int n = min(16, D - d);
    if constexpr (kInt4) {
      const uint2 w = *reinterpret_cast<const uint2 *>(a.cache.pages + (size_t)slot[i] * a.cache.row_bytes + 8 * g);
      const float s = e4m3_value(a.cache.scales[(size_t)slot[i] * G + g]);
      float lo[8], hi[8];
      unpack8(w.x, s, lo);
      unpack8(w.y, s, hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = lo[e], v[8 + e] = hi[e];
    } else {
      load16(reinterpret_cast<const T *>(a.cache.pages) + (size_t)slot[i] * D + d, v, n, vec);
    }
    store16(out + (long long)i * a.row_stride + d, v, n, vec);
  }
}

template <typename T>
cudaError_t launch_rows(const PagedRowsArgs &a, bool append, cudaStream_t stream) {
  const int G = (a.cache.D + 15) / 16;
  // Rows per block: 32 (a pair's sine and cosine serve 4 and more rows), fewer
  // where that leaves less than four blocks per SM; as many rotated rows as
  // the block can hold.
  const long long fill = (long long)a.B * a.n / (4 * device_sm_count());
  int rb = fill < 1 ? 1 : fill > kMaxRows ? kMaxRows : (int)fill;
  if (append && a.rope_dims && rb * a.rope_dims > kRopeElems) rb = kRopeElems / a.rope_dims;
  const long long chunks = (a.n + rb - 1) / rb;
  if (chunks * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
  int threads = (rb * G + 31) / 32 * 32;
  threads = threads > kThreads ? kThreads : threads;
  const bool int4 = a.cache.scales != nullptr;
  const uintptr_t e = sizeof(T);
  const bool vec = a.cache.D % 16 == 0 && a.row_stride * e % 16 == 0 && a.seq_stride * e % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.rows) & 15) == 0 &&
                   (int4 || (reinterpret_cast<uintptr_t>(a.cache.pages) & 15) == 0);
  auto kern = append ? (int4 ? paged_append_kernel<T, true> : paged_append_kernel<T, false>)
                     : (int4 ? paged_read_kernel<T, true> : paged_read_kernel<T, false>);
  return launch_pdl(kern, dim3((unsigned)(chunks * a.B)), dim3(threads), 0, stream, a, rb, (int)chunks, vec);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedRowsArgs &a, bool append, cudaStream_t stream) {
  return a.dtype == CSA_DTYPE_F32 ? launch_rows<float>(a, append, stream) : launch_rows<bf16>(a, append, stream);
}

}  // namespace csa
