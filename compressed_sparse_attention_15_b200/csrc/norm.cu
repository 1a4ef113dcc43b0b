// csa_add_rmsnorm: the residual's addition, RMSNorm, and its 8-bit form.
//
//     h = round(x + residual),  y = h / sqrt(mean h^2 + eps) * weight   (fp32),
//     out = round(y),  or per group of dims s = amax|y| / 448, code = E4M3(y / s).
// h is rounded to the element type before the norm, so that the norm is that
// of the residual stream that the next layer reads; every sum is fp32.
//
// Bytes bound it: x, the residual, h and the output move once each, the row
// staying in registers between the sum of squares and the output.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

namespace {

// 8 consecutive elements as floats.
__device__ __forceinline__ void load8(const bf16 *p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(bf16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Scale of a group whose largest magnitude is amax.
__device__ __forceinline__ float group_scale(float amax) {
  const float s = amax / 448.f;
  return s > 0.f ? s : 1.f;
}

// The codes of 8 values. v / s as v (1 / s), off by 2^-23 of it at most, next to
// the 2^-4 of the rounding to E4M3 that follows: the same code but for quotients
// within 2^-23 of the middle between two. (1 / s overflows for the smallest s: both
// factors are scaled then.)
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s) {
  const float up = s < 0x1p-120f ? 0x1p100f : 1.f, inv = 1.f / (s * up);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x[4] = {v[4 * i] * up * inv, v[4 * i + 1] * up * inv, v[4 * i + 2] * up * inv, v[4 * i + 3] * up * inv};
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// Reduction over the WPR warps of a row (RPB rows per block), the same in
// every thread: op over v, then over the warps through shared memory.
template <int WPR, int RPB, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float (&red)[RPB][WPR], int row, int warp, int lane) {
  v = kMax ? warp_max(v) : warp_sum(v);
  if constexpr (WPR > 1) {
    __syncthreads();  // red's last use
    if (lane == 0) red[row][warp] = v;
    __syncthreads();
    float r = lane < WPR ? red[row][lane] : 0.f;  // (every value is >= 0)
    v = kMax ? warp_max(r) : warp_sum(r);
  }
  return v;
}

// WPR warps per row, NV vectors of 8 dims per thread (vector t + 32 WPR i),
// RPB rows per block.
template <typename T, int WPR, int NV, int RPB, bool kFp8>
__global__ void __launch_bounds__(32 * WPR *RPB) add_rmsnorm_kernel(NormArgs a) {
  __shared__ float red[RPB][WPR];
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, row = w / WPR, warp = w % WPR;
  const int t = warp * 32 + lane, nvec = a.D / 8;
  const long long r = (long long)blockIdx.x * RPB + row;
  const bool live = r < a.rows;
  float v[NV][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    if (live && j < nvec) {
      load8(static_cast<const T *>(a.x) + r * a.x_stride + 8 * j, v[i]);
      if (a.residual) {
        float u[8];
        load8(static_cast<const T *>(a.residual) + r * a.D + 8 * j, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = to_f(from_f<T>(v[i][e] + u[e]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    if (a.residual && live && j < nvec) store8(static_cast<T *>(a.sum_out) + r * a.D + 8 * j, v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
  }
  ss = row_reduce<WPR, RPB, false>(ss, red, row, warp, lane);
  const float rs = 1.f / sqrtf(ss / (float)a.D + a.eps);
  float amax[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    amax[i] = 0.f;
    if (live && j < nvec) {
      float g[8];
      load8(a.weight + 8 * j, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = v[i][e] * rs * g[e];
        amax[i] = fmaxf(amax[i], fabsf(v[i][e]));
      }
      if constexpr (!kFp8) store8(static_cast<T *>(a.out) + r * a.D + 8 * j, v[i]);
    }
  }
  if constexpr (kFp8) {
    uint8_t *out = static_cast<uint8_t *>(a.out) + r * a.D;
    const int lanes = a.group / 8;  // lanes that hold a group (a group of 32..256 dims lies in one warp's vectors)
    if (a.group < a.D) {
      float *scales = a.scales + r * (a.D / a.group);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = t + 32 * WPR * i;
        float m = amax[i];
        for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (live && j < nvec) {
          const float s = group_scale(m);
          *reinterpret_cast<uint2 *>(out + 8 * j) = codes8(v[i], s);
          if (j % lanes == 0) scales[j / lanes] = s;
        }
      }
    } else {
      float m = amax[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, amax[i]);
      m = row_reduce<WPR, RPB, true>(m, red, row, warp, lane);
      const float s = group_scale(m);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = t + 32 * WPR * i;
        if (live && j < nvec) *reinterpret_cast<uint2 *>(out + 8 * j) = codes8(v[i], s);
      }
      if (live && t == 0) a.scales[r] = s;
    }
  }
}

// Any D, stride and alignment: one block per row, h and then y in shared memory.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(256) add_rmsnorm_generic_kernel(NormArgs a) {
  extern __shared__ float h[];
  __shared__ float red[1][8];
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r = blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
  float ss = 0.f;
  for (int d = threadIdx.x; d < a.D; d += 256) {
    float v = to_f(x[d]);
    if (a.residual) {
      const T s = from_f<T>(v + to_f(static_cast<const T *>(a.residual)[r * a.D + d]));
      static_cast<T *>(a.sum_out)[r * a.D + d] = s;
      v = to_f(s);
    }
    h[d] = v;
    ss = fmaf(v, v, ss);
  }
  ss = row_reduce<8, 1, false>(ss, red, 0, warp, lane);
  const float rs = 1.f / sqrtf(ss / (float)a.D + a.eps);
  float m = 0.f;
  for (int d = threadIdx.x; d < a.D; d += 256) {
    const float y = h[d] * rs * a.weight[d];
    h[d] = y;
    m = fmaxf(m, fabsf(y));
    if constexpr (!kFp8) static_cast<T *>(a.out)[r * a.D + d] = from_f<T>(y);
  }
  if constexpr (kFp8) {
    uint8_t *out = static_cast<uint8_t *>(a.out) + r * a.D;
    float *scales = a.scales + r * (a.D / a.group);
    if (a.group == a.D) {
      const float s = group_scale(row_reduce<8, 1, true>(m, red, 0, warp, lane));
      for (int d = threadIdx.x; d < a.D; d += 256) out[d] = __nv_cvt_float_to_fp8(h[d] / s, __NV_SATFINITE, __NV_E4M3);
      if (threadIdx.x == 0) scales[0] = s;
    } else {
      __syncthreads();
      for (int g = warp; g < a.D / a.group; g += 8) {  // a warp per group
        float gm = 0.f;
        for (int d = lane; d < a.group; d += 32) gm = fmaxf(gm, fabsf(h[g * a.group + d]));
        const float s = group_scale(warp_max(gm));
        for (int d = lane; d < a.group; d += 32)
          out[g * a.group + d] = __nv_cvt_float_to_fp8(h[g * a.group + d] / s, __NV_SATFINITE, __NV_E4M3);
        if (lane == 0) scales[g] = s;
      }
    }
  }
}

template <typename T, int WPR, int NV, int RPB>
cudaError_t launch_rows(const NormArgs &a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows + RPB - 1) / RPB)), block(32 * WPR * RPB);
  return a.scales ? launch_pdl(add_rmsnorm_kernel<T, WPR, NV, RPB, true>, grid, block, 0, stream, a)
                  : launch_pdl(add_rmsnorm_kernel<T, WPR, NV, RPB, false>, grid, block, 0, stream, a);
}

template <typename T, bool kFp8>
cudaError_t launch_generic(const NormArgs &a, cudaStream_t stream) {
  static DeviceOnce attr;  // set for the largest D the ABI admits
  once_per_device(attr, [] {
    cudaFuncSetAttribute(add_rmsnorm_generic_kernel<T, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 16384 * 4);
  });
  return launch_pdl(add_rmsnorm_generic_kernel<T, kFp8>, dim3((unsigned)a.rows), dim3(256), (size_t)a.D * 4, stream, a);
}

template <typename T>
cudaError_t launch_t(const NormArgs &a, cudaStream_t stream) {
  if (a.rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                      reinterpret_cast<uintptr_t>(a.sum_out) | reinterpret_cast<uintptr_t>(a.weight);
  const bool vec = a.D % 8 == 0 && a.x_stride % 8 == 0 && (p & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.out) & (a.scales ? 7 : 15)) == 0;
  if (!vec) return a.scales ? launch_generic<T, true>(a, stream) : launch_generic<T, false>(a, stream);
  const int nvec = a.D / 8;
  if (nvec <= 32) return launch_rows<T, 1, 1, 8>(a, stream);
  if (nvec <= 64) return launch_rows<T, 2, 1, 4>(a, stream);
  if (nvec <= 128) return launch_rows<T, 4, 1, 2>(a, stream);
  if (nvec <= 256) return launch_rows<T, 8, 1, 1>(a, stream);
  if (nvec <= 512) return launch_rows<T, 8, 2, 1>(a, stream);
  if (nvec <= 1024) return launch_rows<T, 16, 2, 1>(a, stream);
  return launch_rows<T, 32, 2, 1>(a, stream);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs &a, cudaStream_t stream) {
  return a.dtype == CSA_DTYPE_F32 ? launch_t<float>(a, stream) : launch_t<bf16>(a, stream);
}

}  // namespace csa
