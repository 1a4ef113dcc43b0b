// csa_add_rmsnorm: the residual's addition, RMSNorm, and its 8-bit form.
//
//     h = round(x + residual),  y = h / sqrt(mean h^2 + eps) * weight   (fp32),
//     out = round(y),  or per group of dims s = amax|y| / 448, code = E4M3(y / s).
// h is rounded to the element type before the norm, so that the norm is that
// of the residual stream that the next layer reads; every sum is fp32.
//
// Bytes bound it: x, the residual, h and the output move once each, the row
// staying in registers between the sum of squares and the output. Its instructions
// come close behind (4,096 rows of 4,096 with 8-bit output took 31 us at one
// instruction a value and step, and takes 23.2 packed: 5.1 TB/s; with bf16 output
// 21.8: 6.2 TB/s), so they are packed:
// x + residual as bf16 pairs (a sum of two bf16 numbers rounds the same from its
// exact value as from its fp32 one, as what fp32 drops is below 2^-16 of it), the
// rest as fp32 pairs.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

namespace {

// 8 consecutive elements as they lie in memory, and as pairs of floats.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = u; }
  __device__ __forceinline__ void add(const Raw8 &o) {
    auto f = [](uint32_t &a, uint32_t b) { asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b)); };
    f(u.x, o.u.x), f(u.y, o.u.y), f(u.z, o.u.z), f(u.w, o.u.w);
  }
  __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  __device__ __forceinline__ void add(const Raw8 &o) {
    a = make_float4(a.x + o.a.x, a.y + o.a.y, a.z + o.a.z, a.w + o.a.w);
    b = make_float4(b.x + o.b.x, b.y + o.b.y, b.z + o.b.z, b.w + o.b.w);
  }
  __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const {
    v[0] = pack2(a.x, a.y), v[1] = pack2(a.z, a.w), v[2] = pack2(b.x, b.y), v[3] = pack2(b.z, b.w);
  }
};

__device__ __forceinline__ void store8(bf16 *p, const uint64_t (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v[i]);
    const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const uint64_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2(v[2 * i]), b = unpack2(v[2 * i + 1]);
    reinterpret_cast<float4 *>(p)[i] = make_float4(a.x, a.y, b.x, b.y);
  }
}

// Scale of a group whose largest magnitude is amax.
__device__ __forceinline__ float group_scale(float amax) {
  const float s = amax / 448.f;
  return s > 0.f ? s : 1.f;
}

// The codes of 8 values y, given as -y: E4M3(y / s), the quotient rounded to fp32
// first. q0 = y (1 / s) alone, off by up to 2^-23 of itself, gives another code next
// to a tie (some 2^-20 of all values); one residual step repairs it (Markstein, IBM
// J. Res. Dev. 34, 1990): q = q0 + (y - q0 s) (1 / s), the bracket in one fused step.
// Before its last rounding q is within 3 2^-24 of an fp32 step of y / s, so that it
// can differ from the rounded quotient only where y / s is as near to the middle
// between two fp32 numbers; of those a code depends on the middles beside a tie
// alone, which few significands of y and s come so near to, and q is right for all
// of them. The signs (-y, -1 / s) keep that of a zero. It costs a packed instruction
// a value: 4,096 rows of 4,096 with 8-bit output take 24.8 us a call where 24.6 with q0.
__device__ __forceinline__ uint2 codes8(uint64_t (&ny)[4], float s) {
  if (s < 0x1p-80f) {  // 1 / s or the residual may leave the normal numbers: both up by 2^100, exactly
#pragma unroll
    for (int i = 0; i < 4; ++i) ny[i] = mul2(ny[i], pack2(0x1p100f, 0x1p100f));
    s *= 0x1p100f;
  }
  const float ninv = -1.f / s, sr = s < INFINITY ? s : 0.f;  // (under an infinite scale q0, 0 or NaN, stays)
  const uint64_t ninv2 = pack2(ninv, ninv), s2 = pack2(sr, sr);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q0 = mul2(ny[i], ninv2), q = fma2(fma2(q0, s2, ny[i]), ninv2, q0);
    c[i] = __nv_cvt_float2_to_fp8x2(unpack2(q), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
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

// WPR warps per row, NV vectors of 8 dims per thread (vector t + 32 WPR i), RPB
// rows per block. Two vectors a thread at most, for rows in flight: with four (or
// two rows a block) the 4,096-dim case took 35 to 39 us where it took 31; and all
// of an SM's threads (32 registers each), 30 us for rows of 16,384 where 37 without.
template <typename T, int WPR, int NV, int RPB, bool kFp8>
__global__ void __launch_bounds__(32 * WPR *RPB, 2048 / (32 * WPR * RPB)) add_rmsnorm_kernel(NormArgs a) {
  __shared__ float red[RPB][WPR];
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, row = w / WPR, warp = w % WPR;
  const int t = warp * 32 + lane, nvec = a.D / 8;
  const long long r = (long long)blockIdx.x * RPB + row;
  const bool live = r < a.rows;
  uint64_t v[NV][4], ss2 = pack2(0.f, 0.f);
  Raw8<T> h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    if (live && j < nvec) {
      h[i].load(static_cast<const T *>(a.x) + r * a.x_stride + 8 * j);
      if (a.residual) {
        Raw8<T> u;
        u.load(static_cast<const T *>(a.residual) + r * a.D + 8 * j);
        h[i].add(u);
      }
    } else {
      h[i] = Raw8<T>{};
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    if (a.residual && live && j < nvec) h[i].store(static_cast<T *>(a.sum_out) + r * a.D + 8 * j);
    h[i].pairs(v[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) ss2 = fma2(v[i][e], v[i][e], ss2);
  }
  float ss = unpack2(ss2).x + unpack2(ss2).y;
  ss = row_reduce<WPR, RPB, false>(ss, red, row, warp, lane);
  const float rs = 1.f / sqrtf(ss / (float)a.D + a.eps);
  const uint64_t rs2 = kFp8 ? pack2(-rs, -rs) : pack2(rs, rs);  // (codes8 takes -y)
  float amax[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = t + 32 * WPR * i;
    amax[i] = 0.f;
    if (live && j < nvec) {
      Raw8<float> w;
      w.load(a.weight + 8 * j);
      uint64_t g[4];
      w.pairs(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[i][e] = mul2(mul2(v[i][e], rs2), g[e]);
        const float2 y = unpack2(v[i][e]);
        amax[i] = fmaxf(fmaxf(amax[i], fabsf(y.x)), fabsf(y.y));
      }
      if constexpr (!kFp8) store8(static_cast<T *>(a.out) + r * a.D + 8 * j, v[i]);
    }
  }
  if constexpr (kFp8) {
    uint8_t *out = static_cast<uint8_t *>(a.out) + r * a.D;
    const int lanes = a.group / 8;  // lanes that hold a group (a group of 32..256 dims lies in one warp's vectors)
    const int shift = __ffs(lanes) - 1;  // (a power of two here)
    if (a.group < a.D) {
      float *scales = a.scales + r * (nvec >> shift);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = t + 32 * WPR * i;
        float m = amax[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float other = __shfl_xor_sync(0xffffffffu, m, o);
          if (o < lanes) m = fmaxf(m, other);
        }
        if (live && j < nvec) {
          const float s = group_scale(m);
          if ((j & (lanes - 1)) == 0) scales[j >> shift] = s;
          *reinterpret_cast<uint2 *>(out + 8 * j) = codes8(v[i], s);
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
