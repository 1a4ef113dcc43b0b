// csa_paged_append / csa_paged_read: rows into and out of a paged cache.
//
// append: v = kv[b, i], its last rope_dims dims rotated in adjacent pairs by
//   (pos0[b] + i pos_stride) theta^(-2 j / rope_dims), rounded to its type;
//   stored as it is, or per 16 dims as s = E4M3(amax |v| / 7) and
//   c = 8 + clamp(rint(v / s), -7, 7)  (c = 8 under a zero or NaN scale).
// read: the rows' values, (c - 8) s (exact in bf16: 3 bits times 4).
//
// Bytes bound both: a row of D dims moves 2 D (bf16) and D / 2 + D / 16 bytes.
// A thread takes one group of 16 dims, so that a group's maximum needs no other
// thread. The rotation's angles need double precision (positions beyond 2^20),
// and its dims other threads: blocks of their own take the rotated end of the
// rows, a thread a pair of dims, each forming the cosine and sine of its first
// row's angle and turning them by the step between its rows from there on. 32,767
// rows of 512 dims into 4 bits: 9.1 us without a rotation (4.7 TB/s), 13.4 with 64
// rotated dims, whose chain of lookups, frequency, angle and rows is what is left;
// in one kind of block, through shared memory, it was 21. Reading them back: 10.0 us.
#include "kernels.h"
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 64;       // rows per block
constexpr int kRotElems = 4096;    // rotated elements that a block packs

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

// t / G by a product: m = ceil(2^32 / G), exact while t G < 2^32 (0 for G = 1).
__device__ __forceinline__ int quotient(int t, uint32_t m) { return m ? (int)__umulhi((uint32_t)t, m) : t; }

// Slots of the block's rows [r0, r0 + rb) of sequence b (-1: nothing there).
__device__ __forceinline__ void block_slots(const PagedRowsArgs &a, int b, int r0, int rb, long long *slot) {
  for (int i = threadIdx.x; i < rb; i += blockDim.x) {
    uint32_t *st = r0 == 0 && i == 0 ? a.status : nullptr;
    const int n = a.n_new ? clamp_count(a.n_new[b], a.n, st) : a.n;
    slot[i] = r0 + i < n ? paged_slot(a.cache, b, (long long)a.entry0[b] + r0 + i, a.status) : -1;
  }
}

// theta^(-2 j / rope_dims): the product with log2 theta and what its rounding left.
__device__ __forceinline__ double frequency(const PagedRowsArgs &a, int j) {
  const double e = -2.0 * j / a.rope_dims, x = e * a.log2_theta[0];
  const double rest = fma(e, a.log2_theta[0], -x) + e * a.log2_theta[1];
  const double f = exp2(x);
  return fma(f, rest * 0.693147180559945309417, f);
}

// Cosine and sine of the 64 angles 2 pi k / 64, from their series (the angles of
// the first eighth; the rest by symmetry).
struct Circle {
  double c[64], s[64];
};
constexpr Circle make_circle() {
  Circle t{};
  for (int k = 0; k < 64; ++k) {
    const int q = k / 16, r = k % 16, m = r > 8 ? 16 - r : r;  // quarter, place in it, folded to an eighth
    const double x = 0.098174770424681038702 * m, x2 = x * x;  // 2 pi / 64
    double c = 0.0, s = 0.0;
    for (int n = 20; n >= 1; --n) {
      c = (c + 1.0) * -x2 / ((2 * n - 1) * (2 * n));
      s = (s + 1.0) * -x2 / ((2 * n) * (2 * n + 1));
    }
    c = c + 1.0;
    s = (s + 1.0) * x;
    const double cr = r > 8 ? s : c, sr = r > 8 ? c : s;
    t.c[k] = q == 0 ? cr : q == 1 ? -sr : q == 2 ? -cr : sr;
    t.s[k] = q == 0 ? sr : q == 1 ? cr : q == 2 ? -sr : -cr;
  }
  return t;
}
__device__ constexpr Circle kCircle = make_circle();

// (cos x, sin x) to about 2^-51, at 20 double operations: the nearest of 64 angles
// from the table, turned by the rest t, |t| <= pi / 64, whose series end at t^8 and
// t^7 (2^-60 and 2^-57 off).
__device__ __forceinline__ double2 circle(double x) {
  const double k = rint(x * 10.185916357881302);  // 64 / 2 pi
  double t = fma(-k, 0.09817477042468103, x);    // 2 pi / 64 in two doubles
  t = fma(-k, 3.827021247335479e-18, t);
  const double t2 = t * t;
  const double ct = fma(t2, fma(t2, fma(t2, fma(t2, 1.0 / 40320, -1.0 / 720), 1.0 / 24), -0.5), 1.0);
  const double st = fma(t * t2, fma(t2, fma(t2, -1.0 / 5040, 1.0 / 120), -1.0 / 6), t);
  const int i = (int)((long long)k & 63);
  const double c = kCircle.c[i], s = kCircle.s[i];
  return make_double2(fma(c, ct, -s * st), fma(s, ct, c * st));
}

__device__ __forceinline__ float2 load_pair(const float *p, bool vec) {
  return vec ? *reinterpret_cast<const float2 *>(p) : make_float2(p[0], p[1]);
}
__device__ __forceinline__ float2 load_pair(const bf16 *p, bool vec) {
  if (!vec) return make_float2(to_f(p[0]), to_f(p[1]));
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Of a rope pair: its frequency, and the turn between a thread's rows.
struct Turn {
  double f;
  double2 step;
};
constexpr int kTurns = 128;  // pairs whose turns a block shares; the threads of a wider rope make their own

__device__ __forceinline__ Turn make_turn(const PagedRowsArgs &a, int j, int rows) {
  Turn t;
  t.f = frequency(a, j);
  t.step = circle((double)rows * a.pos_stride * t.f);
  return t;
}

// A group's scale from the bits of its largest magnitude (a NaN's are above every number's).
__device__ __forceinline__ uint8_t group_scale(uint32_t amax) {
  return __nv_cvt_float_to_fp8(__uint_as_float(amax) / 7.f, __NV_SATFINITE, __NV_E4M3);
}

// 16 dims as nibbles and their scale: codes 8 + clamp(rint(v / s), -7, 7), 8 under a
// zero or NaN scale. The quotient has to be rounded as one.
__device__ __forceinline__ uint2 pack16(const float (&v)[16], uint8_t &scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  scale = group_scale(m);
  const float s = e4m3_value(scale);
  uint32_t w[2] = {0x88888888u, 0x88888888u};
  if (s > 0.f) {
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      // 1.5 2^23 + 8 + q, rounded to a whole number (ties to even): its low bits are the code's
      const float q = fminf(fmaxf(v[i] / s, -7.f), 7.f);
      w[i >> 3] |= (__float_as_uint(__fadd_rn(q, 12582920.f)) & 15u) << (4 * ((i & 7) >> 1) + 16 * (i & 1));
    }
  }
  return make_uint2(w[0], w[1]);
}

// The same of bf16 values (x[i]: dims 2 i and 2 i + 1). A value's 8 bits by a
// scale's 4 give a tie (k + 1/2) or a quotient at least 2^-10 away from one, so v
// times 1 / s, off by 2^-24 of it, needs only be rounded to 2^-13 first for ties to
// be ties again: 1536 + v (1 / s) in one fused step has that spacing, and a second
// addition rounds it to a whole number. No quotient needs a clamp unless the scale
// was itself cut off (at 448, or among the subnormals).
__device__ __forceinline__ uint2 pack16(const uint32_t (&x)[8], uint8_t &scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x[i] & 0x7fff7fffu);
  m = max(m << 16, m & 0xffff0000u);
  scale = group_scale(m);
  const float s = e4m3_value(scale), inv = 1.f / s;
  uint32_t w[2] = {0x88888888u, 0x88888888u};
  if (__uint_as_float(m) * inv < 7.49f) {  // (false for a zero or NaN scale)
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float lo = __fadd_rn(__fmaf_rn(__uint_as_float(x[i] << 16), inv, 1536.f), 12581384.f);
      const float hi = __fadd_rn(__fmaf_rn(__uint_as_float(x[i] & 0xffff0000u), inv, 1536.f), 12581384.f);
      w[i >> 2] += (__byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) & 0x000f000fu) << (4 * (i & 3));
    }
  } else if (s > 0.f) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(x[i] << 16);
      v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
    return pack16(v, scale);
  }
  return make_uint2(w[0], w[1]);
}

// 16 elements as pack16 takes them, of which n exist.
__device__ __forceinline__ void load_group(const float *p, float (&v)[16], bool vec) { load16(p, v, 16, vec); }
__device__ __forceinline__ void load_group(const bf16 *p, uint32_t (&x)[8], bool vec) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = reinterpret_cast<const uint4 *>(p)[h];
      x[4 * h] = u.x; x[4 * h + 1] = u.y; x[4 * h + 2] = u.z; x[4 * h + 3] = u.w;
    }
  } else {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
  }
}
template <typename T> struct Group;
template <> struct Group<float> { float v[16]; };
template <> struct Group<bf16> { uint32_t v[8]; };

// Rows [r0, r0 + rb) of sequence b from dim d16 on: the rope dims, and in front of
// them (4 bits, where the rope begins inside a group) 8 dims that are not rotated.
// 4 bits: rotated into rot[rb][D - d16], then packed, a thread a group.
template <typename T, bool kInt4>
__device__ __forceinline__ void append_rotated(const PagedRowsArgs &a, int b, int r0, int rb, int d16, const long long *slot,
                                               Turn *turns, T *rot, bool vec) {
  const int D = a.cache.D, E = D - d16, P = E / 2, lead = P - a.rope_dims / 2;
  const int at_once = max(1, (int)blockDim.x / P);  // rows turned at once
  const bool shared = P - lead <= kTurns;
  if (shared) {
    for (int j = threadIdx.x; j < P - lead; j += blockDim.x) turns[j] = make_turn(a, j, at_once);
    __syncthreads();
  }
  const long long p0 = (a.pos0 ? a.pos0[b] : 0) + (long long)r0 * a.pos_stride;
  const T *rows = static_cast<const T *>(a.rows) + b * a.seq_stride + (long long)r0 * a.row_stride + d16;
  uint8_t *pages = const_cast<uint8_t *>(a.cache.pages);
  for (int t = threadIdx.x; t < at_once * P; t += blockDim.x) {
    const int j = t % P, first = t / P;
    if (first >= rb) continue;
    Turn u{0.0, make_double2(1.0, 0.0)};
    double2 at = u.step;
    if (j >= lead) {
      u = shared ? turns[j - lead] : make_turn(a, j - lead, at_once);
      at = circle((double)(p0 + (long long)first * a.pos_stride) * u.f);
    }
    constexpr int kAhead = 4;  // rows whose loads are in flight together
    for (int i0 = first; i0 < rb; i0 += kAhead * at_once) {
      float2 x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * at_once;
        x[k] = make_float2(0.f, 0.f);
        if (i < rb && slot[i] >= 0) x[k] = load_pair(rows + (long long)i * a.row_stride + 2 * j, vec);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * at_once;
        if (i >= rb) break;
        T y0 = from_f<T>((float)(x[k].x * at.x - x[k].y * at.y)), y1 = from_f<T>((float)(x[k].x * at.y + x[k].y * at.x));
        if (j < lead) y0 = from_f<T>(x[k].x), y1 = from_f<T>(x[k].y);  // (a turn by nothing would make inf * 0 of them)
        at = make_double2(at.x * u.step.x - at.y * u.step.y, at.y * u.step.x + at.x * u.step.y);
        if constexpr (kInt4) {
          rot[i * E + 2 * j] = y0;
          rot[i * E + 2 * j + 1] = y1;
        } else if (slot[i] >= 0) {
          T *o = reinterpret_cast<T *>(pages) + (size_t)slot[i] * D + d16 + 2 * j;
          o[0] = y0;
          o[1] = y1;
        }
      }
    }
  }
  if constexpr (kInt4) {
    __syncthreads();
    const int G = E / 16;
    for (int t = threadIdx.x; t < rb * G; t += blockDim.x) {
      const int i = t / G, g = t - i * G;
      if (slot[i] < 0) continue;
      Group<T> v;
      load_group(rot + i * E + 16 * g, v.v, true);
      uint8_t s;
      const uint2 w = pack16(v.v, s);
      *reinterpret_cast<uint2 *>(pages + (size_t)slot[i] * a.cache.row_bytes + d16 / 2 + 8 * g) = w;
      const_cast<uint8_t *>(a.cache.scales)[(size_t)slot[i] * (D / 16) + d16 / 16 + g] = s;
    }
  }
}

// Blocks [0, turn_blocks) take the rows' ends from dim d16 on, turn_rb rows each; the others the dims before, rb rows each.
template <typename T, bool kInt4>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(PagedRowsArgs a, int rb, int chunks, int turn_rb,
                                                                int turn_chunks, int turn_blocks, int d16, uint32_t per_g,
                                                                bool vec) {
  __shared__ long long slot[kMaxRows];
  __shared__ Turn turns[kTurns];
  __shared__ alignas(16) T rot[kInt4 ? kRotElems : 1];
  pdl_wait();
  pdl_release();
  if ((int)blockIdx.x < turn_blocks) {
    const int b = blockIdx.x / turn_chunks, r0 = (blockIdx.x - b * turn_chunks) * turn_rb;
    block_slots(a, b, r0, turn_rb, slot);
    __syncthreads();
    append_rotated<T, kInt4>(a, b, r0, turn_rb, d16, slot, turns, rot, vec);
    return;
  }
  const int blk = blockIdx.x - turn_blocks;
  const int b = blk / chunks, r0 = (blk - b * chunks) * rb, D = a.cache.D;
  block_slots(a, b, r0, rb, slot);
  __syncthreads();
  const int G = (d16 + 15) / 16;
  const T *rows = static_cast<const T *>(a.rows) + b * a.seq_stride + (long long)r0 * a.row_stride;
  uint8_t *pages = const_cast<uint8_t *>(a.cache.pages);
  for (int t = threadIdx.x; t < rb * G; t += blockDim.x) {
    const int i = quotient(t, per_g), g = t - i * G, d = 16 * g;
    if (slot[i] < 0) continue;
    if constexpr (kInt4) {
      Group<T> v;
      load_group(rows + i * a.row_stride + d, v.v, vec);
      uint8_t s;
      const uint2 w = pack16(v.v, s);
      *reinterpret_cast<uint2 *>(pages + (size_t)slot[i] * a.cache.row_bytes + 8 * g) = w;
      const_cast<uint8_t *>(a.cache.scales)[(size_t)slot[i] * (D / 16) + g] = s;
    } else {
      float v[16];
      const int n = min(16, d16 - d);
      load16(rows + i * a.row_stride + d, v, n, vec && n == 16);
      store16(reinterpret_cast<T *>(pages) + (size_t)slot[i] * D + d, v, n, vec && n == 16);
    }
  }
}

template <typename T, bool kInt4>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(PagedRowsArgs a, int rb, int chunks, uint32_t per_g,
                                                              bool vec) {
  __shared__ long long slot[kMaxRows];
  pdl_wait();
  pdl_release();
  const int b = blockIdx.x / chunks, r0 = (blockIdx.x - b * chunks) * rb, D = a.cache.D;
  block_slots(a, b, r0, rb, slot);
  __syncthreads();
  const int G = (D + 15) / 16;
  T *out = static_cast<T *>(const_cast<void *>(a.rows)) + b * a.seq_stride + (long long)r0 * a.row_stride;
  for (int t = threadIdx.x; t < rb * G; t += blockDim.x) {
    const int i = quotient(t, per_g), g = t - i * G, d = 16 * g;
    if (slot[i] < 0) continue;
    float v[16];
    const int n = min(16, D - d);
    if constexpr (kInt4) {
      const uint2 w = *reinterpret_cast<const uint2 *>(a.cache.pages + (size_t)slot[i] * a.cache.row_bytes + 8 * g);
      const float s = e4m3_value(a.cache.scales[(size_t)slot[i] * G + g]);
      if constexpr (sizeof(T) == 2) {
        if (vec) {  // already the output's type
          const uint32_t sc = bf16x2_dup(s), off = bf16x2_dup(-136.f * s);
          uint32_t lo[4], hi[4];
          widen8(w.x, sc, off, lo);
          widen8(w.y, sc, off, hi);
          uint4 *o = reinterpret_cast<uint4 *>(out + (long long)i * a.row_stride + d);
          o[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          o[1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          continue;
        }
      }
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

// Rows per block: enough to give every thread one of a row's `items`; more, up to
// `most`, where `per_sm` blocks per SM remain.
int rows_per_block(const PagedRowsArgs &a, int items, int per_sm, int most) {
  const long long fill = (long long)a.B * a.n / ((long long)per_sm * device_sm_count());
  long long rb = fill > most ? most : fill;
  if (rb < kThreads / items) rb = kThreads / items;
  if (rb < 1) rb = 1;
  if (rb > kMaxRows) rb = kMaxRows;
  return (int)(rb > a.n ? a.n : rb);
}

template <typename T>
cudaError_t launch_rows(const PagedRowsArgs &a, bool append, cudaStream_t stream) {
  const int D = a.cache.D;
  const bool int4 = a.cache.scales != nullptr;
  const uintptr_t e = sizeof(T);
  const bool vec = D % 16 == 0 && a.row_stride * e % 16 == 0 && a.seq_stride * e % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.rows) & 15) == 0 &&
                   (int4 || (reinterpret_cast<uintptr_t>(a.cache.pages) & 15) == 0);
  const int d_rot = append ? D - a.rope_dims : D, d16 = int4 ? d_rot & ~15 : d_rot;
  // (32,767 rows of 512 dims: into 4 bits 9.1 us with up to 32 rows a block, 9.8 with 16, 10.1 with 64; as they are
  // 12.2, 11.6 and 16.0; out of 4 bits 12.1, 10.1 and 11.0)
  const bool packs = append && int4;
  const int rb = rows_per_block(a, d16 ? (d16 + 15) / 16 : 1, packs ? 4 : 8, packs ? 32 : 16);
  const long long chunks = (a.n + rb - 1) / rb;
  long long blocks = d16 ? chunks * a.B : 0, turn_chunks = 1, turn_blocks = 0;
  int turn_rb = 1;
  if (d_rot < D) {  // (64 rows of 64 dims: a thread's first cosine and sine serve 8; the same rows 13.4 us, with 32 rows 14.7)
    turn_rb = rows_per_block(a, (D - d16) / 2, 2, 64);
    if (int4 && turn_rb * (D - d16) > kRotElems) turn_rb = kRotElems / (D - d16);
    turn_chunks = (a.n + turn_rb - 1) / turn_rb;
    turn_blocks = turn_chunks * a.B;
  }
  blocks += turn_blocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int items = max(rb * ((d16 + 15) / 16), turn_blocks ? turn_rb * ((D - d16) / 2) : 0);
  const int threads = min((items + 31) / 32 * 32, kThreads);
  const int G = (d16 + 15) / 16;
  const uint32_t per_g = G > 1 ? (uint32_t)(((1ull << 32) + G - 1) / G) : 0;
  if (append)
    return launch_pdl(int4 ? paged_append_kernel<T, true> : paged_append_kernel<T, false>, dim3((unsigned)blocks),
                      dim3(threads), 0, stream, a, rb, (int)chunks, turn_rb, (int)turn_chunks, (int)turn_blocks, d16, per_g, vec);
  return launch_pdl(int4 ? paged_read_kernel<T, true> : paged_read_kernel<T, false>, dim3((unsigned)blocks), dim3(threads), 0,
                    stream, a, rb, (int)chunks, per_g, vec);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedRowsArgs &a, bool append, cudaStream_t stream) {
  return a.dtype == CSA_DTYPE_F32 ? launch_rows<float>(a, append, stream) : launch_rows<bf16>(a, append, stream);
}

}  // namespace csa
