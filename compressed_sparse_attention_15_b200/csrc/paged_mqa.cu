// csa_paged_sparse_mqa / csa_paged_hca_mqa: attention over entries of a paged
// cache + sliding window + attention sink.
//
// The mathematics is csa_sparse_mqa's and hca_mqa's (mqa.cu), over rows found
// through a page table and, in the 4-bit form, widened on the way. This file
// holds the fp32-FFMA kernel for every shape, and the merge of its splits; the
// tensor-core kernel (bf16, head_dim a multiple of 128) is in paged_mqa_tc.cu.
//
// One block takes HG heads of a query and one of `splits` runs of 32-row
// chunks of its row list, and keeps the running maximum, sum and output of the
// heads in registers:
//   S: lane = row, warp = an eighth of the dims, every head at once (a row's 4
//      dims are read once for all heads); the warps' parts are added after.
//   O: thread = dim, rows in turn (in as many row groups as the dims leave
//      threads for, added at the end).
// Logits are held in units of log2, so that 2^x is the softmax's exponential.
// Shared-memory reads bound it (S: 12 wavefronts for 32 FFMA instructions of 8
// heads); eight heads a block keep a row's widening and reads common to them, and a
// query of 64 heads reads and widens its rows 8 times. 16 sequences of 8,192 entries,
// 64 heads of 512 dims in fp32: 7.1 ms, 1.7 ms from 4-bit pages (plain fp32 matrix
// products in torch on rows in order: 0.49 ms); from bf16 at 64 dims 0.67 ms.
#include "kernels.h"
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kRC = 32;         // rows per chunk
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDPT = 4;      // dims per thread: D <= 1024
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFloor = -1e30f;  // running maximum of no rows (finite: no inf - inf)

// Row stride in floats: a multiple of 4 whose quarter is odd, so that 32 rows' float4s fall into distinct banks.
__host__ __device__ inline int row_stride(int D) { return (((D + 3) / 4) | 1) * 4; }

template <typename T, int HG>
__global__ void __launch_bounds__(kThreads) paged_mqa_kernel(PagedMqaArgs a, int groups, int splits) {
  extern __shared__ float4 sm4[];
  const int D = a.cache.D, DS = row_stride(D), H = a.H;
  float *qs = reinterpret_cast<float *>(sm4);  // [HG][DS]
  float *rows = qs + HG * DS;                  // [kRC][DS]
  float *part = rows + kRC * DS;               // [kWarps][HG][kRC]
  float *ps = part + kWarps * HG * kRC;        // [kRC][HG]
  __shared__ const uint8_t *rowp[kRC], *scp[kRC];
  __shared__ float m_s[HG], l_s[HG], alpha_s[HG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_release();
  const int split = blockIdx.x % splits, qg = blockIdx.x / splits, qq = qg / groups, h0 = (qg - qq * groups) * HG;
  const int b = qq / a.q_per_seq, nh = min(HG, H - h0);
  uint32_t *st = tid == 0 && split == 0 ? a.status : nullptr;
  const int nsel = a.idx ? a.k : clamp_count(a.n_cmp[qq], (int)a.cache.capacity(), st);
  int wlo = 0, nwin = 0;
  if (a.win_len) {
    int e = a.win_end[qq];
    if (e < 0 || e >= a.T_raw) {
      raise_status(st, CSA_STATUS_BAD_WINDOW);
      e = e < 0 ? 0 : a.T_raw - 1;
    }
    wlo = max(0, e - a.win_len + 1);
    nwin = e - wlo + 1;
  }
  const int R = nsel + nwin, chunks = (R + kRC - 1) / kRC;
  const int c0 = (int)((long long)chunks * split / splits), c1 = (int)((long long)chunks * (split + 1) / splits);
  const T *win = static_cast<const T *>(a.kv_win) + (size_t)b * a.T_raw * D;
  const T *qp = static_cast<const T *>(a.q) + ((size_t)qq * H + h0) * D;
  for (int h = warp; h < HG; h += kWarps)
    for (int d = lane; d < DS; d += 32) qs[h * DS + d] = h < nh && d < D ? to_f(qp[(size_t)h * D + d]) : 0.f;
  if (tid < HG) m_s[tid] = kFloor, l_s[tid] = 0.f;
  // O: threads as (row group, dim)
  int DT = 32;
  while (DT < D && DT < kThreads) DT *= 2;
  const int RG = kThreads / DT, rg = tid / DT, dt = tid - rg * DT;
  float o[HG][kMaxDPT];
#pragma unroll
  for (int h = 0; h < HG; ++h)
#pragma unroll
    for (int i = 0; i < kMaxDPT; ++i) o[h][i] = 0.f;
  const float scale_log2 = a.scale * kLog2e;

  for (int c = c0; c < c1; ++c) {
    __syncthreads();  // the previous chunk's rows and weights are read
    if (tid < kRC) {
      const int r = c * kRC + tid;
      const uint8_t *p = nullptr, *s = nullptr;
      if (r < nsel) {
        const int j = a.idx ? a.idx[(size_t)qq * a.k + r] : r;
        if (j != -1) {
          const long long slot = paged_slot(a.cache, b, j, a.status);
          if (slot >= 0) {
            p = a.cache.pages + (size_t)slot * a.cache.row_bytes;
            if (a.cache.scales) s = a.cache.scales + (size_t)slot * (D / 16);
          }
        }
      } else if (r < R) {
        p = reinterpret_cast<const uint8_t *>(win + (size_t)(wlo + r - nsel) * D);
      }
      rowp[tid] = p;
      scp[tid] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRC / kWarps; ++i) {
      const int rr = warp + kWarps * i;
      const uint8_t *p = rowp[rr], *s = scp[rr];
      float *dst = rows + rr * DS;
      if (s) {
        for (int w = lane; w < D / 8; w += 32) {
          float v[8];
          unpack8(reinterpret_cast<const uint32_t *>(p)[w], e4m3_value(s[w >> 1]), v);
          *reinterpret_cast<float4 *>(dst + 8 * w) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4 *>(dst + 8 * w + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll 4
        for (int d = lane; d < D; d += 32) dst[d] = p ? to_f(reinterpret_cast<const T *>(p)[d]) : 0.f;
      }
      if (lane < DS - D) dst[D + lane] = 0.f;
    }
    __syncthreads();
    {
      const int q4 = DS / 4, v0 = q4 * warp / kWarps, v1 = q4 * (warp + 1) / kWarps;
      float acc[HG];
#pragma unroll
      for (int h = 0; h < HG; ++h) acc[h] = 0.f;
      for (int v = v0; v < v1; ++v) {
        const float4 x = *reinterpret_cast<const float4 *>(rows + lane * DS + 4 * v);
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float4 y = *reinterpret_cast<const float4 *>(qs + h * DS + 4 * v);
          acc[h] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[h]))));
        }
      }
#pragma unroll
      for (int h = 0; h < HG; ++h) part[(warp * HG + h) * kRC + lane] = acc[h];
    }
    __syncthreads();
    if (warp < HG) {
      const int h = warp;
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += part[(w * HG + h) * kRC + lane];
      const bool live = rowp[lane] != nullptr;
      x = live ? x * scale_log2 : -INFINITY;
      const float m_old = m_s[h], m_new = fmaxf(m_old, warp_max(x));
      const float p = live ? exp2f(x - m_new) : 0.f;
      ps[lane * HG + h] = p;
      const float sum = warp_sum(p);
      if (lane == 0) {
        const float al = exp2f(m_old - m_new);
        l_s[h] = l_s[h] * al + sum;
        m_s[h] = m_new;
        alpha_s[h] = al;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxDPT; ++i) {
      const int d = dt + DT * i;
      if (d < D) {
        float acc[HG];
#pragma unroll
        for (int h = 0; h < HG; ++h) acc[h] = o[h][i] * alpha_s[h];
#pragma unroll 4
        for (int rr = rg; rr < kRC; rr += RG) {
          const float v = rows[rr * DS + d];
#pragma unroll
          for (int h = 0; h < HG; ++h) acc[h] = fmaf(ps[rr * HG + h], v, acc[h]);
        }
#pragma unroll
        for (int h = 0; h < HG; ++h) o[h][i] = acc[h];
      }
    }
  }
  __syncthreads();
  if (RG > 1) {  // (one dim per thread: D <= 128)
    float *red = part;  // [HG][kThreads]
#pragma unroll
    for (int h = 0; h < HG; ++h) red[h * kThreads + tid] = o[h][0];
    __syncthreads();
    if (rg == 0) {
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        float s = 0.f;
        for (int g = 0; g < RG; ++g) s += red[h * kThreads + g * DT + dt];
        o[h][0] = s;
      }
    }
  }
  if (rg) return;
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    if (h >= nh) break;
    const size_t qh = (size_t)qq * H + h0 + h;
    float f = 1.f;
    if (splits > 1) {
      if (tid == 0) reinterpret_cast<float2 *>(a.part_ml)[qh * splits + split] = make_float2(m_s[h], l_s[h]);
    } else {
      const float m = m_s[h], sk = a.sink[h0 + h] * kLog2e, M = fmaxf(m, sk), wm = exp2f(m - M);
      const float L = l_s[h] * wm + exp2f(sk - M);
      f = L == 0.f ? 0.f : wm / L;  // (no row and a sink of -inf: nothing to attend, 0)
    }
#pragma unroll
    for (int i = 0; i < kMaxDPT; ++i) {
      const int d = dt + DT * i;
      if (d < D) {
        if (splits > 1)
          a.part_o[(qh * splits + split) * D + d] = o[h][i];
        else
          static_cast<T *>(a.out)[qh * D + d] = from_f<T>(o[h][i] * f);
      }
    }
  }
}

// Merge of a (query, head)'s splits with its sink:
//   M = max(max_s m_s, sink), L = sum_s l_s 2^(m_s - M) + 2^(sink - M),
//   out = sum_s O_s 2^(m_s - M) / L.
// A block takes 512 dims, four a thread, and each thread every split; or (kFew,
// where that leaves few blocks) 128 dims, and warp w of 8 the splits w, w + 8, ...
// Its bytes are the partials', just written, so L2 serves them; eight of a thread's
// are on their way while the first warp forms the weights.
constexpr int kMergeWarps = 8;

template <typename T, bool kVec, bool kFew>
__global__ void __launch_bounds__(kFew ? 32 * kMergeWarps : 128)
    paged_merge_kernel(const float *part_o, const float *part_ml, const float *sink, T *out, int H, int D, int splits) {
  __shared__ float4 acc_s[kFew ? kMergeWarps : 1][32];
  __shared__ float w[kPagedMaxSplits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kStep = kFew ? kMergeWarps : 1;
  const size_t qh = blockIdx.x;
  const int d0 = (kFew ? 128 : 512) * blockIdx.y, d = d0 + 4 * (kFew ? lane : (int)threadIdx.x);
  const int s0 = kFew ? warp : 0;
  pdl_wait();
  pdl_release();
  const float *src = part_o + qh * splits * D + d;
  auto load = [&](int s) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s >= splits) return v;
    const float *p = src + (size_t)s * D;
    if (kVec) {
      if (d < D) v = __ldcg(reinterpret_cast<const float4 *>(p));
    } else {
      if (d < D) v.x = __ldcg(p);
      if (d + 1 < D) v.y = __ldcg(p + 1);
      if (d + 2 < D) v.z = __ldcg(p + 2);
      if (d + 3 < D) v.w = __ldcg(p + 3);
    }
    return v;
  };
  constexpr int kAhead = 8;
  float4 v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) v[i] = load(s0 + kStep * i);
  if (warp == 0) {
    constexpr int kPer = kPagedMaxSplits / 32;
    const float2 *ml = reinterpret_cast<const float2 *>(part_ml) + qh * splits;
    const float sk = sink[qh % H] * kLog2e;
    float2 m[kPer];
    float M = sk, L = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      m[i] = lane + 32 * i < splits ? ml[lane + 32 * i] : make_float2(-INFINITY, 0.f);
      M = fmaxf(M, m[i].x);
    }
    M = warp_max(M);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      m[i].x = lane + 32 * i < splits ? exp2f(m[i].x - M) : 0.f;
      L = fmaf(m[i].y, m[i].x, L);
    }
    L = warp_sum(L) + exp2f(sk - M);
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < splits) w[lane + 32 * i] = m[i].x * inv;
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = s0; s < splits; s += kStep * kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s + kStep * i < splits) {
        const float c = w[s + kStep * i];
        acc.x = fmaf(c, v[i].x, acc.x);
        acc.y = fmaf(c, v[i].y, acc.y);
        acc.z = fmaf(c, v[i].z, acc.z);
        acc.w = fmaf(c, v[i].w, acc.w);
        v[i] = load(s + kStep * (i + kAhead));
      }
    }
  }
  if constexpr (kFew) {
    acc_s[warp][lane] = acc;
    __syncthreads();
    if (threadIdx.x < 128 && d0 + (int)threadIdx.x < D) {
      const float *a = reinterpret_cast<const float *>(acc_s) + threadIdx.x;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kMergeWarps; ++i) sum += a[128 * i];
      out[qh * D + d0 + threadIdx.x] = from_f<T>(sum);
    }
  } else {
    const float o[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d + e < D) out[qh * D + d + e] = from_f<T>(o[e]);
  }
}

template <typename T>
cudaError_t launch_merge(const PagedMqaArgs &a, int splits, cudaStream_t stream) {
  const long long blocks = (long long)a.Q * a.H;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int D = a.cache.D;
  const bool few = blocks < 4 * device_sm_count();
  auto kern = D % 4 ? (few ? paged_merge_kernel<T, false, true> : paged_merge_kernel<T, false, false>)
                    : (few ? paged_merge_kernel<T, true, true> : paged_merge_kernel<T, true, false>);
  const int dims = few ? 128 : 512, threads = few ? 32 * kMergeWarps : 128;
  return launch_pdl(kern, dim3((unsigned)blocks, (D + dims - 1) / dims), dim3(threads), 0, stream, (const float *)a.part_o,
                    (const float *)a.part_ml, a.sink, static_cast<T *>(a.out), a.H, D, splits);
}

int heads_per_block(int H) { return H >= 5 ? 8 : H >= 3 ? 4 : H; }

// Runs of chunks per query: enough blocks for two per SM, no run below two chunks.
int generic_splits(int Q, int H, int rows_max) {
  const int HG = heads_per_block(H), chunks = (rows_max + kRC - 1) / kRC;
  const long long blocks = (long long)Q * ((H + HG - 1) / HG);
  long long s = (2LL * device_sm_count() + blocks - 1) / blocks;
  if (s > (chunks + 1) / 2) s = (chunks + 1) / 2;
  return (int)(s < 1 ? 1 : s > kPagedMaxSplits ? kPagedMaxSplits : s);
}

template <typename T, int HG>
cudaError_t launch_hg(const PagedMqaArgs &a, int splits, cudaStream_t stream) {
  const int DS = row_stride(a.cache.D);
  const size_t floats = (size_t)(HG + kRC) * DS + kWarps * HG * kRC + kRC * HG;
  static DeviceOnce attr;  // set for the largest D the ABI admits
  once_per_device(attr, [] {
    cudaFuncSetAttribute(paged_mqa_kernel<T, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         (int)(((size_t)(HG + kRC) * row_stride(1024) + kWarps * HG * kRC + kRC * HG) * sizeof(float)));
  });
  const int groups = (a.H + HG - 1) / HG;
  const long long blocks = (long long)a.Q * groups * splits;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(paged_mqa_kernel<T, HG>, dim3((unsigned)blocks), dim3(kThreads), floats * sizeof(float), stream, a,
                    groups, splits);
}

template <typename T>
cudaError_t launch_generic(const PagedMqaArgs &a, cudaStream_t stream) {
  const int splits = generic_splits(a.Q, a.H, a.rows_max);
  cudaError_t e;
  switch (heads_per_block(a.H)) {
    case 8: e = launch_hg<T, 8>(a, splits, stream); break;
    case 4: e = launch_hg<T, 4>(a, splits, stream); break;
    case 2: e = launch_hg<T, 2>(a, splits, stream); break;
    default: e = launch_hg<T, 1>(a, splits, stream);
  }
  return e == cudaSuccess && splits > 1 ? launch_paged_merge(a, splits, stream) : e;
}

size_t ml_floats(int Q, int H, int splits) { return ((size_t)Q * H * splits * 2 + 3) & ~(size_t)3; }

size_t partial_floats(int Q, int H, int D, int splits) {
  return splits > 1 ? ml_floats(Q, H, splits) + (size_t)Q * H * splits * D : 0;
}

}  // namespace

cudaError_t launch_paged_merge(const PagedMqaArgs &a, int splits, cudaStream_t stream) {
  return a.dtype == CSA_DTYPE_F32 ? launch_merge<float>(a, splits, stream) : launch_merge<bf16>(a, splits, stream);
}

size_t paged_mqa_partial_bytes(int Q, int H, int D, int rows_max) {
  const int s = generic_splits(Q, H, rows_max), t = paged_mqa_tc_splits(Q, H, D, rows_max);
  return sizeof(float) * partial_floats(Q, H, D, s > t ? s : t);
}

// The workspace's partials: the (m, l) pairs, then the outputs, 16-byte aligned.
void paged_mqa_carve(PagedMqaArgs &a, void *partials, int splits) {
  a.part_ml = static_cast<float *>(partials);
  a.part_o = a.part_ml + ml_floats(a.Q, a.H, splits);
}

cudaError_t launch_paged_mqa(const PagedMqaArgs &args, void *partials, cudaStream_t stream) {
  bool taken = false;
  const cudaError_t e = launch_paged_mqa_tc(args, partials, stream, &taken);
  if (taken) return e;
  PagedMqaArgs a = args;
  paged_mqa_carve(a, partials, generic_splits(a.Q, a.H, a.rows_max));
  return a.dtype == CSA_DTYPE_F32 ? launch_generic<float>(a, stream) : launch_generic<bf16>(a, stream);
}

}  // namespace csa
