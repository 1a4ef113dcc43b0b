// csa_paged_sparse_mqa / csa_paged_hca_mqa on the tensor cores: bf16 queries,
// head_dim 128, 256, 384 or 512, a paged cache in bf16 or 4 bits.
//
// The products are mqa_tc.cu's, transposed, with the heads (64 a block, unused
// ones zero) on N:
//   S^T[r, h]  = sum_d KV[r, d] Q[h, d]      M = 64 rows,  K-major A and B
//   O^T[d, h] += sum_r KV[r, d] P^T[r, h]    M = 128 dims, A = the same tile read MN-major
// and so are the online softmax (running maximum moved only when a logit passes
// it by 2^8), the two tile buffers, and the issue order.
//
// A tile of 4-bit rows is widened to bf16 (exactly, two dims an instruction:
// widen8) on its way into shared memory. A lane takes 32 bytes of a row, the 64 dims of one
// 128-byte swizzled line, and 8 lanes take 8 rows, so that every 16-byte store
// of theirs falls into distinct banks. The packed rows come through a staging
// tile: each warp copies its own rows of the next tile there, asynchronously, once
// it has read those of the current one into registers (loads into registers would
// have to be waited for at the fence that shows a tile to the tensor core). Two
// warps look the rows up (list, page table), each load a tile ahead of its use, and
// publish them two tiles ahead.
//
// Two tiles are in flight (a third does not fit beside the queries), so a
// tile's way through widening, S^T, softmax and P.V bounds the rate as much as
// any one unit does: every widening warp works on every tile; a tile's halves (of
// 256 dims) are handed over one by one, so that S^T starts on the first while
// the second is widened, and the next tile's first half is widened while P.V
// works on the second; and eight softmax warps, a quarter of the rows and half
// of the heads each, take the logits as packed pairs, with one barrier (per half
// of the heads) on the usual path.
//
// The kernel is persistent: a block takes items (one split of the row list of 64
// heads of a query) in turn, and each role runs ahead into the next item, so that
// its loads, its queries' and its first products overlap the end of the last. Row
// lists differ in length (a selection ends at its last used slot), so a block
// claims its next item, by a counter in the workspace, when the lookups of the one
// it works on are done.
//
// What bounds it. A tile's products take the tensor pipe 1,800 cycles (S^T 32 MMAs
// of 32, P.V 16 of 48: their operands' shared-memory reads; with an N of 128 or more
// the same products would be about 1,030), widening it 4,096 words at 13
// instructions; it goes by in about 2,800, at half an instruction a cycle and
// scheduler and the tensor pipe 36 % active, because each tile's way through the five
// roles is a chain of waits and only two tiles fit. Measured: 16 sequences of 8,192
// entries 38 us with the merge of 4 (17.2 GFLOP: 0.27 of the measured tensor peak;
// the same rows in bf16 take 46), 1,024 prefill queries over up to 512 entries each
// 109 us, 32 decode queries over 512 of 16,383 entries 20 us with the merge. Code
// size counts: 130 KB of it, with every wait and loop in line, ran 1.3 times as long.
//
// Roles (640 threads): warps 0-7 widen (or copy bf16 rows), warps 8-15 run the
// softmax and write the output, warp 16 loads the queries and issues S^T, warp
// 17 issues P.V and owns TMEM, warps 18 and 19 look rows up. All
// mbarrier waits are bounded; the softmax warps of a half take every decision to
// stop together.
#include "attn.cuh"
#include "paged.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace csa {

namespace {

constexpr int kH = 64;                              // heads per block
constexpr int kRows = 64;                           // rows per tile
constexpr uint32_t kBoxBytes = kRows * 128;         // 64 rows x 64 dims
constexpr uint32_t kQBoxBytes = kH * 128;           // 64 heads x 64 dims
constexpr uint32_t kPBytes = kRows * kH * 2;
constexpr int kLoadWarps = 8;
constexpr int kRowsPerWarp = kRows / kLoadWarps;    // 8
constexpr int kSoftWarp0 = kLoadWarps;
constexpr int kSoftWarps = 8;
constexpr int kSWarp = kSoftWarp0 + kSoftWarps;
constexpr int kPvWarp = kSWarp + 1;
constexpr int kFetchWarp0 = kPvWarp + 1;
constexpr int kThreads = 32 * (kFetchWarp0 + 2);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kFloor = -1e30f;  // running maximum of no rows (finite: no inf - inf)

struct Small {
  // per tile buffer (and half of the dims): filled, read; per tile buffer: S^T made, P^T written
  uint64_t kv_full[2][2], kv_empty[2][2], s_full[2];
  // The same, of a window tile copied in bulk: its bytes are there. (Barriers of the
  // issuing thread alone: their phases end with the bytes, whichever role gives up.)
  uint64_t win_full[2][2];
  uint64_t p_full;                             // P^T written
  uint64_t slot_full[2], slot_empty[2];        // a tile's slots: published, read
  uint64_t pv_done[4];                         // P.V made, per tile (mod 4)
  uint64_t q_full, q_empty, o_done, o_free;    // per item: queries loaded / read, O^T made / read
  uint64_t norm_full[2];                       // per item (mod 2): norm is there
  uint64_t s_fin, pv_fin;                      // the last products of the block
  uint64_t item_full[4], item_empty[4];        // ring of the block's items
  alignas(16) int item[4][8];                  // of struct Item: qv, t0, ntiles, b, nsel, wlo, nwin, w64
  float red[4][kH];
  float mref[kH];
  float alpha[kH];            // what a rescale multiplies by
  // What an item's output is multiplied by: of its items with tiles in turn, and of
  // one without (an item of one tile gets there before the one before it is written).
  float norm[3][kH];
  uint32_t tmem_base;
  int abort;
  int rescale[2];             // per half of the heads
  uint8_t valid[2][kRows];    // per tile buffer: the row holds a key
  long long slot[2][kRows];   // of a tile (mod 2): row of the window or of the pages, -1: no key
};

// The staging tile: 64 rows of codes, then of scales. Row strides that put 8
// rows' reads (16 and 4 bytes a lane) into distinct banks.
constexpr uint32_t stage_row(int NB) { return 32 * NB + 16; }
constexpr uint32_t kStageScaleRow = 48;
constexpr uint32_t stage_bytes(int NB) { return kRows * (stage_row(NB) + kStageScaleRow); }

// Shared memory, in 64-dim boxes: two KV tiles, Q, P^T; the staging tile.
constexpr size_t smem_bytes(int NB) {
  return 1024 + (size_t)NB * (2 * kBoxBytes + kQBoxBytes) + kPBytes + stage_bytes(NB) + sizeof(Small);
}
static_assert(smem_bytes(8) <= 227 * 1024, "shared memory per block");

// An item: a run of tiles (split blockIdx.y of gridDim.y) of the row list of 64
// heads of a query. The list is the window rows [0, nwin) (kv_win rows wlo ...,
// padded with unused rows to whole tiles: w64), then the compressed rows
// [w64, w64 + nsel).
struct Item {
  int qv;  // query and head group; -1: no more items
  int qq, h0, b;
  int nsel, wlo, nwin, w64;
  int t0, ntiles;

  // Tile li holds 64 rows of the window on end, and is copied in bulk.
  __device__ __forceinline__ bool bulk(int li) const { return (t0 + li + 1) * kRows <= nwin; }
};

// The waits of this kernel: one try in line, the rest (with its limit) out of
// line. Some thirty waits by five roles, each with its own loop, made a kernel of
// 130 KB, more than the instruction caches hold, and every role slower.
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return tc::mbar_wait(bar, parity, abort, status, tc::wait_limit_of(status));
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return tc::mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, status);
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort, status));
}

// Query qv / 2 and its heads 64 (qv % 2) ... where a query has more than 64 heads, else query qv.
__device__ __forceinline__ int query_of(const PagedMqaArgs &a, int qv) { return a.H > kH ? qv >> 1 : qv; }

// Item number k of the block; false if the wait for it gave up. The whole warp takes part.
__device__ __forceinline__ bool take_item(const PagedMqaArgs &a, Small *sm, uint32_t k, volatile int *abort, Item &t) {
  if (!__all_sync(0xffffffffu, wait(&sm->item_full[k & 3], (k >> 2) & 1, abort, a.status))) return false;
  const int4 u = *reinterpret_cast<const int4 *>(sm->item[k & 3]), v = *reinterpret_cast<const int4 *>(sm->item[k & 3] + 4);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&sm->item_empty[k & 3]);
  t.qv = u.x;
  t.t0 = u.y;
  t.ntiles = u.z;
  t.b = u.w;
  t.nsel = v.x;
  t.wlo = v.y;
  t.nwin = v.z;
  t.w64 = v.w;
  t.qq = query_of(a, t.qv);
  t.h0 = a.H > kH ? (t.qv & 1) * kH : 0;
  return true;
}

// (nsel, wlo, nwin) of an item: the count clamped, a selection up to its last used slot.
__device__ __forceinline__ int3 item_rows(const PagedMqaArgs &a, int qv, int lane, uint32_t *status) {
  const int qq = query_of(a, qv);
  int3 v = make_int3(0, 0, 0);
  int e = a.win_len ? a.win_end[qq] : 0;
  if (a.idx) {
#pragma unroll 1
    for (int i0 = a.k - 128; v.x == 0 && i0 > -128; i0 -= 128) {
      int last = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + lane + 32 * u;
        if (i >= 0 && a.idx[(size_t)qq * a.k + i] != -1) last = i + 1;
      }
      v.x = __reduce_max_sync(0xffffffffu, last);
    }
  } else {
    v.x = clamp_count(a.n_cmp[qq], (int)a.cache.capacity(), status);
  }
  if (a.win_len) {
    if (e < 0 || e >= a.T_raw) {
      raise_status(status, CSA_STATUS_BAD_WINDOW);
      e = e < 0 ? 0 : a.T_raw - 1;
    }
    v.y = max(0, e - a.win_len + 1);
    v.z = e - v.y + 1;
  }
  return v;
}

// 32 bytes of codes and 4 of scales: 64 dims of one row.
struct Packed {
  uint32_t w[8];
  uint32_t s;
};

__device__ __forceinline__ void load_packed(Packed &u, uint32_t codes, uint32_t scales) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.w[4 * i]), "=r"(u.w[4 * i + 1]), "=r"(u.w[4 * i + 2]), "=r"(u.w[4 * i + 3])
                 : "r"(codes + 16 * i));
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u.s) : "r"(scales));
}

// 8 or 16 bytes from global memory, or zeros where there is no source. (Zeros are
// stored: a copy of no bytes still asks for its address, the same one everywhere.
// Predicated, as a branch a piece cost 7 % of a prefill chunk.)
template <int kBytes>
__device__ __forceinline__ void copy_piece(uint32_t dst, uint64_t src) {
  if constexpr (kBytes == 16)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u64 p, %1, 0;\n\t"
        "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t@!p st.shared.v4.b32 [%0], {%2, %2, %2, %2};\n\t}" ::"r"(dst),
        "l"(src), "r"(0)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u64 p, %1, 0;\n\t"
        "@p cp.async.ca.shared.global [%0], [%1], 8;\n\t@!p st.shared.v2.b32 [%0], {%2, %2};\n\t}" ::"r"(dst), "l"(src), "r"(0)
        : "memory");
}

// *p, or 0 without reading it where !pred. (One predicated load: no branch at
// whose end its value would be waited for.)
__device__ __forceinline__ int load_if(const int32_t *p, bool pred) {
  int v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.nc.b32 %0, [%1];\n\t}"
               : "=r"(v)
               : "l"(p), "r"((uint32_t)pred));
  return v;
}

// tcgen05.ld of 16 TMEM lanes x 32 columns (16x256b shape, 4 repeats): for
// column group c, thread t gets r[4c + e] = (lane t/4, column 8c + 2(t%4) + e)
// and r[4c + 2 + e] = (lane t/4 + 8, same column), e = 0, 1.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 TMEM lanes x 16 columns: thread i holds lane i of the warp's quarter.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Four 8 x 8 blocks of 16-bit elements: lane i gives the address of row i % 8 of
// block i / 8 and holds row i / 4, columns 2 (i % 4) and the next, of each block.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}

// An 8 x 8 block of 16-bit elements (lane i: row i / 4, columns 2 (i % 4) and the next), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The 64 dims of `u` into the 128-byte line whose chunk 0 is at `chunk0` (16-byte chunks, swizzled).
__device__ __forceinline__ void store_widened(const Packed &u, uint32_t chunk0) {
  // per 16 dims: s and -136 s, in both halves of a register
  uint32_t sc[4], off[4];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u.s >> (16 * p)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    sc[2 * p] = bf16x2_dup(f.x);
    sc[2 * p + 1] = bf16x2_dup(f.y);
    off[2 * p] = bf16x2_dup(-136.f * f.x);
    off[2 * p + 1] = bf16x2_dup(-136.f * f.y);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t v[4];
    widen8(u.w[c], sc[c >> 1], off[c >> 1], v);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk0 ^ (c << 4)), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
  }
}

// The products of dims [256 part, 256 part + 256) of one tile.
template <int NB>
__device__ __forceinline__ void issue_s(uint32_t tmem_s, uint64_t kv, uint64_t q, int part) {
  constexpr uint32_t idesc = tc::idesc_bf16(64, 64, 0, 0);
  const int b0 = 4 * part, b1 = min(NB, b0 + 4);
  kv += (uint64_t)(b0 * (kBoxBytes >> 4));
  q += (uint64_t)(b0 * (kQBoxBytes >> 4));
#pragma unroll 1
  for (int bx = b0; bx < b1; ++bx, kv += kBoxBytes >> 4, q += kQBoxBytes >> 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) tc::mma_bf16(tmem_s, kv + 2 * j, q + 2 * j, idesc, bx > 0 || j > 0);
  }
}
template <int NB>
__device__ __forceinline__ void issue_pv(uint32_t tmem_o, uint64_t v, uint64_t p, bool first, int part) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, 64, 1, 1);
  const int m0 = 2 * part, m1 = min(NB / 2, m0 + 2);
  v += (uint64_t)(m0 * (2 * kBoxBytes >> 4));
  tmem_o += 64 * m0;
#pragma unroll 1
  for (int m = m0; m < m1; ++m, tmem_o += 64, v += 2 * kBoxBytes >> 4) {
#pragma unroll
    for (int j = 0; j < kRows / 16; ++j) tc::mma_bf16(tmem_o, v + 128 * j, p + 128 * j, idesc, j > 0 || !first);
  }
}

// O^T of 64 heads of a query, [32 i, 32 i + 32) of every 128 dims and `heads`
// (up to 32) heads from the query's `qh` on, times norm, to the output or, as it
// is, to the partials. A warp takes blocks m0 .. m1 - 1 of 16 dims (m / 2: the
// 128-dim chunk, m % 2: half of the warp's TMEM quarter), each turned in registers
// so that 4 lanes write a 32-byte sector of a head's row.
template <int NB>
__device__ __noinline__ void write_out(const PagedMqaArgs &a, uint32_t tmem, const float *norm, size_t qh, int heads,
                                          int quarter, int m0, int m1, bool some, uint64_t *o_free) {
  constexpr int kD = 64 * NB;
  const int lane = threadIdx.x & 31, rq = lane >> 2, cq = lane & 3;
  const int splits = gridDim.y;
  uint64_t f[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) f[c] = pack2(norm[8 * c + 2 * cq], norm[8 * c + 2 * cq + 1]);
#pragma unroll 1
  for (int m = m0; m < m1; ++m) {
    uint32_t v[16];
    if (some) {
      tmem_ld_16x256b_x4(tmem + ((uint32_t)(32 * quarter + 16 * (m & 1)) << 16) + 64 * (m >> 1), v);
      tc::tmem_ld_wait();
      if (m == m1 - 1) {  // read: the next item's P.V may overwrite it
        tc::fence_before_sync();
        tc::mbar_arrive(o_free);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) v[c] = 0u;
    }
    const int d0 = 128 * (m >> 1) + 32 * quarter + 16 * (m & 1);
    if (splits > 1) {
      float *po = a.part_o + ((qh + 2 * cq) * splits + blockIdx.y) * kD + d0 + rq;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (8 * c + 2 * cq + e < heads) {
            float *p = po + (size_t)(8 * c + e) * splits * kD;
            p[0] = __uint_as_float(v[4 * c + e]);
            p[8] = __uint_as_float(v[4 * c + 2 + e]);
          }
    } else {
      // lane 4 h + i: dims 0, 8, 4 or 12 and the next three of head 8 c + h
      bf16 *out = static_cast<bf16 *>(a.out) + (qh + rq) * kD + d0 + 8 * (cq & 1) + 2 * (cq & 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t t[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 y = unpack2(mul2(pack2(__uint_as_float(v[4 * c + 2 * r]), __uint_as_float(v[4 * c + 2 * r + 1])), f[c]));
          const __nv_bfloat162 w = __floats2bfloat162_rn(y.x, y.y);
          t[r] = transpose8(*reinterpret_cast<const uint32_t *>(&w));  // dims 8 r + 2 cq, + 1 of head 8 c + rq
        }
        const uint32_t got = __shfl_xor_sync(0xffffffffu, cq & 1 ? t[0] : t[1], 1);
        if (8 * c + rq < heads)
          *reinterpret_cast<uint2 *>(out + (size_t)8 * c * kD) = cq & 1 ? make_uint2(got, t[1]) : make_uint2(t[0], got);
      }
    }
  }
}

// NB: head_dim / 64. kInt4: the cache is in 4 bits.
template <int NB, bool kInt4>
__global__ void __launch_bounds__(kThreads, 1)
    paged_mqa_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_win, PagedMqaArgs a,
                        int qvs, float scale_log2) {
  constexpr int kD = 64 * NB;
  constexpr uint32_t kTileBytes = NB * kBoxBytes, kQBytes = NB * kQBoxBytes;
  constexpr uint32_t kColS = 64 * (NB / 2);  // O^T chunk m at columns 64 m, S^T buffer j at kColS + 64 j
  constexpr uint32_t kTmemCols = kColS + 128 > 256 ? 512 : 256;
  constexpr int kParts = (NB + 3) / 4;       // parts of 256 dims a tile is handed over in
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *kv = smem;                              // [2 tiles][NB boxes][64 rows][128 B]
  uint8_t *qs = smem + 2 * kTileBytes;             // [NB boxes][64 heads][128 B]
  uint8_t *ps = qs + kQBytes;                      // [64 rows][128 B]  (P^T, MN-major)
  uint8_t *stage = ps + kPBytes;
  Small *sm = reinterpret_cast<Small *>(stage + stage_bytes(NB));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        tc::mbar_init(&sm->kv_full[i][j], 32 * kLoadWarps);
        tc::mbar_init(&sm->kv_empty[i][j], 1);
        tc::mbar_init(&sm->win_full[i][j], 1);
      }
      tc::mbar_init(&sm->s_full[i], 1);
    }
    tc::mbar_init(&sm->p_full, 32 * kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm->slot_full[i], kRows);
      tc::mbar_init(&sm->slot_empty[i], kLoadWarps);
    }
    for (int i = 0; i < 4; ++i) tc::mbar_init(&sm->pv_done[i], 1);
    tc::mbar_init(&sm->q_full, 1);
    tc::mbar_init(&sm->q_empty, 1);
    tc::mbar_init(&sm->o_done, 1);
    tc::mbar_init(&sm->o_free, 32 * (kLoadWarps + kSoftWarps));
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm->norm_full[i], kH);
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sm->item_full[i], 1);
      tc::mbar_init(&sm->item_empty[i], kThreads / 32);
    }
    tc::mbar_init(&sm->s_fin, 1);
    tc::mbar_init(&sm->pv_fin, 1);
    sm->abort = 0;
    tc::fence_barrier_init();
  }
  if (threadIdx.x < kH) sm->mref[threadIdx.x] = kFloor;
  if (warp == kPvWarp) tc::tmem_alloc(&sm->tmem_base, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm->tmem_base;
  volatile int *abort = &sm->abort;
  pdl_wait();
  pdl_release();

  if (warp < kLoadWarps) {
    // ------------------------------------------------------------ widening
    // Every warp takes 8 rows of every tile, a lane 64 dims of row lane % 8.
    const uint32_t kv_base = tc::smem_u32(kv), stage_base = tc::smem_u32(stage);
    const int my_row = kRowsPerWarp * warp + (lane & 7);
    const uint32_t codes = stage_base + my_row * stage_row(NB), scales = stage_base + kRows * stage_row(NB) + my_row * kStageScaleRow;
    uint32_t T = 0;  // tiles so far
    bool ok = true;
    // Half of an item's output is these warps' to write. They do so when both
    // tile buffers hold tiles of the items after it, and have nothing else to do.
    uint32_t bulk_made = 0, bulk_phase = 0;  // bit g: tiles copied in bulk into buffer g: some, the parity of their number
    int out_qv = -1;
    uint32_t out_at = 0, done = 0;  // the tile before which it is written; items written
    auto output = [&] {
      ok = ok && wait(&sm->norm_full[done & 1], (done >> 1) & 1, abort, a.status);
      ok = ok && wait(&sm->o_done, done & 1, abort, a.status);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      const int half = warp >> 2, h0 = (a.H > kH ? (out_qv & 1) * kH : 0) + 32 * half;
      if (ok)
        write_out<NB>(a, tmem + 32 * half, sm->norm[done & 1] + 32 * half, (size_t)query_of(a, out_qv) * a.H + h0, a.H - h0, warp & 3,
                      NB / 2, NB, true, &sm->o_free);
      ++done;
      out_qv = -1;
    };
    for (uint32_t k = 0; ok; ++k) {
      Item L;
      ok = take_item(a, sm, k, abort, L);
      if (!ok || L.qv < 0) break;
      // This warp's rows of tile li: their slots, and their packed bytes on their way into the staging tile.
      long long next_slot = -1;
      auto stage_rows = [&](int li, uint32_t t) {
        ok = ok && warp_wait(&sm->slot_full[t & 1], (t >> 1) & 1, abort, a.status);
        if (!ok) return;
        next_slot = sm->slot[t & 1][my_row];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->slot_empty[t & 1]);
        if (kInt4 && (L.t0 + li) * kRows >= L.w64) {
          // this lane's row as an address (0: no key); every lane copies pieces of every row
          const uint64_t code_row = next_slot >= 0 ? reinterpret_cast<uint64_t>(a.cache.pages) + (uint64_t)next_slot * (kD / 2) : 0;
          const uint64_t scale_row = next_slot >= 0 ? reinterpret_cast<uint64_t>(a.cache.scales) + (uint64_t)next_slot * (kD / 16) : 0;
          constexpr int kPer = 2 * NB;  // 16-byte pieces of a row's codes
#pragma unroll
          for (int i = 0; i < kRowsPerWarp * kPer / 32; ++i) {
            const int n = 32 * i + lane, rw = n / kPer, c = n - rw * kPer;
            const uint64_t row = __shfl_sync(0xffffffffu, code_row, rw);
            copy_piece<16>(stage_base + (kRowsPerWarp * warp + rw) * stage_row(NB) + 16 * c, row ? row + 16 * c : 0);
          }
          constexpr int kPiece = NB % 4 ? 8 : 16, kPerS = 4 * NB / kPiece;  // pieces of a row's scales
          const int rw = lane / kPerS, c = lane - rw * kPerS;
          const uint64_t row = __shfl_sync(0xffffffffu, scale_row, rw & 7);
          if (rw < kRowsPerWarp)
            copy_piece<kPiece>(stage_base + kRows * stage_row(NB) + (kRowsPerWarp * warp + rw) * kStageScaleRow + kPiece * c,
                               row ? row + kPiece * c : 0);
        }
      };
      if (L.ntiles > 0) stage_rows(0, T);
      for (int li = 0; li < L.ntiles; ++li, ++T) {
        const int g = T & 1;
        if (out_qv >= 0 && T == out_at) output();
        if (!ok) break;
        const uint32_t free_phase = ((T >> 1) & 1) ^ 1, line = kv_base + g * kTileBytes + my_row * 128 + ((lane & 7) << 4);
        const bool in_win = (L.t0 + li) * kRows < L.w64;
        const long long slot = next_slot;
        if (kInt4 && !in_win) {
          cp_async_wait_all();
          __syncwarp();
          Packed u[kParts];
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            const int s = min((lane >> 3) + 4 * i, NB - 1);  // (a piece past the row is not stored)
            load_packed(u[i], codes + 32 * s, scales + 4 * s);
          }
          __syncwarp();
          if (li + 1 < L.ntiles) stage_rows(li + 1, T + 1);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            ok = warp_wait(&sm->kv_empty[g][i], free_phase, abort, a.status);
            if (!ok) break;
            if (i == 0 && lane < kRowsPerWarp) sm->valid[g][my_row] = slot >= 0;
            const int s = (lane >> 3) + 4 * i;
            if (s < NB) store_widened(u[i], line + s * kBoxBytes);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc::mbar_arrive(&sm->kv_full[g][i]);
          }
        } else {
          if (li + 1 < L.ntiles) stage_rows(li + 1, T + 1);
#pragma unroll
          for (int i = 0; i < kParts; ++i)
            ok = ok && wait(&sm->kv_empty[g][i], free_phase, abort, a.status);
          ok = __all_sync(0xffffffffu, ok);
          const int r0 = (L.t0 + li) * kRows;
          if (ok && L.bulk(li)) {
            // 64 rows of the window on end: bulk copies, which land while the next tile is widened. (Not so where
            // rows of the tile lie outside the window: those must not be read.)
            if (lane < kRowsPerWarp) sm->valid[g][my_row] = 1;
            if (warp == 0 && lane == 0) {
#pragma unroll 1
              for (int i = 0; i < kParts; ++i) {
                const int b0 = 4 * i, b1 = min(NB, b0 + 4);
                tc::mbar_arrive_expect_tx(&sm->win_full[g][i], (b1 - b0) * kBoxBytes);
#pragma unroll 1
                for (int bx = b0; bx < b1; ++bx)
                  tc::tma_load_2d(kv + g * kTileBytes + bx * kBoxBytes, &tm_win, 64 * bx, L.b * a.T_raw + L.wlo + r0,
                                  &sm->win_full[g][i]);
              }
              bulk_made |= 1u << g;
              bulk_phase ^= 1u << g;
            }
#pragma unroll
            for (int i = 0; i < kParts; ++i) tc::mbar_arrive(&sm->kv_full[g][i]);
          } else if (ok) {
            if (lane < kRowsPerWarp) sm->valid[g][my_row] = slot >= 0;
            const bf16 *base = in_win ? static_cast<const bf16 *>(a.kv_win) + (size_t)L.b * a.T_raw * kD
                                      : reinterpret_cast<const bf16 *>(a.cache.pages);
#pragma unroll 4
            for (int rw = 0; rw < kRowsPerWarp; ++rw) {
              const long long at = __shfl_sync(0xffffffffu, slot, rw);
              const uint32_t dst = kv_base + g * kTileBytes + (kRowsPerWarp * warp + rw) * 128;
              const uint64_t src = at >= 0 ? reinterpret_cast<uint64_t>(base + (size_t)at * kD) : 0;
              for (int c16 = lane; c16 < 8 * NB; c16 += 32)  // 16-byte piece c16 of the row
                copy_piece<16>(dst + (c16 >> 3) * kBoxBytes + (((c16 & 7) ^ rw) << 4), src ? src + 16 * c16 : 0);
            }
            cp_async_wait_all();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
            for (int i = 0; i < kParts; ++i) tc::mbar_arrive(&sm->kv_full[g][i]);
          }
        }
        if (!ok) break;
      }
      if (ok && L.ntiles > 0) {
        // (an item of one tile may end before the output of the one before it is due)
        if (out_qv >= 0) output();
        out_qv = L.qv;
        out_at = T + 2;
      }
    }
    if (out_qv >= 0) output();
    cp_async_wait_all();
    // Nothing is in flight when the block ends: a buffer's last bulk copy has landed, or is waited for here (the one
    // before it was used: the buffer was free again).
    for (int g = 0; g < 2; ++g)
      if (bulk_made >> g & 1)
        for (int i = 0; i < kParts; ++i) tc::mbar_drain(&sm->win_full[g][i], ((bulk_phase >> g) & 1) ^ 1);
  } else if (warp >= kFetchWarp0) {
    // ------------------------------------------------------------ lookups
    // A lane looks one row up.
    const int my_row = 32 * (warp - kFetchWarp0) + lane;
    uint32_t T = 0;
    bool ok = true;
    // The first of these warps also makes the block's items, the next when it has
    // fetched the last tile of one: the tiles in flight then last longer than the
    // claim and the loads take, and the blocks end as evenly as may be.
    const bool maker = warp == kFetchWarp0;
    for (uint32_t k = 0; ok; ++k) {
      if (maker) {
        int next = blockIdx.x;  // (the first item is the block's own)
        if (k > 0) {
          next = qvs;
          if (qvs > (int)gridDim.x) next = __shfl_sync(0xffffffffu, lane == 0 ? (int)(gridDim.x + atomicAdd(a.status + 4, 1u)) : 0, 0);
        }
        const int3 v = next < qvs ? item_rows(a, next, lane, blockIdx.y == 0 && lane == 0 ? a.status : nullptr) : make_int3(0, 0, 0);
        ok = warp_wait(&sm->item_empty[k & 3], ((k >> 2) & 1) ^ 1, abort, a.status);
        if (ok && lane == 0) {
          const int w64 = (v.z + kRows - 1) / kRows * kRows, tiles = (w64 + v.x + kRows - 1) / kRows;
          const int splits = gridDim.y, split = blockIdx.y, base = tiles / splits, rest = tiles - base * splits;
          *reinterpret_cast<int4 *>(sm->item[k & 3]) = make_int4(next < qvs ? next : -1, split * base + min(split, rest),
                                                                 base + (split < rest ? 1 : 0), query_of(a, next) / a.q_per_seq);
          *reinterpret_cast<int4 *>(sm->item[k & 3] + 4) = make_int4(v.x, v.y, v.z, w64);
          tc::mbar_arrive(&sm->item_full[k & 3]);
        }
      }
      Item L;
      ok = take_item(a, sm, k, abort, L);
      if (!ok || L.qv < 0) break;
      const int t0 = L.t0, ntiles = L.ntiles, b = L.b, qq = L.qq;
      auto is_win = [&](int li) { return (t0 + li) * kRows < L.w64; };
      // The lookup of this lane's row of tile li in three steps, each one load: the
      // row's entry, or number in the window; ...
      struct Entry {
        int j;
        bool live;
      };
      auto entry_of = [&](int li) -> Entry {
        const int r = (t0 + li) * kRows + my_row, p = r - L.w64;
        const bool mine = li < ntiles;
        if (p < 0) return Entry{L.wlo + r, mine && r < L.nwin};
        const bool live = mine && p < L.nsel;
        return Entry{a.idx ? load_if(a.idx + (size_t)qq * a.k + p, live) : p, live};
      };
      // ... its page and the row there (-1: no key); ...
      auto page_of = [&](int li, Entry e) -> int2 {
        if (is_win(li)) return make_int2(0, e.live ? e.j : -1);
        const bool ok = e.live && e.j >= 0 && e.j < a.cache.capacity();
        if (e.live && !ok && e.j != -1) raise_status(a.status, CSA_STATUS_BAD_INDEX);
        const uint2 at = page_and_row(a.cache, ok ? e.j : 0);
        return make_int2(load_if(a.cache.table + (size_t)b * a.cache.per + at.x, ok), ok ? (int)at.y : -1);
      };
      // ... and the row of the window or of the pages.
      auto row_of = [&](int li, int2 pg) -> long long {
        if (pg.y < 0 || is_win(li)) return pg.y;
        if (pg.x < 0 || pg.x >= a.cache.num_pages) {
          raise_status(a.status, CSA_STATUS_BAD_PAGE);
          return -1;
        }
        return (long long)pg.x * a.cache.page + pg.y;
      };
      const Entry e0 = entry_of(0), e1 = entry_of(1);
      Entry e2 = entry_of(2);
      const int2 p0 = page_of(0, e0);
      int2 p1 = page_of(1, e1);
      long long at = row_of(0, p0);
      for (int li = 0; li < ntiles; ++li, ++T) {
        ok = warp_wait(&sm->slot_empty[T & 1], ((T >> 1) & 1) ^ 1, abort, a.status);
        if (!ok) break;
        sm->slot[T & 1][my_row] = at;
        if ((!kInt4 || is_win(li)) && at >= 0) {  // a bf16 row: into L2, for the copy
          const bf16 *base = is_win(li) ? static_cast<const bf16 *>(a.kv_win) + (size_t)b * a.T_raw * kD
                                        : reinterpret_cast<const bf16 *>(a.cache.pages);
          bulk_prefetch_l2(base + (size_t)at * kD, kD * 2);
        }
        tc::mbar_arrive(&sm->slot_full[T & 1]);
        at = row_of(li + 1, p1);
        p1 = page_of(li + 2, e2);
        e2 = entry_of(li + 3);
      }
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------ queries, S^T
    // (the whole warp runs the loops of the two issuers; one lane issues)
    const uint64_t ad_kv = tc::sw128_desc(tc::smem_u32(kv), 16, 1024), bd_q = tc::sw128_desc(tc::smem_u32(qs), 16, 1024);
    auto ready = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.status); };
    uint32_t T = 0, done = 0;  // tiles and items (with tiles) so far
    uint32_t bulk_phase = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      Item it;
      ok = take_item(a, sm, k, abort, it);
      if (!ok || it.qv < 0) break;
      if (it.ntiles == 0) continue;
      if (done > 0 && !(ok = ready(&sm->q_empty, (done - 1) & 1))) break;
      if (tc::elect_one()) {
        tc::mbar_arrive_expect_tx(&sm->q_full, kQBytes);
#pragma unroll 1
        for (int bx = 0; bx < NB; ++bx) tc::tma_load_3d(qs + bx * kQBoxBytes, &tm_q, bx * 64, it.h0, it.qq, &sm->q_full);
      }
      __syncwarp();
      if (!(ok = ready(&sm->q_full, done & 1))) {
        if (tc::elect_one()) tc::mbar_drain(&sm->q_full, done & 1);  // (nothing is in flight when the block ends)
        break;
      }
      for (int li = 0; li < it.ntiles; ++li, ++T) {
        const int buf = T & 1;
        // (S^T(T) overwrites S^T(T - 2), which has been read: the tile buffer was free for tile T only
        // after P.V(T - 2))
#pragma unroll 1
        for (int i = 0; i < kParts; ++i) {
          if (!(ok = ready(&sm->kv_full[buf][i], (T >> 1) & 1))) break;
          if (it.bulk(li) && !(ok = ready(&sm->win_full[buf][i], (bulk_phase >> buf) & 1))) break;
          tc::fence_after_sync();
          if (tc::elect_one())
            issue_s<NB>(tmem + kColS + 64 * buf, ad_kv + (uint64_t)((buf * kTileBytes) >> 4), bd_q, i);
          __syncwarp();
        }
        if (!ok) break;
        if (it.bulk(li)) bulk_phase ^= 1u << buf;
        if (tc::elect_one()) {
          tc::commit(&sm->s_full[buf]);
          if (li == it.ntiles - 1) tc::commit(&sm->q_empty);
        }
        __syncwarp();
      }
      ++done;
    }
    if (tc::elect_one()) {
      tc::commit(&sm->s_fin);
      tc::mbar_drain(&sm->s_fin, 0);
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ P.V
    const uint64_t ad_v = tc::sw128_desc(tc::smem_u32(kv), kBoxBytes, 1024);
    const uint64_t bd_p = tc::sw128_desc(tc::smem_u32(ps), kPBytes, 1024);
    auto ready = [&](uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity, abort, a.status); };
    uint32_t T = 0, done = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      Item it;
      ok = take_item(a, sm, k, abort, it);
      if (!ok || it.qv < 0) break;
      const int ntiles = it.ntiles;
      if (ntiles == 0) continue;
      if (done > 0 && !(ok = ready(&sm->o_free, (done - 1) & 1))) break;
      for (int li = 0; li < ntiles; ++li, ++T) {
        const int buf = T & 1;
        for (int i = 0; i < kParts; ++i) ok = ok && ready(&sm->kv_full[buf][i], (T >> 1) & 1);  // (the tile's writes; of
        // one copied in bulk S^T has waited for the bytes and read them, and P^T comes after S^T)
        if (!ok || !(ok = ready(&sm->p_full, T & 1))) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll 1
          for (int i = 0; i < kParts; ++i) {
            issue_pv<NB>(tmem, ad_v + (uint64_t)((buf * kTileBytes) >> 4), bd_p, li == 0, i);
            tc::commit(&sm->kv_empty[buf][i]);
          }
          tc::commit(&sm->pv_done[T & 3]);
          if (li == ntiles - 1) tc::commit(&sm->o_done);
        }
        __syncwarp();
      }
      ++done;
    }
    if (tc::elect_one()) {
      tc::commit(&sm->pv_fin);
      tc::mbar_drain(&sm->pv_fin, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // An M = 64 accumulator occupies TMEM lanes 0-15 of each 32-lane quarter: a
    // warp takes the 16 rows of its quarter and 32 heads, read with the 16x256b
    // shape: lane t holds rows rq = t/4 and rq + 8 for heads 8c + 2cq + {0, 1}
    // (c = 0..3, cq = t%4) of its half.
    const int quarter = warp & 3, half = (warp - kSoftWarp0) >> 2;
    const int rq = lane >> 2, cq = lane & 3;
    const int rowA = quarter * 16 + rq, rowB = rowA + 8;  // tile rows of this thread
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    float *red = sm->red[quarter] + 32 * half;
    // the 16-byte chunk of P^T that this lane names to stmatrix (128-byte rows, chunks swizzled by row & 7)
    const int prow = quarter * 16 + (lane & 15);
    const uint32_t pdst = tc::smem_u32(ps) + prow * 128 + (((4 * half + (lane >> 4)) ^ (prow & 7)) << 4);
    const uint64_t scale2 = pack2(scale_log2, scale_log2);
    bool ok = true;
    uint32_t T = 0, done = 0;  // tiles so far, items with tiles so far
    const int splits = gridDim.y, split = blockIdx.y;
    for (uint32_t k = 0;; ++k) {
      Item it;
      ok = ok && take_item(a, sm, k, abort, it);
      // (the warps of a half leave together: whoever stays waits for the others at the barriers below)
      if (bar_any(1 + half, 128, !ok)) {
        ok = false;
        break;
      }
      if (it.qv < 0) break;
      const int nh = min(kH, a.H - it.h0);
      uint64_t nm[4], l[4];  // per pair of heads: minus the reference (of log2 logits), the running sum
      bool fresh = true;     // some of this thread's heads have had no row
#pragma unroll
      for (int c = 0; c < 4; ++c) nm[c] = l[c] = pack2(0.f, 0.f);
      for (int li = 0; li < it.ntiles; ++li, ++T) {
        const int buf = T & 1;
        // (kv_full too: the row flags are the loaders' own writes)
        bool got = wait(&sm->kv_full[buf][0], (T >> 1) & 1, abort, a.status);
        got = got && wait(&sm->s_full[buf], (T >> 1) & 1, abort, a.status);
        got = __all_sync(0xffffffffu, got);
        tc::fence_after_sync();
        const bool validA = sm->valid[buf][rowA], validB = sm->valid[buf][rowB];
        const bool full = __all_sync(0xffffffffu, validA && validB);
        uint32_t v[16];
        tmem_ld_16x256b_x4(tmem + lane_off + kColS + 64 * buf + 32 * half, v);
        tc::tmem_ld_wait();
        // y = logit - reference, in log2 units; rows without a key are -inf. A
        // head's reference moves only when some logit of a tile exceeds it by more
        // than 2^8, and on its first row (it is 0 until then, and not final).
        float2 yA[4], yB[4];
        bool rescale = false;
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            yA[c] = unpack2(fma2(pack2(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1])), scale2, nm[c]));
            yB[c] = unpack2(fma2(pack2(__uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3])), scale2, nm[c]));
          }
          if (!full) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (!validA) yA[c] = make_float2(-INFINITY, -INFINITY);
              if (!validB) yB[c] = make_float2(-INFINITY, -INFINITY);
            }
          }
          if (pass) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) top = fmaxf(fmaxf(top, fmaxf(yA[c].x, yA[c].y)), fmaxf(yB[c].x, yB[c].y));
          if (!bar_any(1 + half, 128, top > kRescaleLog2 || fresh || !(got && ok))) break;
          if (bar_any(1 + half, 128, !(got && ok))) {  // S^T(li) missing, or the previous P.V never completed
            ok = false;
            break;
          }
          // per-head tile maximum: over the thread's two rows, then over the 8
          // lanes of the same cq, then over the 4 warps
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float2 mx = make_float2(fmaxf(yA[c].x, yB[c].x), fmaxf(yA[c].y, yB[c].y));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
              mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
            }
            if (rq == 0) *reinterpret_cast<float2 *>(red + 8 * c + 2 * cq) = mx;
          }
          named_sync(1 + half, 128);
          if (quarter == 0) {
            const int h = 32 * half + lane;
            const float tm = fmaxf(fmaxf(sm->red[0][h], sm->red[1][h]), fmaxf(sm->red[2][h], sm->red[3][h]));
            const float mo = sm->mref[h];
            const bool first = mo == kFloor, up = first ? tm != -INFINITY : tm > kRescaleLog2;
            if (up) sm->mref[h] = first ? tm : mo + tm;
            sm->alpha[h] = up && !first ? ex2_approx(-tm) : 1.f;
            const bool any = __any_sync(0xffffffffu, up && !first);
            if (lane == 0) sm->rescale[half] = any ? 1 : 0;
          }
          named_sync(1 + half, 128);
          rescale = sm->rescale[half] != 0;
          fresh = false;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 m = *reinterpret_cast<const float2 *>(&sm->mref[32 * half + 8 * c + 2 * cq]);
            fresh |= m.x == kFloor || m.y == kFloor;
            nm[c] = pack2(m.x == kFloor ? 0.f : -m.x, m.y == kFloor ? 0.f : -m.y);
            if (rescale) {
              const float2 al = *reinterpret_cast<const float2 *>(&sm->alpha[32 * half + 8 * c + 2 * cq]);
              l[c] = mul2(l[c], pack2(al.x, al.y));
            }
          }
        }
        if (!ok) break;
        // P = 2^y, rounded to bf16 (P.V takes both operands in one type, and V's is
        // bf16; a second product for what the rounding drops would add 768 cycles to
        // a tile's 1,800) and summed per head in fp32. The sums take the same bf16
        // weights as P.V, so that a dominant row's weight (up to 2^8 between rescales)
        // cancels exactly. A weight is off by 2^-8 of it at most, independently of the
        // others: next to the output's own rounding (1.7e-3 of its size, r.m.s.) outputs
        // are off by 1.7e-3 (8,192 rows) to 2.2e-3 (a few rows) in all.
        uint32_t pA[4], pB[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const __nv_bfloat162 ta = __floats2bfloat162_rn(ex2_approx(yA[c].x), ex2_approx(yA[c].y));
          const __nv_bfloat162 tb = __floats2bfloat162_rn(ex2_approx(yB[c].x), ex2_approx(yB[c].y));
          pA[c] = *reinterpret_cast<const uint32_t *>(&ta);
          pB[c] = *reinterpret_cast<const uint32_t *>(&tb);
          l[c] = add2(l[c], pack2(__uint_as_float(pA[c] << 16), __uint_as_float(pA[c] & 0xffff0000u)));
          l[c] = add2(l[c], pack2(__uint_as_float(pB[c] << 16), __uint_as_float(pB[c] & 0xffff0000u)));
        }
        // P.V of the tile before has to be complete before P^T, and where the
        // maximum moved O^T too, are written again.
        if (T > 0) {
          ok = warp_wait(&sm->pv_done[(T - 1) & 3], ((T - 1) >> 2) & 1, abort, a.status);
          tc::fence_after_sync();
        }
        stmatrix_x4(pdst, pA[0], pB[0], pA[1], pB[1]);
        stmatrix_x4(pdst ^ 32, pA[2], pB[2], pA[3], pB[3]);
        if (li > 0 && rescale) {
          if (ok) {
#pragma unroll 1
            for (int m = 0; m < NB; ++m) {  // 16 heads of a 128-dim chunk at a time
              const int h = 32 * half + 16 * (m & 1);
              uint32_t o[16];
              const uint32_t ta = tmem + lane_off + 64 * (m >> 1) + h;
              tmem_ld16(ta, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * sm->alpha[h + c]);
              tmem_st16(ta, o);
            }
            tmem_st_wait();
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::fence_before_sync();
        tc::mbar_arrive(&sm->p_full);
      }
      // Per-head sums, and what the output is multiplied by.
      const int which = it.ntiles > 0 ? done & 1 : 2;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float2 s = unpack2(l[c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
          s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        }
        if (rq == 0) *reinterpret_cast<float2 *>(red + 8 * c + 2 * cq) = s;
      }
      named_sync(1 + half, 128);
      if (quarter == 0) {
        const int h = 32 * half + lane;
        const float ls = (sm->red[0][h] + sm->red[1][h]) + (sm->red[2][h] + sm->red[3][h]);
        const float mr = sm->mref[h];
        if (h < nh) {
          if (splits > 1) {
            reinterpret_cast<float2 *>(a.part_ml)[((size_t)it.qq * a.H + it.h0 + h) * splits + split] = make_float2(mr, ls);
          } else {  // fold in the sink (logit sink[h], value 0) and normalise
            const float sk = a.sink[it.h0 + h] * kLog2e, M = fmaxf(mr, sk), wm = ex2_approx(mr - M);
            const float Ls = ls * wm + ex2_approx(sk - M);
            sm->norm[which][h] = Ls == 0.f ? 0.f : wm / Ls;
          }
        }
        sm->mref[h] = kFloor;  // for the next item, which reads it after a barrier
        if (it.ntiles > 0) tc::mbar_arrive(&sm->norm_full[done & 1]);
      }
      named_sync(1 + half, 128);
      // These warps' half of the output (all of it where the item has no tiles).
      const bool some = it.ntiles > 0;
      if (some) {
        ok = __all_sync(0xffffffffu, ok && wait(&sm->o_done, done & 1, abort, a.status));
        tc::fence_after_sync();
        ++done;
      }
      if (ok)
        write_out<NB>(a, tmem + 32 * half, sm->norm[which] + 32 * half, (size_t)it.qq * a.H + it.h0 + 32 * half, nh - 32 * half, quarter, 0,
                      some ? NB / 2 : NB, some, &sm->o_free);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kPvWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  // the last block returns the counters to zero for the next launch
  if (threadIdx.x == 0 && qvs > (int)gridDim.x && atomicAdd(a.status + 5, 1u) == gridDim.x * gridDim.y - 1) {
    a.status[4] = 0;
    a.status[5] = 0;
  }
}

bool aligned(const void *p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int NB, bool kInt4>
cudaError_t launch_nb(const PagedMqaArgs &a, const CUtensorMap &tm_q, const CUtensorMap &tm_win, int splits, cudaStream_t stream) {
  static DeviceOnce attr;
  once_per_device(attr, [] {
    cudaFuncSetAttribute(paged_mqa_tc_kernel<NB, kInt4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(NB));
  });
  const int groups = (a.H + kH - 1) / kH;
  const long long qvs = (long long)a.Q * groups;
  const int sms = device_sm_count();
  if (qvs > 0x7fffffffLL - sms) return cudaErrorInvalidValue;  // (item numbers pass the last by a grid)
  const long long most = sms / splits > 0 ? sms / splits : 1;
  return launch_pdl(paged_mqa_tc_kernel<NB, kInt4>, dim3((unsigned)(qvs < most ? qvs : most), splits), dim3(kThreads),
                    smem_bytes(NB), stream, tm_q, tm_win, a, (int)qvs, a.scale * kLog2e);
}

}  // namespace

int paged_mqa_tc_splits(int Q, int H, int D, int rows_max) {
  if (D % 128 || D > 512) return 0;
  const int tiles = (rows_max + 2 * kRows - 1) / kRows;  // (the window's padding to whole tiles)
  const long long qv = (long long)Q * ((H + kH - 1) / kH);
  // a block per SM, and no split below two tiles: its partials are as many bytes to write and to merge for half of
  // the work (one query's 130 tiles: 16.7 us with one tile at least, 15.6 with two, 17.9 with three)
  long long s = device_sm_count() / qv;
  if (s > tiles / 2) s = tiles / 2;
  return (int)(s < 1 ? 1 : s > kPagedMaxSplits ? kPagedMaxSplits : s);
}

cudaError_t launch_paged_mqa_tc(const PagedMqaArgs &args, void *partials, cudaStream_t stream, bool *taken) {
  *taken = false;
  PagedMqaArgs a = args;
  const int D = a.cache.D;
  const bool int4 = a.cache.scales != nullptr;
  if (a.dtype != CSA_DTYPE_BF16 || D % 128 || D > 512 || !aligned(a.q, 16) || !aligned(a.kv_win, 16) ||
      !aligned(a.out, 16))
    return cudaSuccess;
  if (!aligned(a.cache.pages, 16) || !aligned(a.cache.scales, 16)) return cudaSuccess;
  CUtensorMap tm_q;
  if (!make_tmap_bf16_3d(&tm_q, a.q, D, a.H, a.Q, 64, kH)) return cudaSuccess;
  CUtensorMap tm_win = tm_q;
  if (a.win_len && !make_tmap_bf16_2d(&tm_win, a.kv_win, D, (uint64_t)a.B * a.T_raw, D * 2, 64, kRows)) return cudaSuccess;
  const int splits = paged_mqa_tc_splits(a.Q, a.H, D, a.rows_max);
  paged_mqa_carve(a, partials, splits);
  *taken = true;
  cudaError_t e = cudaErrorInvalidValue;
  switch (2 * (D / 128) + int4) {
    case 2: e = launch_nb<2, false>(a, tm_q, tm_win, splits, stream); break;
    case 3: e = launch_nb<2, true>(a, tm_q, tm_win, splits, stream); break;
    case 4: e = launch_nb<4, false>(a, tm_q, tm_win, splits, stream); break;
    case 5: e = launch_nb<4, true>(a, tm_q, tm_win, splits, stream); break;
    case 6: e = launch_nb<6, false>(a, tm_q, tm_win, splits, stream); break;
    case 7: e = launch_nb<6, true>(a, tm_q, tm_win, splits, stream); break;
    case 8: e = launch_nb<8, false>(a, tm_q, tm_win, splits, stream); break;
    case 9: e = launch_nb<8, true>(a, tm_q, tm_win, splits, stream); break;
  }
  return e == cudaSuccess && splits > 1 ? launch_paged_merge(a, splits, stream) : e;
}

}  // namespace csa
