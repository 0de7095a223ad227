// Backward pass of range-masked attention on the 5th-generation tensor cores (sm_103a), bf16 inputs.
//
// With x_ij the score (capped, biased by distance; score_fwd.cuh), P = exp(x - LSE), dP = dO V^T, D = dO . O and t the tanh of the
// cap (0 without one):
//   dS = P (dP - D) (1 - t^2),   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO,   over lo_i <= j < hi_i.
//
// Two passes of the plain backward pass's kind (tile_bwd_tc.cu), in one launch: the first CTAs of the grid run dkdv, the others dq,
// each pass persistent over its own units (its own index first, then a counter), decoded by the producer warp and
// published through a two-entry shared-memory ring.  One CTA fills an SM; where both passes together have fewer units than
// there are SMs they run side by side, and otherwise dq's CTAs start as dkdv's end.  Roles, 16 warps:
//   warps 0-7   elementwise: two warps per TMEM lane quadrant, each taking 64 of a block's 128 columns
//   warp 8      MMA issuer, warp 9 producer, warps 10-11 idle
//   warps 12-15 (dq) copy each unit's Q and dO into TMEM, and drain and store dQ
// dkdv (unit = batch, KV head, 128-key block, part): K and V stay in shared memory, the Q and dO blocks of the query blocks
//   that see the key block stream, head of the group after head.  TMEM: S^T | dP^T | dV | dK.
// dq (unit = batch, head, 128-row block, part): Q and dO are copied into TMEM, the K and V blocks that the rows see stream.
//   TMEM: S | dP | dQ | Q | dO.
//
// Masks.  prep_kernel leaves for each 128-row query block the key blocks that it sees and the keys that all of its rows see
// (an elementwise warp masks a block only where it is not inside those), beside D.  A dkdv unit's query blocks are the first to the
// last that see its key block.  In dkdv the columns' ranges travel beside LSE and D through shared memory, clipped to the key
// block, two bytes a column.
// A unit that meets no block is not published: the producer warp writes its zeros.
//
// Bound by the elementwise warps: a block takes dkdv 1.4 us and dq 1.1 (tensor pipe 57 % busy), with a cap 2.3 and 2.1 (39 %).
// Measured, bf16: 8,192 tokens in five documents, 16 heads on 4, d 128, 322 us capped, 233 without a cap; one document 631
// (1,090 TFLOP/s); 2 x 1,000 tokens, 4 heads, d 64, slopes, 23.
//
// D is of O as the forward returned it, in bf16: its rounding reaches every dS of the row, 1e-3 to 2e-3 of the norm of dQ and
// dK, as much as dS's own.  P and dS are rounded to bf16 for their products (2^-8 relative a term at most); sums are fp32; the
// gradients are rounded once. Every mbarrier wait is bounded; a timeout records MESH_ATTN_ERR_DEVICE_TIMEOUT, the CTA stops,
// drains its copies and products and frees its tensor memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "score.cuh"
#include "score_bwd.h"
#include "tmap.h"

namespace mesh {
namespace sbw {

constexpr int BM = 128;  // rows per tile = TMEM lanes = keys / queries per block
constexpr int NUM_THREADS = 512;
constexpr int N_EW = 8;  // elementwise warps: two per TMEM lane quadrant, 64 columns each
constexpr int WARP_MMA = 8;
constexpr int WARP_LOAD = 9;
constexpr int WARP_EPI = 12;
constexpr int N_EPI = 4;
// Register budgets after setmaxnreg, per warpgroup: elementwise (warps 0-7), MMA / producer (8-11),
// epilogue (12-15).  They add up to the 512 x 128 registers of the launch; the launcher checks
// the kernels' register count against that before launching.
constexpr int EW_REGS = 168, MMA_REGS = 104, EPI_REGS = 72;
static_assert(2 * 128 * EW_REGS + 128 * MMA_REGS + 128 * EPI_REGS <= NUM_THREADS * 128, "register split");
// The bf16 P / dS written back into TMEM by column half `hf` land in packed columns
// [64 hf, 64 hf + 32) of their region -- inside the half's own input columns, so the halves never
// overwrite values the other still has to read -- and the MMAs that take them as A read K-step kk
// (16 elements = 8 packed columns) from here:
__device__ __forceinline__ uint32_t packed_col(int kk) { return (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8); }
constexpr int64_t DRAIN_NS = 200000000;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int ROLE_EW = 1, ROLE_MMA = 2, ROLE_LOAD = 3, ROLE_ITEM = 4, ROLE_EPI = 5;

// What prep_kernel leaves of a 128-row query block: the key blocks [kb0, kb1) that its rows see, and the keys [all_lo, all_hi) that
// all of them do.  Where one sees nothing, none are: its weight of 2^(x - inf) is no number when the score x is infinite.
struct alignas(16) Bounds {
  int32_t kb0, kb1, all_lo, all_hi;
};

// Up to so many blocks a row of the batch, prep_kernel also sorts them by length: [masks][nb] query blocks, the longest first, then
// key blocks, and the query blocks [x, y) that see each key block.  Beyond, units are taken as a causal mask wants them: there are
// many more than SMs.
constexpr int ORDER_MAX = 512;

struct Params {
  const float* lse;   // [B, Hq, S]
  const float* dsum;  // [B, Hq, S]
  const Bounds* bounds;  // [B or 1, nb]
  const int32_t* order_q;  // [B or 1, nb], or NULL
  const int32_t* order_kv;
  const int2* seen_by;
  const int32_t* lo;
  const int32_t* hi;
  int64_t mask_bs;
  int32_t bounds_bs;
  const float* slopes;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* dq_part;  // units in parts: [B, Hq, parts, S, D], [B, Hkv, parts, S, D]
  float* dk_part;
  float* dv_part;
  int32_t* status;
  uint32_t* counters;  // of the two passes, 64 apart, zeroed by prep_kernel
  int64_t S;
  int32_t B, Hq, Hkv, g, nb;
  int32_t kv_units, dq_units, kv_ctas, dq_ctas, kv_parts, dq_parts, kv_batch, dq_batch;
  float scale, scale_log2;
  Cap cap;
  int64_t wait_limit_ns;
};

// Shared memory: the resident pair (K, V in dkdv; in dq the landing buffers of Q and dO, which
// the epilogue warps copy into TMEM), NSA stages of stream A (the operand of the S product, which
// the next block's S needs while the current block's dK or dQ still reads it: Q in dkdv, K in
// dq) and NSB stages of stream B (dO in dkdv, V in dq).  226 KB for d = 128 leaves no room to align the base by hand:
// the kernel checks that the dynamic shared window starts 1024-aligned (it does on sm_100-class
// parts, whose window starts at a 1 KB-aligned offset) and reports MESH_ATTN_ERR_INTERNAL if not.
template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // one 128-row bf16 block
  static constexpr uint32_t BOX = BM * 64 * 2;  // one 128 x 64 TMA box
  static constexpr int NSA = 3, NSB = 2;
  static constexpr uint32_t RES0 = 0, RES1 = TILE;
  static constexpr uint32_t A0 = 2 * TILE;             // stream A stage s at A0 + s TILE
  static constexpr uint32_t B0 = A0 + NSA * TILE;      // stream B stage s at B0 + s TILE
  static constexpr uint32_t VEC_OFF = B0 + NSB * TILE;  // dkdv: -LSE (base 2) [2][128], -D [2][128] fp32, ranges [2][128] 2 bytes
  static constexpr uint32_t BAR_OFF = VEC_OFF + 4 * BM * 4 + 2 * BM * 2;
  static constexpr int B_RES = 0, B_AF = 1, B_AE = B_AF + NSA, B_BF = B_AE + NSA, B_BE = B_BF + NSB,
                       B_S = B_BE + NSB, B_DP = B_S + 1, B_P = B_DP + 1, B_DS = B_P + 1, B_ACC = B_DS + 1,
                       B_DRAIN = B_ACC + 1, B_VEC = B_DRAIN + 1, B_RESE = B_VEC + 2, B_ACCE = B_RESE + 1,
                       B_UF = B_ACCE + 1, B_UE = B_UF + 2, B_ACC2 = B_UE + 2, B_ACCE2 = B_ACC2 + 1,
                       B_SREAD = B_ACCE2 + 1, B_QTF = B_SREAD + 1, B_QTE = B_QTF + 1, NBARS = B_QTE + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBARS * 8;  // tmem base, abort flag
  static constexpr uint32_t RING_OFF = MISC_OFF + 8;         // unit ring: 2 decoded units, 8 ints each
  static constexpr uint32_t TOTAL = RING_OFF + 2 * 32;
};
static_assert(Layout<128>::TOTAL <= 232448, "shared memory of a CTA");

__device__ __forceinline__ float4 shfl4(float4 x, int src) {
  x.x = __shfl_sync(0xffffffffu, x.x, src);
  x.y = __shfl_sync(0xffffffffu, x.y, src);
  x.z = __shfl_sync(0xffffffffu, x.z, src);
  x.w = __shfl_sync(0xffffffffu, x.w, src);
  return x;
}

// Store one warp's 32 x 32 fp32 chunk -- lane r holds columns [c, c + 32) of row row0 + r, times
// `mul` -- into a row-major [rows][D] buffer.  Each group of four lanes transposes its 4 x 4
// matrix of 16-byte pieces (two exchange steps: lanes ^ 2, then lanes ^ 1), after which lane
// 4a + i holds piece i of rows 4a .. 4a + 3; so each store instruction writes eight 64-byte row
// segments (whole sectors) instead of 32 scattered 16-byte pieces, without shared memory.  Rows
// from `rows_valid` on are not written.
template <int D>
__device__ __forceinline__ void store_rows(const float (&v)[32], float mul, float* dst, int64_t row0,
                                           int rows_valid, int c, int lane) {
  const int i = lane & 3, rbase = lane & ~3;
  const bool hi = (i & 2) != 0, odd = (i & 1) != 0;
#pragma unroll
  for (int blk = 0; blk < 2; ++blk) {
    float4 e[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = 16 * blk + 4 * q;
      e[q] = make_float4(v[o] * mul, v[o + 1] * mul, v[o + 2] * mul, v[o + 3] * mul);
    }
    {  // swap the off-diagonal 2 x 2 blocks with lane ^ 2
      const float4 r0 = shfl4(hi ? e[0] : e[2], lane ^ 2), r1 = shfl4(hi ? e[1] : e[3], lane ^ 2);
      if (hi) {
        e[0] = r0;
        e[1] = r1;
      } else {
        e[2] = r0;
        e[3] = r1;
      }
    }
    {  // swap within the 2 x 2 blocks with lane ^ 1
      const float4 r0 = shfl4(odd ? e[0] : e[1], lane ^ 1), r1 = shfl4(odd ? e[2] : e[3], lane ^ 1);
      if (odd) {
        e[0] = r0;
        e[2] = r1;
      } else {
        e[1] = r0;
        e[3] = r1;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (rbase + j < rows_valid)
        *reinterpret_cast<float4*>(dst + (row0 + rbase + j) * D + c + 16 * blk + 4 * i) = e[j];
  }
}

// 32 columns of this lane's row, times mul, rounded to bf16: 64 bytes in a row of their own.
__device__ __forceinline__ void store_bf16(const float* v, float mul, __nv_bfloat16* dst) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(dst + 8 * q) =
        make_uint4(pack_bf16x2(v[8 * q] * mul, v[8 * q + 1] * mul), pack_bf16x2(v[8 * q + 2] * mul, v[8 * q + 3] * mul),
                   pack_bf16x2(v[8 * q + 4] * mul, v[8 * q + 5] * mul), pack_bf16x2(v[8 * q + 6] * mul, v[8 * q + 7] * mul));
}

// Descriptor offsets (16-byte units) of a 128-row operand made of 64-column SW128 boxes.
template <int D>
__device__ __forceinline__ uint64_t kmaj_off(int kk) {
  return (uint64_t)((kk >> 2) * (Layout<D>::BOX >> 4) + (kk & 3) * 2);
}

// A unit of either pass: 128-row block `blk` of a (KV) head, part `part` of its streamed blocks: of `per` blocks a head from
// `first` on (dkdv: query blocks, the heads of the group one after another; dq: key blocks, one head), those from
// `start` on, NB of them.
struct Unit {
  int u, blk, h, b, part, first, per, start, NB;
};
__device__ __forceinline__ void put_unit(volatile int32_t* e, const Unit& x) {
  e[0] = x.u;
  e[1] = x.blk, e[2] = x.h, e[3] = x.b | x.part << 16, e[4] = x.first, e[5] = x.per, e[6] = x.start, e[7] = x.NB;
}
__device__ __forceinline__ void get_unit(const volatile int32_t* e, Unit& x) {
  x.u = e[0], x.blk = e[1], x.h = e[2], x.first = e[4], x.per = e[5], x.start = e[6], x.NB = e[7];
  x.b = e[3] & 0xffff, x.part = e[3] >> 16;
}
// Decoded by a whole warp.  Units are numbered batch of (batch, head) lanes by batch, within it block by block, the longest
// first, within those lane by lane, its parts together.
template <bool KV>
__device__ __forceinline__ Unit unit_of(int u, const Params& prm) {
  const int lane = threadIdx.x & 31;
  const int H = KV ? prm.Hkv : prm.Hq, parts = KV ? prm.kv_parts : prm.dq_parts, batch = KV ? prm.kv_batch : prm.dq_batch;
  Unit x;
  x.u = u;
  x.part = u % parts;
  int t = u / parts;
  const int per = batch * prm.nb, first = t / per * batch;
  const int lanes = min(batch, prm.B * H - first);  // the last batch may be smaller
  t %= per;
  const int idx = t / lanes;
  t = first + t % lanes;
  x.h = t % H;
  x.b = t / H;
  const int64_t mask = (int64_t)x.b * prm.bounds_bs;
  int lo = 0x7fffffff, hi = 0;
  if (prm.order_q) {
    x.blk = (KV ? prm.order_kv : prm.order_q)[mask + idx];
  } else {
    x.blk = KV ? idx : prm.nb - 1 - idx;
  }
  if (!KV) {
    lo = prm.bounds[mask + x.blk].kb0;
    hi = prm.bounds[mask + x.blk].kb1;
  } else if (prm.order_q) {
    lo = prm.seen_by[mask + x.blk].x;
    hi = prm.seen_by[mask + x.blk].y;
  } else {  // the query blocks from the first to the last that see key block blk
    const Bounds* bd = prm.bounds + mask;
    for (int q = lane; q < prm.nb; q += 32)
      if (bd[q].kb0 <= x.blk && x.blk < bd[q].kb1) {
        lo = min(lo, q);
        hi = q + 1;
      }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
  }
  x.first = lo < hi ? lo : 0;
  x.per = lo < hi ? hi - lo : 0;
  const int n = x.per * (KV ? prm.g : 1), k = max(1, min(parts, n));
  x.start = (int)((int64_t)min(x.part, k) * n / k);
  x.NB = (int)((int64_t)min(x.part + 1, k) * n / k) - x.start;
  return x;
}

// Streamed blocks of a unit: head within the group (dkdv), block.
struct Cursor {
  int h, blk, first, end;
  __device__ __forceinline__ void start(const Unit& x) {
    first = x.first;
    end = x.first + x.per;
    h = x.per > 0 ? x.start / x.per : 0;
    blk = first + x.start - h * x.per;
  }
  __device__ __forceinline__ void step() {
    if (++blk < end) return;
    blk = first;
    ++h;
  }
};

// A row's bound as the nearest that there is: it may be any 32-bit number, from which a block's first key or another bound could not
// be taken.
__device__ __forceinline__ int clip(int bound, int64_t S) { return min(max(bound, 0), (int)S); }

// 64 scores of consecutive columns to weights, MODE 0 plain, 1 slopes, 2 cap (and slopes where given); `reload` fetches the scores
// again for a higher tier of the cap:
//   P = 2^(x + nl(c)), nl(c) being -LSE in base 2 of columns c and c + 1, and |i - j| = |c + off|.
// Leaves P (1 - t^2) in s and, with PACK, P in bf16 pairs in pk.
template <int MODE, bool PACK, typename F, typename L>
__device__ __forceinline__ void weights(const Params& prm, float (&s)[64], uint32_t* pk, float slope2, int off, int& tier, F&& nl,
                                        L&& reload) {
  const uint64_t sc2 = f2_pack(prm.scale_log2, prm.scale_log2);
  const bool slopes = MODE == 1 || (MODE == 2 && prm.slopes);
  const float o = (float)off;
  // -slope |i - j| of columns c, c + 1 on top of -LSE
  auto base = [&](int c) -> uint64_t {
    uint64_t n = nl(c);
    if (MODE >= 1 && slopes) {
      float n0, n1;
      f2_unpack(n, n0, n1);
      n = f2_pack(fmaf(-slope2, fabsf(o + (float)c), n0), fmaf(-slope2, fabsf(o + (float)(c + 1)), n1));
    }
    return n;
  };
  if (MODE < 2) {
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sc2, base(c)), x0, x1);
      s[c] = fast_exp2(x0);
      s[c + 1] = fast_exp2(x1);
      if (PACK) pk[c / 2] = pack_bf16x2(s[c], s[c + 1]);
    }
    return;
  }
  cap_scores(prm.cap, s, tier, true, reload);
  const uint64_t i2 = f2_pack(-prm.cap.inv2, -prm.cap.inv2), one = f2_pack(1.f, 1.f);
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    const uint64_t y = f2_pack(s[c], s[c + 1]);
    float x0, x1;
    f2_unpack(f2_add(y, base(c)), x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    if (PACK) pk[c / 2] = pack_bf16x2(p0, p1);
    f2_unpack(f2_mul(f2_pack(p0, p1), f2_fma(f2_mul(y, y), i2, one)), s[c], s[c + 1]);  // t = y / (cap log2 e)
  }
}

// What both passes share: barrier set-up, the unit ring and the exit.
template <int D, int MODE, bool KV>
__device__ __forceinline__ void run_pass(const CUtensorMap& tmR0, const CUtensorMap& tmR1, const CUtensorMap& tmA,
                                         const CUtensorMap& tmB, const Params& prm, int cta, int n_ctas) {
  // R0, R1: the resident blocks' tensors (dkdv: K, V; dq: Q, dO); A, B: the streamed ones (Q, dO; K, V)
  using Ly = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {  // 128-byte swizzle atoms need 1024-aligned operands (see Layout)
    if (threadIdx.x == 0) record_error(prm.status, MESH_ATTN_ERR_INTERNAL, ROLE_ITEM, (int32_t)blockIdx.x);
    return;
  }
  uint8_t* smem = smem_raw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + Ly::BAR_OFF + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::MISC_OFF);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC_OFF + 4);
  volatile int32_t* ring = reinterpret_cast<volatile int32_t*>(smem + Ly::RING_OFF);
  const int64_t S = prm.S;

  if (threadIdx.x == 0) {
    mbar_init(bar(Ly::B_RES), 1);
    mbar_init(bar(Ly::B_RESE), KV ? 1 : N_EPI);  // dq: the epilogue warps have copied Q and dO into TMEM
    for (int s = 0; s < Ly::NSA; ++s) {
      mbar_init(bar(Ly::B_AF + s), 1);
      mbar_init(bar(Ly::B_AE + s), 1);
    }
    for (int s = 0; s < Ly::NSB; ++s) {
      mbar_init(bar(Ly::B_BF + s), 1);
      mbar_init(bar(Ly::B_BE + s), 1);
    }
    mbar_init(bar(Ly::B_S), 1);
    mbar_init(bar(Ly::B_SREAD), N_EW);  // dq: S has been loaded by every elementwise warp
    mbar_init(bar(Ly::B_DP), 1);
    mbar_init(bar(Ly::B_P), N_EW);  // one lane of each elementwise warp
    mbar_init(bar(Ly::B_DS), N_EW);
    mbar_init(bar(Ly::B_ACC), 1);
    mbar_init(bar(Ly::B_ACCE), KV ? N_EW : N_EPI);
    mbar_init(bar(Ly::B_ACC2), 1);
    mbar_init(bar(Ly::B_ACCE2), N_EW);
    mbar_init(bar(Ly::B_DRAIN), 1);
    mbar_init(bar(Ly::B_VEC), BM);  // every thread of the first column half has written its column's values
    mbar_init(bar(Ly::B_VEC + 1), BM);
    mbar_init(bar(Ly::B_QTF), N_EPI);  // dq: Q and dO of the unit are in TMEM
    mbar_init(bar(Ly::B_QTE), 1);      // dq: the unit's last S and dP products are done with them
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Ly::B_UF + s), 1);
      mbar_init(bar(Ly::B_UE + s), N_EW + 1 + (KV ? 0 : N_EPI));  // the warps that read a unit
    }
    wait_for_kernel_before();
    // without any time to wait there is nothing to start: the first load would be waited for
    if (prm.wait_limit_ns <= 0) record_error(prm.status, MESH_ATTN_ERR_DEVICE_TIMEOUT, ROLE_LOAD, -1);
    *abort_flag = (*reinterpret_cast<volatile int32_t*>(prm.status) != 0) ? 1 : 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  wait_for_kernel_before();  // and before tensor memory is taken, which that kernel may still want
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == WARP_LOAD && lane == 0) {
    tma_prefetch_desc(&tmR0);
    tma_prefetch_desc(&tmR1);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = *abort_flag == 0;

  // the next unit from the ring (every lane of the warp waits, one lane frees the slot)
  int nu = 0;
  auto take = [&](Unit& y, int role) -> bool {
    const int slot = nu & 1;
    const bool r = mbar_wait_warp(bar(Ly::B_UF + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status, role, -1);
    if (!r) return false;
    get_unit(ring + 8 * slot, y);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Ly::B_UE + slot));
    ++nu;
    return true;
  };
  auto wait_all = [&](int b, uint32_t parity, int role, int unit) -> bool {  // warp-uniform
    const bool r = mbar_wait(bar(b), parity, prm.wait_limit_ns, abort_flag, prm.status, role, unit);
    return __all_sync(0xffffffffu, r);
  };
  auto arrive = [&](int b) {  // after this warp's TMEM accesses
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };

  if (warp < N_EW) {
    // ================================================================ elementwise
    regs_inc<EW_REGS>();
    const int wq = warp & 3, hf = warp >> 2;  // TMEM lane quadrant, column half
    const int row = wq * 32 + lane;           // TMEM lane: a key row (dkdv) or a query row (dq) of the block
    const int c_base = hf * 64;               // this warp's columns [c_base, c_base + 64)
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tm_s = tmem + lane_base + (uint32_t)c_base;         // S, then P (bf16) in dkdv
    const uint32_t tm_dp = tmem + lane_base + 128u + (uint32_t)c_base;  // dP, then dS (bf16)
    bool ok = run;
    Unit x;
    x.u = -1;
    if (ok) ok = take(x, ROLE_EW);
    int64_t g0 = 0;  // global index of the unit's first block
    int k_unit = 0;
    int tier = 0;  // of the cap
    if constexpr (KV) {
      // ---------------------------------------------------------------- dK and dV
      float* nlse_s = reinterpret_cast<float*>(smem + Ly::VEC_OFF);  // [2][BM] -LSE log2 e of the query columns
      float* ndsum_s = nlse_s + 2 * BM;                              // [2][BM] -D
      uint16_t* rng_s = reinterpret_cast<uint16_t*>(ndsum_s + 2 * BM);  // [2][BM] first key row | keys << 8
      // What query column `row` of the next block is, loaded raw one block ahead by the first column half and only used (scaled,
      // published) at the top of the next iteration, so that the loads never stall the block in flight; across
      // units, the next unit's first block is loaded before this unit's epilogue.  Beside it the keys that all rows
      // of the query block see, and the head's slope.
      float raw_lse = 0.f, raw_d = 0.f, raw_slope = 0.f;
      int raw_lo = 0, raw_hi = 0, raw_all_lo = 0, raw_all_hi = 0;
      bool raw_in = false;
      auto fetch = [&](const Unit& y, const Cursor& c) {
        const int64_t ql = (int64_t)c.blk * BM + row;
        const int h = y.h * prm.g + c.h;
        const Bounds* bd = prm.bounds + (int64_t)y.b * prm.bounds_bs + c.blk;
        raw_all_lo = bd->all_lo;
        raw_all_hi = bd->all_hi;
        if (MODE >= 1 && prm.slopes) raw_slope = prm.slopes[h] * LOG2E;
        raw_in = ql < S;
        if (hf == 0 && raw_in) {
          const int64_t at = ((int64_t)y.b * prm.Hq + h) * S + ql;
          raw_lse = prm.lse[at];
          raw_d = prm.dsum[at];
          raw_lo = prm.lo[y.b * prm.mask_bs + ql];
          raw_hi = prm.hi[y.b * prm.mask_bs + ql];
        }
      };
      Cursor cur, nxt;
      if (ok && x.u >= 0) {
        cur.start(x);
        fetch(x, cur);
      }
      while (ok && x.u >= 0) {
        const int kb = x.blk, NB = x.NB, k0 = kb * BM;
        nxt = cur;
        for (int i = 0; i < NB && ok; ++i) {
          const int64_t gi = g0 + i;
          const int vb = (int)(gi & 1);
          if (i > 0) cur = nxt;
          if (i + 1 < NB) nxt.step();
          // publish this column's values, then wait (bounded) until all 128 columns are written; a
          // buffer is rewritten two blocks later, after every writer has arrived for the block between
          const bool edge = raw_all_lo > k0 || raw_all_hi < k0 + BM;
          const float slope2 = raw_slope;
          if (hf == 0) {
            // no such query row: exp2(0 - inf) = 0, so it needs no mask
            nlse_s[vb * BM + row] = raw_in && raw_lse != -INFINITY ? -raw_lse * LOG2E : -INFINITY;
            ndsum_s[vb * BM + row] = raw_in ? -raw_d : 0.f;
            const int a = min(max(clip(raw_lo, S) - k0, 0), BM), z = min(max(clip(raw_hi, S) - k0, a), BM);
            rng_s[vb * BM + row] = (uint16_t)(a | (z - a) << 8);
            mbar_arrive(bar(Ly::B_VEC + vb));
          }
          const int qb = cur.blk;
          if (i + 1 < NB) fetch(x, nxt);
          ok = wait_all(Ly::B_VEC + vb, (uint32_t)((gi >> 1) & 1), ROLE_EW, i);
          if (!ok) break;
          ok = wait_all(Ly::B_S, (uint32_t)(gi & 1), ROLE_EW, i);
          if (!ok) break;
          tc_fence_after();
          float pv[64];
          auto load_s = [&]() {
            tmem_ld32(tm_s, pv);
            tmem_ld32(tm_s + 32u, pv + 32);
            tc_wait_ld();
          };
          load_s();
          const float* lv = nlse_s + vb * BM + c_base;
          uint32_t pk[32];
          weights<MODE, true>(
              prm, pv, pk, slope2, qb * BM + c_base - (k0 + row), tier,
              [&](int c) {
                const float2 l2 = *reinterpret_cast<const float2*>(lv + c);
                return f2_pack(l2.x, l2.y);
              },
              load_s);
          if (edge) {
            asm volatile("" ::: "memory");  // a branch, not selects that every block would run
            const uint4* rv = reinterpret_cast<const uint4*>(rng_s + vb * BM + c_base);
            // all columns may have one range, as behind a document's start: this thread's key then counts or is dropped as a whole
            const uint32_t one = (rv[0].x & 0xffffu) * 0x10001u;
            uint32_t differ = 0u;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 r4 = rv[c];
              differ |= (r4.x ^ one) | (r4.y ^ one) | (r4.z ^ one) | (r4.w ^ one);
            }
            if (differ == 0u) {
              asm volatile("" ::: "memory");
              const bool in = (uint32_t)(row - (int)(one & 255u)) < (one >> 24);
#pragma unroll
              for (int c = 0; c < 32; ++c) pk[c] = in ? pk[c] : 0u;
#pragma unroll
              for (int c = 0; c < 64; ++c) pv[c] = in ? pv[c] : 0.f;
            } else {
#pragma unroll
              for (int c = 0; c < 64; c += 8) {
                const uint4 r4 = rv[c / 8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t r2 = e == 0 ? r4.x : e == 1 ? r4.y : e == 2 ? r4.z : r4.w;
                  const bool in0 = (uint32_t)(row - (int)(r2 & 255u)) < ((r2 >> 8) & 255u);
                  const bool in1 = (uint32_t)(row - (int)((r2 >> 16) & 255u)) < (r2 >> 24);
                  pk[c / 2 + e] &= (in0 ? 0xffffu : 0u) | (in1 ? 0xffff0000u : 0u);
                  if (!in0) pv[c + 2 * e] = 0.f;
                  if (!in1) pv[c + 2 * e + 1] = 0.f;
                }
              }
            }
          }
          tmem_st32(tm_s, pk);  // P^T columns of this half (see packed_col)
          tc_wait_st();
          arrive(Ly::B_P);
          ok = wait_all(Ly::B_DP, (uint32_t)(gi & 1), ROLE_EW, i);
          if (!ok) break;
          tc_fence_after();
          {
            float dp[64];
            tmem_ld32(tm_dp, dp);
            tmem_ld32(tm_dp + 32u, dp + 32);
            tc_wait_ld();
            const float4* dv_ = reinterpret_cast<const float4*>(ndsum_s + vb * BM + c_base);
            uint32_t ds2[32];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const float4 d4 = dv_[c / 4];
              float a0, a1, a2, a3;
              f2_unpack(f2_mul(f2_add(f2_pack(dp[c], dp[c + 1]), f2_pack(d4.x, d4.y)), f2_pack(pv[c], pv[c + 1])), a0, a1);
              f2_unpack(f2_mul(f2_add(f2_pack(dp[c + 2], dp[c + 3]), f2_pack(d4.z, d4.w)), f2_pack(pv[c + 2], pv[c + 3])), a2, a3);
              ds2[c / 2] = pack_bf16x2(a0, a1);
              ds2[c / 2 + 1] = pack_bf16x2(a2, a3);
            }
            tmem_st32(tm_dp, ds2);  // dS^T columns of this half
          }
          tc_wait_st();
          arrive(Ly::B_DS);
        }
        if (!ok) break;
        // the next unit, and its first block's values, before this unit's epilogue
        Unit xn;
        ok = take(xn, ROLE_EW);
        if (!ok) break;
        if (xn.u >= 0) {
          cur.start(xn);
          fetch(xn, cur);
        }
        // ---- epilogue: this half's columns of the dV and dK rows of this key block, at the unit boundary where the tensor
        // pipe has little else to do
        ok = wait_all(Ly::B_ACC2, (uint32_t)(k_unit & 1), ROLE_EW, -1);  // dK's last product, and so dV's, has completed
        if (!ok) break;
        tc_fence_after();
        {
          const uint32_t tm_dv = tmem + lane_base + 256u + (uint32_t)(hf * (D / 2));
          const int64_t rl = (int64_t)k0 + row;
          float acc[D / 2];
#pragma unroll
          for (int which = 0; which < 2; ++which) {  // dV, then dK
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) tmem_ld32(tm_dv + (uint32_t)(which * D + c), acc + c);
            tc_wait_ld();
            if (which) {  // both accumulators are copied out: the next unit may overwrite them
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(bar(Ly::B_ACCE));
                mbar_arrive(bar(Ly::B_ACCE2));
              }
            }
            const float mul = which ? prm.scale : 1.f;
            if (prm.kv_parts > 1) {
              const int64_t row0 = (((int64_t)x.b * prm.Hkv + x.h) * prm.kv_parts + x.part) * S + k0 + wq * 32;
              const int rows_valid = (int)max((int64_t)0, min((int64_t)32, S - (k0 + wq * 32)));
#pragma unroll
              for (int c = 0; c < D / 2; c += 32)
                store_rows<D>(*reinterpret_cast<const float(*)[32]>(acc + c), mul, which ? prm.dk_part : prm.dv_part, row0,
                              rows_valid, hf * (D / 2) + c, lane);
            } else if (rl < S) {
              __nv_bfloat16* dst = (which ? prm.dk : prm.dv) + (((int64_t)x.b * prm.Hkv + x.h) * S + rl) * D + hf * (D / 2);
#pragma unroll
              for (int c = 0; c < D / 2; c += 32) store_bf16(acc + c, mul, dst + c);
            }
          }
        }
        ++k_unit;
        tier = 0;
        g0 += NB;
        x = xn;
      }
    } else {
      // ---------------------------------------------------------------- dQ
      // this thread's row, loaded as soon as the unit is known and used a phase later
      float raw_lse = 0.f, raw_d = 0.f, raw_slope = 0.f;
      int raw_lo = 0, raw_hi = 0, raw_all_lo = 0, raw_all_hi = 0;
      bool row_in = false;
      auto fetch = [&](const Unit& y) {
        const int64_t ql = (int64_t)y.blk * BM + row;
        const Bounds* bd = prm.bounds + (int64_t)y.b * prm.bounds_bs + y.blk;
        raw_all_lo = bd->all_lo;
        raw_all_hi = bd->all_hi;
        if (MODE >= 1 && prm.slopes) raw_slope = prm.slopes[y.h] * LOG2E;
        row_in = ql < S;
        if (row_in) {
          const int64_t at = ((int64_t)y.b * prm.Hq + y.h) * S + ql;
          raw_lse = prm.lse[at];
          raw_d = prm.dsum[at];
          raw_lo = prm.lo[y.b * prm.mask_bs + ql];
          raw_hi = prm.hi[y.b * prm.mask_bs + ql];
        }
      };
      if (ok && x.u >= 0) fetch(x);
      while (ok && x.u >= 0) {
        // a row that is not there, or sees nothing: weights of 0
        const float nlse = row_in && raw_lse != -INFINITY ? -raw_lse * LOG2E : -INFINITY;
        const float dsum = row_in ? raw_d : 0.f, slope2 = raw_slope;
        const int lo = clip(raw_lo, S), hi = clip(raw_hi, S), all_lo = raw_all_lo, all_hi = raw_all_hi;
        const int q = x.blk * BM + row;
        const uint64_t nl2 = f2_pack(nlse, nlse), nd2 = f2_pack(-dsum, -dsum);
        for (int j = 0; j < x.NB && ok; ++j) {
          const int64_t gi = g0 + j;
          const int k0 = (x.first + x.start + j) * BM;
          ok = wait_all(Ly::B_S, (uint32_t)(gi & 1), ROLE_EW, j);
          if (!ok) break;
          tc_fence_after();
          float pv[64];
          auto load_s = [&]() {
            tmem_ld32(tm_s, pv);
            tmem_ld32(tm_s + 32u, pv + 32);
            tc_wait_ld();
          };
          load_s();
          if (MODE < 2) arrive(Ly::B_SREAD);  // S(g) is in registers: the next block's S may overwrite it
          weights<MODE, false>(prm, pv, nullptr, slope2, k0 + c_base - q, tier, [&](int) { return nl2; }, load_s);
          // with a cap it may be read again until here (picking the tier by the scores' maximum first instead: 10 % slower)
          if (MODE == 2) arrive(Ly::B_SREAD);
          if (all_lo > k0 || all_hi < k0 + BM) {
            asm volatile("" ::: "memory");
            const int a = lo - k0 - c_base, n = max(hi - lo, 0);
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if ((uint32_t)(c - a) >= (uint32_t)n) pv[c] = 0.f;
          }
          ok = wait_all(Ly::B_DP, (uint32_t)(gi & 1), ROLE_EW, j);
          if (!ok) break;
          tc_fence_after();
          {
            float dp[64];
            tmem_ld32(tm_dp, dp);
            tmem_ld32(tm_dp + 32u, dp + 32);
            tc_wait_ld();
            uint32_t ds2[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float a0, a1;
              f2_unpack(f2_mul(f2_add(f2_pack(dp[c], dp[c + 1]), nd2), f2_pack(pv[c], pv[c + 1])), a0, a1);
              ds2[c / 2] = pack_bf16x2(a0, a1);
            }
            tmem_st32(tm_dp, ds2);  // dS columns of this half (see packed_col)
          }
          tc_wait_st();
          arrive(Ly::B_DS);
        }
        if (!ok) break;
        // the next unit, and its row's values (the epilogue warps drain this one)
        Unit xn;
        ok = take(xn, ROLE_EW);
        if (!ok) break;
        if (xn.u >= 0) fetch(xn);
        tier = 0;
        g0 += x.NB;
        x = xn;
      }
    }
  } else if (warp < WARP_EPI) {
    regs_dec<MMA_REGS>();
    if (warp == WARP_MMA) {
      // ================================================================ MMA issuer
      constexpr uint32_t idesc_sk = idesc_bf16_f32(BM, BM, false);  // S, dP: K-major A and B
      constexpr uint32_t idesc_ts = idesc_bf16_f32(BM, D, true);    // dV, dK, dQ: B MN-major
      constexpr uint64_t TILE16 = Ly::TILE >> 4;
      const uint64_t r0_desc = smem_desc_sw128(sb + Ly::RES0, 16u, 1024u);
      const uint64_t r1_desc = smem_desc_sw128(sb + Ly::RES1, 16u, 1024u);
      const uint64_t a_kmaj = smem_desc_sw128(sb + Ly::A0, 16u, 1024u);
      const uint64_t a_mn = smem_desc_sw128(sb + Ly::A0, Ly::BOX, 1024u);
      const uint64_t b_kmaj = smem_desc_sw128(sb + Ly::B0, 16u, 1024u);
      const uint64_t b_mn = smem_desc_sw128(sb + Ly::B0, Ly::BOX, 1024u);
      const uint32_t tm_qt = tmem + 384u, tm_gt = tmem + 384u + (uint32_t)(D / 2);  // dq: Q and dO (bf16)
      auto issue_s = [&](int64_t gi) {  // dkdv: S^T = K Q(gi)^T; dq: S = Q K(gi)^T
        const uint64_t ad = a_kmaj + (uint64_t)(gi % Ly::NSA) * TILE16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (KV) tc_mma_ss_warp(tmem, r0_desc + kmaj_off<D>(kk), ad + kmaj_off<D>(kk), idesc_sk, kk > 0);
          else tc_mma_ts_warp(tmem, tm_qt + (uint32_t)(kk * 8), ad + kmaj_off<D>(kk), idesc_sk, kk > 0 ? 1u : 0u);
        }
        tc_commit_warp(bar(Ly::B_S));
      };
      auto issue_dp = [&](int64_t gi) {  // dkdv: dP^T = V dO(gi)^T; dq: dP = dO V(gi)^T, V(gi)'s only reader
        const int s = (int)(gi % Ly::NSB);
        const uint64_t bd = b_kmaj + (uint64_t)s * TILE16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (KV) tc_mma_ss_warp(tmem + 128u, r1_desc + kmaj_off<D>(kk), bd + kmaj_off<D>(kk), idesc_sk, kk > 0);
          else tc_mma_ts_warp(tmem + 128u, tm_gt + (uint32_t)(kk * 8), bd + kmaj_off<D>(kk), idesc_sk, kk > 0 ? 1u : 0u);
        }
        tc_commit_warp(bar(Ly::B_DP));
        if (!KV) tc_commit_warp(bar(Ly::B_BE + s));
      };
      auto issue_dv = [&](int64_t gi, bool first) {  // dV += P^T dO(gi)
        const int s = (int)(gi % Ly::NSB);
        const uint64_t gd = b_mn + (uint64_t)s * TILE16;
#pragma unroll
        for (int kk = 0; kk < BM / 16; ++kk)
          tc_mma_ts_warp(tmem + 256u, tmem + packed_col(kk), gd + (uint64_t)(kk * 128), idesc_ts, (!first || kk > 0) ? 1u : 0u);
        tc_commit_warp(bar(Ly::B_BE + s));  // dO(gi): read by dP^T(gi) and dV(gi)
      };
      auto issue_acc = [&](int64_t gi, bool first) {  // dkdv: dK += dS^T Q(gi); dq: dQ += dS K(gi)
        const int s = (int)(gi % Ly::NSA);
        const uint64_t ad = a_mn + (uint64_t)s * TILE16;
#pragma unroll
        for (int kk = 0; kk < BM / 16; ++kk)
          tc_mma_ts_warp(tmem + 256u + (KV ? (uint32_t)D : 0u), tmem + 128u + packed_col(kk), ad + (uint64_t)(kk * 128), idesc_ts,
                         (!first || kk > 0) ? 1u : 0u);
        tc_commit_warp(bar(Ly::B_AE + s));  // read by S(gi) and this
      };
      auto wait = [&](int b, uint32_t parity, int64_t g) {
        return mbar_wait_warp(bar(b), parity, prm.wait_limit_ns, abort_flag, prm.status, ROLE_MMA, (int32_t)g);
      };
      auto wait_a = [&](int64_t g) { return wait(Ly::B_AF + (int)(g % Ly::NSA), (uint32_t)((g / Ly::NSA) & 1), g); };
      auto wait_b = [&](int64_t g) { return wait(Ly::B_BF + (int)(g % Ly::NSB), (uint32_t)((g / Ly::NSB) & 1), g); };
      int nres = 0;
      // S(0) and dP(0) of a unit whose first block is g, as soon as its resident blocks are there (dq: in TMEM); for
      // every unit but the first, after the previous unit's last dK or dQ
      auto start_unit = [&](const Unit& y, int64_t g) -> bool {
        if (!wait(KV ? Ly::B_RES : Ly::B_QTF, (uint32_t)(nres & 1), -1)) return false;
        ++nres;
        if (!wait_a(g)) return false;
        tc_fence_after();
        issue_s(g);
        if (!wait_b(g)) return false;
        tc_fence_after();
        issue_dp(g);
        if (y.NB == 1) tc_commit_warp(bar(KV ? Ly::B_RESE : Ly::B_QTE));  // the unit's last S and dP are issued
        return true;
      };
      bool ok = run;
      Unit x;
      x.u = -1;
      if (ok) ok = take(x, ROLE_MMA);
      if (ok && x.u >= 0) ok = start_unit(x, 0);
      int64_t g0 = 0;
      int k_unit = 0;
      while (ok && x.u >= 0) {
        const int NB = x.NB;
        for (int i = 0; i < NB && ok; ++i) {
          const int64_t gi = g0 + i;
          if (KV) {
            ok = wait(Ly::B_P, (uint32_t)(gi & 1), i);
            if (!ok) break;
            if (i == 0 && k_unit > 0) {  // the previous unit's dV has been copied out of TMEM
              ok = wait(Ly::B_ACCE, (uint32_t)((k_unit - 1) & 1), -1);
              if (!ok) break;
            }
            tc_fence_after();
            issue_dv(gi, i == 0);
            if (i + 1 < NB) {
              ok = wait_a(gi + 1);
              if (!ok) break;
              tc_fence_after();
              issue_s(gi + 1);
            }
          } else if (i + 1 < NB) {
            // S(gi) has been read into registers: S(gi + 1) may overwrite it.  (The next block's S is
            // issued only after this wait, so the barrier cannot run a phase ahead of it.)
            ok = wait(Ly::B_SREAD, (uint32_t)(gi & 1), i);
            if (ok) ok = wait_a(gi + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(gi + 1);
          }
          ok = wait(Ly::B_DS, (uint32_t)(gi & 1), i);
          if (!ok) break;
          if (i == 0 && k_unit > 0) {  // the previous unit's dK or dQ has been copied out of TMEM
            ok = wait(KV ? Ly::B_ACCE2 : Ly::B_ACCE, (uint32_t)((k_unit - 1) & 1), -1);
            if (!ok) break;
          }
          tc_fence_after();
          issue_acc(gi, i == 0);
          if (i + 1 == NB) tc_commit_warp(bar(KV ? Ly::B_ACC2 : Ly::B_ACC));
          if (i + 1 < NB) {
            ok = wait_b(gi + 1);
            if (!ok) break;
            tc_fence_after();
            issue_dp(gi + 1);
            if (i + 2 == NB) tc_commit_warp(bar(KV ? Ly::B_RESE : Ly::B_QTE));  // the unit's last S and dP are issued
          }
        }
        if (!ok) break;
        g0 += NB;
        ++k_unit;
        ok = take(x, ROLE_MMA);
        if (!ok || x.u < 0) break;
        ok = start_unit(x, g0);
      }
      // exit-path drain: every MMA issued completes before TMEM is freed
      tc_commit_warp(bar(Ly::B_DRAIN));
      mbar_drain(bar(Ly::B_DRAIN), 0u, DRAIN_NS);
    } else if (warp == WARP_LOAD) {
      // ================================================================ producer: the whole warp, converged; lane 0 loads
      bool ok = run;
      int np = 0;   // units published
      int taken = 0;
      const int n_units = KV ? prm.kv_units : prm.dq_units;
      uint32_t* counter = prm.counters + (KV ? 0 : 64);
      Unit next;
      // the next unit with blocks: a CTA's first is its own index, the others come from the counter.  What meets no block is
      // zeros, written here
      auto publish = [&]() {
        const int slot = np & 1;
        ok = mbar_wait_warp(bar(Ly::B_UE + slot), (uint32_t)(((np >> 1) & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status,
                            ROLE_LOAD, -1);
        if (!ok) return;
        for (;;) {
          int v = cta;
          if (taken++ > 0) {
            v = n_units;
            if (n_units > n_ctas) {
              if (lane == 0) v = (int)(n_ctas + atomicAdd(counter, 1u));
              v = __shfl_sync(0xffffffffu, v, 0);
            }
          }
          next.u = -1;
          if (v >= n_units) break;
          next = unit_of<KV>(v, prm);
          if (next.NB > 0) break;
          const int parts = KV ? prm.kv_parts : prm.dq_parts;
          const int64_t head = (int64_t)next.b * (KV ? prm.Hkv : prm.Hq) + next.h;
          const int64_t rows = min((int64_t)BM, S - (int64_t)next.blk * BM);
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          if (parts > 1) {
            const int64_t at = ((head * parts + next.part) * S + (int64_t)next.blk * BM) * D / 4;
            for (int64_t i = lane; i < rows * D / 4; i += 32)
              for (float* p : {KV ? prm.dk_part : prm.dq_part, KV ? prm.dv_part : nullptr})
                if (p) reinterpret_cast<uint4*>(p)[at + i] = zero;
          } else {
            const int64_t at = (head * S + (int64_t)next.blk * BM) * D / 8;
            for (int64_t i = lane; i < rows * D / 8; i += 32)
              for (__nv_bfloat16* p : {KV ? prm.dk : prm.dq, KV ? prm.dv : nullptr})
                if (p) reinterpret_cast<uint4*>(p)[at + i] = zero;
          }
        }
        if (lane == 0) {
          put_unit(ring + 8 * slot, next);
          mbar_arrive(bar(Ly::B_UF + slot));
        }
        __syncwarp();
        ++np;
      };
      int nres = 0;
      int64_t ga = 0, gb = 0;  // blocks of the two streams issued
      if (ok) publish();
      while (ok && next.u >= 0) {
        const Unit x = next;
        publish();  // the following unit
        if (!ok) break;
        // resident blocks: the previous unit's last products must be done with them (dq: they are copied into TMEM)
        ok = mbar_wait_warp(bar(Ly::B_RESE), (uint32_t)((nres & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, x.u);
        if (!ok) break;
        const int32_t res_head = x.b * (KV ? prm.Hkv : prm.Hq) + x.h;
        const int32_t str_head = KV ? x.b * prm.Hq + x.h * prm.g : x.b * prm.Hkv + x.h / prm.g;
        if (lane == 0) {
          mbar_expect_tx(bar(Ly::B_RES), 2 * Ly::TILE);
          for (int c = 0; c < D / 64; ++c) {
            tma_load_3d(sb + Ly::RES0 + (uint32_t)c * Ly::BOX, &tmR0, c * 64, x.blk * BM, res_head, bar(Ly::B_RES));
            tma_load_3d(sb + Ly::RES1 + (uint32_t)c * Ly::BOX, &tmR1, c * 64, x.blk * BM, res_head, bar(Ly::B_RES));
          }
        }
        __syncwarp();
        ++nres;
        Cursor cur;
        cur.start(x);
        for (int i = 0; i < x.NB && ok; ++i) {
          if (i > 0) cur.step();
          const int sa = (int)(ga % Ly::NSA), sbb = (int)(gb % Ly::NSB);
          if (ga >= Ly::NSA) {
            ok = mbar_wait_warp(bar(Ly::B_AE + sa), (uint32_t)((ga / Ly::NSA - 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                                ROLE_LOAD, i);
            if (!ok) break;
          }
          if (lane == 0) {
            mbar_expect_tx(bar(Ly::B_AF + sa), Ly::TILE);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sb + Ly::A0 + (uint32_t)sa * Ly::TILE + (uint32_t)c * Ly::BOX, &tmA, c * 64, cur.blk * BM,
                          str_head + cur.h, bar(Ly::B_AF + sa));
          }
          __syncwarp();
          ++ga;
          if (gb >= Ly::NSB) {
            ok = mbar_wait_warp(bar(Ly::B_BE + sbb), (uint32_t)((gb / Ly::NSB - 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                                ROLE_LOAD, i);
            if (!ok) break;
          }
          if (lane == 0) {
            mbar_expect_tx(bar(Ly::B_BF + sbb), Ly::TILE);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sb + Ly::B0 + (uint32_t)sbb * Ly::TILE + (uint32_t)c * Ly::BOX, &tmB, c * 64, cur.blk * BM,
                          str_head + cur.h, bar(Ly::B_BF + sbb));
          }
          __syncwarp();
          ++gb;
        }
      }
      // exit-path drain: every load issued lands before the CTA exits
      if (nres > 0) mbar_drain(bar(Ly::B_RES), (uint32_t)((nres - 1) & 1), DRAIN_NS);
      for (int64_t j = (ga > Ly::NSA ? ga - Ly::NSA : 0); j < ga; ++j)
        mbar_drain(bar(Ly::B_AF + (int)(j % Ly::NSA)), (uint32_t)((j / Ly::NSA) & 1), DRAIN_NS);
      for (int64_t j = (gb > Ly::NSB ? gb - Ly::NSB : 0); j < gb; ++j)
        mbar_drain(bar(Ly::B_BF + (int)(j % Ly::NSB)), (uint32_t)((j / Ly::NSB) & 1), DRAIN_NS);
    }
  } else {
    // ================================================================ epilogue warps (dq)
    regs_dec<EPI_REGS>();
    if constexpr (!KV) {
      // Per unit: copy its resident Q and dO from shared memory into TMEM (as the A operands of S
      // and dP) as soon as the previous unit's last S and dP products are done with the TMEM copy,
      // releasing the shared buffers to the producer; then drain the previous unit's dQ while the
      // other roles run this one, releasing it (so the next unit may overwrite it) once its last
      // TMEM load has completed.
      const int wq = warp & 3;  // TMEM lane quadrant
      const int r = wq * 32 + lane;  // this thread's row of the 128-row block
      const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
      const uint32_t tm_dq = tmem + lane_base + 256u;
      const uint32_t tm_qt = tmem + lane_base + 384u, tm_gt = tm_qt + (uint32_t)(D / 2);
      bool ok = run;
      int k_unit = 0, ncopy = 0;
      // row r of a 128 x D bf16 block landed by TMA in 64-column boxes with 128-byte swizzle (the
      // 16-byte chunk j of a 128-byte row sits at chunk j ^ (r mod 8)), packed two columns per TMEM
      // column from column `dst`
      auto copy_row = [&](uint32_t src_off, uint32_t dst) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          const uint8_t* rowp = smem + src_off + (uint32_t)c * Ly::BOX + (uint32_t)r * 128u;
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 q = *reinterpret_cast<const uint4*>(rowp + ((j ^ (r & 7)) << 4));
            w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
          }
          tmem_st32(dst + (uint32_t)(32 * c), w);
        }
      };
      auto copy_in = [&]() -> bool {
        if (!mbar_wait_warp(bar(Ly::B_RES), (uint32_t)(ncopy & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_EPI, -1))
          return false;
        if (ncopy > 0 && !mbar_wait_warp(bar(Ly::B_QTE), (uint32_t)((ncopy - 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                                         ROLE_EPI, -1))
          return false;
        tc_fence_after();
        copy_row(Ly::RES0, tm_qt);
        copy_row(Ly::RES1, tm_gt);
        tc_wait_st();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // reads done before the next TMA write
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(Ly::B_QTF));
          mbar_arrive(bar(Ly::B_RESE));
        }
        ++ncopy;
        return true;
      };
      Unit x;
      x.u = -1;
      if (ok) ok = take(x, ROLE_EPI);
      if (ok && x.u >= 0) ok = copy_in();
      while (ok && x.u >= 0) {
        Unit xn;
        ok = take(xn, ROLE_EPI);
        if (!ok) break;
        if (xn.u >= 0) {
          ok = copy_in();
          if (!ok) break;
        }
        const int64_t head = (int64_t)x.b * prm.Hq + x.h, q0 = (int64_t)x.blk * BM + wq * 32;
        const int rows_valid = (int)max((int64_t)0, min((int64_t)32, S - q0));
        ok = mbar_wait_warp(bar(Ly::B_ACC), (uint32_t)(k_unit & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_EPI, -1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float t[32];
          tmem_ld32(tm_dq + (uint32_t)c, t);
          tc_wait_ld();
          if (c + 32 == D) arrive(Ly::B_ACCE);
          if (prm.dq_parts > 1) store_rows<D>(t, prm.scale, prm.dq_part, (head * prm.dq_parts + x.part) * S + q0, rows_valid, c, lane);
          else if (lane < rows_valid) store_bf16(t, prm.scale, prm.dq + (head * S + q0 + lane) * D + c);
        }
        ++k_unit;
        x = xn;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
               const __grid_constant__ Params prm) {
  if ((int)blockIdx.x < prm.kv_ctas)
    run_pass<D, MODE, true>(tmK, tmV, tmQ, tmG, prm, (int)blockIdx.x, prm.kv_ctas);
  else
    run_pass<D, MODE, false>(tmQ, tmG, tmK, tmV, prm, (int)blockIdx.x - prm.kv_ctas, prm.dq_ctas);
}

// D = dO . O by rows, the query blocks' bounds, the order of the blocks, and the unit counters at zero, in one launch: the
// first CTAs of the grid take a mask each (beyond ORDER_MAX blocks: eight query blocks each), the others 16-byte pieces of
// rows, D / 8 lanes a row (four pieces a thread: 1 to 2 % slower for the pass as a whole).
constexpr int PREP_THREADS = 256;
struct PrepParams {
  const uint4* o;
  const uint4* go;
  float* dsum;
  Bounds* bounds;
  int32_t* order_q;  // or NULL
  int32_t* order_kv;
  int2* seen_by;
  const int32_t* lo;
  const int32_t* hi;
  uint32_t* counters;
  int32_t* status;
  int64_t mask_bs, S, rows;
  int32_t nb, bounds_blocks, n_bounds;  // n_bounds = nb times the masks
};
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  float s = 0.f;
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
    s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
  }
  return s;
}
template <int D>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(const __grid_constant__ PrepParams p) {
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(p.status) != 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int WARPS = PREP_THREADS / 32;
  if ((int)blockIdx.x < p.bounds_blocks) {
    __shared__ int2 see[ORDER_MAX], seen[ORDER_MAX];  // key blocks of a query block, and the other way round
    if (blockIdx.x == 0 && threadIdx.x < 2) p.counters[threadIdx.x * 64] = 0u;
    const int first = p.order_q ? (int)blockIdx.x * p.nb : (int)blockIdx.x * WARPS;
    const int end = p.order_q ? first + p.nb : min(first + WARPS, p.n_bounds);
    constexpr int U = 4;  // query blocks of a warp whose loads are in flight together
    for (int i0 = first + warp; i0 < end; i0 += WARPS * U) {
      int a[U][BM / 32], z[U][BM / 32];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * WARPS, m = i / p.nb, qb = i - m * p.nb;
#pragma unroll
        for (int e = 0; e < BM / 32; ++e) {
          const int64_t q = (int64_t)qb * BM + e * 32 + lane;
          const bool in = i < end && q < p.S;
          a[u][e] = in ? p.lo[m * p.mask_bs + q] : 0;
          z[u][e] = in ? p.hi[m * p.mask_bs + q] : 0;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * WARPS, qb = i % p.nb;
        if (i >= end) continue;
        int kmin = 0x7fffffff, kmax = 0, all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
        for (int e = 0; e < BM / 32; ++e) {
          const int x = max(a[u][e], 0), y = (int)min((int64_t)z[u][e], p.S);
          if (x < y) {
            kmin = min(kmin, x), kmax = max(kmax, y);
            all_lo = max(all_lo, x), all_hi = min(all_hi, y);
          } else if ((int64_t)qb * BM + e * 32 + lane < p.S) {
            all_hi = 0;
          }
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        Bounds b{0, 0, all_lo, all_hi};
        if (kmin < kmax) b.kb0 = kmin / BM, b.kb1 = (kmax + BM - 1) / BM;
        if (lane == 0) {
          p.bounds[i] = b;
          if (p.order_q) see[qb] = make_int2(b.kb0, b.kb1);
        }
      }
    }
    if (!p.order_q) return;
    __syncthreads();
    for (int k = threadIdx.x; k < p.nb; k += PREP_THREADS) {
      int a = 0, z = 0;
      for (int q = 0; q < p.nb; ++q)
        if (see[q].x <= k && k < see[q].y) {
          if (z == 0) a = q;
          z = q + 1;
        }
      seen[k] = make_int2(a, z);
      p.seen_by[first + k] = seen[k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.nb; i += PREP_THREADS) {
      const int2* r = i < p.nb ? see : seen;
      const int e = i < p.nb ? i : i - p.nb, n = r[e].y - r[e].x;
      int rank = 0;
      for (int j = 0; j < p.nb; ++j) {
        const int m = r[j].y - r[j].x;
        rank += m > n || (m == n && j < e);
      }
      (i < p.nb ? p.order_q : p.order_kv)[first + rank] = e;
    }
    return;
  }
  constexpr int L = D / 8;  // lanes a row
  const int64_t at = ((int64_t)blockIdx.x - p.bounds_blocks) * PREP_THREADS + threadIdx.x, row = at / L;
  float s = 0.f;
  if (row < p.rows) s = dot8(__ldcs(p.o + at), p.go[at]);
#pragma unroll
  for (int w = L / 2; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  if (row < p.rows && at % L == 0) p.dsum[row] = s;
}

// Sums of units in parts, in order: out[b, h] = sum over the parts of part[b, h, part].
struct SumParams {
  const float4* part[3];
  uint2* out[3];
  int64_t n[3];        // 4-column pieces of a tensor
  int64_t per_head;    // of a head
  int32_t parts[3];
  int32_t* status;
};
static __global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumParams p) {
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(p.status) != 0) return;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
#pragma unroll 1
  for (int w = 0; w < 3; ++w) {
    if (i >= p.n[w]) {
      i -= p.n[w];
      continue;
    }
    const float4* src = p.part[w] + i / p.per_head * p.per_head * p.parts[w] + i % p.per_head;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < p.parts[w]; ++k) {
      const float4 y = __ldcs(src + k * p.per_head);
      s.x += y.x, s.y += y.y, s.z += y.z, s.w += y.w;
    }
    p.out[w][i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    return;
  }
}

// ------------------------------------------------------------------ host side
template <int D, int MODE>
static cudaError_t launch_main(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mg,
                               const Params& prm, cudaStream_t st, std::string* err) {
  auto kern = bwd_kernel<D, MODE>;
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  cudaError_t e = cudaSuccess;
  if (once.pending(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::TOTAL);
    // setmaxnreg hands registers between warpgroups within the launch's pool: the split must fit
    // the registers the kernel is launched with, or a raising warpgroup would wait forever
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess && fa.numRegs * NUM_THREADS < 2 * 128 * EW_REGS + 128 * MMA_REGS + 128 * EPI_REGS) {
      *err = "range backward built with " + std::to_string(fa.numRegs) +
             " registers per thread, fewer than its warpgroups' register split needs";
      return cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) once.mark(dev);
  }
  if (e != cudaSuccess) return e;
  // not launch_behind: begun beside the end of prep_kernel, the whole took 404 us where this takes 322 (8,192 tokens in five
  // documents, 16 heads on 4, capped; without a cap 252 and 233), for 2 us less where there is little to do
  kern<<<dim3((unsigned)(prm.kv_ctas + prm.dq_ctas)), NUM_THREADS, Layout<D>::TOTAL, st>>>(mq, mk, mv, mg, prm);
  return cudaGetLastError();
}

template <int D>
static int launch(const RangeArgs& a, const RangeBwdShape& z, int sms, cudaStream_t st, std::string* err) {
  const int64_t nb = (a.S + BM - 1) / BM, kv_units = nb * a.B * a.Hkv * z.kv_parts, dq_units = nb * a.B * a.Hq * z.dq_parts;
  const int64_t rows = (int64_t)a.B * a.Hq * a.S, masks = a.mask_bs ? a.B : 1;
  if (kv_units > 0x3fffffff || dq_units > 0x3fffffff || nb * masks > 0x3fffffff) {
    *err = "too many work units for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  PrepParams pp{};
  pp.o = static_cast<const uint4*>(a.o);
  pp.go = static_cast<const uint4*>(a.go);
  pp.dsum = reinterpret_cast<float*>(a.ws + z.dsum);
  pp.bounds = reinterpret_cast<Bounds*>(a.ws + z.bounds);
  pp.lo = a.lo;
  pp.hi = a.hi;
  pp.counters = reinterpret_cast<uint32_t*>(a.ws + z.counters);
  pp.status = a.status;
  pp.mask_bs = a.mask_bs;
  pp.S = a.S;
  pp.rows = rows;
  pp.nb = (int32_t)nb;
  pp.n_bounds = (int32_t)(nb * masks);
  pp.bounds_blocks = (pp.n_bounds + PREP_THREADS / 32 - 1) / (PREP_THREADS / 32);
  if (nb <= ORDER_MAX) {
    pp.order_q = reinterpret_cast<int32_t*>(a.ws + z.order);
    pp.order_kv = pp.order_q + pp.n_bounds;
    pp.seen_by = reinterpret_cast<int2*>(pp.order_kv + pp.n_bounds);
    pp.bounds_blocks = (int32_t)masks;
  }
  const int64_t prep_blocks = pp.bounds_blocks + (rows * (D / 8) + PREP_THREADS - 1) / PREP_THREADS;
  Params prm{};
  prm.lse = a.lse;
  prm.dsum = pp.dsum;
  prm.bounds = pp.bounds;
  prm.order_q = pp.order_q;
  prm.order_kv = pp.order_kv;
  prm.seen_by = pp.seen_by;
  prm.lo = a.lo;
  prm.hi = a.hi;
  prm.mask_bs = a.mask_bs;
  prm.bounds_bs = a.mask_bs ? (int32_t)nb : 0;
  prm.slopes = a.slopes;
  prm.dq = static_cast<__nv_bfloat16*>(a.dq);
  prm.dk = static_cast<__nv_bfloat16*>(a.dk);
  prm.dv = static_cast<__nv_bfloat16*>(a.dv);
  prm.dq_part = reinterpret_cast<float*>(a.ws + z.dq_part);
  prm.dk_part = reinterpret_cast<float*>(a.ws + z.dk_part);
  prm.dv_part = reinterpret_cast<float*>(a.ws + z.dv_part);
  prm.status = a.status;
  prm.counters = pp.counters;
  prm.S = a.S;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.g = a.Hq / a.Hkv;
  prm.nb = (int32_t)nb;
  prm.kv_units = (int32_t)kv_units;
  prm.dq_units = (int32_t)dq_units;
  prm.kv_ctas = (int32_t)std::min<int64_t>(kv_units, sms);
  prm.dq_ctas = (int32_t)std::min<int64_t>(dq_units, sms);
  prm.kv_parts = z.kv_parts;
  prm.dq_parts = z.dq_parts;
  // lanes numbered together: enough for about three times the grid, so that the last units are short where lengths differ
  prm.kv_batch = (int32_t)std::min<int64_t>((int64_t)a.B * a.Hkv, (3LL * sms + nb - 1) / nb);
  prm.dq_batch = (int32_t)std::min<int64_t>((int64_t)a.B * a.Hq, (3LL * sms + nb - 1) / nb);
  prm.scale = a.scale;
  prm.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  prm.cap = make_cap(a.scale, a.cap);
  prm.wait_limit_ns = a.wait_limit_ns;
  CUtensorMap mq, mk, mv, mg;
  const uint64_t qd[3] = {D, (uint64_t)a.S, (uint64_t)a.B * a.Hq}, kd[3] = {D, (uint64_t)a.S, (uint64_t)a.B * a.Hkv};
  const int64_t str[2] = {D, a.S * D};
  const uint32_t box[3] = {64, BM, 1};
  if (!encode_bf16_map(&mq, a.q, 3, qd, str, box, err) || !encode_bf16_map(&mk, a.k, 3, kd, str, box, err) ||
      !encode_bf16_map(&mv, a.v, 3, kd, str, box, err) || !encode_bf16_map(&mg, a.go, 3, qd, str, box, err))
    return (int)cudaErrorInvalidValue;
  cudaError_t e = launch_behind(prep_kernel<D>, dim3((unsigned)prep_blocks), PREP_THREADS, 0, st, pp);
  if (e == cudaSuccess)
    e = a.cap > 0.f    ? launch_main<D, 2>(mq, mk, mv, mg, prm, st, err)
        : a.slopes ? launch_main<D, 1>(mq, mk, mv, mg, prm, st, err)
                   : launch_main<D, 0>(mq, mk, mv, mg, prm, st, err);
  if (e == cudaSuccess && (z.kv_parts > 1 || z.dq_parts > 1)) {
    SumParams sp{};
    const float* parts[3] = {prm.dq_part, prm.dk_part, prm.dv_part};
    void* outs[3] = {a.dq, a.dk, a.dv};
    int64_t n = 0;
    for (int w = 0; w < 3; ++w) {
      sp.parts[w] = w ? z.kv_parts : z.dq_parts;
      sp.part[w] = reinterpret_cast<const float4*>(parts[w]);
      sp.out[w] = static_cast<uint2*>(outs[w]);
      sp.n[w] = sp.parts[w] > 1 ? (int64_t)a.B * (w ? a.Hkv : a.Hq) * a.S * (D / 4) : 0;
      n += sp.n[w];
    }
    sp.per_head = a.S * (D / 4);
    sp.status = a.status;
    e = launch_behind(sum_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, st, sp);
  }
  if (e != cudaSuccess && err->empty()) *err = std::string("range backward launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace sbw

}  // namespace mesh
