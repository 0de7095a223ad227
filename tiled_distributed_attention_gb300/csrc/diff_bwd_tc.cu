// Differential attention backward on the 5th-generation tensor cores (sm_103a), bf16 inputs.
//
// With P_m = exp(scale q_m.k_m - LSE_m), dP = dO V^T (one product for both maps) and D_m = dO . O_m:
//   A = P_1 - lam P_2,            dV = A^T dO,
//   dS_1 = P_1 (dP - D_1),        dS_2 = -lam P_2 (dP - D_2),
//   dq_m = scale dS_m k_m,        dk_m = scale dS_m^T q_m,        dlam = -sum P_2 dP.
// Both maps of a block share dP, and their halves of the columns fill one product of the plain backward
// pass, so a block costs the tensor cores what plain attention of the same d costs; the exponentials
// are twice as many.  (The last sum is D_2 summed over the rows, taken from fp32 products instead of
// the rounded O_2: it nearly cancels over a batch, which a rounded operand would show.)
//
// Two passes after the plain backward pass's pattern, in one launch: the first CTAs of the grid run dkdv, the
// others dq, each pass persistent over its own units (its own index first, then a counter), published
// through a two-entry shared-memory ring.  One CTA fills an SM; where both passes together have fewer
// units than there are SMs they run side by side, and otherwise dq's CTAs start as dkdv's end.
// Every role has warps of its own:
//   warps 0-7   elementwise: two warps per TMEM lane quadrant, each taking 32 of a block's 64 columns
//   warp 8      MMA issuer, warp 9 producer (TMA), warps 10-11 idle
//   warps 12-15 (dq) copy each unit's Q and dO into TMEM, and drain and store dQ
// The streamed blocks are 64 rows deep, half of the plain pass's: two score maps, dP and the
// accumulators then fit the 512 TMEM columns at d = 128.
//
// dkdv (unit = batch, KV head, 128-key block, part): K and V stay in shared memory, Q and dO blocks
// of 64 query rows stream.  TMEM: S_1^T | S_2^T | dP^T | A^T (two buffers) | dV | dK_1 | dK_2.
//   Issue order per block i: [S(i) read] S(i+1)   [dS(i) and A(i) ready] dK(i), dP(i+1), dV(i).
//   dS_1 and dS_2 (bf16) replace dP in its own columns.
// dq (unit = batch, head, 128-row block, part): Q and dO are copied into TMEM once per unit and
// feed the products as A operands; K and V blocks of 64 keys stream.  TMEM: S_1 | S_2 | dP (two
// buffers) | dQ_1 | dQ_2 | Q | dO.
//   Issue order per block j: [S(j) read] S(j+1), dP(j+1)   [dS(j) ready] dQ(j).
// At d = 64 a map's half is 32 columns: dK_m and dQ_m are computed 64 wide and half of them is used.
//
// The gradients are written from the accumulators, rounded once, where the blocks alone fill the GPU.  With
// fewer, a unit is cut into parts of its streamed blocks (diff_bwd_parts), which leave fp32 sums that
// sum_parts adds in order.  Rows past the end are loaded as zeros.
// A, dS_1 and dS_2 are rounded to bf16 for their products (2^-8 relative a term at most); sums are fp32.
// Every mbarrier wait is bounded; a timeout records MESH_ATTN_ERR_DEVICE_TIMEOUT, the CTA stops,
// drains its copies and products and frees its tensor memory.
//
// Measured (16 heads on 4, 8,192 tokens, d = 128, causal): 0.98 ms, 700 TFLOP/s of the formulas' five
// products (seven are computed).  Bound by the elementwise warps' chain (scores in, exponentials, dP in,
// A and dS out): 1,700-1,900 cycles a 128 x 64 block against 1,300 (dkdv) and 780 (dq) of products; the
// tensor pipe is 42 % busy.  Slower: 16 elementwise warps (1.15 ms where 8 took 1.11).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace dbtc {

constexpr int BM = 128;  // resident rows = TMEM lanes
constexpr int BS = 64;   // streamed rows per block = columns of a score block
constexpr int NUM_THREADS = 512;
constexpr int N_EW = 8;  // elementwise warps: two per TMEM lane quadrant, 32 columns each
constexpr int WARP_MMA = 8;
constexpr int WARP_LOAD = 9;
constexpr int WARP_EPI = 12;
constexpr int N_EPI = 4;
// Register budgets after setmaxnreg, per warpgroup: elementwise (warps 0-7), MMA / producer (8-11),
// epilogue (12-15).  They add up to the 512 x 128 registers of the launch; the launcher checks
// the kernels' register count against that before launching.
constexpr int EW_REGS = 168, MMA_REGS = 104, EPI_REGS = 72;
static_assert(2 * 128 * EW_REGS + 128 * MMA_REGS + 128 * EPI_REGS <= NUM_THREADS * 128, "register split");
constexpr int64_t DRAIN_NS = 200000000;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int ROLE_EW = 1, ROLE_MMA = 2, ROLE_LOAD = 3, ROLE_ITEM = 4, ROLE_EPI = 5;
// TMEM columns
constexpr uint32_t COL_S = 0;     // S_1 [64], S_2 [64]
constexpr uint32_t COL_DP = 128;  // dP [64] (dq: two buffers); dS_1, dS_2 (bf16) in its place
constexpr uint32_t COL_A = 192;   // dkdv: A^T (bf16), two buffers of 32
constexpr uint32_t COL_ACC = 256; // dkdv: dV [D]; dq: dQ_1 [64], dQ_2 [64]
constexpr uint32_t COL_DK = 384;  // dkdv: dK_1 [64], dK_2 [64]
constexpr uint32_t COL_Q = 384;   // dq: Q [D / 2], then dO [D / 2] (bf16)
// dS_m of column half hf (32 columns) lies in packed columns [32 hf + 16 m, + 16) of its dP region: inside
// the half's own input columns.  K-step kk (16 elements, 8 packed columns) of dS_m:
__device__ __forceinline__ uint32_t ds_col(int m, int kk) { return (uint32_t)((kk >> 1) * 32 + m * 16 + (kk & 1) * 8); }

struct Params {
  const float* lse;   // [B, Hq, 2, S]
  const float* dsum;  // [B, Hq, 2, S]
  const __nv_bfloat16* lam;
  __nv_bfloat16* out0;  // dQ, or dK
  __nv_bfloat16* out1;  //         dV
  float* part0;         // of units in parts, [B, H, parts, S, D]: dQ, or dK
  float* part1;         //                                              dV
  float* dlam_part;     // [B, Hq, parts, nb, N_EW]
  int32_t* status;
  uint32_t* counter;
  int64_t S;
  int32_t B, Hq, Hkv, parts, nb, ns, causal, n_tiles, n_units, lam_n;  // nb 128-row blocks, ns 64-row blocks
  int32_t batch;  // heads whose units are numbered together (unit_of)
  float scale, scale_log2;
  int64_t wait_limit_ns;
};

template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // resident 128-row block
  static constexpr uint32_t BOX = BM * 64 * 2;  // its 64-column boxes
  static constexpr uint32_t SBLK = BS * D * 2;  // streamed 64-row block
  static constexpr uint32_t SBOX = BS * 64 * 2;
  static constexpr int NSA = 4, NSB = 4;
  static constexpr uint32_t RES0 = 0, RES1 = TILE;
  static constexpr uint32_t A0 = 2 * TILE;              // Q (dkdv) or K (dq) stages
  static constexpr uint32_t B0 = A0 + NSA * SBLK;       // dO (dkdv) or V (dq) stages
  static constexpr uint32_t VEC_OFF = B0 + NSB * SBLK;  // dkdv: -LSE_1, -LSE_2 (base 2), -D_1, lam D_2: [3][4][64] fp32
  static constexpr uint32_t BAR_OFF = VEC_OFF + 3 * 4 * BS * 4;
  static constexpr int B_RES = 0, B_AF = 1, B_AE = B_AF + NSA, B_BF = B_AE + NSA, B_BE = B_BF + NSB,
                       B_S = B_BE + NSB, B_SREAD = B_S + 1, B_DP = B_SREAD + 1, B_DS = B_DP + 2,
                       B_ACC = B_DS + 2, B_ACCE = B_ACC + 1, B_DRAIN = B_ACCE + 1, B_VEC = B_DRAIN + 1,
                       B_RESE = B_VEC + 3, B_UF = B_RESE + 1, B_UE = B_UF + 2, B_QTF = B_UE + 2, B_QTE = B_QTF + 1,
                       NBARS = B_QTE + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBARS * 8 + (NBARS % 2) * 8;  // tmem base, abort flag
  static constexpr uint32_t RING_OFF = MISC_OFF + 16;  // unit ring: 2 decoded units, 16 ints each
  static constexpr uint32_t TOTAL = RING_OFF + 2 * 64;
};

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

__device__ __forceinline__ float lam_of(const Params& prm, int h) {
  return __bfloat162float(prm.lam[prm.lam_n == 1 ? 0 : h]);
}

// A unit of either pass: 128-row block `blk` of a (KV) head, and of its streamed blocks [start, start + NB).  A dq
// unit streams 64-key blocks, a dkdv unit the 64-row blocks of the group's query heads, head after head; causal
// units up to, or from, the diagonal.
struct Unit {
  int blk, h, b, part, start, NB;
};
template <bool KV>
__device__ __forceinline__ int blocks_of(int blk, int ns, int causal, int group) {
  if (KV) return (ns - (causal ? 2 * blk : 0)) * group;
  return causal ? min(ns, 2 * blk + 2) : ns;
}
template <bool KV>
__device__ __forceinline__ Unit unit_of(int u, const Params& prm) {
  Unit x;
  const int H = KV ? prm.Hkv : prm.Hq, g = prm.Hq / prm.Hkv;
  x.part = u % prm.parts;
  int t = u / prm.parts;
  // numbered batch of (batch, head) lanes by batch, within it block by block from the longest
  const int per = prm.batch * prm.nb, first = t / per * prm.batch;
  const int lanes = min(prm.batch, prm.n_tiles / prm.nb - first);  // the last batch may be smaller
  t %= per;
  x.blk = t / lanes;
  if (!KV && prm.causal) x.blk = prm.nb - 1 - x.blk;
  t = first + t % lanes;
  x.h = t % H;
  x.b = t / H;
  const int n = blocks_of<KV>(x.blk, prm.ns, prm.causal, g), k = min(prm.parts, n);
  x.start = (int)((int64_t)min(x.part, k) * n / k);
  x.NB = (int)((int64_t)min(x.part + 1, k) * n / k) - x.start;  // none where there are fewer blocks than parts
  return x;
}
// A unit travels through the shared-memory ring decoded.
__device__ __forceinline__ void put_unit(volatile int32_t* e, int u, const Unit& x) {
  e[0] = u;
  e[1] = x.blk, e[2] = x.h, e[3] = x.b, e[4] = x.NB, e[5] = x.part, e[6] = x.start;
}
__device__ __forceinline__ int get_unit(const volatile int32_t* e, Unit& x) {
  x.blk = e[1], x.h = e[2], x.b = e[3], x.NB = e[4], x.part = e[5], x.start = e[6];
  return e[0];
}

// Query blocks of a dkdv unit: heads of the group, then a head's blocks.
struct QCursor {
  int h, qb, begin;
  __device__ __forceinline__ void start(const Params& prm, const Unit& x) {
    begin = prm.causal ? 2 * x.blk : 0;
    const int n = prm.ns - begin;
    h = x.h * (prm.Hq / prm.Hkv) + x.start / n;
    qb = begin + x.start % n;
  }
  __device__ __forceinline__ void step(const Params& prm) {
    if (++qb < prm.ns) return;
    qb = begin;
    ++h;
  }
};

// What both kernels share: barrier set-up, the unit ring and the exit.
template <int D, bool KV>
__device__ __forceinline__ void run_pass(const CUtensorMap& tmR0, const CUtensorMap& tmR1, const CUtensorMap& tmA,
                                         const CUtensorMap& tmB, const Params& prm, int cta, int n_ctas) {
  // R0, R1: the resident blocks' tensors (dkdv: K, V; dq: Q, dO); A, B: the streamed ones (Q, dO; K, V)
  using Ly = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = smem_u32(smem_raw);
  if (sb & 1023u) {  // 128-byte swizzle atoms need 1024-aligned operands; the window starts so on this part
    if (threadIdx.x == 0) record_error(prm.status, MESH_ATTN_ERR_INTERNAL, ROLE_ITEM, (int32_t)blockIdx.x);
    return;
  }
  uint8_t* smem = smem_raw;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + Ly::BAR_OFF + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::MISC_OFF);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC_OFF + 4);
  volatile int32_t* unit_ring = reinterpret_cast<volatile int32_t*>(smem + Ly::RING_OFF);
  const int64_t S = prm.S;
  const int g = prm.Hq / prm.Hkv;

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
    mbar_init(bar(Ly::B_SREAD), N_EW);  // one lane of each elementwise warp
    mbar_init(bar(Ly::B_DP), 1);
    mbar_init(bar(Ly::B_DP + 1), 1);
    // two, like dP's: in dq the elementwise warps may finish dS(g + 1) before the issuer has looked at dS(g),
    // and a barrier two phases ahead looks like one that is not there yet
    mbar_init(bar(Ly::B_DS), N_EW);
    mbar_init(bar(Ly::B_DS + 1), N_EW);
    mbar_init(bar(Ly::B_ACC), 1);
    mbar_init(bar(Ly::B_ACCE), KV ? N_EW : N_EPI);
    mbar_init(bar(Ly::B_DRAIN), 1);
    mbar_init(bar(Ly::B_VEC), N_EW * 32);  // every elementwise thread has written its LSE or D value
    mbar_init(bar(Ly::B_VEC + 1), N_EW * 32);
    mbar_init(bar(Ly::B_VEC + 2), N_EW * 32);
    mbar_init(bar(Ly::B_QTF), N_EPI);
    mbar_init(bar(Ly::B_QTE), 1);
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
  auto take = [&](int& v, Unit& y, int role) -> bool {
    const int slot = nu & 1;
    bool r = mbar_wait_warp(bar(Ly::B_UF + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status, role, -1);
    if (!r) return false;
    v = get_unit(unit_ring + 16 * slot, y);
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
    const int c_base = hf * 32;               // this warp's columns [c_base, c_base + 32)
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tm_s = tmem + lane_base + COL_S + (uint32_t)c_base;
    const uint32_t tm_dp = tmem + lane_base + COL_DP + (uint32_t)c_base;
    const uint64_t sc2 = f2_pack(prm.scale_log2, prm.scale_log2);
    bool ok = run;
    int v = -1;
    Unit x;
    if (ok) ok = take(v, x, ROLE_EW);
    int64_t g0 = 0;  // global index of the unit's first block
    int k_unit = 0;
    if constexpr (KV) {
      // ---------------------------------------------------------------- dK and dV
      // Vector `vec` (LSE_1, LSE_2, D_1, D_2) of query column `vq`: loaded raw two blocks ahead, scaled and
      // published one block ahead, so that neither the load nor the other threads' writes are waited
      // for.  Three buffers: a warp that publishes block i + 1 has seen dP(i - 1), which was issued
      // after every warp's dS(i - 2), so nobody reads the buffer of block i - 2 any more.
      float* vec_s = reinterpret_cast<float*>(smem + Ly::VEC_OFF);
      const int tid = threadIdx.x, vec = tid >> 6, vq = tid & 63;
      float raw = 0.f;
      bool raw_in = false;
      float raw_lam = 0.f;  // lam of the head whose value `raw` is
      int lam_h = -1;
      auto fetch = [&](const Unit& y, const QCursor& c) {
        const int64_t ql = (int64_t)c.qb * BS + vq;
        raw_in = ql < S;
        if (raw_in) {
          const int64_t at = (((int64_t)y.b * prm.Hq + c.h) * 2 + (vec & 1)) * S + ql;
          raw = (vec < 2 ? prm.lse : prm.dsum)[at];
        }
        if (c.h != lam_h) {
          lam_h = c.h;
          raw_lam = lam_of(prm, c.h);
        }
      };
      // block n of the launch; no such query row (or one without a visible key): exp2(s - inf) = 0, so it
      // needs no mask
      auto publish = [&](int64_t n) {
        const int vb = (int)(n % 3);
        float val = vec < 2 ? -INFINITY : 0.f;
        if (raw_in) val = vec == 2 ? -raw : vec == 3 ? raw_lam * raw : raw == -INFINITY ? -INFINITY : -raw * LOG2E;
        vec_s[(vb * 4 + vec) * BS + vq] = val;
        mbar_arrive(bar(Ly::B_VEC + vb));
      };
      // cursors: block i, and the next one to fetch (i + 2, or the next unit's first)
      QCursor cur, nxt;
      float lam_cur = 0.f, lam_pub = 0.f;  // lam of block i and of the block published last
      if (ok && v >= 0) {
        cur.start(prm, x);
        fetch(x, cur);
        lam_pub = raw_lam;
        publish(0);
        nxt = cur;
        if (x.NB > 1) {
          nxt.step(prm);
          fetch(x, nxt);
        }
      }
      while (ok && v >= 0) {
        const int kb = x.blk, NB = x.NB;
        QCursor c1 = nxt;  // block i + 1
        for (int i = 0; i < NB && ok; ++i) {
          const int64_t gi = g0 + i;
          const int vb = (int)(gi % 3);
          if (i > 0) {
            cur = c1;
            c1 = nxt;
          }
          lam_cur = lam_pub;
          if (i + 1 < NB) {
            lam_pub = raw_lam;
            publish(gi + 1);
            if (i + 2 < NB) {
              nxt.step(prm);
              fetch(x, nxt);
            }
          }
          const float nl = -lam_cur;
          ok = wait_all(Ly::B_VEC + vb, (uint32_t)((gi / 3) & 1), ROLE_EW, i);
          if (!ok) break;
          // causal diagonal: query columns before this key row are masked
          const int lo = prm.causal ? kb * BM + row - cur.qb * BS - c_base : 0;
          ok = wait_all(Ly::B_S, (uint32_t)(gi & 1), ROLE_EW, i);
          if (!ok) break;
          tc_fence_after();
          float p1[32], p2[32];
          tmem_ld32(tm_s, p1);
          tmem_ld32(tm_s + 64u, p2);
          tc_wait_ld();
          arrive(Ly::B_SREAD);  // the next block's S may overwrite it
          if (__any_sync(0xffffffffu, lo > 0)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c < lo) p1[c] = p2[c] = -INFINITY;
          }
          const float4* l1 = reinterpret_cast<const float4*>(vec_s + (vb * 4 + 0) * BS + c_base);
          const float4* l2 = reinterpret_cast<const float4*>(vec_s + (vb * 4 + 1) * BS + c_base);
          const float4* d1 = reinterpret_cast<const float4*>(vec_s + (vb * 4 + 2) * BS + c_base);
          const float4* d2 = reinterpret_cast<const float4*>(vec_s + (vb * 4 + 3) * BS + c_base);
          const uint64_t nl2 = f2_pack(nl, nl);
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 a = l1[c / 4], b = l2[c / 4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              float x0, x1, y0, y1;
              f2_unpack(f2_fma(f2_pack(p1[c + e], p1[c + e + 1]), sc2, e ? f2_pack(a.z, a.w) : f2_pack(a.x, a.y)), x0, x1);
              f2_unpack(f2_fma(f2_pack(p2[c + e], p2[c + e + 1]), sc2, e ? f2_pack(b.z, b.w) : f2_pack(b.x, b.y)), y0, y1);
              p1[c + e] = fast_exp2(x0);
              p1[c + e + 1] = fast_exp2(x1);
              p2[c + e] = fast_exp2(y0);
              p2[c + e + 1] = fast_exp2(y1);
              float a0, a1;  // A = P_1 - lam P_2
              f2_unpack(f2_fma(f2_pack(p2[c + e], p2[c + e + 1]), nl2, f2_pack(p1[c + e], p1[c + e + 1])), a0, a1);
              pk[(c + e) / 2] = pack_bf16x2(a0, a1);
            }
          }
          tmem_st16(tmem + lane_base + COL_A + (uint32_t)((gi & 1) * 32 + hf * 16), pk);  // complete by this block's DS
          ok = wait_all(Ly::B_DP, (uint32_t)(gi & 1), ROLE_EW, i);
          if (!ok) break;
          tc_fence_after();
          float dp[32];
          tmem_ld32(tm_dp, dp);
          tc_wait_ld();
          uint32_t s1[16], s2[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 a = d1[c / 4], b = d2[c / 4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t d = f2_pack(dp[c + e], dp[c + e + 1]);
              float a0, a1;
              f2_unpack(f2_mul(f2_add(d, e ? f2_pack(a.z, a.w) : f2_pack(a.x, a.y)), f2_pack(p1[c + e], p1[c + e + 1])), a0, a1);
              s1[(c + e) / 2] = pack_bf16x2(a0, a1);
              // -lam (dP - D_2) P_2
              f2_unpack(f2_mul(f2_fma(d, nl2, e ? f2_pack(b.z, b.w) : f2_pack(b.x, b.y)), f2_pack(p2[c + e], p2[c + e + 1])), a0, a1);
              s2[(c + e) / 2] = pack_bf16x2(a0, a1);
            }
          }
          tmem_st16(tm_dp, s1);
          tmem_st16(tm_dp + 16u, s2);
          tc_wait_st();
          arrive(Ly::B_DS + (int)(gi & 1));
        }
        if (!ok) break;
        // the next unit, and its first block's values, before this unit's epilogue
        int vn = -1;
        Unit xn;
        ok = take(vn, xn, ROLE_EW);
        if (!ok) break;
        if (vn >= 0) {
          cur.start(prm, xn);
          fetch(xn, cur);
        }
        // ---- epilogue: this half's columns of the dV and dK rows of this key block
        ok = wait_all(Ly::B_ACC, (uint32_t)(k_unit & 1), ROLE_EW, -1);
        if (!ok) break;
        tc_fence_after();
        {
          const uint32_t tm_dv = tmem + lane_base + COL_ACC + (uint32_t)(hf * (D / 2));
          // map hf's dK: columns [hf D / 2, + D / 2), at d = 64 the half of its 64-wide product that is its own
          const uint32_t tm_dk = tmem + lane_base + COL_DK + (uint32_t)(hf * 64 + (D == 64 ? hf * 32 : 0));
          const int64_t rl = (int64_t)kb * BM + row;
          float acc[D / 2];
#pragma unroll
          for (int which = 0; which < 2; ++which) {  // dV, then dK
            const uint32_t tm = which ? tm_dk : tm_dv;
            const float mul = which ? prm.scale : 1.f;
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) tmem_ld32(tm + (uint32_t)c, acc + c);
            tc_wait_ld();
            if (which) arrive(Ly::B_ACCE);  // both accumulators are copied out: the next unit may overwrite them
            if (prm.parts > 1) {
              const int64_t row0 = (((int64_t)x.b * prm.Hkv + x.h) * prm.parts + x.part) * S + (int64_t)kb * BM + wq * 32;
              const int rows_valid = (int)max((int64_t)0, min((int64_t)32, S - ((int64_t)kb * BM + wq * 32)));
#pragma unroll
              for (int c = 0; c < D / 2; c += 32)
                store_rows<D>(*reinterpret_cast<const float(*)[32]>(acc + c), mul, which ? prm.part0 : prm.part1, row0,
                              rows_valid, hf * (D / 2) + c, lane);
            } else if (rl < S) {
              __nv_bfloat16* dst = (which ? prm.out0 : prm.out1) +
                                   (((int64_t)x.b * prm.Hkv + x.h) * S + rl) * D + hf * (D / 2);
#pragma unroll
              for (int c = 0; c < D / 2; c += 32) store_bf16(acc + c, mul, dst + c);
            }
          }
        }
        ++k_unit;
        g0 += NB;
        v = vn;
        x = xn;
        if (v >= 0) {
          lam_pub = raw_lam;
          publish(g0);
          nxt = cur;
          if (x.NB > 1) {
            nxt.step(prm);
            fetch(x, nxt);
          }
        }
      }
    } else {
      // ---------------------------------------------------------------- dQ
      // LSEs and Ds of this thread's row, loaded as soon as the unit is known and used a phase later
      float raw_l[2] = {0.f, 0.f}, raw_d[2] = {0.f, 0.f}, raw_nl = 0.f;
      bool row_in = false;
      auto fetch = [&](const Unit& y) {
        const int64_t ql = (int64_t)y.blk * BM + row;
        row_in = ql < S;
        raw_nl = -lam_of(prm, y.h);
        if (row_in) {
          const int64_t at = (((int64_t)y.b * prm.Hq + y.h) * 2) * S + ql;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            raw_l[m] = prm.lse[at + m * S];
            raw_d[m] = prm.dsum[at + m * S];
          }
        }
      };
      if (ok && v >= 0) fetch(x);
      while (ok && v >= 0) {
        const int qb = x.blk;
        float nl[2], nd[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          nl[m] = row_in && raw_l[m] != -INFINITY ? -raw_l[m] * LOG2E : -INFINITY;
          nd[m] = row_in ? -raw_d[m] : 0.f;
        }
        const uint64_t l1 = f2_pack(nl[0], nl[0]), l2 = f2_pack(nl[1], nl[1]);
        const float lam_d2 = raw_nl * nd[1];
        const uint64_t d1 = f2_pack(nd[0], nd[0]), ld2 = f2_pack(lam_d2, lam_d2), nlam2 = f2_pack(raw_nl, raw_nl);
        uint64_t t2[2] = {0ull, 0ull};  // sum of P_2 dP
        const int n_keys = (int)S, diag_keys = qb * BM + row + 1;  // keys; those up to the row's own
        for (int j = 0; j < x.NB && ok; ++j) {
          const int kb = x.start + j;
          const int64_t gi = g0 + j;
          const uint32_t dpb = tm_dp + (uint32_t)((gi & 1) * 64);
          // keys past the end, or behind the row, are masked
          const int hi = (prm.causal ? min(n_keys, diag_keys) : n_keys) - kb * BS - c_base;
          const bool any_mask = (kb + 1) * BS > (prm.causal ? min(n_keys, qb * BM) : n_keys);
          ok = wait_all(Ly::B_S, (uint32_t)(gi & 1), ROLE_EW, j);
          if (!ok) break;
          tc_fence_after();
          float p1[32], p2[32];
          tmem_ld32(tm_s, p1);
          tmem_ld32(tm_s + 64u, p2);
          tc_wait_ld();
          arrive(Ly::B_SREAD);  // the next block's S may overwrite it
          if (any_mask) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= hi) p1[c] = p2[c] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(p1[c], p1[c + 1]), sc2, l1), x0, x1);
            p1[c] = fast_exp2(x0);
            p1[c + 1] = fast_exp2(x1);
            f2_unpack(f2_fma(f2_pack(p2[c], p2[c + 1]), sc2, l2), x0, x1);
            p2[c] = fast_exp2(x0);
            p2[c + 1] = fast_exp2(x1);
          }
          ok = wait_all(Ly::B_DP + (int)(gi & 1), (uint32_t)((gi >> 1) & 1), ROLE_EW, j);
          if (!ok) break;
          tc_fence_after();
          float dp[32];
          tmem_ld32(dpb, dp);
          tc_wait_ld();
          uint32_t s1[16], s2[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const uint64_t d = f2_pack(dp[c], dp[c + 1]);
            const uint64_t q2 = f2_pack(p2[c], p2[c + 1]);
            float a0, a1;
            f2_unpack(f2_mul(f2_add(d, d1), f2_pack(p1[c], p1[c + 1])), a0, a1);
            s1[c / 2] = pack_bf16x2(a0, a1);
            t2[(c >> 1) & 1] = f2_fma(q2, d, t2[(c >> 1) & 1]);
            f2_unpack(f2_mul(f2_fma(d, nlam2, ld2), q2), a0, a1);  // -lam (dP - D_2) P_2
            s2[c / 2] = pack_bf16x2(a0, a1);
          }
          tmem_st16(dpb, s1);
          tmem_st16(dpb + 16u, s2);
          tc_wait_st();
          arrive(Ly::B_DS + (int)(gi & 1));
        }
        if (!ok) break;
        {
          float a0, a1;
          f2_unpack(f2_add(t2[0], t2[1]), a0, a1);
          float t = a0 + a1;
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
          if (lane == 0)
            prm.dlam_part[((((int64_t)x.b * prm.Hq + x.h) * prm.parts + x.part) * prm.nb + qb) * N_EW + warp] = -t;
        }
        // the next unit and its row's values (the epilogue warps drain this one)
        int vn = -1;
        Unit xn;
        ok = take(vn, xn, ROLE_EW);
        if (!ok) break;
        if (vn >= 0) fetch(xn);
        g0 += x.NB;
        v = vn;
        x = xn;
      }
    }
  } else if (warp < WARP_EPI) {
    regs_dec<MMA_REGS>();
    if (warp == WARP_MMA) {
      // ================================================================ MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BS, false);   // S, dP: N = 64, K-major B
      constexpr uint32_t idesc_h = idesc_bf16_f32(BM, 64, true);    // dK_m, dQ_m: N = 64, MN-major B
      constexpr uint32_t idesc_dv = idesc_bf16_f32(BM, D, true);    // dV
      constexpr uint64_t SBLK16 = Ly::SBLK >> 4, SBOX16 = Ly::SBOX >> 4, BOX16 = Ly::BOX >> 4;
      const uint64_t r0 = smem_desc_sw128(sb + Ly::RES0, 16u, 1024u), r1 = smem_desc_sw128(sb + Ly::RES1, 16u, 1024u);
      const uint64_t a_kmaj = smem_desc_sw128(sb + Ly::A0, 16u, 1024u);
      const uint64_t a_mn = smem_desc_sw128(sb + Ly::A0, Ly::SBOX, 1024u);
      const uint64_t b_kmaj = smem_desc_sw128(sb + Ly::B0, 16u, 1024u);
      const uint64_t b_mn = smem_desc_sw128(sb + Ly::B0, Ly::SBOX, 1024u);
      // K-step kk of a K-major operand: 16 columns, box kk / 4, byte 32 (kk mod 4)
      auto res_off = [](int kk) { return (uint64_t)((kk >> 2) * BOX16 + (kk & 3) * 2); };
      auto str_off = [](int kk) { return (uint64_t)((kk >> 2) * SBOX16 + (kk & 3) * 2); };
      const uint32_t tm_qt = tmem + COL_Q, tm_gt = tm_qt + (uint32_t)(D / 2);
      auto issue_s = [&](int64_t gi) {  // both maps
        const uint64_t sd = a_kmaj + (uint64_t)(gi % Ly::NSA) * SBLK16;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            const int c = m * (D / 32) + kk;
            if (KV) tc_mma_ss_warp(tmem + COL_S + 64u * m, r0 + res_off(c), sd + str_off(c), idesc_s, kk > 0);
            else tc_mma_ts_warp(tmem + COL_S + 64u * m, tm_qt + (uint32_t)(c * 8), sd + str_off(c), idesc_s, kk > 0);
          }
        tc_commit_warp(bar(Ly::B_S));
      };
      auto issue_dp = [&](int64_t gi) {
        const int st = (int)(gi % Ly::NSB);
        const uint64_t sd = b_kmaj + (uint64_t)st * SBLK16;
        const uint32_t d = tmem + COL_DP + (KV ? 0u : (uint32_t)((gi & 1) * 64));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (KV) tc_mma_ss_warp(d, r1 + res_off(kk), sd + str_off(kk), idesc_s, kk > 0);
          else tc_mma_ts_warp(d, tm_gt + (uint32_t)(kk * 8), sd + str_off(kk), idesc_s, kk > 0);
        }
        tc_commit_warp(bar(Ly::B_DP + (KV ? 0 : (int)(gi & 1))));
        if (!KV) tc_commit_warp(bar(Ly::B_BE + st));  // V(gi) is read by this product only
      };
      auto issue_dv = [&](int64_t gi, bool first) {  // dV += A^T dO(gi)
        const int st = (int)(gi % Ly::NSB);
        const uint64_t sd = b_mn + (uint64_t)st * SBLK16;
#pragma unroll
        for (int kk = 0; kk < BS / 16; ++kk)
          tc_mma_ts_warp(tmem + COL_ACC, tmem + COL_A + (uint32_t)((gi & 1) * 32 + kk * 8), sd + (uint64_t)(kk * 128), idesc_dv,
                         (!first || kk > 0) ? 1u : 0u);
        tc_commit_warp(bar(Ly::B_BE + st));  // dO(gi): read by dP(gi) and dV(gi)
      };
      auto issue_half = [&](int64_t gi, bool first) {  // dK_m += dS_m^T Q_m(gi), or dQ_m += dS_m K_m(gi)
        const int st = (int)(gi % Ly::NSA);
        const uint32_t acc = tmem + (KV ? COL_DK : COL_ACC);
        const uint32_t ds = tmem + COL_DP + (KV ? 0u : (uint32_t)((gi & 1) * 64));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          // the map's 64-column box; at d = 64 both maps share one box and half of each product is used
          const uint64_t sd = a_mn + (uint64_t)st * SBLK16 + (D == 128 ? (uint64_t)m * SBOX16 : 0ull);
#pragma unroll
          for (int kk = 0; kk < BS / 16; ++kk)
            tc_mma_ts_warp(acc + 64u * m, ds + ds_col(m, kk), sd + (uint64_t)(kk * 128), idesc_h, (!first || kk > 0) ? 1u : 0u);
        }
        tc_commit_warp(bar(Ly::B_AE + st));  // Q(gi) or K(gi): read by S(gi) and here
      };
      auto wait_a = [&](int64_t gi) {
        return mbar_wait_warp(bar(Ly::B_AF + (int)(gi % Ly::NSA)), (uint32_t)((gi / Ly::NSA) & 1), prm.wait_limit_ns,
                              abort_flag, prm.status, ROLE_MMA, (int32_t)gi);
      };
      auto wait_b = [&](int64_t gi) {
        return mbar_wait_warp(bar(Ly::B_BF + (int)(gi % Ly::NSB)), (uint32_t)((gi / Ly::NSB) & 1), prm.wait_limit_ns,
                              abort_flag, prm.status, ROLE_MMA, (int32_t)gi);
      };
      auto wait1 = [&](int b, uint32_t parity) {
        return mbar_wait_warp(bar(b), parity, prm.wait_limit_ns, abort_flag, prm.status, ROLE_MMA, -1);
      };
      int nres = 0;
      // S and dP of a unit's first block, as soon as its resident operands are there
      auto start_unit = [&](const Unit& y, int64_t gi) -> bool {
        if (!wait1(KV ? Ly::B_RES : Ly::B_QTF, (uint32_t)(nres & 1))) return false;
        ++nres;
        if (!wait_a(gi)) return false;
        tc_fence_after();
        issue_s(gi);
        if (!wait_b(gi)) return false;
        tc_fence_after();
        issue_dp(gi);
        if (y.NB == 1) tc_commit_warp(bar(KV ? Ly::B_RESE : Ly::B_QTE));  // the unit's last S and dP are issued
        return true;
      };
      bool ok = run;
      int v = -1;
      Unit x;
      if (ok) ok = take(v, x, ROLE_MMA);
      if (ok && v >= 0) {
        ok = start_unit(x, 0);
      }
      int64_t g0 = 0;
      int k_unit = 0;
      while (ok && v >= 0) {
        const int NB = x.NB;
        for (int i = 0; i < NB && ok; ++i) {
          const int64_t gi = g0 + i;
          // S(gi) is in registers: S(gi + 1) may overwrite it.  (The last block's phase of this barrier is
          // not waited for, but it precedes the DS arrivals that are.)
          if (i + 1 < NB) {
            ok = wait1(Ly::B_SREAD, (uint32_t)(gi & 1)) && wait_a(gi + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(gi + 1);
            if (!KV) {  // the other dP buffer: dS(gi - 1) in it has been read by dQ(gi - 1), issued before
              ok = wait_b(gi + 1);
              if (!ok) break;
              tc_fence_after();
              issue_dp(gi + 1);
              if (i + 2 == NB) tc_commit_warp(bar(Ly::B_QTE));
            }
          }
          ok = wait1(Ly::B_DS + (int)(gi & 1), (uint32_t)((gi >> 1) & 1));  // (dkdv: and A)
          if (ok && i == 0 && k_unit > 0) ok = wait1(Ly::B_ACCE, (uint32_t)((k_unit - 1) & 1));  // accumulators copied out
          if (!ok) break;
          tc_fence_after();
          issue_half(gi, i == 0);
          if (KV) {
            if (i + 1 < NB) {  // in place of dS(gi), which dK(gi) has read; the elementwise warps wait for it next
              ok = wait_b(gi + 1);
              if (!ok) break;
              tc_fence_after();
              issue_dp(gi + 1);
              if (i + 2 == NB) tc_commit_warp(bar(Ly::B_RESE));  // the unit's last S and dP are issued
            }
            // A's buffer is written again at gi + 2, after S(gi + 2), which follows this product
            issue_dv(gi, i == 0);
          }
          if (i + 1 == NB) tc_commit_warp(bar(Ly::B_ACC));  // the unit's accumulators are complete
        }
        if (!ok) break;
        int vn = -1;
        ok = take(vn, x, ROLE_MMA);
        if (!ok) break;
        g0 += NB;
        ++k_unit;
        v = vn;
        if (v < 0) break;
        ok = start_unit(x, g0);
      }
      // exit-path drain: every MMA issued completes before TMEM is freed
      tc_commit_warp(bar(Ly::B_DRAIN));
      mbar_drain(bar(Ly::B_DRAIN), 0u, DRAIN_NS);
    } else if (warp == WARP_LOAD && lane == 0) {
      // ================================================================ producer
      bool ok = run;
      int np = 0;  // units published
      // a CTA's first unit is its own index, the others come from the counter; units without blocks are passed over
      auto next = [&]() { return prm.n_units > n_ctas ? (int)(n_ctas + atomicAdd(prm.counter, 1u)) : prm.n_units; };
      auto publish = [&](Unit& y) -> int {
        const int slot = np & 1;
        ok = mbar_wait(bar(Ly::B_UE + slot), (uint32_t)(((np >> 1) & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status,
                       ROLE_LOAD, -1);
        if (!ok) return -1;
        int u = np > 0 ? next() : cta;
        for (; u < prm.n_units; u = next()) {
          y = unit_of<KV>(u, prm);
          if (y.NB > 0) break;
          if (!KV)  // its share of lam's gradient
            for (int w = 0; w < N_EW; ++w)
              prm.dlam_part[((((int64_t)y.b * prm.Hq + y.h) * prm.parts + y.part) * prm.nb + y.blk) * N_EW + w] = 0.f;
        }
        if (u >= prm.n_units) u = -1;
        put_unit(unit_ring + 16 * slot, u, y);
        mbar_arrive(bar(Ly::B_UF + slot));
        ++np;
        return u;
      };
      int nres = 0;
      int64_t ga = 0, gb = 0;  // streamed blocks issued
      Unit x{}, y{};
      int u = ok ? publish(x) : -1;
      while (ok && u >= 0) {
        // publish the following unit now and pull its resident rows into L2
        const int un = publish(y);
        if (!ok) break;
        const int H = KV ? prm.Hkv : prm.Hq;
        if (un >= 0) {
          const int32_t pn = y.b * H + y.h;
          for (int c = 0; c < D / 64; ++c) {
            tma_prefetch_l2_3d(&tmR0, c * 64, y.blk * BM, pn);
            tma_prefetch_l2_3d(&tmR1, c * 64, y.blk * BM, pn);
          }
        }
        // resident operands: the previous unit's must have been used (dkdv) or copied into TMEM (dq)
        ok = mbar_wait(bar(Ly::B_RESE), (uint32_t)((nres & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, u);
        if (!ok) break;
        const int32_t res = x.b * H + x.h;
        mbar_expect_tx(bar(Ly::B_RES), 2 * Ly::TILE);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(sb + Ly::RES0 + (uint32_t)c * Ly::BOX, &tmR0, c * 64, x.blk * BM, res, bar(Ly::B_RES));
          tma_load_3d(sb + Ly::RES1 + (uint32_t)c * Ly::BOX, &tmR1, c * 64, x.blk * BM, res, bar(Ly::B_RES));
        }
        ++nres;
        QCursor qc;
        if (KV) qc.start(prm, x);
        for (int i = 0; i < x.NB && ok; ++i) {
          if (KV && i > 0) qc.step(prm);
          const int blk = KV ? qc.qb : x.start + i;
          const int32_t z = KV ? x.b * prm.Hq + qc.h : x.b * prm.Hkv + x.h / g;
          const int sa = (int)(ga % Ly::NSA), st = (int)(gb % Ly::NSB);
          if (ga >= Ly::NSA) {
            ok = mbar_wait(bar(Ly::B_AE + sa), (uint32_t)((ga / Ly::NSA - 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                           ROLE_LOAD, i);
            if (!ok) break;
          }
          mbar_expect_tx(bar(Ly::B_AF + sa), Ly::SBLK);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sb + Ly::A0 + (uint32_t)sa * Ly::SBLK + (uint32_t)c * Ly::SBOX, &tmA, c * 64, blk * BS, z, bar(Ly::B_AF + sa));
          ++ga;
          if (gb >= Ly::NSB) {
            ok = mbar_wait(bar(Ly::B_BE + st), (uint32_t)((gb / Ly::NSB - 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                           ROLE_LOAD, i);
            if (!ok) break;
          }
          mbar_expect_tx(bar(Ly::B_BF + st), Ly::SBLK);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sb + Ly::B0 + (uint32_t)st * Ly::SBLK + (uint32_t)c * Ly::SBOX, &tmB, c * 64, blk * BS, z, bar(Ly::B_BF + st));
          ++gb;
        }
        u = un;
        x = y;
      }
      // exit-path drain: every load issued lands before the CTA exits
      if (nres > 0) mbar_drain(bar(Ly::B_RES), (uint32_t)((nres - 1) & 1), DRAIN_NS);
      for (int64_t j = (ga > Ly::NSA ? ga - Ly::NSA : 0); j < ga; ++j)
        mbar_drain(bar(Ly::B_AF + (int)(j % Ly::NSA)), (uint32_t)((j / Ly::NSA) & 1), DRAIN_NS);
      for (int64_t j = (gb > Ly::NSB ? gb - Ly::NSB : 0); j < gb; ++j)
        mbar_drain(bar(Ly::B_BF + (int)(j % Ly::NSB)), (uint32_t)((j / Ly::NSB) & 1), DRAIN_NS);
    }
  } else {
    regs_dec<EPI_REGS>();
    if constexpr (!KV) {
      // ================================================================ epilogue (dq)
      // Per unit: copy its Q and dO from shared memory into TMEM as soon as the previous unit's last S
      // and dP are done with the TMEM copy, releasing the shared buffers to the producer; then drain
      // the previous unit's dQ while the other roles run this one.
      const int wq = warp & 3;
      const int r = wq * 32 + lane;  // this thread's row of the block
      const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
      const uint32_t tm_dq = tmem + lane_base + COL_ACC;
      const uint32_t tm_qt = tmem + lane_base + COL_Q, tm_gt = tm_qt + (uint32_t)(D / 2);
      bool ok = run;
      int v = -1, k_unit = 0, ncopy = 0;
      Unit x;
      // row r of a 128 x D block in 64-column boxes with 128-byte swizzle (16-byte chunk j of a row at
      // chunk j ^ (r mod 8)), packed two columns per TMEM column
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
        if (ncopy > 0 && !mbar_wait_warp(bar(Ly::B_QTE), (uint32_t)((ncopy - 1) & 1), prm.wait_limit_ns, abort_flag,
                                         prm.status, ROLE_EPI, -1))
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
      if (ok) ok = take(v, x, ROLE_EPI);
      if (ok && v >= 0) ok = copy_in();
      while (ok && v >= 0) {
        int vn = -1;
        Unit xn;
        ok = take(vn, xn, ROLE_EPI);
        if (!ok) break;
        if (vn >= 0) {
          ok = copy_in();
          if (!ok) break;
        }
        const int64_t row0 = (((int64_t)x.b * prm.Hq + x.h) * prm.parts + x.part) * S + (int64_t)x.blk * BM + wq * 32;
        const int rows_valid = (int)max((int64_t)0, min((int64_t)32, S - ((int64_t)x.blk * BM + wq * 32)));
        __nv_bfloat16* dst = prm.out0 + (((int64_t)x.b * prm.Hq + x.h) * S + (int64_t)x.blk * BM + r) * D;
        ok = mbar_wait_warp(bar(Ly::B_ACC), (uint32_t)(k_unit & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_EPI, -1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float t[32];
          // at d = 64 the second map's half lies in the second half of its 64-wide product
          tmem_ld32(tm_dq + (uint32_t)(D == 64 ? c * 3 : c), t);
          tc_wait_ld();
          if (c + 32 == D) arrive(Ly::B_ACCE);
          if (prm.parts > 1) store_rows<D>(t, prm.scale, prm.part0, row0, rows_valid, c, lane);
          else if (lane < rows_valid) store_bf16(t, prm.scale, dst + c);
        }
        ++k_unit;
        v = vn;
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

// Tensor maps of a 128-row and of a 64-row box for each of Q, K, V and dO.
struct Maps {
  CUtensorMap q, k, v, g;
};
template <int D>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    diff_bwd_kernel(const __grid_constant__ Maps rows128, const __grid_constant__ Maps rows64,
                    const __grid_constant__ Params kv, const __grid_constant__ Params dq, const int kv_ctas) {
  if ((int)blockIdx.x < kv_ctas)
    run_pass<D, true>(rows128.k, rows128.v, rows64.q, rows64.g, kv, (int)blockIdx.x, kv_ctas);
  else
    run_pass<D, false>(rows128.q, rows128.g, rows64.k, rows64.v, dq, (int)blockIdx.x - kv_ctas, (int)gridDim.x - kv_ctas);
}

// out[head][row] = sum over its block's parts, in order, rounded once; blockIdx.y picks one of up to three tensors
struct SumArgs {
  const float4* part[3];  // [head][parts][S][D]
  uint2* out[3];
  int64_t heads[3];
  int32_t parts[3], kv[3];
  int64_t S;
  int32_t row4, ns, causal, group;  // 16-byte pieces of a row
  const int32_t* status;
};
__global__ void __launch_bounds__(256) sum_parts(const SumArgs a) {
  wait_for_kernel_before();
  if (*reinterpret_cast<const volatile int32_t*>(a.status) != 0) return;
  const int w = blockIdx.y;
  const int64_t per = a.S * a.row4, total = a.heads[w] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t head = i / per, at = i - head * per;
    const int blk = (int)(at / a.row4 / BM);
    const int n = a.kv[w] ? blocks_of<true>(blk, a.ns, a.causal, a.group) : blocks_of<false>(blk, a.ns, a.causal, a.group);
    const int k = min(a.parts[w], n);
    const float4* src = a.part[w] + head * a.parts[w] * per + at;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < k; ++p) {
      const float4 x = __ldcs(src + p * per);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    a.out[w][i] = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
  }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode(std::string* err) {
  static EncodeTiledFn fn = nullptr;
  if (fn) return fn;
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !ptr) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return nullptr;
  }
  fn = reinterpret_cast<EncodeTiledFn>(ptr);
  return fn;
}

// [parts][L][d] bf16 rows, boxes of box_rows x 64 columns with 128-byte swizzle; rows of a box past L
// are zeros.
static bool make_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, uint64_t L, uint64_t parts, int d, int box_rows,
                     std::string* err) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)L * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *err = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

static int64_t fill(Params& prm, const DiffArgs& a, const DiffWorkspace& w, int sms, bool kv, int parts) {
  prm.lse = a.LSE;
  prm.dsum = reinterpret_cast<const float*>(a.ws + w.dsum);
  prm.lam = static_cast<const __nv_bfloat16*>(a.lam);
  prm.out0 = static_cast<__nv_bfloat16*>(kv ? a.dK : a.dQ);
  prm.out1 = static_cast<__nv_bfloat16*>(a.dV);
  prm.part0 = reinterpret_cast<float*>(a.ws + (kv ? w.dk_part : w.dq_part));
  prm.part1 = reinterpret_cast<float*>(a.ws + w.dv_part);
  prm.dlam_part = reinterpret_cast<float*>(a.ws + w.dlam_part);
  prm.status = a.status;
  prm.counter = reinterpret_cast<uint32_t*>(a.ws + w.counters) + (kv ? 0 : 64);
  prm.S = a.S;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.parts = parts;
  prm.nb = (int32_t)((a.S + BM - 1) / BM);
  prm.ns = (int32_t)((a.S + BS - 1) / BS);
  const int64_t tiles = (int64_t)prm.nb * a.B * (kv ? a.Hkv : a.Hq);
  prm.n_tiles = (int32_t)tiles;
  prm.n_units = (int32_t)(tiles * parts);
  prm.causal = a.causal;
  // causal units differ in length: enough lanes together for about three times the grid, so that the last ones are short
  prm.batch = a.causal ? (int32_t)std::min<int64_t>(tiles / prm.nb, (3LL * sms + prm.nb - 1) / prm.nb) : 1;
  prm.lam_n = a.lam_n;
  prm.scale = a.scale;
  prm.scale_log2 = a.scale_log2;
  prm.wait_limit_ns = a.wait_limit_ns;
  return tiles * parts;
}

static bool make_maps(EncodeTiledFn enc, Maps* m, const DiffArgs& a, int box_rows, std::string* err) {
  const uint64_t S = (uint64_t)a.S, nq = (uint64_t)a.B * a.Hq, nk = (uint64_t)a.B * a.Hkv;
  return make_map(enc, &m->q, a.Q, S, nq, a.d, box_rows, err) && make_map(enc, &m->g, a.dO, S, nq, a.d, box_rows, err) &&
         make_map(enc, &m->k, a.K, S, nk, a.d, box_rows, err) && make_map(enc, &m->v, a.V, S, nk, a.d, box_rows, err);
}

template <int D>
static int launch(const DiffArgs& a, const DiffWorkspace& w, int sms, BwdParts parts, cudaStream_t st, std::string* err) {
  Params kv{}, dq{};
  const int64_t kv_units = fill(kv, a, w, sms, true, parts.kv), dq_units = fill(dq, a, w, sms, false, parts.dq);
  if (kv_units > 0x3fffffff || dq_units > 0x3fffffff) {
    *err = "too many work units for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  EncodeTiledFn enc = get_encode(err);
  if (!enc) return (int)cudaErrorNotSupported;
  Maps rows128{}, rows64{};
  if (!make_maps(enc, &rows128, a, BM, err) || !make_maps(enc, &rows64, a, BS, err)) return (int)cudaErrorInvalidValue;
  auto kern = diff_bwd_kernel<D>;
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
      *err = "differential backward built with " + std::to_string(fa.numRegs) +
             " registers per thread, fewer than its warpgroups' register split needs";
      return (int)cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) once.mark(dev);
  }
  // with a CTA for every unit a pass does not read its counter
  if (e == cudaSuccess && (kv_units > sms || dq_units > sms)) e = cudaMemsetAsync(kv.counter, 0, 512, st);
  if (e == cudaSuccess) {
    const int kv_ctas = (int)std::min<int64_t>(kv_units, sms), dq_ctas = (int)std::min<int64_t>(dq_units, sms);
    e = launch_behind(kern, dim3((unsigned)(kv_ctas + dq_ctas)), NUM_THREADS, Layout<D>::TOTAL, st, rows128, rows64, kv, dq, kv_ctas);
  }
  if (e == cudaSuccess && (parts.kv > 1 || parts.dq > 1)) {
    SumArgs s{};
    int n = 0;
    auto add = [&](float* part, void* out, int heads, int p, bool is_kv) {
      s.part[n] = reinterpret_cast<const float4*>(part);
      s.out[n] = static_cast<uint2*>(out);
      s.heads[n] = (int64_t)a.B * heads;
      s.parts[n] = p;
      s.kv[n++] = is_kv;
    };
    if (parts.kv > 1) {
      add(kv.part0, a.dK, a.Hkv, parts.kv, true);
      add(kv.part1, a.dV, a.Hkv, parts.kv, true);
    }
    if (parts.dq > 1) add(dq.part0, a.dQ, a.Hq, parts.dq, false);
    s.S = a.S;
    s.row4 = D / 4;
    s.ns = kv.ns;
    s.causal = a.causal;
    s.group = a.Hq / a.Hkv;
    s.status = a.status;
    const int64_t most = (int64_t)a.B * a.Hq * a.S * s.row4;
    e = launch_behind(sum_parts, dim3((unsigned)std::min<int64_t>((most + 255) / 256, 152 * 8), (unsigned)n), 256, 0, st, s);
  }
  if (e != cudaSuccess) *err = std::string("diff_bwd launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace dbtc

// Parts of the passes' units: those with the least estimated time, in streamed blocks (about 1 us each).  A unit
// takes UNIT blocks besides its own; the parts' sums SUM, and what their 8 bytes a value (written and read) take at
// 5 TB/s for d = 128.  With an SM for every unit the longest decides; with
// more units than that, their whole work shared out, and half a unit for the uneven end.  Measured, us of the
// backward call, whole / cut: 16 heads on one, 1,192 tokens 372 / 81; one head of 8,192 161 / 114, of 2,304 54 / 37;
// 2 x 4 heads of 1,000 tokens, where whole units just fill the GPU, 31 / 35 in halves.
BwdParts diff_bwd_parts(int64_t S, int32_t B, int32_t Hq, int32_t Hkv, bool causal) {
  constexpr int SMS = 152;  // the whole GPU's: so the workspace's size needs no device
  constexpr double UNIT = 10, SUM = 3, ROW = 128 * 8 / 5e6;
  const int64_t nb = (S + dbtc::BM - 1) / dbtc::BM, ns = (S + dbtc::BS - 1) / dbtc::BS, group = std::max(1, Hq / Hkv);
  const double tiles_kv = (double)nb * B * Hkv, tiles_dq = (double)nb * B * Hq;
  if (tiles_kv > SMS) return {1, 1};  // several waves of whole units
  const double blocks = 2.0 * (double)(causal ? nb * (nb + 1) : nb * ns) * B * Hq;  // of both passes: the same pairs
  BwdParts best{1, 1};
  double least = 1e300;
  constexpr int ks[] = {1, 2, 3, 4, 6, 8, 11, 16};
  for (int kv : ks) {
    const double len_kv = (double)((ns * group + kv - 1) / kv);
    for (int dq : ks) {
      const double unit = UNIT + std::max(len_kv, (double)((ns + dq - 1) / dq)), units = tiles_kv * kv + tiles_dq * dq;
      const double shared = (units * UNIT + blocks) / SMS;
      const double rows = (kv > 1 ? 2.0 * kv * B * Hkv * S : 0) + (dq > 1 ? (double)dq * B * Hq * S : 0);
      const double t = (units <= SMS ? unit : std::max(unit, shared) + unit / 2) + (rows > 0 ? SUM + rows * ROW : 0);
      if (t < least) least = t, best = {kv, dq};
    }
  }
  return best;
}

int launch_diff_bwd_tc(const DiffArgs& a, const DiffWorkspace& w, int sms, BwdParts parts, void* stream, std::string* err) {
  cudaStream_t st = (cudaStream_t)stream;
  return a.d == 128 ? dbtc::launch<128>(a, w, sms, parts, st, err) : dbtc::launch<64>(a, w, sms, parts, st, err);
}

}  // namespace mesh
