// Differential attention forward on the 5th-generation tensor cores (sm_103a), bf16 inputs.
//
//   O = P_1 V - lam P_2 V,  P_m = softmax(scale q_m k_m^T),  q = [q_1 | q_2], k = [k_1 | k_2] by columns.
//
// The two maps of a query tile take the places that two query tiles have in the plain tile kernel: both
// warpgroups of softmax warps own the same 128 query rows, one map each, with the online softmax
// of that kernel (a running reference that moves only when a block's maximum outgrows it by 2^8).
// One K block and one V block in shared memory serve both maps: the score products take the half of
// Q's and K's columns that is their map's (K = d/2 each), the P_m V products take the same V.
// At the end both accumulators lie in the same TMEM lanes, so each warpgroup reads both of them
// for one half of the columns and writes O = O_1 / l_1 - lam O_2 / l_2 (and O_2 for the backward
// pass) rounded once.
//
// A work unit is (batch, KV head, query head of the group, 128-row query tile); causal units go heaviest
// first within batches of heads that fill the grid a few times (Params::batch).  Where tiles would
// leave most SMs idle, all of them (few tiles) or those of the last, mostly empty wave (equal tiles without a
// mask) are cut into parts of their keys: a part leaves its normalised outputs and LSEs, which
// merge_parts_kernel adds up (choose_parts).
//
// Per 128 x 128 block and head: 2 x 4 score products and 2 x 8 PV products of 64 cycles each at
// d = 128 (1,536 cycles), 32,768 exponentials.  P is rounded to bf16 for its product (2^-8 relative
// a term), everything else is fp32.  That rounding costs 1.9e-3 of O's norm beside the 1.7e-3 of O's own (2.6e-3
// together, as the same rounding in 64-bit arithmetic gives); a second piece of P would take it away for 1,024 cycles of
// products more a block, 2,560 against the softmax's 2,400.
//
// Measured (d = 128, 16 heads, 16,384 tokens, calls in a row): causal 1.13 to 1.18 ms, 1,400 to 1,460 TFLOP/s; without a
// mask, on 4 KV heads, 2.18 ms, 1,510 TFLOP/s (0.80 of the bf16 burst rate).  Bound by the softmax warps: a block takes them
// 2,350-2,450 cycles for its 1,536 cycles of products, though no pipe is full (MUFU 40 % busy, FMA 22 %): both softmax
// warps of a sub-partition run the same phase, and in the sub-partition of the MMA warp, whose products' issue takes
// dispatch slots, the exponentials of 64 keys take 1,000 cycles where they take 640 in the others.
// Slower (no mask): two warps a row 2.70 ms, 64-key steps with two score buffers a map 2.70 ms, P handed
// over in halves 2.53 ms, an MMA issuer for each map 2.78 ms, products issued in paced groups of four 2.57 ms.
//
// Persistent grid, one CTA per SM; warps 0-7 softmax, warp 8 MMA issuer, warp 9 producer, warps 10-11
// idle.  TMEM (512 columns): S_1 | S_2 | O_1 | O_2; P_m overwrites S_m.  K, V and Q tiles come by head
// ([heads][rows][d] tensor maps): rows past a head's end are zeros.
// Every mbarrier wait is bounded: a timeout records MESH_ATTN_ERR_DEVICE_TIMEOUT in the status
// block, every role of the CTA stops, in-flight copies and MMAs are drained and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace dtc {

constexpr int BM = 128;  // query rows per tile = TMEM lanes
constexpr int BN = 128;  // keys per KV block
constexpr int NST = 2;   // K/V ring stages
constexpr int NUM_THREADS = 384;
constexpr int SOFTMAX_REGS = 200;  // 2 x 128 x 200 + 128 x 104 <= 384 x 168 registers at launch
constexpr int OTHER_REGS = 104;
constexpr int WARP_MMA = 8;
constexpr int WARP_LOAD = 9;
constexpr float LOG2_RESCALE = 8.0f;
// Row sum of one block accepted without a max pass: every term is then at most 2^16, and a sum
// this large implies a row maximum more than 2^LOG2_RESCALE above the reference (2^16 / BN > 2^8).
constexpr float SUM_ACCEPT = 65536.0f;
constexpr int MAX_PARTS = 16;          // of a tile (choose_parts)
constexpr int64_t DRAIN_NS = 200000000;  // exit-path waits for copies in flight

// roles recorded with an error
constexpr int ROLE_SOFTMAX = 1, ROLE_MMA = 2, ROLE_LOAD = 3;

template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // bytes of one Q tile / K block / V block
  static constexpr uint32_t BOX = BM * 64 * 2;  // one 128 x 64 bf16 TMA box (16 KB)
  static constexpr uint32_t Q_OFF = 0;          // two Q tiles: a unit's and the next unit's
  static constexpr uint32_t K_OFF = Q_OFF + 2 * TILE;
  static constexpr uint32_t V_OFF = K_OFF + NST * TILE;
  static constexpr uint32_t EPI_OFF = V_OFF + NST * TILE;  // 8 softmax warps x 4 KB
  static constexpr uint32_t BAR_OFF = EPI_OFF + 8 * 4096;
  static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_KEMPTY = B_KFULL + NST,
                       B_VFULL = B_KEMPTY + NST, B_VEMPTY = B_VFULL + NST, B_SFULL = B_VEMPTY + NST,
                       B_PFULL = B_SFULL + 2, B_OFINAL = B_PFULL + 2, B_OFREE = B_OFINAL + 1,
                       B_INV = B_OFREE + 1, B_UFULL = B_INV + 1, B_UEMPTY = B_UFULL + 2, B_DRAIN = B_UEMPTY + 2,
                       NBARS = B_DRAIN + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBARS * 8;  // tmem base, abort flag, unit ring[2]
  static constexpr uint32_t INV_OFF = MISC_OFF + 16;         // 1 / l of both maps, [2][128] fp32
  static constexpr uint32_t TOTAL = INV_OFF + 2 * BM * 4;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
};

struct Params {
  const TablesHeader* header;
  uint64_t tag;
  const __nv_bfloat16* lam;
  __nv_bfloat16* o;  // O, O2 (or NULL) and LSE
  __nv_bfloat16* o2;
  float* lse;
  float* part_o;  // of the tiles in parts: [part][map][128][D], and their LSEs [part][map][128]
  float* part_lse;
  int32_t* status;
  uint32_t* counter;
  int64_t S;
  int32_t B, Hq, Hkv, nqt, n_tiles, n_whole, parts, n_units, causal, lam_n;
  int32_t batch;  // heads whose tiles are numbered together
  float scale_log2;
  int64_t wait_limit_ns;
};

// What every role derives from a unit index: the first n_whole units are whole tiles, of the other tiles
// each has `parts`.  A lane is (batch, query head); tiles are numbered batch of lanes by batch, within it
// row by row (causal: from the longest), within a row lane by lane.  With batch = 1 the units running
// at once share one KV head's keys in L2; a few lanes together keep the last units short where
// their lengths differ.
struct Unit {
  int b, h, hk, qt;
  int part;      // index of its partial outputs, or -1: a whole tile
  int blk0, NB;  // its 128-key blocks; a part may be left without
};

// Parts of a tile that sees nbk blocks, and what tile x is.
__device__ __forceinline__ int parts_of(int nbk, const Params& prm) { return min(prm.parts, nbk); }
__device__ __forceinline__ Unit decode_tile(int t, const Params& prm) {
  Unit x;
  const int per = prm.batch * prm.nqt, first = t / per * prm.batch;
  const int lanes = min(prm.batch, prm.n_tiles / prm.nqt - first);  // the last batch may be smaller
  t %= per;
  x.qt = t / lanes;
  if (prm.causal) x.qt = prm.nqt - 1 - x.qt;
  t = first + t % lanes;
  x.h = t % prm.Hq;
  x.b = t / prm.Hq;
  x.hk = x.h / (prm.Hq / prm.Hkv);
  x.part = -1;
  x.blk0 = 0;
  x.NB = prm.causal ? min(prm.nqt, x.qt + 1) : prm.nqt;
  return x;
}
__device__ __forceinline__ Unit decode(int u, const Params& prm) {
  if (u < prm.n_whole) return decode_tile(u, prm);
  const int e = u - prm.n_whole;
  Unit x = decode_tile(prm.n_whole + e / prm.parts, prm);
  const int k = parts_of(x.NB, prm), i = e % prm.parts, nbk = x.NB;
  x.part = e;
  x.blk0 = min(i, k) * nbk / k;
  x.NB = min(i + 1, k) * nbk / k - x.blk0;
  return x;
}

template <int D>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    diff_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const Params prm) {
  using Ly = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;  // 1024-aligned base (128-byte swizzle atoms)
  uint8_t* smem = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + Ly::BAR_OFF + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::MISC_OFF);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC_OFF + 4);
  volatile int32_t* unit_ring = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC_OFF + 8);
  const int64_t S = prm.S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(Ly::B_KFULL + s), 1);
      mbar_init(bar(Ly::B_KEMPTY + s), 1);
      mbar_init(bar(Ly::B_VFULL + s), 1);
      mbar_init(bar(Ly::B_VEMPTY + s), 1);
    }
    mbar_init(bar(Ly::B_OFINAL), 1);
    mbar_init(bar(Ly::B_OFREE), 2 * BM);  // every softmax thread has copied what it needs of O_1 and O_2
    mbar_init(bar(Ly::B_INV), 2 * BM);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(Ly::B_QFULL + t), 1);
      mbar_init(bar(Ly::B_QEMPTY + t), 1);
      mbar_init(bar(Ly::B_SFULL + t), 1);
      mbar_init(bar(Ly::B_PFULL + t), BM);
      mbar_init(bar(Ly::B_UFULL + t), 1);
      mbar_init(bar(Ly::B_UEMPTY + t), 1 + 8);  // one lane of the MMA warp and of each softmax warp
    }
    mbar_init(bar(Ly::B_DRAIN), 1);
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
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ================================================================ softmax warpgroups
    regs_inc<SOFTMAX_REGS>();
    const int t = warp >> 2;  // map
    const int wq = warp & 3;
    const int row = wq * 32 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tm_s = tmem + lane_base + (uint32_t)(t * 128);
    const uint32_t tm_o = tmem + lane_base + 256u + (uint32_t)(t * 128);
    float* epi = reinterpret_cast<float*>(smem + Ly::EPI_OFF + (uint32_t)warp * 4096u);
    float* inv_s = reinterpret_cast<float*>(smem + Ly::INV_OFF);
    int nu = 0, cnt = 0, uses = 0;
    bool ok = true;
    while (ok) {
      const int slot = nu & 1;
      ok = mbar_wait(bar(Ly::B_UFULL + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                     ROLE_SOFTMAX, -1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int u = unit_ring[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_UEMPTY + slot));
      ++nu;
      if (u < 0) break;
      const Unit x = decode(u, prm);
      if (x.NB == 0) continue;
      const int a_t = x.qt;
      float m_used = -INFINITY, l_sum = 0.f;
      {
        for (int jb = x.blk0; jb < x.blk0 + x.NB; ++jb, ++cnt) {
          ok = mbar_wait(bar(Ly::B_SFULL + t), (uint32_t)(cnt & 1), prm.wait_limit_ns, abort_flag, prm.status,
                         ROLE_SOFTMAX, u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          // mask: causal diagonal block (key column > query row) and keys past the end
          const int kv_valid = (int)min((int64_t)BN, S - (int64_t)jb * BN);
          int lim = prm.causal && jb == a_t ? row : BN - 1;
          lim = min(lim, kv_valid - 1);
          // The exponentials use the row's running reference m_used, which only ever grows.  A
          // block whose row maximum stays within 2^LOG2_RESCALE of it needs no maximum at all, so
          // the common case skips the max pass: exponentiate against m_used and accept the block
          // when its row sum is at most SUM_ACCEPT (every term is then bounded as well).  A row
          // without a reference yet (first block of the unit), or a block whose sum is too large
          // or not finite, takes the row maximum first, raising m_used (and rescaling O and l)
          // when it grew by more than 2^LOG2_RESCALE, and the exponentials are redone.
          bool need_max = __any_sync(0xffffffffu, m_used == -INFINITY);
          float factor = 1.f, blk = 0.f;
          uint32_t pk[BN / 2];
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            // S_t stays in TMEM until P_t is written, so a second pass reloads it rather than
            // keeping 128 scores live across the pass
            float s[BN];
#pragma unroll
            for (int c = 0; c < BN; c += 32) tmem_ld32(tm_s + (uint32_t)c, s + c);
            tc_wait_ld();
            if (lim < BN - 1) {
#pragma unroll
              for (int c = 0; c < BN; ++c)
                if (c > lim) s[c] = -INFINITY;
            }
            if (need_max) {
              // row max: four independent chains of 3-input max
              float mc[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float v = max3f(s[32 * q], s[32 * q + 1], s[32 * q + 2]);
#pragma unroll
                for (int i = 3; i + 1 < 32; i += 2) v = max3f(v, s[32 * q + i], s[32 * q + i + 1]);
                mc[q] = fmaxf(v, s[32 * q + 31]);
              }
              const float m_new = fmaxf(max3f(mc[0], mc[1], mc[2]), mc[3]) * prm.scale_log2;
              if (m_new > -INFINITY) {
                if (m_used == -INFINITY) {
                  m_used = m_new;
                } else if (m_new > m_used + LOG2_RESCALE) {
                  factor *= fast_exp2(m_used - m_new);
                  m_used = m_new;
                }
              }
            }
            const float mref = (m_used == -INFINITY) ? 0.f : m_used;
            // p = 2^(s * scale * log2 e - m): two elements per FMA, four independent sum chains
            const uint64_t sc2 = f2_pack(prm.scale_log2, prm.scale_log2);
            const uint64_t nm2 = f2_pack(-mref, -mref);
            uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c = 0; c < BN / 2; ++c) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[2 * c], s[2 * c + 1]), sc2, nm2), x0, x1);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              acc2[c & 3] = f2_add(acc2[c & 3], f2_pack(p0, p1));
              pk[c] = pack_bf16x2(p0, p1);
            }
            float sa, sb2;
            f2_unpack(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])), sa, sb2);
            blk = sa + sb2;
            // NaN fails the comparison: a NaN row takes the max pass once and is then accepted
            if (pass == 1 || __all_sync(0xffffffffu, blk <= SUM_ACCEPT)) break;
            need_max = true;
          }
          if (__any_sync(0xffffffffu, factor != 1.f)) {
            // O_t holds every earlier PV product of this unit: S_t(j) was issued after
            // PV_t(j-1) and its completion covers all earlier tensor-core work.
            l_sum *= factor;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(tm_o + (uint32_t)c, o);
              tc_wait_ld();
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * factor);
              tmem_st32(tm_o + (uint32_t)c, w);
            }
          }
          l_sum += blk;
          tmem_st32(tm_s, pk);
          tmem_st32(tm_s + 32u, pk + 32);
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(bar(Ly::B_PFULL + t));
        }
      }
      if (!ok) break;
      ok = mbar_wait(bar(Ly::B_OFINAL), (uint32_t)(uses & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_SOFTMAX, u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const int64_t row_local = (int64_t)a_t * BM + row;
      const int64_t wrow0 = row_local - lane;  // warp's first row
      // a row without a visible key: O_m = 0, LSE = -inf (a NaN sum stays NaN)
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      const float lse = l_sum == 0.f ? -INFINITY : (m_used + log2f(l_sum)) * 0.69314718055994531f;
      if (x.part < 0) {
        // ---- a whole tile: this warpgroup's half of the columns of both maps.  1 / l of the other map comes
        // through shared memory; it is written after OFINAL, which the previous unit's readers precede
        // (the products behind OFINAL waited for their OFREE).
        constexpr int CW = D / 2, NC = CW / 8;  // columns, 16-byte pieces of a row
        inv_s[t * BM + row] = inv;
        mbar_arrive(bar(Ly::B_INV));
        ok = mbar_wait(bar(Ly::B_INV), (uint32_t)(uses & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_SOFTMAX, u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float i1 = inv_s[row], i2 = inv_s[BM + row];
        float o1[CW], o2[CW];
        const uint32_t tm = tmem + lane_base + 256u + (uint32_t)(t * CW);
#pragma unroll
        for (int c = 0; c < CW; c += 32) {
          tmem_ld32(tm + (uint32_t)c, o1 + c);
          tmem_ld32(tm + 128u + (uint32_t)c, o2 + c);
        }
        tc_wait_ld();
        tc_fence_before();
        mbar_arrive(bar(Ly::B_OFREE));
        ++uses;
        const float lam = __bfloat162float(prm.lam[prm.lam_n == 1 ? 0 : x.h]);
        const int64_t grow = ((int64_t)x.b * prm.Hq + x.h) * S;  // the head's first row
        uint32_t w[CW / 2];
        uint4* stage = reinterpret_cast<uint4*>(epi);
        // 32 rows through the shared stage, so that each store writes whole 128-byte (64 at d = 64) row pieces
        auto put = [&](__nv_bfloat16* out) {
          __syncwarp();
#pragma unroll
          for (int q = 0; q < NC; ++q)
            stage[lane * NC + (q ^ (lane & (NC - 1)))] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int r = i * (32 / NC) + lane / NC, q = lane % NC;
            const uint4 v = stage[r * NC + (q ^ (r & (NC - 1)))];
            if (wrow0 + r < S)
              *reinterpret_cast<uint4*>(out + (grow + wrow0 + r) * D + t * CW + q * 8) = v;
          }
        };
#pragma unroll
        for (int c = 0; c < CW; c += 2) {
          o2[c] *= i2;
          o2[c + 1] *= i2;
          w[c / 2] = pack_bf16x2(fmaf(-lam, o2[c], o1[c] * i1), fmaf(-lam, o2[c + 1], o1[c + 1] * i1));
        }
        put(prm.o);
        if (prm.o2) {
#pragma unroll
          for (int c = 0; c < CW; c += 2) w[c / 2] = pack_bf16x2(o2[c], o2[c + 1]);
          put(prm.o2);
        }
        if (row_local < S) prm.lse[(((int64_t)x.b * prm.Hq + x.h) * 2 + t) * S + row_local] = lse;
        continue;
      }
      // ---- a part: this map's normalised output of it
      float o[D];
#pragma unroll
      for (int c = 0; c < D; c += 32) tmem_ld32(tm_o + (uint32_t)c, o + c);
      tc_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(Ly::B_OFREE));
      ++uses;
      const int64_t prow = ((int64_t)x.part * 2 + t) * BM + row;
      float* dst0 = prm.part_o + (prow - lane) * D;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        // 32 rows x 32 columns: 16-byte chunks swizzled by row, read back 4 rows per store
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(epi + lane * 32 + ((q ^ (lane & 7)) * 4)) =
              make_float4(o[c + 4 * q] * inv, o[c + 4 * q + 1] * inv, o[c + 4 * q + 2] * inv, o[c + 4 * q + 3] * inv);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3), qq = lane & 7;
          const float4 v = *reinterpret_cast<const float4*>(epi + r * 32 + ((qq ^ (r & 7)) * 4));
          if (wrow0 + r < S) *reinterpret_cast<float4*>(dst0 + (int64_t)r * D + c + qq * 4) = v;
        }
        __syncwarp();
      }
      if (row_local < S) prm.part_lse[prow] = lse;
    }
  } else {
    regs_dec<OTHER_REGS>();
    if (warp == WARP_MMA) {
      // ================================================================ MMA issuer
      // The whole warp runs this loop converged; tcgen05.mma and tcgen05.commit are issued by
      // one elected lane (tc_*_warp), every wait is warp-uniform (mbar_wait_warp).
      constexpr uint32_t idesc_qk = idesc_bf16_f32(BM, BN, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, true);
      // Base descriptors are built once; per instruction only the start-address field (the
      // low 14 bits, address / 16) advances by a compile-time offset.  Shared addresses stay
      // below 256 KB, so the addition never carries out of that field.  Keeping the issuing
      // warp's work per MMA to a few independent adds on uniform values is what lets one warp
      // keep the tensor pipe fed.
      const uint64_t q_desc0 = smem_desc_sw128(sb + Ly::Q_OFF, 16u, 1024u);
      const uint64_t k_desc0 = smem_desc_sw128(sb + Ly::K_OFF, 16u, 1024u);
      const uint64_t v_desc0 = smem_desc_sw128(sb + Ly::V_OFF, Ly::BOX, 1024u);
      constexpr uint64_t TILE16 = Ly::TILE >> 4, BOX16 = Ly::BOX >> 4;
      // K-major operand (Q or K): K-step kk of 16 elements sits in box kk/4 at byte 32*(kk%4)
      auto kmaj_off = [](int kk) { return (uint64_t)((kk >> 2) * BOX16 + (kk & 3) * 2); };
      // MN-major V: K-step kk covers key rows 16kk..16kk+15 (two 8-row swizzle atoms, 2048
      // bytes); the second 64-column half of d is the next box (leading byte offset)
      auto issue_s = [&](int t, int qbuf, int stage) {  // map t: its half of the columns of Q and K
        const uint64_t qd = q_desc0 + (uint64_t)qbuf * TILE16 + kmaj_off(t * (D / 32));
        const uint64_t kd = k_desc0 + (uint64_t)stage * TILE16 + kmaj_off(t * (D / 32));
        const uint32_t d_tm = tmem + (uint32_t)(t * 128);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) tc_mma_ss_warp(d_tm, qd + kmaj_off(kk), kd + kmaj_off(kk), idesc_qk, kk > 0);
        tc_commit_warp(bar(Ly::B_SFULL + t));
      };
      auto issue_pv = [&](int t, int stage, bool first) {
        const uint64_t vd = v_desc0 + (uint64_t)stage * TILE16;
        const uint32_t tm_p = tmem + (uint32_t)(t * 128);
        const uint32_t tm_o = tmem + 256u + (uint32_t)(t * 128);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          tc_mma_ts_warp(tm_o, tm_p + (uint32_t)(kk * 8), vd + (uint64_t)(kk * 128), idesc_pv, (!first || kk > 0) ? 1u : 0u);
      };
      int nu = 0, nq = 0, nblk = 0, cnt = 0;
      bool ok = true;
      while (ok) {
        const int slot = nu & 1;
        ok = mbar_wait_warp(bar(Ly::B_UFULL + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                       ROLE_MMA, -1);
        if (!ok) break;
        const int u = unit_ring[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_UEMPTY + slot));
        __syncwarp();
        ++nu;
        if (u < 0) break;
        const int NB = decode(u, prm).NB;
        if (NB == 0) continue;
        const int uidx = nq++;  // units with work
        const int qb = uidx & 1;
        ok = mbar_wait_warp(bar(Ly::B_QFULL + qb), (uint32_t)((uidx >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                            ROLE_MMA, u);
        if (ok)
          ok = mbar_wait_warp(bar(Ly::B_KFULL + nblk % NST), (uint32_t)((nblk / NST) & 1), prm.wait_limit_ns, abort_flag,
                         prm.status, ROLE_MMA, u);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < 2; ++t) issue_s(t, qb, nblk % NST);
        if (NB == 1) tc_commit_warp(bar(Ly::B_QEMPTY + qb));
        tc_commit_warp(bar(Ly::B_KEMPTY + nblk % NST));
        for (int j = 0; j < NB && ok; ++j) {
          const int g = nblk + j;
          const int st = g % NST;
          ok = mbar_wait_warp(bar(Ly::B_VFULL + st), (uint32_t)((g / NST) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                         ROLE_MMA, u);
          for (int t = 0; t < 2 && ok; ++t) {
            ok = mbar_wait_warp(bar(Ly::B_PFULL + t), (uint32_t)(cnt & 1), prm.wait_limit_ns, abort_flag, prm.status,
                           ROLE_MMA, u);
            if (ok && t == 0 && j == 0 && uidx > 0)  // the previous unit's epilogue has copied O_1 and O_2 out
              ok = mbar_wait_warp(bar(Ly::B_OFREE), (uint32_t)((uidx - 1) & 1), prm.wait_limit_ns, abort_flag,
                             prm.status, ROLE_MMA, u);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, st, j == 0);
            if (j + 1 < NB) {
              const int sn = (g + 1) % NST;
              if (t == 0) {
                ok = mbar_wait_warp(bar(Ly::B_KFULL + sn), (uint32_t)(((g + 1) / NST) & 1), prm.wait_limit_ns, abort_flag,
                               prm.status, ROLE_MMA, u);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(t, qb, sn);
            }
          }
          if (!ok) break;
          ++cnt;
          if (j + 1 == NB) tc_commit_warp(bar(Ly::B_OFINAL));  // the unit's last products: its epilogue may start
          if (j + 1 < NB) tc_commit_warp(bar(Ly::B_KEMPTY + (g + 1) % NST));
          if (j + 2 == NB) tc_commit_warp(bar(Ly::B_QEMPTY + qb));  // the unit's last S products are issued
          tc_commit_warp(bar(Ly::B_VEMPTY + st));
        }
        if (!ok) break;
        nblk += NB;
      }
      // exit-path drain: every MMA issued completes before TMEM is freed
      tc_commit_warp(bar(Ly::B_DRAIN));
      mbar_drain(bar(Ly::B_DRAIN), 0u, DRAIN_NS);
    } else if (warp == WARP_LOAD && lane == 0) {
      // ================================================================ producer
      int nu = 0, nq = 0, nk = 0, nv = 0;
      bool ok = *abort_flag == 0;
      if (ok && (prm.header->magic != TABLES_MAGIC || prm.header->tag != prm.tag)) {  // another plan's tables
        record_error(prm.status, MESH_ATTN_ERR_INVALID_ARG, ROLE_LOAD, 0);
        *abort_flag = 1;
        ok = false;
      }
      // a CTA's first unit is its own index, the others come from the counter; published to the
      // consumers' ring
      auto publish = [&]() -> int {
        const int slot = nu & 1;
        ok = mbar_wait(bar(Ly::B_UEMPTY + slot), (uint32_t)(((nu >> 1) & 1) ^ 1), prm.wait_limit_ns, abort_flag,
                       prm.status, ROLE_LOAD, -1);
        if (!ok) return -1;
        int v = (int)blockIdx.x;
        if (nu > 0) v = prm.n_units > (int)gridDim.x ? (int)(gridDim.x + atomicAdd(prm.counter, 1u)) : prm.n_units;
        if (v >= prm.n_units) v = -1;
        unit_ring[slot] = v;
        mbar_arrive(bar(Ly::B_UFULL + slot));
        ++nu;
        return v;
      };
      int u = ok ? publish() : -1;
      while (ok && u >= 0) {
        const Unit x = decode(u, prm);
        // publish the following unit now and pull its Q tile and first K/V block into L2, so
        // the unit boundary does not wait on DRAM
        const int un = publish();
        if (!ok) break;
        if (un >= 0) {
          const Unit xn = decode(un, prm);
          const int32_t qp = xn.b * prm.Hq + xn.h, kp = xn.b * prm.Hkv + xn.hk;
          for (int c = 0; c < D / 64; ++c) {
            tma_prefetch_l2_3d(&tmQ, c * 64, xn.qt * BM, qp);
            tma_prefetch_l2_3d(&tmK, c * 64, xn.blk0 * BN, kp);
            tma_prefetch_l2_3d(&tmV, c * 64, xn.blk0 * BN, kp);
          }
        }
        if (x.NB == 0) {
          u = un;
          continue;
        }
        // Q tile: the last S products of the unit before last must be done with this buffer
        const int qb = nq & 1;
        ok = mbar_wait(bar(Ly::B_QEMPTY + qb), (uint32_t)(((nq >> 1) & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status,
                       ROLE_LOAD, u);
        if (!ok) break;
        const int32_t qp = x.b * prm.Hq + x.h, kp = x.b * prm.Hkv + x.hk;
        mbar_expect_tx(bar(Ly::B_QFULL + qb), Ly::TILE);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sb + Ly::Q_OFF + (uint32_t)qb * Ly::TILE + (uint32_t)c * Ly::BOX, &tmQ, c * 64, x.qt * BM, qp,
                      bar(Ly::B_QFULL + qb));
        ++nq;
        {
          for (int jb = x.blk0; jb < x.blk0 + x.NB; ++jb) {
            const int st = nk % NST;
            const uint32_t ph = (uint32_t)((nk / NST) & 1);
            ok = mbar_wait(bar(Ly::B_KEMPTY + st), ph ^ 1u, prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, u);
            if (!ok) break;
            mbar_expect_tx(bar(Ly::B_KFULL + st), Ly::TILE);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sb + Ly::K_OFF + (uint32_t)st * Ly::TILE + (uint32_t)c * Ly::BOX, &tmK, c * 64, jb * BN, kp,
                          bar(Ly::B_KFULL + st));
            ++nk;
            ok = mbar_wait(bar(Ly::B_VEMPTY + st), ph ^ 1u, prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, u);
            if (!ok) break;
            mbar_expect_tx(bar(Ly::B_VFULL + st), Ly::TILE);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sb + Ly::V_OFF + (uint32_t)st * Ly::TILE + (uint32_t)c * Ly::BOX, &tmV, c * 64, jb * BN, kp,
                          bar(Ly::B_VFULL + st));
            ++nv;
          }
        }
        u = un;
      }
      // exit-path drain: every load issued lands before the CTA exits
      for (int jj = (nq > 2 ? nq - 2 : 0); jj < nq; ++jj)
        mbar_drain(bar(Ly::B_QFULL + (jj & 1)), (uint32_t)((jj >> 1) & 1), DRAIN_NS);
      for (int jj = (nk > NST ? nk - NST : 0); jj < nk; ++jj)
        mbar_drain(bar(Ly::B_KFULL + jj % NST), (uint32_t)((jj / NST) & 1), DRAIN_NS);
      for (int jj = (nv > NST ? nv - NST : 0); jj < nv; ++jj)
        mbar_drain(bar(Ly::B_VFULL + jj % NST), (uint32_t)((jj / NST) & 1), DRAIN_NS);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// O = sum_t w1_t O1_t - lam sum_t w2_t O2_t over a tile's parts, w = exp(lse_t - lse) of each map, O2 and the LSEs.
// A thread takes a 16-byte piece of one map's row, all parts' loads in flight together; a CTA a few rows, so
// that the few tiles there are still fill the GPU.
constexpr int MERGE_THREADS = 256;
template <int D>
constexpr int MERGE_ROWS = MERGE_THREADS / (D / 2);
template <int D>
__global__ void __launch_bounds__(MERGE_THREADS) merge_parts_kernel(const Params prm) {
  constexpr int Q4 = D / 4, ROWS = MERGE_ROWS<D>, PER_TILE = BM / ROWS;
  __shared__ float4 o2_s[ROWS * Q4];
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(prm.status) != 0) return;
  const int i = (int)blockIdx.x / PER_TILE, r0 = (int)blockIdx.x % PER_TILE * ROWS;
  const int m = (int)threadIdx.x / (ROWS * Q4), at = (int)threadIdx.x % (ROWS * Q4), r = r0 + at / Q4, c = at % Q4 * 4;
  const Unit x = decode_tile(prm.n_whole + i, prm);
  const int k = parts_of(x.NB, prm);
  const int64_t row = (int64_t)x.qt * BM + r, head = (int64_t)x.b * prm.Hq + x.h;
  const bool in = row < prm.S;
  const int64_t base = ((int64_t)i * prm.parts * 2 + m) * BM + r;  // row of part t: base + 2 t BM
  float w[MAX_PARTS];
  float4 v[MAX_PARTS];
#pragma unroll
  for (int t = 0; t < MAX_PARTS; ++t) {
    const bool there = in && t < k;
    w[t] = there ? prm.part_lse[base + 2 * t * BM] : -INFINITY;
    v[t] = there ? __ldcs(reinterpret_cast<const float4*>(prm.part_o + (base + 2 * t * BM) * D + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY, W = 0.f;
#pragma unroll
  for (int t = 0; t < MAX_PARTS; ++t) M = fmaxf(M, w[t]);
  const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int t = 0; t < MAX_PARTS; ++t) {
    w[t] = __expf(w[t] - Ms);
    W += w[t];
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;  // a NaN sum stays NaN
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int t = 0; t < MAX_PARTS; ++t) {
    const float f = t < k ? w[t] * inv : 0.f;
    o.x = fmaf(f, v[t].x, o.x);
    o.y = fmaf(f, v[t].y, o.y);
    o.z = fmaf(f, v[t].z, o.z);
    o.w = fmaf(f, v[t].w, o.w);
  }
  const int64_t dst = (head * prm.S + row) * D + c;
  if (m == 1) {
    o2_s[at] = o;
    if (in && prm.o2) *reinterpret_cast<uint2*>(prm.o2 + dst) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  if (in && c == 0) prm.lse[(2 * head + m) * prm.S + row] = W == 0.f ? -INFINITY : Ms + logf(W);
  __syncthreads();
  if (m == 0 && in) {
    const float lam = __bfloat162float(prm.lam[prm.lam_n == 1 ? 0 : x.h]);
    const float4 y = o2_s[at];
    *reinterpret_cast<uint2*>(prm.o + dst) = make_uint2(pack_bf16x2(fmaf(-lam, y.x, o.x), fmaf(-lam, y.y, o.y)),
                                                        pack_bf16x2(fmaf(-lam, y.z, o.z), fmaf(-lam, y.w, o.w)));
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

// [parts][L][d] bf16 rows, boxes of 128 rows x 64 columns with 128-byte swizzle; rows of a box past L
// are zeros.
static bool make_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, uint64_t L, uint64_t parts, int d,
                     std::string* err) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)L * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)BM, 1};
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

// Which tiles are cut into parts.  A part costs its tile's share of the blocks; the parts and their merge cost
// about as much as four blocks (5 us at 1.25 us a block), so a cut has to save more.  All tiles: where at
// most half of the SMs would have one (18 tiles of up to 18 blocks, causal: 31 -> 19 us).  The last wave's:
// tiles without a mask all take the same time, and a wave with few of them takes as long as a full one (320 tiles
// of 20 blocks on 152 SMs: 90 -> 79 us).
struct Parts {
  int64_t whole, parts;  // tiles in one piece; parts of each of the others
};
static Parts choose_parts(int64_t tiles, int64_t nb, bool causal, int sms) {
  const int64_t tail = 2 * tiles <= sms ? tiles : causal || tiles < sms ? 0 : tiles % sms;
  if (tail == 0 || 2 * tail > sms) return {tiles, 1};
  const int64_t parts = std::min<int64_t>({sms / tail, nb / 2, MAX_PARTS});
  if (parts < 2 || nb - nb / parts <= 4) return {tiles, 1};
  return {tiles - tail, parts};
}

template <int D>
static int launch(const DiffArgs& a, const DiffWorkspace& w, int sms, cudaStream_t st, std::string* err) {
  Params prm{};
  prm.header = static_cast<const TablesHeader*>(a.tables);
  prm.tag = a.tag;
  prm.lam = static_cast<const __nv_bfloat16*>(a.lam);
  prm.o = static_cast<__nv_bfloat16*>(a.O);
  prm.o2 = static_cast<__nv_bfloat16*>(a.O2);
  prm.lse = a.LSE;
  prm.part_o = reinterpret_cast<float*>(a.ws + w.part_o);
  prm.part_lse = reinterpret_cast<float*>(a.ws + w.part_lse);
  prm.status = a.status;
  prm.counter = reinterpret_cast<uint32_t*>(a.ws + w.counters);
  prm.S = a.S;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  const int64_t nqt = (a.S + BM - 1) / BM, tiles = nqt * a.B * a.Hq;
  if (tiles > 0x3fffffff) {
    *err = "too many work units for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  const Parts cut = choose_parts(tiles, nqt, a.causal, sms);
  const int64_t n_cut = tiles - cut.whole, units = cut.whole + n_cut * cut.parts;
  prm.nqt = (int32_t)nqt;
  prm.n_tiles = (int32_t)tiles;
  prm.n_whole = (int32_t)cut.whole;
  prm.parts = (int32_t)cut.parts;
  prm.n_units = (int32_t)units;
  prm.causal = a.causal;
  // enough lanes for about three times the grid
  prm.batch = a.causal ? (int32_t)std::min<int64_t>(tiles / nqt, (3LL * sms + nqt - 1) / nqt) : 1;
  prm.lam_n = a.lam_n;
  prm.scale_log2 = a.scale_log2;
  prm.wait_limit_ns = a.wait_limit_ns;
  EncodeTiledFn enc = get_encode(err);
  if (!enc) return (int)cudaErrorNotSupported;
  CUtensorMap mq, mk, mv;
  if (!make_map(enc, &mq, a.Q, (uint64_t)a.S, (uint64_t)a.B * a.Hq, D, err) ||
      !make_map(enc, &mk, a.K, (uint64_t)a.S, (uint64_t)a.B * a.Hkv, D, err) ||
      !make_map(enc, &mv, a.V, (uint64_t)a.S, (uint64_t)a.B * a.Hkv, D, err))
    return (int)cudaErrorInvalidValue;
  auto kern = diff_fwd_tc_kernel<D>;
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  cudaError_t e = cudaSuccess;
  if (once.pending(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::ALLOC);
    // a warpgroup that raises its registers beyond what the launch has would wait for ever
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess && fa.numRegs * NUM_THREADS < 2 * 128 * SOFTMAX_REGS + 128 * OTHER_REGS) {
      *err = "differential forward built with " + std::to_string(fa.numRegs) +
             " registers a thread, fewer than its warpgroups' register split needs";
      return (int)cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) once.mark(dev);
  }
  // with a CTA for every unit the counter is not read
  if (e == cudaSuccess && units > sms) e = cudaMemsetAsync(prm.counter, 0, 4, st);
  if (e != cudaSuccess) {
    *err = std::string("diff_fwd_tc: ") + cudaGetErrorString(e);
    return (int)e;
  }
  const unsigned grid = (unsigned)std::min<int64_t>(units, sms);  // persistent: one CTA per SM
  e = launch_behind(kern, dim3(grid), NUM_THREADS, Layout<D>::ALLOC, st, mq, mk, mv, prm);
  if (e == cudaSuccess && n_cut > 0) {
    const int64_t blocks = n_cut * (BM / MERGE_ROWS<D>);
    e = launch_behind(merge_parts_kernel<D>, dim3((unsigned)blocks), MERGE_THREADS, 0, st, prm);
  }
  if (e != cudaSuccess) *err = std::string("diff_fwd_tc launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace dtc

int launch_diff_fwd_tc(const DiffArgs& a, const DiffWorkspace& w, int sms, void* stream, std::string* err) {
  cudaStream_t st = (cudaStream_t)stream;
  return a.d == 128 ? dtc::launch<128>(a, w, sms, st, err) : dtc::launch<64>(a, w, sms, st, err);
}

// Parts there may be, whatever the number of SMs.
int64_t diff_fwd_max_parts(int64_t S, int32_t B, int32_t Hq, bool causal) {
  const int64_t nb = (S + dtc::BM - 1) / dtc::BM, tiles = nb * B * Hq;
  if (nb <= 4 || (causal && 2 * tiles > MAX_SMS)) return 0;
  return std::min<int64_t>(MAX_SMS, tiles * dtc::MAX_PARTS);
}

}  // namespace mesh
