// Differential attention backward for fp32 inputs, on the tensor cores (sm_103a).
//
// With P_m = exp(scale q_m.k_m - LSE_m), dP = dO V^T and D_m = dO . O_m:
//   A = P_1 - lam P_2,  dS_1 = P_1 (dP - D_1),  dS_2 = -lam P_2 (dP - D_2),
//   dq_m = scale dS_m k_m,  dk_m = scale dS_m^T q_m,  dV = A^T dO.
// Every operand is the sum of three bf16 pieces (exact: 3 x 8 significant bits), and every product the six
// piece products that are not below 2^-24 of it, summed in fp32, as in the fp32 forward.
//
// Three passes of one shape in one launch, pass p of a CTA keeping 128 resident rows (R0, R1) of one head
// and streaming 64-row blocks of the other side (C0, C1):
//   dQ: R = Q, dO;  C = K, V      dK: R = K, V;  C = Q, dO      dV: R = K;  C = Q, dO
//   S_m = R0_m C0_m^T,  dP = R1 C1^T,  acc_m += dS_m C0_m  (dV: acc += A C1)
// dV has a pass of its own, with the scores once more, since its accumulators and A's pieces do not fit the 512
// TMEM columns beside dK's: eight products where seven would do.  R1's pieces lie in TMEM (the operand
// of dP, split by the elementwise warps straight from fp32), R0's in shared memory with one stage of C0 and
// C1 (two at d = 64); they come by TMA from pieces that pieces_kernel writes.
//   TMEM: R1's pieces [0, 192) (dV: A's, two buffers) | S_1, S_2, dP [192, 384), later the pieces of dS_1 and
//   dS_2 in their place | accumulators [384, 512).
//   warps 0-7   elementwise: two warps per TMEM lane quadrant, each taking 32 of a block's 64 columns
//   warp 8      MMA issuer, warp 9 producer (TMA), warps 10-11 idle
// In dQ and dK a block's steps follow one another (dP and S, the elementwise part, dS C0), TMEM being full; in dV
// the next block's scores run while A is made.  At d = 64 a map's half is 32 columns: its product with C0
// is computed 64 wide and half of it is used.
//
// Few rows leave SMs idle, so the streamed axis is split between CTAs (`splits`); the splits, and for dK and
// dV the query heads of a KV head, leave partial sums that sum_parts adds in order.  Rows past the end are
// loaded as zeros.  Every mbarrier wait is bounded, as in the other kernels.
//
// Measured (the backward call, us): 2 x 8 heads on one of 801 tokens, d = 128: 306, 43 TFLOP/s of the formulas' five
// products (a kernel on the CUDA cores took 824); 4 heads on 2 of 777, d = 64, causal: 56 (74).  Bound by the chain of a
// block's steps: at d = 128 about 11,000 cycles for dQ and dK, 7,500 of products (48 each of S, dP and the
// accumulators', 45-62 cycles) and 2,500-4,000 of the elementwise warps; 7,300 for dV.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace db32 {

constexpr int BM = 128;  // resident rows = TMEM lanes
constexpr int BS = 64;   // streamed rows per block
constexpr int N_EW = 8;
constexpr int WARP_MMA = 8;
constexpr int WARP_LOAD = 9;
constexpr int NUM_THREADS = 384;
// Registers after setmaxnreg: the elementwise warpgroups, and the one of the MMA and load warps.  They add up to the
// launch's 384 x 168, which the launcher checks.
constexpr int EW_REGS = 200, OTHER_REGS = 104;
constexpr int64_t DRAIN_NS = 200000000;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int ROLE_EW = 1, ROLE_MMA = 2, ROLE_LOAD = 3;
constexpr uint32_t COL_R1 = 0, COL_A = 0, COL_S = 192, COL_DP = 320, COL_ACC = 384;
enum Pass { DQ = 0, DK = 1, DV = 2 };

// piece pairs (a, b) of a product, smallest first
constexpr int N_PAIR = 6;
__device__ __forceinline__ constexpr int pair_a(int i) { return i == 0 ? 2 : i == 2 || i == 3 ? 1 : 0; }
__device__ __forceinline__ constexpr int pair_b(int i) { return i == 1 ? 2 : i == 2 || i == 4 ? 1 : 0; }

template <int D>
struct Layout {
  static constexpr int NST = D == 64 ? 2 : 1;
  static constexpr uint32_t RBOX = BM * 128, CBOX = BS * 128;  // 64 columns of bf16, 128-byte swizzle
  static constexpr uint32_t RP = (D / 64) * RBOX, CP = (D / 64) * CBOX;  // a piece
  static constexpr uint32_t R0 = 0;
  static constexpr uint32_t C0 = R0 + 3 * RP;         // [NST][3 pieces]
  static constexpr uint32_t C1 = C0 + NST * 3 * CP;   // [NST][3 pieces]
  static constexpr uint32_t VEC = C1 + NST * 3 * CP;  // [2][64][4]: LSE_1, LSE_2, D_1, D_2 of a block's query rows
  static constexpr uint32_t BAR = VEC + 2 * BS * 16;
  static constexpr int B_RF = 0, B_R1 = 1, B_C0F = 2, B_C0E = B_C0F + 2, B_C1F = B_C0E + 2, B_C1E = B_C1F + 2, B_S = B_C1E + 2,
                       B_SR = B_S + 1, B_DS = B_SR + 1, B_ACC = B_DS + 2, B_DRAIN = B_ACC + 1, NBARS = B_DRAIN + 1;
  static constexpr uint32_t MISC = BAR + NBARS * 8;  // tmem base, abort flag, whether to run at all
  static constexpr uint32_t ALLOC = MISC + 16 + 1024;
};

struct Maps {
  CUtensorMap q128, k128, q64, k64, v64, g64;  // pieces as [3 B H][S][d]; boxes of 128 or 64 rows x 64 columns
};

struct Params {
  const float* v;
  const float* g;     // dO
  const float* lse;   // [B, Hq, 2, S]
  const float* dsum;  // [B, Hq, 2, S]
  const float* lam;
  float* out[3];      // dQ, dK, dV: [B, heads, parts, S, D]
  int32_t* status;
  int64_t S, wait_limit_ns;
  int32_t B, Hq, Hkv, lam_n, causal, splits;
  float scale, scale_log2;
};

// Two values as three packed pieces: x1 = x with the low 16 bits cleared, then the same of what is left (exact).
__device__ __forceinline__ void split3(float x, float y, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  const uint32_t u0 = __float_as_uint(x), u1 = __float_as_uint(y);
  const float r0 = x - __uint_as_float(u0 & 0xffff0000u), r1 = y - __uint_as_float(u1 & 0xffff0000u);
  const uint32_t w0 = __float_as_uint(r0), w1 = __float_as_uint(r1);
  const float t0 = r0 - __uint_as_float(w0 & 0xffff0000u), t1 = r1 - __uint_as_float(w1 & 0xffff0000u);
  p1 = __byte_perm(u0, u1, 0x7632u);
  p2 = __byte_perm(w0, w1, 0x7632u);
  p3 = __byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x7632u);
}

// Q, K, V and dO as pieces, [3][rows][d] each; blockIdx.y picks the tensor.
struct PiecesArgs {
  const float4* x[4];
  uint2* out[4];
  int64_t n4[4];
  const int32_t* status;
};
__global__ void __launch_bounds__(256) pieces_kernel(const PiecesArgs a) {
  wait_for_kernel_before();
  if (*reinterpret_cast<const volatile int32_t*>(a.status) != 0) return;
  const int w = blockIdx.y;
  const int64_t n = a.n4[w];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const float4 v = a.x[w][i];
    uint2 p[3];
    split3(v.x, v.y, p[0].x, p[1].x, p[2].x);
    split3(v.z, v.w, p[0].y, p[1].y, p[2].y);
#pragma unroll
    for (int k = 0; k < 3; ++k) a.out[w][k * n + i] = p[k];
  }
}

template <int D, int PASS>
__device__ __forceinline__ void run_pass(const Maps& maps, const Params& prm, int bh, int rb, int split, uint32_t sb,
                                         uint8_t* smem, uint32_t tmem) {
  using Ly = Layout<D>;
  constexpr bool KV = PASS != DQ;
  constexpr int NST = Ly::NST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + Ly::BAR + 8u * (uint32_t)i; };
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC + 4);
  const int64_t S = prm.S;
  const int b = bh / prm.Hq, h = bh % prm.Hq, group = prm.Hq / prm.Hkv, hk = h / group, bk = b * prm.Hkv + hk;
  const int64_t r0 = (int64_t)rb * BM;
  // this CTA's streamed blocks: its share of those a resident row sees
  const int n_all = (int)((S + BS - 1) / BS);
  const int first = KV && prm.causal ? 2 * rb : 0, last = !KV && prm.causal ? min(n_all, 2 * rb + 2) : n_all;
  const int per = (last - first + prm.splits - 1) / prm.splits;
  const int c_begin = min(last, first + split * per), NB = min(last, c_begin + per) - c_begin;
  // The same for all warps: the elementwise warps meet at named barriers, which wait without a limit.  (The abort
  // flag may be set by a warp that is ahead; the vote in the block loop carries such an abort to all of them.)
  const bool run = *reinterpret_cast<const volatile int32_t*>(smem + Ly::MISC + 8) != 0 && NB > 0;

  if (warp < N_EW) {
    // ================================================================ elementwise
    regs_inc<EW_REGS>();
    const int wq = warp & 3, hf = warp >> 2;  // lane quadrant, half of a block's columns
    const int64_t row = r0 + wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    float* vec = reinterpret_cast<float*>(smem + Ly::VEC);
    const int64_t vrow = (int64_t)bh * 2 * S;
    // value w (LSE_1, LSE_2, D_1, D_2) of query row s as it enters the FMAs; a row past the end, or without a
    // visible key, gets exp2(x - inf) = 0
    auto fetch = [&](int w, int64_t s) {
      return s < S ? (w < 2 ? prm.lse : prm.dsum)[vrow + (w & 1) * S + s] : w < 2 ? -INFINITY : 0.f;
    };
    auto value = [&](int w, float x) { return w >= 2 ? -x : x == -INFINITY ? -INFINITY : -x * LOG2E; };
    bool ok = run;
    float rv[4];
    if (ok) {
      if (!KV)
#pragma unroll
        for (int w = 0; w < 4; ++w) rv[w] = value(w, fetch(w, row));
      if (PASS != DV) {  // R1's pieces to TMEM, this warp's half of the columns
        const float* src = PASS == DQ ? prm.g + ((int64_t)bh * S + row) * D : prm.v + ((int64_t)bk * S + row) * D;
#pragma unroll
        for (int c = 0; c < D / 2; c += 32) {
          uint32_t p1[16], p2[16], p3[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 x = row < S ? reinterpret_cast<const float4*>(src + hf * (D / 2) + c)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
            split3(x.x, x.y, p1[2 * e], p2[2 * e], p3[2 * e]);
            split3(x.z, x.w, p1[2 * e + 1], p2[2 * e + 1], p3[2 * e + 1]);
          }
          const uint32_t at = lanes + COL_R1 + (uint32_t)(hf * (D / 4) + c / 2);
          tmem_st16(at, p1);
          tmem_st16(at + D / 2, p2);
          tmem_st16(at + D, p3);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_R1));
      }
    }
    // where this warp's half of the columns of its rows goes: [B, head, part, S, D]
    auto out_row = [&]() {
      const int64_t head = KV ? bk : bh;
      const int n_part = KV ? group * prm.splits : prm.splits, part = KV ? (h % group) * prm.splits + split : split;
      return prm.out[PASS] + ((head * n_part + part) * S + row) * D + hf * (D / 2);
    };
    const float f = PASS == DV ? 1.f : prm.scale;
    // d = 64: the second map's accumulator is 64 columns behind, its half of the columns in the second 32
    const uint32_t acc = lanes + COL_ACC + (uint32_t)(hf * (D == 64 && PASS != DV ? 96 : D / 2));
    const float nlam = -prm.lam[prm.lam_n == 1 ? 0 : h];
    // The tensor cores' fp32 sums truncate, so a long accumulation loses digits whatever its terms' signs (4e-6 of dK's
    // norm at 800 queries, 8e-6 at 4,096): only a block's products are summed there, and the blocks here, with rounding
    // (5e-7 at any length; at d = 128 up to 6 % slower).  In dQ and dK that is done while the next block's scores and dP
    // are computed; in dV, whose next scores are there already, at the end of the next block.
    float sums[D / 2] = {};
    auto add_block = [&](int j) -> bool {
      if (!mbar_wait_warp(bar(Ly::B_ACC), (uint32_t)(j & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_EW, j)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        tmem_ld32(acc + (uint32_t)c, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) sums[c + e] += o[e];
      }
      return true;
    };
    const int vw = threadIdx.x >> 6, vc = threadIdx.x & 63;  // the value this thread fetches for a block
    float vnext = KV && ok ? fetch(vw, (int64_t)c_begin * BS + vc) : 0.f;
    bool added = true;  // false: add_block's wait failed, which the next vote tells the others
    for (int j = 0; j < NB && ok; ++j) {
      const int64_t c0 = (int64_t)(c_begin + j) * BS;
      const float4* bv = reinterpret_cast<const float4*>(vec + (j & 1) * 4 * BS);
      if (KV) {  // (the buffer's readers of two blocks ago have passed the last block's barrier)
        vec[(j & 1) * 4 * BS + vc * 4 + vw] = value(vw, vnext);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (j + 1 < NB) vnext = fetch(vw, c0 + BS + vc);
      }
      if (PASS != DV && j > 0) added = add_block(j - 1);
      ok = added && mbar_wait_warp(bar(Ly::B_S), (uint32_t)(j & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_EW, j);
      // an abort ends all warps' loops: none may wait for another below
      float s1[32], s2[32], dp[32];
      if (ok) {
        tc_fence_after();
        tmem_ld32(lanes + COL_S + (uint32_t)(32 * hf), s1);
        tmem_ld32(lanes + COL_S + 64u + (uint32_t)(32 * hf), s2);
        if (PASS != DV) tmem_ld32(lanes + COL_DP + (uint32_t)(32 * hf), dp);
        tc_wait_ld();
        if (PASS == DV) {  // the next block's scores may come
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Ly::B_SR));
        }
      }
      // everyone has read before anyone writes in the scores' place; the vote keeps the warps together
      int all;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 2, 256, p;\n\t"
          "selp.b32 %0, 1, 0, q;\n\t}"
          : "=r"(all)
          : "r"((int)ok)
          : "memory");
      ok = all != 0;
      if (!ok) break;
      uint32_t p1[16], p2[16], p3[16];
      // this thread's columns with a visible pair are [lo, hi): keys up to the query's and inside the sequence (query
      // rows past the end have weights 0 already)
      const int64_t cb = c0 + 32 * hf;
      const int lo = !KV ? 0 : row >= S ? 32 : prm.causal ? (int)max((int64_t)0, min((int64_t)32, row - cb)) : 0;
      const int hi = KV ? 32 : (int)max((int64_t)0, min((int64_t)32, min(prm.causal ? row + 1 : S, S) - cb));
      const auto weights = [&](auto masked) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const bool off = decltype(masked)::value && (c < lo || c >= hi);
          float l1, l2, d1, d2;
          if (KV) {
            const float4 x = bv[32 * hf + c];
            l1 = x.x, l2 = x.y, d1 = x.z, d2 = x.w;
          } else {
            l1 = rv[0], l2 = rv[1], d1 = rv[2], d2 = rv[3];
          }
          const float e1 = fast_exp2(fmaf(s1[c], prm.scale_log2, l1));
          const float e2 = nlam * fast_exp2(fmaf(s2[c], prm.scale_log2, l2));
          if (PASS == DV) {
            s1[c] = off ? 0.f : e1 + e2;
          } else {
            s1[c] = off ? 0.f : e1 * (dp[c] + d1);
            s2[c] = off ? 0.f : e2 * (dp[c] + d2);
          }
        }
      };
      if (__any_sync(0xffffffffu, lo > 0 || hi < 32)) weights(std::true_type{});
      else weights(std::false_type{});
      // (A's buffer of two blocks ago has been read: that product precedes the scores just waited for)
      const uint32_t at = lanes + (PASS == DV ? COL_A + 96u * (uint32_t)(j & 1) : COL_S) + (uint32_t)(16 * hf);
#pragma unroll
      for (int c = 0; c < 16; ++c) split3(s1[2 * c], s1[2 * c + 1], p1[c], p2[c], p3[c]);
      tmem_st16(at, p1);
      tmem_st16(at + 32u, p2);
      tmem_st16(at + 64u, p3);
      if (PASS != DV) {
#pragma unroll
        for (int c = 0; c < 16; ++c) split3(s2[2 * c], s2[2 * c + 1], p1[c], p2[c], p3[c]);
        tmem_st16(at + 96u, p1);
        tmem_st16(at + 128u, p2);
        tmem_st16(at + 160u, p3);
      }
      tc_wait_st();
      if (PASS == DV && j > 0) added = add_block(j - 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_DS + (j & 1)));
    }
    if (ok) ok = added && add_block(NB - 1);
    if (ok || (NB == 0 && *abort_flag == 0)) {
      float* const dst = out_row();
      // 32 rows x 32 columns at a time through shared memory (C0's, whose last reader is done), 16-byte pieces
      // swizzled by row, so that a store writes whole 128-byte row pieces
      float* stage = reinterpret_cast<float*>(smem + Ly::C0 + (uint32_t)warp * 4096u);
      const int rows = (int)max((int64_t)0, min((int64_t)32, S - (row - lane)));  // of this warp, inside the sequence
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(stage + lane * 32 + ((e ^ (lane & 7)) * 4)) =
              make_float4(sums[c + 4 * e] * f, sums[c + 4 * e + 1] * f, sums[c + 4 * e + 2] * f, sums[c + 4 * e + 3] * f);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3), e = lane & 7;
          const float4 x = *reinterpret_cast<const float4*>(stage + r * 32 + ((e ^ (r & 7)) * 4));
          if (r < rows) *reinterpret_cast<float4*>(dst + (int64_t)(r - lane) * D + c + e * 4) = x;
        }
      }
    }
    return;
  }
  regs_dec<OTHER_REGS>();
  if (warp == WARP_MMA) {
    // ================================================================ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BS, false);                       // S, dP: N = 64, K-major B
    constexpr uint32_t idesc_a = idesc_bf16_f32(BM, PASS == DV ? D : 64, true);       // accumulators: MN-major B
    const uint64_t rd = smem_desc_sw128(sb + Ly::R0, 16u, 1024u);
    const uint64_t c0d = smem_desc_sw128(sb + Ly::C0, 16u, 1024u), c1d = smem_desc_sw128(sb + Ly::C1, 16u, 1024u);
    const uint64_t c0m = smem_desc_sw128(sb + Ly::C0, Ly::CBOX, 1024u), c1m = smem_desc_sw128(sb + Ly::C1, Ly::CBOX, 1024u);
    // K-step kk of a K-major operand: 16 columns, box kk / 4, byte 32 (kk mod 4)
    auto r_off = [](int p, int kk) { return (uint64_t)((p * Ly::RP + (kk >> 2) * Ly::RBOX) >> 4) + (uint64_t)((kk & 3) * 2); };
    auto c_off = [](int p, int kk) { return (uint64_t)((p * Ly::CP + (kk >> 2) * Ly::CBOX) >> 4) + (uint64_t)((kk & 3) * 2); };
    // The pairs' loops are unrolled: offsets are then constants, and the issue costs a few cycles a product (130 with
    // offsets computed from a loop variable).
    auto wait = [&](int i, uint32_t parity, int j) {
      return mbar_wait_warp(bar(i), parity, prm.wait_limit_ns, abort_flag, prm.status, ROLE_MMA, j);
    };
    bool ok = run;
    if (ok) ok = wait(Ly::B_RF, 0u, -1);
    if (ok && PASS != DV) ok = wait(Ly::B_R1, 0u, -1);
    auto issue_s = [&](int j) -> bool {  // S_1 and S_2 of block j
      const int st = j % NST;
      if (!wait(Ly::B_C0F + st, (uint32_t)((j / NST) & 1), j)) return false;
      tc_fence_after();
      const uint64_t c = c0d + (uint64_t)st * ((3 * Ly::CP) >> 4);
#pragma unroll
      for (int pr = 0; pr < N_PAIR; ++pr)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int m = kk / (D / 32);  // a map's half of the columns
          tc_mma_ss_warp(tmem + COL_S + 64u * m, rd + r_off(pair_a(pr), kk), c + c_off(pair_b(pr), kk), idesc_s,
                         (pr > 0 || kk % (D / 32) > 0) ? 1u : 0u);
        }
      if (PASS == DV) tc_commit_warp(bar(Ly::B_C0E + st));
      tc_commit_warp(bar(Ly::B_S));
      return true;
    };
    auto issue_dp = [&](int j) -> bool {
      const int st = j % NST;
      if (!wait(Ly::B_C1F + st, (uint32_t)((j / NST) & 1), j)) return false;
      tc_fence_after();
      const uint64_t c = c1d + (uint64_t)st * ((3 * Ly::CP) >> 4);
#pragma unroll
      for (int pr = 0; pr < N_PAIR; ++pr)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ts_warp(tmem + COL_DP, tmem + COL_R1 + (uint32_t)(pair_a(pr) * (D / 2) + kk * 8), c + c_off(pair_b(pr), kk), idesc_s,
                         (pr > 0 || kk > 0) ? 1u : 0u);
      tc_commit_warp(bar(Ly::B_C1E + st));
      return true;
    };
    auto sum = [&](uint32_t acc, uint32_t a, uint64_t c) {  // acc = the pieces at a times a block's rows, MN-major
#pragma unroll
      for (int pr = 0; pr < N_PAIR; ++pr)
#pragma unroll
        for (int kk = 0; kk < BS / 16; ++kk)
          tc_mma_ts_warp(acc, a + (uint32_t)(pair_a(pr) * 32 + kk * 8), c + (c_off(pair_b(pr), 0) + (uint64_t)(kk * 128)), idesc_a,
                         (pr > 0 || kk > 0) ? 1u : 0u);
    };
    // dP before the scores: C1's stage is free before C0's, whose next load then overlaps this product
    if (ok) ok = (PASS == DV || issue_dp(0)) && issue_s(0);
    for (int j = 0; j < NB && ok; ++j) {
      const int st = j % NST;
      const uint64_t stage = (uint64_t)st * ((3 * Ly::CP) >> 4);
      if (PASS == DV) {  // the next scores run while A(j) is made
        if (j + 1 < NB && !(ok = wait(Ly::B_SR, (uint32_t)(j & 1), j) && issue_s(j + 1))) break;
        if (!(ok = wait(Ly::B_C1F + st, (uint32_t)((j / NST) & 1), j))) break;
      }
      if (!(ok = wait(Ly::B_DS + (j & 1), (uint32_t)((j >> 1) & 1), j))) break;
      tc_fence_after();
      if (PASS == DV) {
        sum(tmem + COL_ACC, tmem + COL_A + 96u * (uint32_t)(j & 1), c1m + stage);
        tc_commit_warp(bar(Ly::B_C1E + st));
        tc_commit_warp(bar(Ly::B_ACC));
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m)  // the map's box of 64 columns; at d = 64 both maps share one
          sum(tmem + COL_ACC + 64u * m, tmem + COL_S + 96u * m, c0m + stage + (D == 128 ? (uint64_t)m * (Ly::CBOX >> 4) : 0ull));
        tc_commit_warp(bar(Ly::B_C0E + st));
        tc_commit_warp(bar(Ly::B_ACC));
        // into the place of dS(j)'s pieces, which those products have read
        if (j + 1 < NB) ok = issue_dp(j + 1) && issue_s(j + 1);
      }
    }
    // exit-path drain: every MMA issued completes before TMEM is freed
    tc_commit_warp(bar(Ly::B_DRAIN));
    mbar_drain(bar(Ly::B_DRAIN), 0u, DRAIN_NS);
  } else if (warp == WARP_LOAD && lane == 0) {
    // ================================================================ producer
    const CUtensorMap* mr = PASS == DQ ? &maps.q128 : &maps.k128;
    const CUtensorMap* m0 = PASS == DQ ? &maps.k64 : &maps.q64;
    const CUtensorMap* m1 = PASS == DQ ? &maps.v64 : &maps.g64;
    const int nq = prm.B * prm.Hq, nk = prm.B * prm.Hkv;  // heads of a piece
    bool ok = run;
    bool loaded_r = false;
    int n0 = 0, n1 = 0;
    if (ok) {
      mbar_expect_tx(bar(Ly::B_RF), 3 * Ly::RP);
      for (int p = 0; p < 3; ++p)
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sb + Ly::R0 + p * Ly::RP + c * Ly::RBOX, mr, c * 64, (int32_t)r0, PASS == DQ ? p * nq + bh : p * nk + bk, bar(Ly::B_RF));
      loaded_r = true;
    }
    for (int j = 0; j < NB && ok; ++j) {
      const int st = j % NST;
      const uint32_t ph = (uint32_t)((j / NST) & 1);
      const int32_t s0 = (c_begin + j) * BS;
      for (int i = 0; i < 2 && ok; ++i) {
        const int w = PASS == DV ? i : 1 - i;  // in the order in which the stages become free
        const int full = (w ? Ly::B_C1F : Ly::B_C0F) + st, empty = (w ? Ly::B_C1E : Ly::B_C0E) + st;
        ok = mbar_wait(bar(empty), ph ^ 1u, prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, j);
        if (!ok) break;
        mbar_expect_tx(bar(full), 3 * Ly::CP);
        for (int p = 0; p < 3; ++p)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sb + (w ? Ly::C1 : Ly::C0) + (uint32_t)(st * 3 + p) * Ly::CP + c * Ly::CBOX, w ? m1 : m0, c * 64, s0,
                        PASS == DQ ? p * nk + bk : p * nq + bh, bar(full));
        ++(w ? n1 : n0);
      }
    }
    // exit-path drain: every load issued lands before the CTA exits
    if (loaded_r) mbar_drain(bar(Ly::B_RF), 0u, DRAIN_NS);
    for (int w = 0; w < 2; ++w) {
      const int n = w ? n1 : n0;
      for (int j = (n > NST ? n - NST : 0); j < n; ++j)
        mbar_drain(bar((w ? Ly::B_C1F : Ly::B_C0F) + j % NST), (uint32_t)((j / NST) & 1), DRAIN_NS);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(NUM_THREADS, 1) diff_bwd32_kernel(const __grid_constant__ Maps maps, const Params prm) {
  using Ly = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;  // 1024-aligned base (128-byte swizzle atoms)
  uint8_t* smem = smem_raw + (sb - raw);
  const int warp = threadIdx.x >> 5;
  auto bar = [&](int i) { return sb + Ly::BAR + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::MISC);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC + 4);
  if (threadIdx.x == 0) {
    mbar_init(bar(Ly::B_RF), 1);
    mbar_init(bar(Ly::B_R1), N_EW);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Ly::B_C0F + s), 1);
      mbar_init(bar(Ly::B_C0E + s), 1);
      mbar_init(bar(Ly::B_C1F + s), 1);
      mbar_init(bar(Ly::B_C1E + s), 1);
    }
    mbar_init(bar(Ly::B_S), 1);
    mbar_init(bar(Ly::B_SR), N_EW);
    mbar_init(bar(Ly::B_DS), N_EW);  // two: dV's A(j + 1) may be there before the issuer has looked at A(j)
    mbar_init(bar(Ly::B_DS + 1), N_EW);
    mbar_init(bar(Ly::B_ACC), 1);
    mbar_init(bar(Ly::B_DRAIN), 1);
    wait_for_kernel_before();
    // without any time to wait there is nothing to start: the first load would be waited for
    if (prm.wait_limit_ns <= 0) record_error(prm.status, MESH_ATTN_ERR_DEVICE_TIMEOUT, ROLE_LOAD, -1);
    const bool stop = *reinterpret_cast<volatile int32_t*>(prm.status) != 0;
    *abort_flag = stop ? 1 : 0;
    *reinterpret_cast<volatile int32_t*>(smem + Ly::MISC + 8) = stop ? 0 : 1;  // nobody writes it again
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  wait_for_kernel_before();  // and before tensor memory is taken, which that kernel may still want
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // heads vary fastest, then the pass, the split and the row block, the longest first
  const int n_bh = prm.B * prm.Hq, nrb = (int)((prm.S + BM - 1) / BM);
  int t = (int)blockIdx.x;
  const int bh = t % n_bh;
  t /= n_bh;
  const int pass = t % 3;
  t /= 3;
  const int split = t % prm.splits, rbi = t / prm.splits;
  const int rb = pass == DQ && prm.causal ? nrb - 1 - rbi : rbi;
  if (pass == DQ) run_pass<D, DQ>(maps, prm, bh, rb, split, sb, smem, tmem);
  else if (pass == DK) run_pass<D, DK>(maps, prm, bh, rb, split, sb, smem, tmem);
  else run_pass<D, DV>(maps, prm, bh, rb, split, sb, smem, tmem);

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// out[head][i] = sum over the parts, in order; blockIdx.y picks one of up to three tensors
struct SumArgs {
  const float4* part[3];
  float4* out[3];
  int64_t heads[3];
  int32_t n[3];
  int64_t row4;  // S * D / 4
  const int32_t* status;
};
__global__ void __launch_bounds__(256) sum_parts(const SumArgs a) {
  wait_for_kernel_before();
  if (*reinterpret_cast<const volatile int32_t*>(a.status) != 0) return;
  const int w = blockIdx.y;
  const int64_t total = a.heads[w] * a.row4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t head = i / a.row4, at = i - head * a.row4;
    const float4* src = a.part[w] + head * a.n[w] * a.row4 + at;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < a.n[w]; ++k) {
      const float4 x = __ldcs(src + k * a.row4);
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    a.out[w][i] = t;
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

// [parts][S][d] bf16, boxes of box_rows x 64 columns with 128-byte swizzle; rows of a box past S are zeros.
static bool make_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, uint64_t S, uint64_t parts, int d, int box_rows,
                     std::string* err) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)S, (cuuint64_t)parts};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)S * d * 2};
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

template <int D>
static cudaError_t launch(const Maps& maps, const Params& prm, unsigned grid, cudaStream_t st, std::string* err) {
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  auto kern = diff_bwd32_kernel<D>;
  if (once.pending(dev)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::ALLOC);
    // a warpgroup that raises its registers beyond what the launch has would wait for ever
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess && fa.numRegs * NUM_THREADS < 2 * 128 * EW_REGS + 128 * OTHER_REGS) {
      *err = "fp32 differential backward built with " + std::to_string(fa.numRegs) +
             " registers a thread, fewer than its warpgroups' register split needs";
      return cudaErrorInvalidConfiguration;
    }
    if (e != cudaSuccess) return e;
    once.mark(dev);
  }
  return launch_behind(kern, dim3(grid), NUM_THREADS, Layout<D>::ALLOC, st, maps, prm);
}

}  // namespace db32

// Parts of the streamed axis: until every SM has a CTA, eight at most, none shorter than two blocks.
int diff_bwd32_splits(int64_t S, int32_t B, int32_t Hq, int sms) {
  const int64_t ctas = std::max<int64_t>(1, 3 * ((S + db32::BM - 1) / db32::BM) * B * Hq);
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(8, (S + 2 * db32::BS - 1) / (2 * db32::BS)));
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, (sms + ctas - 1) / ctas));
}

BwdPieces bwd32_pieces_layout(int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t q = up((size_t)6 * B * Hq * (size_t)S * d), kv = up((size_t)6 * B * Hkv * (size_t)S * d);
  return {0, q, q + kv, q + 2 * kv, 2 * q + 2 * kv};
}

int launch_diff_bwd_tc32(const DiffArgs& a, const DiffWorkspace& w, int sms, void* stream, std::string* err) {
  using namespace db32;
  cudaStream_t st = (cudaStream_t)stream;
  const int splits = diff_bwd32_splits(a.S, a.B, a.Hq, sms), group = a.Hq / a.Hkv;
  const int64_t q_rows = (int64_t)a.B * a.Hq * a.S, kv_rows = (int64_t)a.B * a.Hkv * a.S;
  const int64_t ctas = 3 * ((a.S + BM - 1) / BM) * a.B * a.Hq * splits;
  if (ctas > 0x7fffffff) {
    *err = "too many rows for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  const BwdPieces pc = bwd32_pieces_layout(a.B, a.Hq, a.Hkv, a.S, a.d);
  char* base = a.ws + w.pieces;
  PiecesArgs x{};
  const void* src[4] = {a.Q, a.K, a.V, a.dO};
  const size_t off[4] = {pc.q, pc.k, pc.v, pc.g};
  for (int i = 0; i < 4; ++i) {
    x.x[i] = static_cast<const float4*>(src[i]);
    x.out[i] = reinterpret_cast<uint2*>(base + off[i]);
    x.n4[i] = (i == 0 || i == 3 ? q_rows : kv_rows) * (a.d / 4);
  }
  x.status = a.status;
  cudaError_t e = launch_behind(pieces_kernel, dim3((unsigned)std::min<int64_t>((x.n4[0] + 255) / 256, 152 * 16), 4), 256, 0, st, x);
  if (e != cudaSuccess) {
    *err = std::string("diff_bwd_tc32 launch: ") + cudaGetErrorString(e);
    return (int)e;
  }
  EncodeTiledFn enc = get_encode(err);
  if (!enc) return (int)cudaErrorNotSupported;
  const uint64_t nq = (uint64_t)3 * a.B * a.Hq, nk = (uint64_t)3 * a.B * a.Hkv, S = (uint64_t)a.S;
  Maps m;
  if (!make_map(enc, &m.q128, base + pc.q, S, nq, a.d, BM, err) || !make_map(enc, &m.k128, base + pc.k, S, nk, a.d, BM, err) ||
      !make_map(enc, &m.q64, base + pc.q, S, nq, a.d, BS, err) || !make_map(enc, &m.k64, base + pc.k, S, nk, a.d, BS, err) ||
      !make_map(enc, &m.v64, base + pc.v, S, nk, a.d, BS, err) || !make_map(enc, &m.g64, base + pc.g, S, nq, a.d, BS, err))
    return (int)cudaErrorInvalidValue;
  const bool q_parts = splits > 1, kv_parts = splits * group > 1;
  Params p{};
  p.v = static_cast<const float*>(a.V);
  p.g = static_cast<const float*>(a.dO);
  p.lse = a.LSE;
  p.dsum = reinterpret_cast<const float*>(a.ws + w.dsum);
  p.lam = static_cast<const float*>(a.lam);
  p.out[DQ] = q_parts ? reinterpret_cast<float*>(a.ws + w.dq_part) : static_cast<float*>(a.dQ);
  p.out[DK] = kv_parts ? reinterpret_cast<float*>(a.ws + w.dk_part) : static_cast<float*>(a.dK);
  p.out[DV] = kv_parts ? reinterpret_cast<float*>(a.ws + w.dv_part) : static_cast<float*>(a.dV);
  p.status = a.status;
  p.S = a.S;
  p.wait_limit_ns = a.wait_limit_ns;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.lam_n = a.lam_n;
  p.causal = a.causal;
  p.splits = splits;
  p.scale = a.scale;
  p.scale_log2 = a.scale_log2;
  e = a.d == 128 ? launch<128>(m, p, (unsigned)ctas, st, err) : launch<64>(m, p, (unsigned)ctas, st, err);
  if (e == cudaSuccess && (q_parts || kv_parts)) {
    SumArgs s{};
    int n = 0;
    auto add = [&](size_t part, void* out, int64_t heads, int parts) {
      s.part[n] = reinterpret_cast<const float4*>(a.ws + part);
      s.out[n] = static_cast<float4*>(out);
      s.heads[n] = heads;
      s.n[n++] = parts;
    };
    if (kv_parts) {
      add(w.dk_part, a.dK, (int64_t)a.B * a.Hkv, splits * group);
      add(w.dv_part, a.dV, (int64_t)a.B * a.Hkv, splits * group);
    }
    if (q_parts) add(w.dq_part, a.dQ, (int64_t)a.B * a.Hq, splits);
    s.row4 = a.S * a.d / 4;
    s.status = a.status;
    const int64_t most = (int64_t)a.B * a.Hq * s.row4;
    e = launch_behind(sum_parts, dim3((unsigned)std::min<int64_t>((most + 255) / 256, 152 * 8), (unsigned)n), 256, 0, st, s);
  }
  if (e != cudaSuccess && err->empty()) *err = std::string("diff_bwd_tc32 launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace mesh
