// Attention forward whose scores are capped, biased by distance and masked by a range of keys a row, bf16 inputs, on the
// 5th-generation tensor cores (sm_103a): of a dense batch with ranges given (range-masked attention), or of the new tokens of
// sequences in a paged cache, whose ranges follow from their places (a chunk of a prompt).
//   x_ij = cap tanh(s q_i.k_j / cap) (or s q_i.k_j) - slope_h |i - j|,  lo_i <= j < hi_i,   O_i = sum_j softmax(x_i)_j v_j.
//
// A tile is 128 rows: gh query heads of one KV head times tt of their tokens, so that a tile's rows share its keys
// and few tokens still fill it; a unit is two tiles, one softmax warpgroup each, tokens after tokens, which stream
// the K and V blocks (128 keys) from the first to the last that any of its rows sees, in shared memory.  Roles, ring, online
// softmax with its lazy reference, and the O accumulators in tensor memory are the plain tile kernel's (tile_fwd_tc.cu):
//   warps 0-7  softmax, warp 8 MMA issuer, warp 9 producer (unit decode and TMA), warps 10-11 idle
//   TMEM (512 columns): S_0 | S_1 | O_0 | O_1; P_t overwrites S_t
// Rows see ranges: a warp masks a block only where it is not inside all of its rows' ranges, and a row that has met no key yet
// takes no maximum pass for a block that it does not see.
//
// Cap (MODE 2, with slopes 3).  tanh by a polynomial while the whole warp's scores of a block stay below the cap, of fewer
// steps below half of it, else by exponentials (score.cuh).  Slopes (MODE 1 and 3): one more FMA where a block lies on one side
// of all of the warp's rows, |i - j| only on the diagonal.
//
// Pages.  A block's keys are boxes of as many rows as a page (a power of two that divides it, 16 to 128), one lane of the producer
// warp a box and 64-column half; each lane looks the next block's page up a block ahead.  Boxes behind the last token, or
// before the first that any row's window holds, load a page that does not exist, which arrives as zeros; the other rows of the
// last token's box and of the first one's are zeroed in V before the product (a weight of 0 times NaN is NaN), and masked in S.
//
// Few units are cut into parts of their keys (score_fwd_shape), whose normalised outputs and LSEs merge_kernel adds up in order.
// P is rounded to bf16 for its product (2^-8 relative a term at most), everything else is fp32.
//
// Bound by the softmax warps: a block of 256 rows takes them 1.45 us plain (tensor pipe 74 % busy) and 2.3 to 2.5 with a cap
// (24 %).  Measured, bf16, d 128: 1,024 new tokens over 65,536 cached, 32 heads on 8, 740-760 us (1,440-1,470 TFLOP/s, 128 units
// on 152 SMs); 16,384 tokens of 16 heads, causal, one document 700 us (1,560), six documents 208 (1,030: units of 17 blocks, of
// which the change from one to the next costs five, and masked blocks at documents' edges); 2 x 2,500 with prefixes,
// capped, 52.
//
// Every mbarrier wait is bounded: a timeout records MESH_ATTN_ERR_DEVICE_TIMEOUT in the status
// block, every role of the CTA stops, in-flight copies and MMAs are drained and TMEM is freed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "score.cuh"
#include "score_fwd.h"
#include "tmap.h"

namespace mesh {
namespace sfw {

constexpr int BM = 128;  // rows per tile = TMEM lanes
constexpr int BN = 128;  // keys per KV block
constexpr int NST = 2;   // K/V ring stages
constexpr int NUM_THREADS = 384;
constexpr int SOFTMAX_REGS = 200;  // 2 x 128 x 200 + 128 x 104 <= 384 x 168 registers at launch
constexpr int OTHER_REGS = 104;
constexpr int WARP_MMA = 8;
constexpr int WARP_LOAD = 9;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;
constexpr float LOG2_RESCALE = 8.0f;
// Row sum of one block accepted without a max pass: every term is then at most 2^16, and a sum
// this large implies a row maximum more than 2^LOG2_RESCALE above the reference (2^16 / BN > 2^8).
constexpr float SUM_ACCEPT = 65536.0f;
constexpr int MAX_PARTS = MAX_FWD_PARTS;
constexpr int64_t DRAIN_NS = 200000000;  // exit-path waits for copies in flight
constexpr int ROLE_SOFTMAX = 1, ROLE_MMA = 2, ROLE_LOAD = 3, ROLE_SEQ = 4, ROLE_PAGE = 5;

template <int D>
struct Layout {
  static constexpr uint32_t TILE = BM * D * 2;  // bytes of one Q tile / K block / V block
  static constexpr uint32_t BOX = BM * 64 * 2;  // its 64-column half
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t K_OFF = Q_OFF + 2 * TILE;
  static constexpr uint32_t V_OFF = K_OFF + NST * TILE;
  static constexpr uint32_t EPI_OFF = V_OFF + NST * TILE;  // 8 softmax warps x 4 KB
  static constexpr uint32_t BAR_OFF = EPI_OFF + 8 * 4096;
  static constexpr int B_QFULL = 0, B_QEMPTY = 1, B_KFULL = 2, B_KEMPTY = B_KFULL + NST,
                       B_VFULL = B_KEMPTY + NST, B_VEMPTY = B_VFULL + NST, B_SFULL = B_VEMPTY + NST,
                       B_PFULL = B_SFULL + 2, B_OFINAL = B_PFULL + 2, B_OFREE = B_OFINAL + 2,
                       B_UFULL = B_OFREE + 2, B_UEMPTY = B_UFULL + 2, B_DRAIN = B_UEMPTY + 2,
                       NBARS = B_DRAIN + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBARS * 8 + (NBARS % 2) * 8;  // tmem base, abort flag
  static constexpr uint32_t RING_OFF = MISC_OFF + 16;  // unit ring: 2 decoded units, 16 ints each
  static constexpr uint32_t MINE_OFF = RING_OFF + 2 * 64;    // each softmax warp's unit, 16 ints
  static constexpr uint32_t TOTAL = MINE_OFF + 8 * 64;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
};
static_assert(Layout<128>::ALLOC <= 232448, "shared memory of a CTA");

struct Plan;
struct Params {
  const float* slopes;
  __nv_bfloat16* o;
  int64_t os[3];  // batch, head, token strides of O
  float* lse;
  int64_t ls[3];
  float* part_o;  // units in parts: [unit][part][tile][128][D] and [unit][part][tile][128]
  float* part_lse;
  int32_t* status;
  uint32_t* counter;
  const int32_t* lo;
  const int32_t* hi;
  int64_t mask_bs;
  const int32_t* offsets;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_s;
  int64_t S;
  int32_t N, B, Hq, Hkv, g, gh, tt, tu, hc, groups, lanes, batch, n_units, parts;
  int32_t n_pages, page, max_pages, max_new, window, box_rows;
  Plan* plan;  // paged, or NULL
  int32_t slots;  // parts that part_o has room for
  float scale_log2;
  Cap cap;
  int64_t wait_limit_ns;
};

// Paged, up to PLAN_GROUPS groups of tokens: what plan_kernel leaves.  The groups in the order of work, the longest first; each
// in k parts, of which the first of a lane is part first of all.
struct Group {
  int32_t b, tok0, k, slot;  // slot: parts of a lane's split groups before it
};
struct Plan {
  int32_t pieces, groups, split, pad;  // parts of a lane, groups with work, those of them in more than one part (the first ones)
  int32_t first[PLAN_GROUPS];
  Group group[PLAN_GROUPS];
};
static_assert(sizeof(Plan) == PLAN_BYTES, "the plan in the workspace");

// A unit: its rows are the tokens [tok0, tok0 + 2 tt) below n_tok of query heads h0 .. h0 + gh - 1 (below h_end), its keys the
// blocks [blk0, blk0 + NB).  Paged: the sequence's first new token is row `row0` of the batch and has the place pos0.
struct Unit {
  int u, b, hk, h0, h_end, tok0, n_tok, row0, pos0, len, blk0, NB;
  int slot;  // of a part of its keys' output in part_o, -1 for all of them
  int kmin;  // the first key that any row sees
  __device__ __forceinline__ int ntiles(int tt) const { return tok0 + tt < n_tok ? 2 : 1; }
  // Its i-th block: from the one of its last token's own key down to the first, then up from behind it.  So rows meet their own key
  // early, where a causal document or a slope has its largest weights, and the running maximum seldom grows (blocks from the first
  // on: 352 us where this takes 219, 16 heads on 4 of 8,192 tokens with slopes).
  __device__ __forceinline__ int mid(int tt) const {
    return min(max((pos0 + min(tok0 + 2 * tt, n_tok) - 1) / BN, blk0), blk0 + NB - 1);
  }
  __device__ __forceinline__ int block(int i, int tt) const {
    const int m = mid(tt);
    return i <= m - blk0 ? m - i : blk0 + i;
  }
};
template <bool PAGED>
__device__ __forceinline__ void put_unit(volatile int32_t* e, const Unit& x) {
  e[0] = x.u, e[1] = x.b, e[2] = x.hk, e[3] = x.h0, e[4] = x.h_end, e[5] = x.tok0, e[6] = x.n_tok, e[7] = x.row0;
  e[8] = x.pos0, e[9] = x.len, e[10] = x.blk0, e[11] = x.NB, e[12] = x.slot;
  if (PAGED) e[13] = x.kmin;  // for the MMA warp, else the producer's own
}
template <bool KMIN = false>
__device__ __forceinline__ Unit get_unit(const volatile int32_t* e) {
  Unit x;
  x.u = e[0], x.b = e[1], x.hk = e[2], x.h0 = e[3], x.h_end = e[4], x.tok0 = e[5], x.n_tok = e[6], x.row0 = e[7];
  x.pos0 = e[8], x.len = e[9], x.blk0 = e[10], x.NB = e[11], x.slot = e[12], x.kmin = KMIN ? e[13] : 0;
  return x;
}

// Sequence b of a batch over pages: its rows and keys, with what does not fit recorded (where `report`).
__device__ __forceinline__ void sequence(const Params& prm, int b, bool report, Unit& x) {
  const Asked s = asked(prm.offsets, prm.lens, b, prm.N, prm.max_new, prm.max_pages, prm.page);
  if (report && s.bad) record_error(prm.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_SEQ, b);
  x.b = b;
  x.row0 = s.begin;
  x.n_tok = s.n;
  x.len = s.len;
  x.pos0 = s.len - s.n;
}
__device__ __forceinline__ void keys_of(const Params& prm, Unit& x) {  // paged: of its group of tokens
  const int kmax = x.pos0 + min(x.tok0 + prm.tu, x.n_tok);
  x.kmin = prm.window ? max(0, x.pos0 + x.tok0 + 1 - prm.window) : 0;
  x.blk0 = x.kmin / BN;
  x.NB = (kmax + BN - 1) / BN - x.blk0;
}
// Part `part` of k of its blocks.
__device__ __forceinline__ void cut(Unit& x, int part, int k) {
  k = max(1, min(k, x.NB));
  const int n = x.NB, i = min(part, k), j = min(part + 1, k);
  x.blk0 += (int)((int64_t)i * n / k);
  x.NB = (int)((int64_t)j * n / k) - (int)((int64_t)i * n / k);
}
__device__ __forceinline__ void heads_of(const Params& prm, int ln, Unit& x) {  // of a lane
  const int c = ln % prm.hc;
  ln /= prm.hc;
  x.hk = ln % prm.Hkv;
  x.b = ln / prm.Hkv;
  x.h0 = x.hk * prm.g + c * prm.gh;
  x.h_end = min(x.h0 + prm.gh, (x.hk + 1) * prm.g);
}

// Unit u of a launch, decoded by a whole warp (without bounds: its rows alone).  Units are numbered batch of lanes by batch,
// within it from the last tokens (the most keys where the mask is causal) to the first, or in the plan's order, within those
// lane by lane, its parts together.  A lane is a (batch, KV head, chunk of heads); paged: a (KV head, chunk), whose groups are
// those of all sequences, sequence b's from offsets[b] / (2 tt) + b on: each has room for its own there, and a few are empty
// (n_tok = 0).
template <bool PAGED>
__device__ __forceinline__ Unit decode(int u, const Params& prm, bool bounds, const Plan* plan) {
  Unit x;
  const int lane = threadIdx.x & 31, tu = prm.tu;
  x.u = u;
  int groups = prm.groups, batch = prm.batch;
  if (PAGED && plan) {
    groups = plan->pieces;
    batch = min(prm.lanes, (3 * (int)gridDim.x + groups - 1) / groups);
  }
  int t = prm.parts > 1 ? u / prm.parts : u;
  const int per = batch * groups, first = t / per * batch;
  const int lanes = min(batch, prm.lanes - first);  // the last batch may be smaller
  t %= per;
  const int idx = t / lanes, grp = prm.groups - 1 - idx, ln = first + t % lanes;
  heads_of(prm, ln, x);
  x.slot = prm.parts > 1 ? u : -1;
  x.blk0 = x.NB = x.kmin = 0;
  if (PAGED && plan) {
    const int e = last_begun_warp(plan->first, plan->groups, idx);
    const Group g = plan->group[e];
    sequence(prm, g.b, false, x);
    x.tok0 = g.tok0;
    keys_of(prm, x);
    if (g.k > 1) {
      const int part = idx - plan->first[e];
      x.slot = g.slot * prm.lanes + ln * g.k + part;
      cut(x, part, g.k);
    }
    return x;
  }
  if (PAGED) {
    // the last b with offsets[b] / tu + b <= grp
    int a = 0, n = prm.B;
    while (n > 0) {
      const int step = (n + 31) / 32, at = a + lane * step;
      const bool in = at < a + n;
      const unsigned m = __ballot_sync(0xffffffffu, in && max(prm.offsets[in ? at : 0], 0) / tu + at <= grp);
      const int k = __popc(m);
      if (k == 0) break;
      const int end = a + n;
      a += (k - 1) * step + 1;
      n = min(step - 1, end - a);
    }
    if (a == 0) {
      x.b = 0, x.tok0 = x.n_tok = x.row0 = x.pos0 = x.len = 0;
      return x;
    }
    sequence(prm, a - 1, bounds && lane == 0, x);
    x.tok0 = (grp - (x.row0 / tu + x.b)) * tu;
    if (x.tok0 < 0 || x.tok0 >= x.n_tok) {  // below 0 where offsets do not ascend
      x.tok0 = x.n_tok = 0;
      return x;
    }
    if (bounds) keys_of(prm, x);
    x.n_tok = min(x.n_tok, x.tok0 + tu);
    return x;
  }
  x.tok0 = grp * tu;
  x.n_tok = min((int)prm.S, x.tok0 + tu);
  x.row0 = x.pos0 = 0;
  x.len = (int)prm.S;
  if (!bounds) return x;
  const int32_t* lo = prm.lo + x.b * prm.mask_bs;
  const int32_t* hi = prm.hi + x.b * prm.mask_bs;
  int kmin = 0x7fffffff, kmax = 0;              // keys that some row sees
  int a[2 * BM / 32], z[2 * BM / 32];  // all loads in flight together
#pragma unroll
  for (int e = 0; e < 2 * BM / 32; ++e) {
    const int i = e * 32 + lane;
    const bool in = i < tu && x.tok0 + i < x.n_tok;
    a[e] = in ? lo[x.tok0 + i] : 0;
    z[e] = in ? hi[x.tok0 + i] : 0;
  }
#pragma unroll
  for (int e = 0; e < 2 * BM / 32; ++e) {
    a[e] = max(a[e], 0);
    z[e] = min(z[e], x.len);
    if (a[e] < z[e]) {
      kmin = min(kmin, a[e]);
      kmax = max(kmax, z[e]);
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (kmin < kmax) {
    x.kmin = kmin;
    x.blk0 = kmin / BN;
    x.NB = (kmax + BN - 1) / BN - x.blk0;
  }
  if (x.slot >= 0) cut(x, u % prm.parts, prm.parts);
  return x;
}

// The plan of a batch over pages, by one CTA, a thread a group; it also puts the unit counter to zero.  A batch of chunks and
// single tokens ends when its longest units do, so those start first: 16 sequences of up to 4,096 tokens, 2,048 new ones in
// four of them, 16 heads on 4, capped, 91-95 us, where units as they come take 108-130.  The kernel itself costs a call 3 us.
//
// Parts.  The SMs' share of all blocks, three more a group for its start (5 us at 1.6 us a block), is what a group should take.
// Those of twice that and more, and of eight blocks or more, are cut into parts of a share, whose outputs merge_kernel adds up
// (200 new tokens of three sequences of up to 16,000: 63 us; 288 whole).  Parts that save less than half of the longest unit do
// not pay for their fp32 rows' way through memory.
template <bool PAGED>
__global__ void __launch_bounds__(PLAN_GROUPS) plan_kernel(const __grid_constant__ Params prm, int sms) {
  __shared__ __align__(16) int32_t nb[PLAN_GROUPS];  // blocks of a group, 0 for one without work
  __shared__ int32_t parts[PLAN_GROUPS], sums[PLAN_GROUPS / 32];  // parts in the order of work; sums of the warps
  __shared__ unsigned long long total;
  __shared__ int32_t split, split_parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = prm.groups, tu = prm.tu;
  if (tid == 0) total = 0ull, split = split_parts = 0;
  nb[tid] = 0;
  __syncthreads();
  wait_for_kernel_before();
  if (tid == 0) *prm.counter = 0u;
  Unit x;
  x.NB = 0;
  {
    int a = 0, z = tid < n ? prm.B : 0;  // the last b with offsets[b] / tu + b <= tid, or 0
    while (z - a > 1) {
      const int c = (a + z) >> 1;
      if (max(prm.offsets[c], 0) / tu + c <= tid) a = c;
      else z = c;
    }
    if (tid < n) {
      sequence(prm, a, true, x);
      const int64_t t0 = ((int64_t)tid - (x.row0 / tu + a)) * tu;
      if (t0 >= 0 && t0 < x.n_tok) {
        x.tok0 = (int)t0;
        keys_of(prm, x);
        nb[tid] = x.NB;
      }
    }
    const unsigned c = __reduce_add_sync(0xffffffffu, x.NB ? (unsigned)x.NB + 3u : 0u);
    if (lane == 0 && c) atomicAdd(&total, (unsigned long long)c);
  }
  const int have = __syncthreads_count(x.NB > 0), mine = x.NB;
  const int64_t share = ((int64_t)total * prm.lanes + sms - 1) / sms;
  int rank = 0;  // groups with more blocks, or as many and a higher number
  if (mine) {
    for (int i = 0; i < n; i += 4) {
      const int4 o = *reinterpret_cast<const int4*>(nb + i);
      rank += (o.x > mine || (o.x == mine && i > tid)) + (o.y > mine || (o.y == mine && i + 1 > tid)) +
              (o.z > mine || (o.z == mine && i + 2 > tid)) + (o.w > mine || (o.w == mine && i + 3 > tid));
    }
    parts[rank] = mine >= 8 ? (int)max((int64_t)1, min((int64_t)MAX_PARTS, mine / share)) : 1;
  }
  __syncthreads();
  // those to be split come first, as many as part_o has room for
  int k = tid < have ? parts[tid] : 1;
  const int want = k > 1 ? k : 0;
  int before = want;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) sums[warp] = before;
  __syncthreads();
  before -= want;
  for (int w = 0; w < warp; ++w) before += sums[w];
  if (k > 1 && (int64_t)(before + k) * prm.lanes > prm.slots) k = 1;
  if (k > 1) {
    atomicAdd(&split, 1);
    atomicAdd(&split_parts, k);
  }
  __syncthreads();
  Plan* plan = prm.plan;
  if (tid < have) {
    plan->first[tid] = k > 1 ? before : split_parts + tid - split;
    plan->group[tid].k = k;
    plan->group[tid].slot = before;
  }
  if (mine) plan->group[rank].b = x.b, plan->group[rank].tok0 = x.tok0;
  if (tid == 0) plan->pieces = split_parts + have - split, plan->groups = have, plan->split = split;
}

// Keys of a row by its token.
template <bool PAGED>
__device__ __forceinline__ void range_of(const Params& prm, const Unit& x, int tok, int& lo, int& hi, int& pos) {
  if (PAGED) {
    pos = x.pos0 + tok;
    hi = pos + 1;
    lo = prm.window ? max(0, hi - prm.window) : 0;
  } else {
    pos = tok;
    lo = max(prm.lo[x.b * prm.mask_bs + tok], 0);
    hi = min(prm.hi[x.b * prm.mask_bs + tok], x.len);
    if (lo >= hi) lo = hi = 0;
  }
}

// What is computed from x stays behind this: the columns' 128 biases, alike in both passes over a block, would else be kept in
// registers that are not there.
__device__ __forceinline__ void keep_here(float& x) { asm volatile("" : "+f"(x)); }

template <int D, int MODE, bool PAGED>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params prm) {
  using Ly = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;  // 1024-aligned base (128-byte swizzle atoms)
  uint8_t* smem = smem_raw + (sb - raw);
  constexpr bool SLOPES = MODE == 1 || MODE == 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + Ly::BAR_OFF + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::MISC_OFF);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(smem + Ly::MISC_OFF + 4);
  volatile int32_t* ring = reinterpret_cast<volatile int32_t*>(smem + Ly::RING_OFF);

  if (threadIdx.x == 0) {
    mbar_init(bar(Ly::B_QFULL), 1);
    mbar_init(bar(Ly::B_QEMPTY), 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(Ly::B_KFULL + s), 1);
      mbar_init(bar(Ly::B_KEMPTY + s), 1);
      mbar_init(bar(Ly::B_VFULL + s), 1);
      mbar_init(bar(Ly::B_VEMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(Ly::B_SFULL + t), 1);
      mbar_init(bar(Ly::B_PFULL + t), BM);
      mbar_init(bar(Ly::B_OFINAL + t), 1);
      mbar_init(bar(Ly::B_OFREE + t), BM);
      mbar_init(bar(Ly::B_UFULL + t), 1);
      mbar_init(bar(Ly::B_UEMPTY + t), 1 + 8);  // one lane of the MMA warp and of each softmax warp
    }
    mbar_init(bar(Ly::B_DRAIN), 1);
    wait_for_kernel_before();
    // without any time to wait there is nothing to start: the first load would be waited for
    if (prm.wait_limit_ns <= 0) {
      record_error(prm.status, MESH_ATTN_ERR_DEVICE_TIMEOUT, ROLE_LOAD, -1);
      if (PAGED) timeout_takes_over(prm.status);
    }
    *abort_flag = stopped<PAGED>(prm.status) ? 1 : 0;
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
    const int t = warp >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t tm_s = tmem + lane_base + (uint32_t)(t * 128);
    const uint32_t tm_o = tmem + lane_base + 256u + (uint32_t)(t * 128);
    float* epi = reinterpret_cast<float*>(smem + Ly::EPI_OFF + (uint32_t)warp * 4096u);
    const int row_h = row / prm.tt, row_t = row - row_h * prm.tt;  // its head and token within the tile
    volatile int32_t* mine = reinterpret_cast<volatile int32_t*>(smem + Ly::MINE_OFF + (uint32_t)warp * 64u);
    int nu = 0, cnt = 0, uses = 0;
    bool ok = true;
    while (ok) {
      const int slot = nu & 1;
      ok = mbar_wait(bar(Ly::B_UFULL + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                     ROLE_SOFTMAX, -1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the unit stays in shared memory, the warp's own copy: the block loop has no registers to spare
      if (lane < 13) mine[lane] = ring[16 * slot + lane];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_UEMPTY + slot));
      ++nu;
      int NB, blk0, mid;  // its blocks: mid down to blk0, then up from mid + 1
      bool valid;
      int lo = 0, hi = 0, pos = 0;
      float slope2 = 0.f;
      {
        const Unit x = get_unit(mine);
        if (x.u < 0) break;
        if (t >= x.ntiles(prm.tt) || x.n_tok == 0) continue;
        NB = __reduce_max_sync(0xffffffffu, x.NB);  // in uniform registers
        blk0 = __reduce_max_sync(0xffffffffu, x.blk0);
        mid = __reduce_max_sync(0xffffffffu, x.mid(prm.tt));
        const int tok = x.tok0 + t * prm.tt + row_t, h = x.h0 + row_h;
        valid = row_h < prm.gh && h < x.h_end && tok < x.n_tok;
        if (valid) {
          range_of<PAGED>(prm, x, tok, lo, hi, pos);
          if (SLOPES) slope2 = prm.slopes[h] * LOG2E;
        }
      }
      // keys that all of the warp's rows see, and the places between which its rows lie
      const int all_lo = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
      const int all_hi = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
      int pmin = 0, pmax = 0;
      if (SLOPES) {
        pmin = __reduce_min_sync(0xffffffffu, valid ? pos : 0x7fffffff);
        pmax = __reduce_max_sync(0xffffffffu, valid ? pos : -1);
      }
      float m_used = valid ? -INFINITY : 0.f, l_sum = 0.f;
      int tier = 0;  // of the cap
      for (int j = 0; j < NB; ++j, ++cnt) {
        ok = mbar_wait(bar(Ly::B_SFULL + t), (uint32_t)(cnt & 1), prm.wait_limit_ns, abort_flag, prm.status,
                       ROLE_SOFTMAX, j);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int j0 = (j <= mid - blk0 ? mid - j : blk0 + j) * BN;
        const bool edge = all_lo > j0 || all_hi < j0 + BN;
        const bool sees = lo < j0 + BN && hi > j0;
        // The exponentials use the row's running reference m_used, which only ever grows.  A
        // block whose row maximum stays within 2^LOG2_RESCALE of it needs no maximum at all, so
        // the common case skips the max pass: exponentiate against m_used and accept the block
        // when its row sum is at most SUM_ACCEPT (every term is then bounded as well).  A row
        // without a reference yet that sees a key of the block, or a block whose sum is too large
        // or not finite, takes the row maximum first, raising m_used (and rescaling O and l)
        // when it grew by more than 2^LOG2_RESCALE, and the exponentials are redone.
        bool need_max = __any_sync(0xffffffffu, m_used == -INFINITY && sees);
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
          if (MODE >= 2) {
            cap_scores(prm.cap, s, tier, valid, [&]() {
#pragma unroll
              for (int c = 0; c < BN; c += 32) tmem_ld32(tm_s + (uint32_t)c, s + c);
              tc_wait_ld();
            });
          }
          if (SLOPES) {
            const float sc = MODE == 3 ? 1.f : prm.scale_log2;
            const bool before = j0 + BN - 1 <= pmin, behind = j0 >= pmax;
            if (before || behind) {  // |i - j| = +-(i - j): linear in the column
              const float sl = before ? slope2 : -slope2;
              float base = sl * (float)(j0 - pos);
              keep_here(base);
#pragma unroll
              for (int c = 0; c < BN; ++c) s[c] = fmaf(s[c], sc, fmaf(sl, (float)c, base));
            } else {
              float off = (float)(j0 - pos);
              keep_here(off);
#pragma unroll
              for (int c = 0; c < BN; ++c) s[c] = fmaf(s[c], sc, -slope2 * fabsf(off + (float)c));
            }
          }
          if (edge) {
            asm volatile("" ::: "memory");  // a branch, not selects that every block would run
            const int a = lo - j0, n = hi - lo;
#pragma unroll
            for (int c = 0; c < BN; ++c)
              if ((uint32_t)(c - a) >= (uint32_t)n) s[c] = -INFINITY;
          }
          constexpr bool RAW = MODE == 0;  // s is not scaled yet
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
            const float mx = fmaxf(max3f(mc[0], mc[1], mc[2]), mc[3]);
            const float m_new = RAW ? mx * prm.scale_log2 : mx;
            if (valid && m_new > -INFINITY) {
              if (m_used == -INFINITY) {
                m_used = m_new;
              } else if (m_new > m_used + LOG2_RESCALE) {
                factor *= fast_exp2(m_used - m_new);
                m_used = m_new;
              }
            }
          }
          const float mref = (m_used == -INFINITY) ? 0.f : m_used;
          // p = 2^(x - m): two elements per FMA or ADD, four independent sum chains
          const uint64_t sc2 = f2_pack(prm.scale_log2, prm.scale_log2);
          const uint64_t nm2 = f2_pack(-mref, -mref);
          uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int c = 0; c < BN / 2; ++c) {
            float x0, x1;
            const uint64_t s2 = f2_pack(s[2 * c], s[2 * c + 1]);
            f2_unpack(RAW ? f2_fma(s2, sc2, nm2) : f2_add(s2, nm2), x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            acc2[c & 3] = f2_add(acc2[c & 3], f2_pack(p0, p1));
            pk[c] = pack_bf16x2(p0, p1);
          }
          float sa, sb2;
          f2_unpack(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])), sa, sb2);
          blk = sa + sb2;
          // NaN fails the comparison: a NaN row takes the max pass once and is then accepted
          if (pass == 1 || __all_sync(0xffffffffu, !valid || blk <= SUM_ACCEPT)) break;
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
      if (!ok) break;
      // ---- epilogue: O_t out of TMEM
      const Unit x = get_unit(mine);
      const int tok = x.tok0 + t * prm.tt + row_t, h = x.h0 + row_h;
      // a row without a visible key: O = 0, LSE = -inf (a NaN sum stays NaN).  What its accumulator holds is a sum of
      // zeros, or nothing where the unit has no blocks
      const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
      const float lse = l_sum == 0.f ? -INFINITY : (m_used + log2f(l_sum)) * LN2;
      if (x.NB > 0) {
        ok = mbar_wait(bar(Ly::B_OFINAL + t), (uint32_t)(uses & 1), prm.wait_limit_ns, abort_flag, prm.status,
                       ROLE_SOFTMAX, x.u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      if (x.slot < 0) {
        uint32_t w[D / 2];
#pragma unroll
        for (int c = 0; c < D / 2; ++c) w[c] = 0u;
        if (x.NB > 0) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tm_o + (uint32_t)c, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              w[(c + e) / 2] = l_sum == 0.f ? 0u : pack_bf16x2(o[e] * inv, o[e + 1] * inv);
          }
          tc_fence_before();
          mbar_arrive(bar(Ly::B_OFREE + t));
          ++uses;
        }
        const int64_t bo = PAGED ? 0 : x.b, to = (int64_t)x.row0 + tok;
        const int64_t at = valid ? bo * prm.os[0] + h * prm.os[1] + to * prm.os[2] : -1;
        uint4* stage = reinterpret_cast<uint4*>(epi);
        // 32 rows x 64 columns through the stage, 16-byte pieces swizzled by row: a store writes four whole 128-byte lines
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            stage[lane * 8 + (q ^ (lane & 7))] =
                make_uint4(w[c / 2 + 4 * q], w[c / 2 + 4 * q + 1], w[c / 2 + 4 * q + 2], w[c / 2 + 4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), q = lane & 7;
            const int64_t ra = __shfl_sync(0xffffffffu, at, r);
            const uint4 v = stage[r * 8 + (q ^ (r & 7))];
            if (ra >= 0) *reinterpret_cast<uint4*>(prm.o + ra + c + q * 8) = v;
          }
        }
        if (valid) prm.lse[bo * prm.ls[0] + h * prm.ls[1] + to * prm.ls[2]] = lse;
        continue;
      }
      // ---- a part: its normalised output, in fp32
      const int64_t prow = ((int64_t)x.slot * 2 + t) * BM + row;
      if (x.NB > 0) {
        float* dst0 = prm.part_o + (prow - lane) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tm_o + (uint32_t)c, o);
          tc_wait_ld();
          __syncwarp();
          // 32 rows x 32 columns: 16-byte chunks swizzled by row, read back 4 rows per store
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(epi + lane * 32 + ((q ^ (lane & 7)) * 4)) =
                make_float4(o[4 * q] * inv, o[4 * q + 1] * inv, o[4 * q + 2] * inv, o[4 * q + 3] * inv);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), qq = lane & 7;
            const float4 v = *reinterpret_cast<const float4*>(epi + r * 32 + ((qq ^ (r & 7)) * 4));
            *reinterpret_cast<float4*>(dst0 + (int64_t)r * D + c + qq * 4) = v;
          }
        }
        tc_fence_before();
        mbar_arrive(bar(Ly::B_OFREE + t));
        ++uses;
      }
      prm.part_lse[prow] = valid ? lse : -INFINITY;
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
      // low 14 bits, address / 16) advances by a compile-time offset.
      const uint64_t q_desc0 = smem_desc_sw128(sb + Ly::Q_OFF, 16u, 1024u);
      const uint64_t k_desc0 = smem_desc_sw128(sb + Ly::K_OFF, 16u, 1024u);
      const uint64_t v_desc0 = smem_desc_sw128(sb + Ly::V_OFF, Ly::BOX, 1024u);
      constexpr uint64_t TILE16 = Ly::TILE >> 4, BOX16 = Ly::BOX >> 4;
      // K-major operand (Q or K): K-step kk of 16 elements sits in box kk/4 at byte 32*(kk%4)
      auto kmaj_off = [](int kk) { return (uint64_t)((kk >> 2) * BOX16 + (kk & 3) * 2); };
      // MN-major V: K-step kk covers key rows 16kk..16kk+15 (two 8-row swizzle atoms, 2048
      // bytes); the second 64-column half of d is the next box (leading byte offset)
      auto issue_s = [&](int t, int stage) {
        const uint64_t qd = q_desc0 + (uint64_t)t * TILE16;
        const uint64_t kd = k_desc0 + (uint64_t)stage * TILE16;
        const uint32_t d_tm = tmem + (uint32_t)(t * 128);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) tc_mma_ss_warp(d_tm, qd + kmaj_off(kk), kd + kmaj_off(kk), idesc_qk, kk > 0);
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
      int nu = 0, nq = 0, nblk = 0;
      int cnt[2] = {0, 0}, uses[2] = {0, 0};
      bool ok = true;
      while (ok) {
        const int slot = nu & 1;
        ok = mbar_wait_warp(bar(Ly::B_UFULL + slot), (uint32_t)((nu >> 1) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                            ROLE_MMA, -1);
        if (!ok) break;
        const Unit x = get_unit<PAGED>(ring + 16 * slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_UEMPTY + slot));
        __syncwarp();
        ++nu;
        const int u = x.u;
        if (u < 0) break;
        const int NB = x.NB;
        if (NB == 0 || x.n_tok == 0) continue;
        const int ntiles = x.ntiles(prm.tt);
        // paged: the blocks whose boxes hold rows behind the last token or before all windows, or -1
        const int ragged_end = (x.len & (prm.box_rows - 1)) ? x.len / BN : -1;
        const int ragged_first = (x.kmin & (prm.box_rows - 1)) ? x.kmin / BN : -1;
        const int uidx = nq++;
        ok = mbar_wait_warp(bar(Ly::B_QFULL), (uint32_t)(uidx & 1), prm.wait_limit_ns, abort_flag, prm.status, ROLE_MMA, u);
        if (ok)
          ok = mbar_wait_warp(bar(Ly::B_KFULL + nblk % NST), (uint32_t)((nblk / NST) & 1), prm.wait_limit_ns, abort_flag,
                              prm.status, ROLE_MMA, u);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < ntiles; ++t) issue_s(t, nblk % NST);
        if (NB == 1) tc_commit_warp(bar(Ly::B_QEMPTY));
        tc_commit_warp(bar(Ly::B_KEMPTY + nblk % NST));
        for (int j = 0; j < NB && ok; ++j) {
          const int g = nblk + j;
          const int st = g % NST;
          ok = mbar_wait_warp(bar(Ly::B_VFULL + st), (uint32_t)((g / NST) & 1), prm.wait_limit_ns, abort_flag, prm.status,
                              ROLE_MMA, u);
          if (PAGED && ok) {
            // the last token's box may go on behind it, with whatever an earlier owner left, and the first one's begin before any
            // row's window: zeros there
            const int jb = x.block(j, prm.tt);
            if (jb == ragged_end || jb == ragged_first) {
              uint8_t* vs = smem + Ly::V_OFF + (uint32_t)st * Ly::TILE;
#pragma unroll 1
              for (int i = lane; i < BN * 8; i += 32) {
                const int key = jb * BN + (i >> 3);
                if (key >= x.kmin && key < x.len) continue;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  *reinterpret_cast<uint4*>(vs + (uint32_t)c * Ly::BOX + (uint32_t)i * 16u) = make_uint4(0u, 0u, 0u, 0u);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
          for (int t = 0; t < ntiles && ok; ++t) {
            ok = mbar_wait_warp(bar(Ly::B_PFULL + t), (uint32_t)(cnt[t] & 1), prm.wait_limit_ns, abort_flag, prm.status,
                                ROLE_MMA, u);
            if (ok && j == 0 && uses[t] > 0)  // the previous unit's epilogue has copied O_t out
              ok = mbar_wait_warp(bar(Ly::B_OFREE + t), (uint32_t)((uses[t] - 1) & 1), prm.wait_limit_ns, abort_flag,
                                  prm.status, ROLE_MMA, u);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, st, j == 0);
            ++cnt[t];
            if (j + 1 == NB) {  // tile t's last product of the unit: its epilogue may start
              tc_commit_warp(bar(Ly::B_OFINAL + t));
              ++uses[t];
            }
            if (j + 1 < NB) {
              const int sn = (g + 1) % NST;
              if (t == 0) {
                ok = mbar_wait_warp(bar(Ly::B_KFULL + sn), (uint32_t)(((g + 1) / NST) & 1), prm.wait_limit_ns, abort_flag,
                                    prm.status, ROLE_MMA, u);
                if (!ok) break;
                tc_fence_after();
              }
              issue_s(t, sn);
            }
          }
          if (!ok) break;
          if (j + 1 < NB) tc_commit_warp(bar(Ly::B_KEMPTY + (g + 1) % NST));
          if (j + 2 == NB) tc_commit_warp(bar(Ly::B_QEMPTY));  // the unit's last S products are issued
          tc_commit_warp(bar(Ly::B_VEMPTY + st));
        }
        if (!ok) break;
        nblk += NB;
      }
      // exit-path drain: every MMA issued completes before TMEM is freed
      tc_commit_warp(bar(Ly::B_DRAIN));
      mbar_drain(bar(Ly::B_DRAIN), 0u, DRAIN_NS);
    } else if (warp == WARP_LOAD) {
      // ================================================================ producer: the whole warp, converged
      int nu = 0, nq = 0, nk = 0;
      bool ok = __all_sync(0xffffffffu, *abort_flag == 0);
      Unit next;
      const Plan* plan = PAGED ? prm.plan : nullptr;
      const int n_units = PAGED && plan ? plan->pieces * prm.lanes : prm.n_units;
      // a CTA's first unit is its own index, the others come from the counter; decoded and published to the consumers' ring
      auto publish = [&]() {
        const int slot = nu & 1;
        ok = mbar_wait_warp(bar(Ly::B_UEMPTY + slot), (uint32_t)(((nu >> 1) & 1) ^ 1), prm.wait_limit_ns, abort_flag,
                            prm.status, ROLE_LOAD, -1);
        if (!ok) return;
        int v = (int)blockIdx.x;
        if (nu > 0) {
          v = n_units;
          if (n_units > (int)gridDim.x) {
            if (lane == 0) v = (int)(gridDim.x + atomicAdd(prm.counter, 1u));
            v = __shfl_sync(0xffffffffu, v, 0);
          }
        }
        if (v < n_units) {
          next = decode<PAGED>(v, prm, true, plan);
        } else {
          next.u = -1;
        }
        if (lane == 0) {
          put_unit<PAGED>(ring + 16 * slot, next);
          mbar_arrive(bar(Ly::B_UFULL + slot));
        }
        __syncwarp();
        ++nu;
      };
      // this lane's box of a block: 64-column half `bc`, rows [br, br + box_rows)
      const int n_box = (D / 64) * (BN / prm.box_rows);
      const int bc = lane % (D / 64), br = lane / (D / 64) * prm.box_rows;
      // where that box of block jb lies: {row, page or batch}
      auto where = [&](const Unit& x, int jb, int& r, int& p) {
        const int key = jb * BN + br;
        if (!PAGED) {
          r = key;
          p = x.b;
          return;
        }
        r = 0;
        p = prm.n_pages;  // no such page: zeros
        if (lane < n_box && key < x.len && key + prm.box_rows > x.kmin) {  // pages before a window need not be there any more
          const int at = key / prm.page;
          r = key - at * prm.page;
          p = prm.table[x.b * prm.table_s + at];
          if (p < 0 || p >= prm.n_pages) {
            record_error(prm.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_PAGE, x.b);
            p = prm.n_pages;
          }
        }
      };
      if (ok) publish();
      while (ok && next.u >= 0) {
        const Unit x = next;
        // the following unit, once this one's first loads are on their way
        auto follow = [&]() {
          publish();
          if (ok && next.u >= 0 && next.NB > 0 && next.n_tok > 0) {
            // its Q tiles and first K and V block into L2, so that the unit boundary does not wait on DRAM
            if (lane < next.ntiles(prm.tt) * (D / 64))
              tma_prefetch_l2_3d(&tmQ, lane % (D / 64) * 64, next.row0 + next.tok0 + lane / (D / 64) * prm.tt,
                                 (PAGED ? 0 : next.b * prm.Hq) + next.h0);
            int rn, pn;
            where(next, next.block(0, prm.tt), rn, pn);
            if (lane < n_box) {
              tma_prefetch_l2_4d(&tmK, bc * 64, rn, next.hk, pn);
              tma_prefetch_l2_4d(&tmV, bc * 64, rn, next.hk, pn);
            }
          }
        };
        if (x.NB == 0 || x.n_tok == 0) {
          follow();
          continue;
        }
        int r, p;
        where(x, x.block(0, prm.tt), r, p);
        // Q tiles: the previous unit's last S products must be done with the Q buffer
        ok = mbar_wait_warp(bar(Ly::B_QEMPTY), (uint32_t)((nq & 1) ^ 1), prm.wait_limit_ns, abort_flag, prm.status,
                            ROLE_LOAD, x.u);
        if (!ok) break;
        const int ntiles = x.ntiles(prm.tt);
        if (lane == 0) mbar_expect_tx(bar(Ly::B_QFULL), (uint32_t)(ntiles * prm.gh * prm.tt) * D * 2u);
        __syncwarp();
        if (lane < ntiles * (D / 64)) {
          const int t = lane / (D / 64), c = lane % (D / 64);
          tma_load_3d(sb + Ly::Q_OFF + (uint32_t)t * Ly::TILE + (uint32_t)c * Ly::BOX, &tmQ, c * 64,
                      x.row0 + x.tok0 + t * prm.tt, (PAGED ? 0 : x.b * prm.Hq) + x.h0, bar(Ly::B_QFULL));
        }
        ++nq;
        for (int j = 0; j < x.NB; ++j) {
          const int st = nk % NST;
          const uint32_t ph = (uint32_t)((nk / NST) & 1);
          const int r0 = r, p0 = p;
          if (j + 1 < x.NB) where(x, x.block(j + 1, prm.tt), r, p);
          ok = mbar_wait_warp(bar(Ly::B_KEMPTY + st), ph ^ 1u, prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, x.u);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(Ly::B_KFULL + st), Ly::TILE);
          __syncwarp();
          const uint32_t at = (uint32_t)st * Ly::TILE + (uint32_t)bc * Ly::BOX + (uint32_t)br * 128u;
          if (lane < n_box) tma_load_4d(sb + Ly::K_OFF + at, &tmK, bc * 64, r0, x.hk, p0, bar(Ly::B_KFULL + st));
          ok = mbar_wait_warp(bar(Ly::B_VEMPTY + st), ph ^ 1u, prm.wait_limit_ns, abort_flag, prm.status, ROLE_LOAD, x.u);
          if (!ok) {  // K's block is on its way, V's is not
            mbar_drain(bar(Ly::B_KFULL + st), ph, DRAIN_NS);
            break;
          }
          if (lane == 0) mbar_expect_tx(bar(Ly::B_VFULL + st), Ly::TILE);
          __syncwarp();
          if (lane < n_box) tma_load_4d(sb + Ly::V_OFF + at, &tmV, bc * 64, r0, x.hk, p0, bar(Ly::B_VFULL + st));
          ++nk;
          if (j == 0) {
            follow();
            if (!ok) break;
          }
        }
      }
      // exit-path drain: every load issued lands before the CTA exits
      __syncwarp();
      if (nq > 0) mbar_drain(bar(Ly::B_QFULL), (uint32_t)((nq - 1) & 1), DRAIN_NS);
      for (int jj = (nk > NST ? nk - NST : 0); jj < nk; ++jj) {
        mbar_drain(bar(Ly::B_KFULL + jj % NST), (uint32_t)((jj / NST) & 1), DRAIN_NS);
        mbar_drain(bar(Ly::B_VFULL + jj % NST), (uint32_t)((jj / NST) & 1), DRAIN_NS);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (PAGED && threadIdx.x == 0 && *abort_flag) timeout_takes_over(prm.status);
}

// O = sum_t w_t O_t over a unit's parts, w_t = exp(lse_t - lse), and the LSE.  A thread takes a 16-byte piece of a row,
// all parts' loads in flight together; a CTA a few rows, so that the few units there are still fill the GPU.
constexpr int MERGE_THREADS = 256;
template <int D>
constexpr int MERGE_ROWS = MERGE_THREADS / (D / 4);
// A row's 16 bytes: `base` its row of the first of k parts, h and tok its head and token.
template <int D, bool PAGED>
__device__ __forceinline__ void merge_row(const Params& prm, const Unit& x, int64_t base, int parts, int h, int tok, int c) {
  float w[MAX_PARTS];
  float4 v[MAX_PARTS];
  float M = -INFINITY;
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k) {
    w[k] = k < parts ? prm.part_lse[base + (int64_t)2 * k * BM] : -INFINITY;
    M = fmaxf(M, w[k]);
  }
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k)
    v[k] = w[k] != -INFINITY ? __ldcs(reinterpret_cast<const float4*>(prm.part_o + (base + (int64_t)2 * k * BM) * D + c))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
  const float Ms = M == -INFINITY ? 0.f : M;
  float W = 0.f;
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k) {
    w[k] = __expf(w[k] - Ms);
    W += w[k];
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;  // a NaN sum stays NaN
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k) {
    const float f = w[k] * inv;
    o.x = fmaf(f, v[k].x, o.x);
    o.y = fmaf(f, v[k].y, o.y);
    o.z = fmaf(f, v[k].z, o.z);
    o.w = fmaf(f, v[k].w, o.w);
  }
  const int64_t bo = PAGED ? 0 : x.b, to = (int64_t)x.row0 + tok;
  *reinterpret_cast<uint2*>(prm.o + bo * prm.os[0] + h * prm.os[1] + to * prm.os[2] + c) =
      make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (c == 0) prm.lse[bo * prm.ls[0] + h * prm.ls[1] + to * prm.ls[2]] = W == 0.f ? -INFINITY : Ms + logf(W);
}
template <int D, bool PAGED>
__global__ void __launch_bounds__(MERGE_THREADS) merge_kernel(const __grid_constant__ Params prm) {
  constexpr int Q4 = D / 4, ROWS = MERGE_ROWS<D>, PER_UNIT = 2 * BM / ROWS;
  wait_for_kernel_before();
  if (stopped<PAGED>(prm.status)) return;
  const Plan* plan = prm.plan;
  const int n = PAGED ? plan->split * prm.lanes * PER_UNIT : (int)gridDim.x;
  for (int i = (int)blockIdx.x; i < n; i += (int)gridDim.x) {
    const int unit = i / PER_UNIT;  // before the cut
    const int r = i % PER_UNIT * ROWS + (int)threadIdx.x / Q4, c = (int)threadIdx.x % Q4 * 4;
    Unit x;
    int64_t slot;
    int parts;
    if (PAGED) {
      const Group g = plan->group[unit / prm.lanes];
      const int ln = unit % prm.lanes;
      heads_of(prm, ln, x);
      sequence(prm, g.b, false, x);
      x.tok0 = g.tok0;
      slot = (int64_t)g.slot * prm.lanes + ln * g.k;
      parts = g.k;
    } else {
      x = decode<PAGED>(unit * prm.parts, prm, false, nullptr);
      slot = (int64_t)unit * prm.parts;
      parts = prm.parts;
    }
    const int t = r / BM, row = r % BM, row_h = row / prm.tt;
    const int tok = x.tok0 + t * prm.tt + row - row_h * prm.tt, h = x.h0 + row_h;
    if (row_h < prm.gh && h < x.h_end && tok < x.n_tok)
      merge_row<D, PAGED>(prm, x, (slot * 2 + t) * BM + row, parts, h, tok, c);
  }
}

// ------------------------------------------------------------------ host side
template <int D, int MODE, bool PAGED>
static int launch_mode(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Params& prm, int sms,
                       cudaStream_t st, std::string* err) {
  auto kern = fwd_kernel<D, MODE, PAGED>;
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  cudaError_t e = cudaSuccess;
  if (once.pending(dev)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::ALLOC);
    // a warpgroup that raises its registers beyond what the launch has would wait for ever
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess && fa.numRegs * NUM_THREADS < 2 * 128 * SOFTMAX_REGS + 128 * OTHER_REGS) {
      *err = "score forward built with " + std::to_string(fa.numRegs) +
             " registers a thread, fewer than its warpgroups' register split needs";
      return (int)cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess) once.mark(dev);
  }
  if constexpr (PAGED)
    if (e == cudaSuccess && prm.plan) e = launch_behind(plan_kernel<PAGED>, dim3(1), PLAN_GROUPS, 0, st, prm, sms);
  // with a CTA for every unit the counter is not read
  if (e == cudaSuccess && !prm.plan && prm.n_units > sms) e = cudaMemsetAsync(prm.counter, 0, 4, st);
  if (e != cudaSuccess) {
    *err = std::string("score_fwd: ") + cudaGetErrorString(e);
    return (int)e;
  }
  // persistent: one CTA per SM
  const unsigned grid = (unsigned)std::min<int64_t>((int64_t)prm.n_units * (prm.plan ? MAX_PARTS : 1), sms);
  e = launch_behind(kern, dim3(grid), NUM_THREADS, Layout<D>::ALLOC, st, mq, mk, mv, prm);
  if (e == cudaSuccess && (prm.parts > 1 || prm.slots > 0))
    e = launch_behind(merge_kernel<D, PAGED>,
                      dim3((unsigned)(PAGED ? 8 * sms : prm.n_units / prm.parts * (2 * BM / MERGE_ROWS<D>))), MERGE_THREADS, 0, st, prm);
  if (e != cudaSuccess) *err = std::string("score_fwd launch: ") + cudaGetErrorString(e);
  return (int)e;
}

template <int D, bool PAGED>
static int launch(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err) {
  Params prm{};
  prm.slopes = a.slopes;
  prm.o = static_cast<__nv_bfloat16*>(a.o);
  prm.lse = a.lse;
  if (PAGED) {
    prm.os[1] = D, prm.os[2] = (int64_t)a.Hq * D;
    prm.ls[1] = 1, prm.ls[2] = a.Hq;
  } else {
    prm.os[0] = (int64_t)a.Hq * a.S * D, prm.os[1] = a.S * D, prm.os[2] = D;
    prm.ls[0] = (int64_t)a.Hq * a.S, prm.ls[1] = a.S, prm.ls[2] = 1;
  }
  prm.part_o = reinterpret_cast<float*>(a.ws + z.part_o);
  prm.part_lse = reinterpret_cast<float*>(a.ws + z.part_lse);
  prm.status = a.status;
  prm.counter = reinterpret_cast<uint32_t*>(a.ws + z.counter);
  prm.lo = a.lo;
  prm.hi = a.hi;
  prm.mask_bs = a.mask_bs;
  prm.offsets = a.offsets;
  prm.lens = a.lens;
  prm.table = a.table;
  prm.table_s = a.table_s;
  prm.S = a.S;
  prm.N = a.N;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.g = a.Hq / a.Hkv;
  prm.gh = z.gh;
  prm.tt = z.tt;
  prm.tu = z.tu;
  prm.hc = z.hc;
  prm.groups = z.groups;
  prm.lanes = z.lanes;
  prm.parts = z.parts;
  prm.plan = z.plan ? reinterpret_cast<Plan*>(a.ws + z.plan) : nullptr;
  prm.slots = z.slots;
  const int64_t units = (int64_t)z.lanes * z.groups * z.parts;
  if (units > 0x3fffffff) {
    *err = "too many work units for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  prm.n_units = (int32_t)units;
  // lanes numbered together: enough for about three times the grid, so that the last units are short where lengths differ
  prm.batch = (int32_t)std::min<int64_t>(z.lanes, (3LL * sms + z.groups - 1) / z.groups);
  prm.n_pages = a.n_pages;
  prm.page = a.page;
  prm.max_pages = a.max_pages;
  prm.max_new = a.max_new;
  prm.window = a.window;
  prm.box_rows = BN;
  if (PAGED)
    while (a.page % prm.box_rows != 0) prm.box_rows /= 2;
  prm.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  prm.cap = make_cap(a.scale, a.cap);
  prm.wait_limit_ns = a.wait_limit_ns;
  CUtensorMap mq, mk, mv;
  bool ok;
  if (PAGED) {
    const uint64_t qd[3] = {D, (uint64_t)a.N, (uint64_t)a.Hq};
    const int64_t qst[2] = {a.qs[0], a.qs[1]};
    const uint64_t kd[4] = {D, (uint64_t)a.page, (uint64_t)a.Hkv, (uint64_t)a.n_pages};
    const int64_t kst[3] = {a.ks[2], a.ks[1], a.ks[0]}, vst[3] = {a.vs[2], a.vs[1], a.vs[0]};
    const uint32_t qb[3] = {64, (uint32_t)z.tt, (uint32_t)z.gh}, kb[4] = {64, (uint32_t)prm.box_rows, 1, 1};
    ok = encode_bf16_map(&mq, a.q, 3, qd, qst, qb, err) && encode_bf16_map(&mk, a.k, 4, kd, kst, kb, err) &&
         encode_bf16_map(&mv, a.v, 4, kd, vst, kb, err);
  } else {
    const uint64_t qd[3] = {D, (uint64_t)a.S, (uint64_t)a.B * a.Hq};
    const int64_t qst[2] = {D, a.S * D};
    const uint64_t kd[4] = {D, (uint64_t)a.S, (uint64_t)a.Hkv, (uint64_t)a.B};
    const int64_t kst[3] = {D, a.S * D, (int64_t)a.Hkv * a.S * D};
    const uint32_t qb[3] = {64, (uint32_t)z.tt, (uint32_t)z.gh}, kb[4] = {64, BN, 1, 1};
    ok = encode_bf16_map(&mq, a.q, 3, qd, qst, qb, err) && encode_bf16_map(&mk, a.k, 4, kd, kst, kb, err) &&
         encode_bf16_map(&mv, a.v, 4, kd, kst, kb, err);
  }
  if (!ok) return (int)cudaErrorInvalidValue;
  if (a.cap > 0.f && a.slopes) return launch_mode<D, 3, PAGED>(mq, mk, mv, prm, sms, st, err);
  if (a.cap > 0.f) return launch_mode<D, 2, PAGED>(mq, mk, mv, prm, sms, st, err);
  if (a.slopes) return launch_mode<D, 1, PAGED>(mq, mk, mv, prm, sms, st, err);
  return launch_mode<D, 0, PAGED>(mq, mk, mv, prm, sms, st, err);
}

}  // namespace sfw
}  // namespace mesh
