// Attention over a paged cache for few new tokens a sequence: one of a decoding step, or a few guessed ones.
//   x = cap tanh(s q.k / cap) (or s q.k) - slope_h (i - j) over the keys j of i - window < j <= i,  O = softmax(x) V.
//
// A sequence's rows are its new tokens times the query heads of a KV head, row t g + h, 16 at most in bf16 (one M = 16 product)
// and 8 in fp32.  Bound by memory: 16 rows are 32 flops a byte.
//
// Work split.  The batch's cached tokens, in tiles of 128 over the segments (sequence, KV head), are one long list that the
// CTAs share out evenly: CTA i takes the units [i W / G, (i + 1) W / G), a unit being a tile, or one of the SEG_COST units that
// stand before each segment for what a segment costs besides its tiles.  So the split does not depend on how ragged the batch
// is, one long sequence fills the GPU as well as many short ones, and short ones do not pile up in one CTA.  Lengths are read
// on the device: a captured graph replays with other lengths, tables and pages.  A segment whose tiles fall into one CTA is
// finished there; of the others every CTA leaves unnormalised sums with their running maxima in a slot of its own (two a CTA:
// the piece that began before it and the piece that goes on behind it), and the last CTA to arrive adds them up in order, so
// results do not depend on the arrival order.  At most one segment begins in a CTA and goes on behind it, so a segment's
// arrival counter is that CTA's: one a CTA, zero between calls (the last CTA puts them back).
//
// Measured: 64 sequences of up to 8,192 tokens, 32 heads on 8, bf16, d 128, 171 us = 6.4 TB/s, 95 % of a plain copy (d 64: 98 us,
// 5.6); one of 131,072, 16 heads on 4, 50 us = 5.4 TB/s, 9 us of it the start, the SMs' spread and the merge.  fp32, the same 64:
// 624 us at d 128 and 321 at d 64, 3.5 and 3.4 TB/s: not memory but the warps bound it (EngineF32).
//
// A row's statistics are fp32; sums of P V are fp32.  A warp's 16 tokens of a tile lie in one page (pages are multiples of
// 16), so a tile costs a warp one look at the table, one tile ahead.  What lies behind a sequence's last token, in its
// last page or in pages of the table behind it, and what lies before all windows, is never read: its places in shared memory
// are zero-filled, so NaN there does not reach a sum.  Lengths, offsets and pages that do not fit are recorded in the status
// block and taken as the nearest that do (a page that does not exist: zeros); the kernel never skips on the status block, since
// a CTA that skipped would leave its counters and slots half done.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace mesh {
namespace prow {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int WT = 16;            // tokens of a warp in a tile, all in one page
constexpr int TILE = WARPS * WT;  // tokens of a tile
constexpr int ROWS = PAGED_FEW_BF16;  // rows of a segment in the buffers (fp32 uses 8 of them)
constexpr int HALF_ROWS = 8;
// CTAs an SM: one with 192 KB of ring at d = 128; two at d = 64, whose tiles are half as long and keep one CTA's warps from the
// memory's rate (64 sequences up to 8,192 tokens, 32 heads on 8: 134 us with one CTA of either depth of ring, 99 with two).
template <int D>
constexpr int CTAS = D == 128 ? 1 : 2;
constexpr int MAX_CTAS = 2 * MAX_SMS;
// Filling the ring and adding up the warps' sums at a segment's end take about as long as three tiles
// (4 us; a tile is 64 KB at d = 128, 1.45 us at the memory's rate).
constexpr int SEG_COST = 3;
constexpr int ROLE_SEQ = 1, ROLE_PAGE = 2;
constexpr float LN2 = 0.69314718055994531f;
constexpr float LOG2E = 1.4426950408889634f;

struct Params {
  const void* q;  // [N, Hq, D], token and head strides
  int64_t qs[2];
  const void* k;  // pages [n_pages, Hkv, page, D]: page, head, row strides
  const void* v;
  int64_t ks[3], vs[3];
  const int32_t* table;
  int64_t table_s;
  const int32_t* offsets;
  const int32_t* lens;
  const float* slopes;  // [Hq] or NULL
  void* o;
  float* lse;
  float* part;         // [2 G][ROWS * D + 2 ROWS]
  uint32_t* counters;  // [G], zero between calls
  int32_t* status;
  int32_t N, B, Hq, Hkv, g, n_pages, page, max_pages, max_new, window;
  float scale, scale_log2, cap;
};

__host__ __device__ constexpr int part_floats(int D) { return ROWS * D + 2 * ROWS; }
// Floats from row to row of the warps' sums in shared memory: the eight rows that a warp's lanes write at once lie in other banks.
__host__ __device__ constexpr int sum_ld(int D) { return D + 8; }

__device__ __forceinline__ Asked seq_of(const Params& p, int b) {
  return asked(p.offsets, p.lens, b, p.N, p.max_new, p.max_pages, p.page);
}
// The first tile that a segment of it reads.
__device__ __forceinline__ int first_tile(const Params& p, const Asked& s) {
  return p.window ? max(s.len - s.n - p.window + 1, 0) / TILE : 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;  // 0: the 16 bytes are zero-filled and src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One piece of a segment as the engines see it.
template <typename T>
struct Piece {
  const T *kb, *vb;          // the KV head of page 0
  const int32_t* pages;      // the sequence's row of the table
  const T* q;                // the sequence's first new token, the KV head's first query head
  const float* slopes;       // of the KV head's query heads, or NULL
  int b, nr;                 // its rows
  int t0, t1;                // tiles
  int len, pos0;             // cached tokens; the place of the first new token
  int lo;                    // the first token that any of the sequence's rows sees
};

// A row's keys [lo, hi), its own place, its slope in base 2.
struct RowMask {
  int lo, hi, pos;
  float slope2;
};
template <typename T>
__device__ __forceinline__ RowMask mask_of(const Params& p, const Piece<T>& c, int r) {
  RowMask m{0, 0, 0, 0.f};
  if (r < c.nr) {
    const int t = r / p.g;
    m.pos = c.pos0 + t;
    m.hi = m.pos + 1;
    m.lo = p.window ? max(0, m.hi - p.window) : 0;
    if (c.slopes) m.slope2 = c.slopes[r - t * p.g] * LOG2E;
  }
  return m;
}
template <typename T>
__device__ __forceinline__ const T* q_row(const Params& p, const Piece<T>& c, int r) {
  const int t = r / p.g;
  return c.q + t * p.qs[0] + (r - t * p.g) * p.qs[1];
}
// The page of the WT tokens from tok0 on, or -1 where none of them is seen (behind the last token, or before a window, whose
// pages need not be there any more) or where the table names none that exists: recorded, and read as zeros.
template <typename T>
__device__ __forceinline__ int page_at(const Params& p, const Piece<T>& c, int tok0, int lane) {
  if (tok0 >= c.len || tok0 / WT * WT + WT <= c.lo) return -1;
  const int pg = c.pages[tok0 / p.page];
  if (pg >= 0 && pg < p.n_pages) return pg;
  if (lane == 0) record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_PAGE, c.b);
  return -1;
}
// A score q.k in base 2: scaled, capped, biased.
__device__ __forceinline__ float score2(const Params& p, float dot, int far, float slope2) {
  float x = p.cap > 0.f ? p.cap * LOG2E * tanhf(dot * (p.scale / p.cap)) : dot * p.scale_log2;
  if (slope2 != 0.f) x = fmaf(-slope2, (float)far, x);
  return x;
}

// What a warp has of a piece: sums [rows][columns] in the engine's own register layout, and the
// running maximum (base 2) and sum of each row, written for the merge by put().

// bf16: products on the tensor cores (mma.sync: 16 rows are far below what a tcgen05 tile wants, and the kernel is
// bound by memory).  Each warp streams its own 16 tokens of every tile through its own cp.async ring, so
// no barrier stands in the loop.
template <int D>
struct EngineBf16 {
  using T = __nv_bfloat16;
  static constexpr int R = PAGED_FEW_BF16;            // rows of a segment, at most
  static constexpr int CH = D / 8;                    // 16-byte chunks of a row
  static constexpr uint32_t HALF = WT * D * 2;        // K or V of a warp's stage
  static constexpr uint32_t STAGE = 2 * HALF;
  static constexpr int STAGES = 3;
  static constexpr uint32_t SMEM = WARPS * STAGES * STAGE;
  uint32_t qf[D / 16][4];
  float acc[D / 8][4];
  float m[2], l[2];  // of rows lane / 4 and 8 + lane / 4; l of this lane's columns
  uint32_t base;     // this warp's ring

  __device__ __forceinline__ void init(uint32_t smem, int warp) { base = smem + (uint32_t)(warp * STAGES) * STAGE; }

  __device__ __forceinline__ void load(const Params& p, const Piece<T>& c, int stage, int tok0, int pg, int lane) {
    const uint32_t dst = base + (uint32_t)stage * STAGE;
    const int row0 = tok0 % p.page;
    const T* kp = c.kb + (int64_t)max(pg, 0) * p.ks[0] + (int64_t)row0 * p.ks[2];
    const T* vp = c.vb + (int64_t)max(pg, 0) * p.vs[0] + (int64_t)row0 * p.vs[2];
#pragma unroll
    for (int i = 0; i < WT * CH / 32; ++i) {
      const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
      const uint32_t at = dst + (uint32_t)(row * D * 2) + (uint32_t)((ch ^ (row & 7)) << 4);
      const bool in = pg >= 0 && tok0 + row < c.len && tok0 + row >= c.lo;
      const int64_t t = in ? row : 0;  // a safe address where nothing is read
      cp_async16(at, in ? kp + t * p.ks[2] + ch * 8 : static_cast<const T*>(p.k), in);
      cp_async16(at + HALF, in ? vp + t * p.vs[2] + ch * 8 : static_cast<const T*>(p.v), in);
    }
  }

  __device__ __forceinline__ void piece(const Params& p, const Piece<T>& c, int warp, int lane) {
    const int c2 = (lane & 3) * 2;
    auto tok_of = [&](int t) { return t * TILE + warp * WT; };
    int pg_next = page_at(p, c, tok_of(c.t0), lane);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      if (c.t0 + s < c.t1) {
        const int pg = pg_next;
        if (c.t0 + s + 1 < c.t1) pg_next = page_at(p, c, tok_of(c.t0 + s + 1), lane);
        load(p, c, s, tok_of(c.t0 + s), pg, lane);
      }
      cp_commit();
    }
    const int ra = lane >> 2, rb = ra + 8;
    {
      const T* qa = q_row(p, c, min(ra, c.nr - 1));
      const T* qb = q_row(p, c, min(rb, c.nr - 1));
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][0] = ra < c.nr ? *reinterpret_cast<const uint32_t*>(qa + s * 16 + c2) : 0u;
        qf[s][1] = rb < c.nr ? *reinterpret_cast<const uint32_t*>(qb + s * 16 + c2) : 0u;
        qf[s][2] = ra < c.nr ? *reinterpret_cast<const uint32_t*>(qa + s * 16 + c2 + 8) : 0u;
        qf[s][3] = rb < c.nr ? *reinterpret_cast<const uint32_t*>(qb + s * 16 + c2 + 8) : 0u;
      }
    }
    const RowMask mk[2] = {mask_of(p, c, ra), mask_of(p, c, rb)};
    // tokens that every row sees: no mask there
    const int all_lo = p.window ? max(0, c.pos0 + (c.nr - 1) / p.g + 1 - p.window) : 0, all_hi = c.pos0 + 1;
    const bool plain = p.cap <= 0.f && !c.slopes;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    const int krow = ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;   // K: 16 tokens x 16 columns
    const int vrow = (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;  // V, transposed
    int stage = 0;
    for (int t = c.t0; t < c.t1; ++t) {
      {
        const int ahead = t + STAGES - 1;
        int s = stage + STAGES - 1;
        if (s >= STAGES) s -= STAGES;
        if (ahead < c.t1) {
          const int pg = pg_next;
          if (ahead + 1 < c.t1) pg_next = page_at(p, c, tok_of(ahead + 1), lane);
          load(p, c, s, tok_of(ahead), pg, lane);
        }
        cp_commit();
      }
      cp_wait<STAGES - 1>();
      __syncwarp();
      const int tok0 = tok_of(t);
      if (tok0 < c.len) {
        const uint32_t ka = base + (uint32_t)stage * STAGE, va = ka + HALF;
        float sc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          uint32_t r[4];
          ldsm4(ka + (uint32_t)(krow * D * 2) + (uint32_t)(((2 * s + kch) ^ (krow & 7)) << 4), r);
#pragma unroll
          for (int n = 0; n < 2; ++n) mma16816(sc[n], qf[s][0], qf[s][1], qf[s][2], qf[s][3], r[2 * n], r[2 * n + 1]);
        }
        if (plain) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] *= p.scale_log2;
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const RowMask& w = mk[e >> 1];
              sc[n][e] = score2(p, sc[n][e], w.pos - (tok0 + n * 8 + c2 + (e & 1)), w.slope2);
            }
        }
        if (tok0 + WT > all_hi || tok0 < all_lo) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = tok0 + n * 8 + c2 + (e & 1);
              if (j < mk[e >> 1].lo || j >= mk[e >> 1].hi) sc[n][e] = -INFINITY;
            }
        }
        float f[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float mx = fmaxf(fmaxf(sc[0][2 * w], sc[0][2 * w + 1]), fmaxf(sc[1][2 * w], sc[1][2 * w + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[w], mx);
          const float ref = mn == -INFINITY ? 0.f : mn;
          f[w] = exp2f(m[w] - ref);
          m[w] = mn;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = fast_exp2(sc[n][2 * w + e] - ref);
              sc[n][2 * w + e] = x;
              sum += x;
            }
          l[w] = l[w] * f[w] + sum;
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][0] *= f[0];
            acc[i][1] *= f[0];
            acc[i][2] *= f[1];
            acc[i][3] *= f[1];
          }
        }
        // P as two bf16 pieces (the second takes what the first rounds off, 2^-17 relative together): the
        // tensor cores have time to spare here, and the output keeps fp32's digits until its own rounding
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = sc[i >> 1][2 * (i & 1)], x1 = sc[i >> 1][2 * (i & 1) + 1];
          ph[i] = pack_bf16x2(x0, x1);
          pl[i] = pack_bf16x2(x0 - __uint_as_float(ph[i] << 16), x1 - __uint_as_float(ph[i] & 0xffff0000u));
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t r[4];
          ldsm4t(va + (uint32_t)(vrow * D * 2) + (uint32_t)(((2 * i + vch) ^ (vrow & 7)) << 4), r);
          mma16816(acc[2 * i], ph[0], ph[1], ph[2], ph[3], r[0], r[1]);
          mma16816(acc[2 * i + 1], ph[0], ph[1], ph[2], ph[3], r[2], r[3]);
          mma16816(acc[2 * i], pl[0], pl[1], pl[2], pl[3], r[0], r[1]);
          mma16816(acc[2 * i + 1], pl[0], pl[1], pl[2], pl[3], r[2], r[3]);
        }
      }
      __syncwarp();  // every lane is done with the stage before the next load overwrites it
      if (++stage == STAGES) stage = 0;
    }
    cp_wait<0>();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
      l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
    }
  }

  __device__ __forceinline__ void put_stats(float* ms, float* ls, int lane) const {
    if ((lane & 3) == 0) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        ms[w * HALF_ROWS + (lane >> 2)] = m[w];
        ls[w * HALF_ROWS + (lane >> 2)] = l[w];
      }
    }
  }
  // buf[row][sum_ld(D)] = sums * 2^(m - M[row]), of the first nr rows
  __device__ __forceinline__ void put(float* buf, const float* M, int nr, int lane) const {
    const int c2 = (lane & 3) * 2;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int row = w * HALF_ROWS + (lane >> 2);
      if (row >= nr) continue;
      const float f = m[w] == -INFINITY ? 0.f : exp2f(m[w] - M[row]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(buf + row * sum_ld(D) + i * 8 + c2) = make_float2(acc[i][2 * w] * f, acc[i][2 * w + 1] * f);
    }
  }
};

// fp32: CUDA cores.  A lane owns D / 32 columns.  A warp takes four tokens at a time from its own ring; the
// reduction over the lanes transposes as it goes (two values, then one, travel), so that afterwards a lane holds one
// token's score and takes one exponential, and four shuffles hand the weights to all lanes.  Bound by the latency
// of that chain, twelve shuffles and a vote a row and four tokens, with two warps a scheduler: it issues in 40 % of the cycles, and
// waits for results of fixed latency in 31 % of a warp's time and for shuffles and shared memory in 26 % (d 128).
template <int D, int G>
struct EngineF32 {
  using T = float;
  static constexpr int R = G;
  static constexpr int E = D / 32;
  static constexpr int U = 4;  // tokens of a stage
  static constexpr int NS = 6;
  static constexpr uint32_t ROWB = U * D * 4;  // K or V of a stage
  static constexpr uint32_t STAGE = 2 * ROWB;
  static constexpr uint32_t SMEM = WARPS * NS * STAGE;
  float acc[G][E];
  float m[G], l[G];  // l of this lane's tokens
  uint32_t base;
  const uint8_t* ring;

  __device__ __forceinline__ void init(uint32_t smem, int warp) {
    base = smem + (uint32_t)(warp * NS) * STAGE;
    extern __shared__ __align__(128) uint8_t smem_bytes[];
    ring = smem_bytes + (size_t)(warp * NS) * STAGE;
  }

  __device__ __forceinline__ void load(const Params& p, const Piece<T>& c, int stage, int tok0, int pg, int lane) {
    const uint32_t dst = base + (uint32_t)stage * STAGE;
    constexpr int CH = D / 4;  // 16-byte chunks of a row
    const int row0 = tok0 % p.page;
    const T* kp = c.kb + (int64_t)max(pg, 0) * p.ks[0] + (int64_t)row0 * p.ks[2];
    const T* vp = c.vb + (int64_t)max(pg, 0) * p.vs[0] + (int64_t)row0 * p.vs[2];
#pragma unroll
    for (int i = 0; i < U * CH / 32; ++i) {
      const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
      const bool in = pg >= 0 && tok0 + row < c.len && tok0 + row >= c.lo;
      const int64_t t = in ? row : 0;  // a safe address where nothing is read
      cp_async16(dst + (uint32_t)idx * 16u, in ? kp + t * p.ks[2] + ch * 4 : static_cast<const T*>(p.k), in);
      cp_async16(dst + ROWB + (uint32_t)idx * 16u, in ? vp + t * p.vs[2] + ch * 4 : static_cast<const T*>(p.v), in);
    }
  }

  __device__ __forceinline__ void piece(const Params& p, const Piece<T>& c, int warp, int lane) {
    const int n = (c.t1 - c.t0) * (WT / U);  // groups of four tokens
    auto tok_of = [&](int g) { return (c.t0 + g / (WT / U)) * TILE + warp * WT + g % (WT / U) * U; };
    int pg = -1;  // the page of the groups of a tile being loaded
    auto load_group = [&](int g, int s) {
      if (g < n) {
        if (g % (WT / U) == 0) pg = page_at(p, c, tok_of(g), lane);
        load(p, c, s, tok_of(g), pg, lane);
      }
      cp_commit();
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) load_group(s, s);
    float q[G][E];
    RowMask mk[G];
    int all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const T* qp = q_row(p, c, min(i, c.nr - 1)) + lane * E;
      mk[i] = mask_of(p, c, i);
      if (i < c.nr) {
        all_lo = max(all_lo, mk[i].lo);
        all_hi = min(all_hi, mk[i].hi);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[i][e] = i < c.nr ? qp[e] : 0.f;
        acc[i][e] = 0.f;
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    const bool b4 = lane & 16, b3 = lane & 8;
    const int mine = (b4 ? 2 : 0) + (b3 ? 1 : 0);  // this lane's token of a group
    int stage = 0;
    for (int g = 0; g < n; ++g) {
      {
        int s = stage + NS - 1;
        if (s >= NS) s -= NS;
        load_group(g + NS - 1, s);
      }
      cp_wait<NS - 1>();
      __syncwarp();
      const int tok = tok_of(g);
      if (tok < c.len) {
        const float* kr = reinterpret_cast<const float*>(ring + (size_t)stage * STAGE) + lane * E;
        const float* vr = kr + U * D;
        float kx[U][E], vx[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            kx[u][e] = kr[u * D + e];
            vx[u][e] = vr[u * D + e];
          }
        const bool edge = tok + U > all_hi || tok < all_lo;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float s[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s[u] = fmaf(q[i][e], kx[u][e], s[u]);
          }
          float k0 = b4 ? s[2] : s[0], k1 = b4 ? s[3] : s[1];
          k0 += __shfl_xor_sync(0xffffffffu, b4 ? s[0] : s[2], 16);
          k1 += __shfl_xor_sync(0xffffffffu, b4 ? s[1] : s[3], 16);
          float x = b3 ? k1 : k0;
          x += __shfl_xor_sync(0xffffffffu, b3 ? k0 : k1, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x = score2(p, x, mk[i].pos - (tok + mine), mk[i].slope2);
          if (edge && (tok + mine < mk[i].lo || tok + mine >= mk[i].hi)) x = -INFINITY;
          float mx = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx = fmaxf(m[i], fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8)));
          const float ref = mx == -INFINITY ? 0.f : mx;
          const float f = exp2f(m[i] - ref);
          m[i] = mx;
          x = exp2f(x - ref);
          l[i] = l[i] * f + x;
          if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] *= f;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float w = __shfl_sync(0xffffffffu, x, (u >> 1) * 16 + (u & 1) * 8);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = fmaf(w, vx[u][e], acc[i][e]);
          }
        }
      }
      __syncwarp();  // every lane is done with the stage before the next load overwrites it
      if (++stage == NS) stage = 0;
    }
    cp_wait<0>();
#pragma unroll
    for (int i = 0; i < G; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
    }
  }

  __device__ __forceinline__ void put_stats(float* ms, float* ls, int lane) const {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        ms[i] = i < G ? m[i < G ? i : 0] : -INFINITY;
        ls[i] = i < G ? l[i < G ? i : 0] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void put(float* buf, const float* M, int, int lane) const {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - M[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) buf[i * sum_ld(D) + lane * E + e] = acc[i][e] * f;
    }
  }
};

// The last CTA of a segment adds its pieces up, in order: row r's weights 2^(m - M) into wts [n_p][ROWS] and its maximum and
// sum, sixteen threads a row; then every thread takes one or two 16-byte columns of the rows over all pieces, or over every
// GR-th of them where there are fewer columns than threads, into part [GR][nr][D].  Returns GR.  The first loads of both are in
// flight together.  A function of its own: its registers would else cost the loop over the tokens some of its loads in flight
// (185 us where it takes 174, 64 sequences).
template <int D>
__device__ __noinline__ int merge_pieces(const float* slots, int64_t i0, int n_p, int nr, float* wts, float* part, float* Ms, float* Ls) {
  const int tid = threadIdx.x;
  auto slot_of = [&](int k) { return slots + ((i0 + k) * 2 + (k == 0 ? 1 : 0)) * part_floats(D); };
  const int cols = nr * (D / 4), GR = cols >= THREADS ? 1 : THREADS / cols;
  constexpr int PRE = 20;
  float4 pre[PRE];
  {
    const int grp = tid / cols, q = tid - grp * cols, r = q / (D / 4), at = q % (D / 4) * 4;
#pragma unroll
    for (int u = 0; u < PRE; ++u) {
      const int k = grp + u * GR;
      pre[u] = tid < cols * GR && k < n_p ? __ldcg(reinterpret_cast<const float4*>(slot_of(k) + r * D + at)) : make_float4(0, 0, 0, 0);
    }
  }
  {
    const int r = tid >> 4, k0 = tid & 15;
    constexpr int PER = MAX_SMS * CTAS<D> / 16;
    float m[PER], l[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int k = k0 + 16 * u;
      const float* st = slot_of(k) + ROWS * D + r;
      m[u] = k < n_p ? __ldcg(st) : -INFINITY;
      l[u] = k < n_p ? __ldcg(st + ROWS) : 0.f;
    }
    float M = -INFINITY;
#pragma unroll
    for (int u = 0; u < PER; ++u) M = fmaxf(M, m[u]);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const float f = m[u] == -INFINITY ? 0.f : exp2f(m[u] - M);
      if (k0 + 16 * u < n_p) wts[(k0 + 16 * u) * ROWS + r] = f;
      L += m[u] == -INFINITY ? l[u] : l[u] * f;  // l is 0 there, or NaN
    }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (k0 == 0) {
      Ms[r] = M;
      Ls[r] = L;
    }
  }
  __syncthreads();
  for (int o = tid; o < cols * GR; o += THREADS) {
    const int grp = o / cols, q = o - grp * cols, r = q / (D / 4), at = q % (D / 4) * 4;
    float4 t = make_float4(0, 0, 0, 0);
    int k = grp;
    if (o == tid) {
#pragma unroll
      for (int u = 0; u < PRE; ++u, k += GR) {
        const float f = k < n_p ? wts[k * ROWS + r] : 0.f;
        t.x = fmaf(pre[u].x, f, t.x), t.y = fmaf(pre[u].y, f, t.y), t.z = fmaf(pre[u].z, f, t.z), t.w = fmaf(pre[u].w, f, t.w);
      }
    }
#pragma unroll 16
    for (; k < n_p; k += GR) {
      const float4 y = __ldcg(reinterpret_cast<const float4*>(slot_of(k) + r * D + at));
      const float f = wts[k * ROWS + r];
      t.x = fmaf(y.x, f, t.x), t.y = fmaf(y.y, f, t.y), t.z = fmaf(y.z, f, t.z), t.w = fmaf(y.w, f, t.w);
    }
    *reinterpret_cast<float4*>(part + (grp * nr + r) * D + at) = t;
  }
  return GR;
}

// Bytes of the engine's ring, or of the warps' sums that take its place at a piece's end.
template <typename Engine, int D>
struct Big {
  static constexpr uint32_t SUMS = (uint32_t)(WARPS * ROWS * sum_ld(D) * 4);
  static constexpr uint32_t BYTES = Engine::SMEM > SUMS ? Engine::SMEM : SUMS;
  // the last CTA's weights, and its columns' sums by group of pieces
  static_assert(MAX_SMS * CTAS<D> * ROWS * 4 + 2 * THREADS * 16 <= BYTES, "room for the merge");
};
// behind the ring: warps' maxima and sums, M, L, the scan
constexpr uint32_t STATS = 4 * (2 * WARPS * ROWS + 2 * ROWS) + 8 * (WARPS + 2);

template <typename Engine, int D>
__global__ void __launch_bounds__(THREADS, CTAS<D>) rows_kernel(const Params p) {
  using T = typename Engine::T;
  constexpr int R = Engine::R;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr uint32_t BIG = Big<Engine, D>::BYTES;
  float* sums = reinterpret_cast<float*>(smem);
  float* ms = reinterpret_cast<float*>(smem + BIG);
  float* ls = ms + WARPS * ROWS;
  float* Ms = ls + WARPS * ROWS;
  float* Ls = Ms + ROWS;
  int64_t* scan = reinterpret_cast<int64_t*>(Ls + ROWS);                // [WARPS + 2]
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + BIG + STATS);     // [B + 1] units
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_kernel_before();

  // units before each sequence, of one KV head
  {
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + tid;
      int64_t n = 0;
      if (b < p.B) {
        const Asked s = seq_of(p, b);
        if (s.bad && blockIdx.x == 0) record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_SEQ, b);
        if (s.n > 0) n = (s.len + TILE - 1) / TILE - first_tile(p, s) + SEG_COST;
      }
      int64_t x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      int64_t before = 0, all = 0;
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
      }
      if (b < p.B) prefix[b] = carry + before + x - n;
      carry += all;
      __syncthreads();
    }
    if (tid == 0) prefix[p.B] = carry;
    __syncthreads();
  }
  const int per = p.Hkv;
  const int64_t W = prefix[p.B] * per;
  // no more CTAs than units: every CTA between a segment's first and last then has a piece of it
  const int64_t G = max((int64_t)1, min((int64_t)gridDim.x, W));
  auto begin_of = [&](int64_t i) { return W * i / G; };
  // the CTA whose range holds unit x
  auto owner_of = [&](int64_t x) {
    int64_t i = x * G / W;
    while (begin_of(i + 1) <= x) ++i;
    while (begin_of(i) > x) --i;
    return i;
  };
  const int64_t lo = blockIdx.x < G ? begin_of(blockIdx.x) : W, hi = blockIdx.x < G ? begin_of(blockIdx.x + 1) : W;

  Engine eng;
  eng.init(smem_u32(smem), warp);
  int64_t x = lo;
  while (x < hi) {
    // the sequence of unit x: the last b with prefix[b] * per <= x (those without work share its prefix)
    int b;
    {
      int a = 0, z = p.B;
      while (z - a > 1) {
        const int c = (a + z) >> 1;
        if (prefix[c] * per <= x) a = c;
        else z = c;
      }
      b = a;
    }
    const Asked s = seq_of(p, b);
    const int64_t n = prefix[b + 1] - prefix[b];  // of a segment, > SEG_COST
    const int hk = (int)((x - prefix[b] * per) / n);
    const int64_t s1 = prefix[b] * per + (hk + 1) * n, s0 = s1 - n + SEG_COST;  // the segment's tiles are [s0, s1)
    const int64_t end = min(hi, s1);
    if (end <= s0) {  // nothing of it but the units before its tiles
      x = end;
      continue;
    }
    x = max(x, s0);
    Piece<T> c;
    c.b = b;
    c.kb = static_cast<const T*>(p.k) + hk * p.ks[1];
    c.vb = static_cast<const T*>(p.v) + hk * p.vs[1];
    c.pages = p.table + b * p.table_s;
    c.q = static_cast<const T*>(p.q) + s.begin * p.qs[0] + (int64_t)hk * p.g * p.qs[1];
    c.slopes = p.slopes ? p.slopes + hk * p.g : nullptr;
    c.nr = s.n * p.g;
    const int tile0 = first_tile(p, s);
    c.t0 = tile0 + (int)(x - s0);
    c.t1 = tile0 + (int)(end - s0);
    c.len = s.len;
    c.pos0 = s.len - s.n;
    c.lo = p.window ? max(0, c.pos0 + 1 - p.window) : 0;
    const bool whole = s0 >= lo && s1 <= hi;
    const int64_t i0 = whole ? 0 : owner_of(s0), i1 = whole ? 0 : owner_of(s1 - 1);  // the CTAs that have pieces of the segment
    eng.piece(p, c, warp, lane);

    // a row's output: sums / l, and its LSE
    auto finish = [&](int r, int c4, float4 a, float m, float l) {
      const int t = r / p.g, h = hk * p.g + r - t * p.g;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible token: O = 0 (a NaN sum stays NaN)
      const int64_t at = ((int64_t)(s.begin + t) * p.Hq + h) * D + c4;
      if constexpr (sizeof(T) == 2) {
        uint2 w;
        w.x = pack_bf16x2(a.x * inv, a.y * inv);
        w.y = pack_bf16x2(a.z * inv, a.w * inv);
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at) = w;
      } else {
        *reinterpret_cast<float4*>(static_cast<T*>(p.o) + at) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      }
      if (c4 == 0) p.lse[(int64_t)(s.begin + t) * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    };

    // the warps' sums as one
    eng.put_stats(ms + warp * ROWS, ls + warp * ROWS, lane);
    __syncthreads();  // also: every warp is done with its ring, whose memory the sums take
    if (tid < ROWS) {
      float M = -INFINITY;
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ms[w * ROWS + tid]);
      float L = 0.f;
      for (int w = 0; w < WARPS; ++w) {
        const float mw = ms[w * ROWS + tid], lw = ls[w * ROWS + tid];
        L += mw == -INFINITY ? lw : lw * exp2f(mw - M);  // lw is 0, or NaN
      }
      Ms[tid] = M;
      Ls[tid] = L;
    }
    __syncthreads();
    eng.put(sums + warp * ROWS * sum_ld(D), Ms, c.nr, lane);
    __syncthreads();
    constexpr int RP = THREADS / (D / 4);  // rows that the threads take at once: 8, or 16 at d = 64
    const int r_at = tid / (D / 4), c4 = tid % (D / 4) * 4;
    // a piece: slot 1 where the segment begins here and goes on, slot 0 where it began before
    float* slot = p.part + ((int64_t)blockIdx.x * 2 + (s0 >= lo ? 1 : 0)) * part_floats(D);
    for (int r = r_at; r < c.nr; r += RP) {
      float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(sums + (w * ROWS + r) * sum_ld(D) + c4);
        a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
      }
      if (whole) finish(r, c4, a, Ms[r], Ls[r]);
      else *reinterpret_cast<float4*>(slot + r * D + c4) = a;
    }
    if (!whole) {
      if (tid < ROWS) {
        slot[ROWS * D + tid] = Ms[tid];
        slot[ROWS * D + ROWS + tid] = Ls[tid];
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        uint32_t* ctr = p.counters + i0;
        const bool last = atomicAdd(ctr, 1u) == (uint32_t)(i1 - i0);
        if (last) *ctr = 0u;
        scan[WARPS] = last;
      }
      __syncthreads();
      if (scan[WARPS]) {
        __threadfence();
        float* part = sums + MAX_SMS * CTAS<D> * ROWS;  // [GR][nr][D]
        const int GR = merge_pieces<D>(p.part, i0, (int)(i1 - i0 + 1), c.nr, sums, part, Ms, Ls);
        __syncthreads();
        for (int r = r_at; r < c.nr; r += RP) {
          float4 a = make_float4(0, 0, 0, 0);
          for (int g = 0; g < GR; ++g) {
            const float4 y = *reinterpret_cast<const float4*>(part + (g * c.nr + r) * D + c4);
            a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
          }
          finish(r, c4, a, Ms[r], Ls[r]);
        }
      }
    }
    __syncthreads();  // the sums' memory is the ring's again
    x = end;
  }
}

template <typename Engine, int D>
static int launch(const Params& p, int grid, cudaStream_t st, std::string* err) {
  auto kern = rows_kernel<Engine, D>;
  const size_t fixed = Big<Engine, D>::BYTES + STATS, smem = fixed + 8 * ((size_t)p.B + 1);
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  cudaError_t e = cudaSuccess;
  if (once.pending(dev)) {  // the most that any batch takes
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(fixed + 8 * (size_t)(PAGED_MAX_B + 1)));
    if (e == cudaSuccess) once.mark(dev);
  }
  if (e == cudaSuccess) e = launch_behind(kern, dim3((unsigned)grid), THREADS, smem, st, p);
  if (e != cudaSuccess) *err = std::string("paged rows launch: ") + cudaGetErrorString(e);
  return (int)e;
}

template <int D>
static int launch_f32(const Params& p, int64_t rows, int grid, cudaStream_t st, std::string* err) {
  if (rows <= 1) return launch<EngineF32<D, 1>, D>(p, grid, st, err);
  if (rows <= 2) return launch<EngineF32<D, 2>, D>(p, grid, st, err);
  if (rows <= 4) return launch<EngineF32<D, 4>, D>(p, grid, st, err);
  return launch<EngineF32<D, 8>, D>(p, grid, st, err);
}

}  // namespace prow

static_assert(PAGED_WS_HEAD >= prow::MAX_CTAS * 4, "room for the counters");
// two slots a CTA
size_t paged_rows_slots() { return (size_t)2 * 4 * std::max(MAX_SMS * prow::CTAS<128> * prow::part_floats(128), MAX_SMS * prow::CTAS<64> * prow::part_floats(64)); }

int launch_paged_rows(const PagedArgs& a, int sms, cudaStream_t st, std::string* err) {
  using namespace prow;
  Params p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  for (int i = 0; i < 2; ++i) p.qs[i] = a.qs[i];
  for (int i = 0; i < 3; ++i) p.ks[i] = a.ks[i], p.vs[i] = a.vs[i];
  p.table = a.table;
  p.table_s = a.table_s;
  p.offsets = a.offsets;
  p.lens = a.lens;
  p.slopes = a.slopes;
  p.o = a.o;
  p.lse = a.lse;
  p.part = reinterpret_cast<float*>(a.ws + PAGED_WS_HEAD);
  p.counters = reinterpret_cast<uint32_t*>(a.ws);
  p.status = a.status;
  p.N = a.N;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.g = a.Hq / a.Hkv;
  p.n_pages = a.n_pages;
  p.page = a.page;
  p.max_pages = a.max_pages;
  p.max_new = a.max_new;
  p.window = a.window;
  p.scale = a.scale;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.cap = a.cap;
  // a CTA for every tile there may be, no more than are resident
  const int64_t rows = (int64_t)a.max_new * p.g;  // of a sequence and KV head, at most
  const int64_t tiles = ((int64_t)a.max_pages * a.page + TILE - 1) / TILE * a.B * a.Hkv;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, std::min(sms, MAX_SMS) * (a.d == 128 ? CTAS<128> : CTAS<64>)));
  if (a.bf16)
    return a.d == 128 ? launch<EngineBf16<128>, 128>(p, grid, st, err) : launch<EngineBf16<64>, 64>(p, grid, st, err);
  return a.d == 128 ? launch_f32<128>(p, rows, grid, st, err) : launch_f32<64>(p, rows, grid, st, err);
}

}  // namespace mesh
