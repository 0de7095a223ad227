// Differential attention of one new token a sequence over a cache with lengths of its own:
//   O_h = softmax(s q1 K1^T) V - lam_h softmax(s q2 K2^T) V,   q = [q1 | q2], K = [K1 | K2] by columns,
// over the first lens[b] tokens of sequence b's cache.
//
// Bound by memory: a KV head's cache serves eight query heads of its group and both maps in one read, at 12
// flops a byte and query head or fewer.  A group of more than eight is cut into chunks of eight heads, segments
// of their own that read the cache once each: 16 query heads on one KV head read it twice, from L2 where it fits.
//
// Work split.  The batch's cached tokens, in tiles of 128 over the segments (sequence, KV head, head chunk),
// are one long list that the CTAs share out evenly: CTA i takes the units [i W / G, (i + 1) W / G), a
// unit being a tile, or one of the SEG_COST units that stand before each segment for what a segment
// costs besides its tiles.  So the split does not depend on how ragged the batch is, one long sequence
// fills the GPU as well as many short ones, and short ones do not pile up in one CTA.  The lengths are
// read on the device: a captured graph replays with other lengths.  A (sequence, head) whose tiles fall
// into one CTA is finished there; of the others every CTA leaves unnormalised sums with their running maxima in a slot of its own (two a CTA: the piece
// that began before it and the piece that goes on behind it), and the last CTA to arrive
// adds them up in order, so results do not depend on the arrival order.  The arrival counters are
// zero between calls (the last CTA puts them back).
//
// A row's statistics are fp32; sums of P V are fp32.  Cached tokens from lens[b] on are never
// read: their places in shared memory are zero-filled, so NaN there does not reach a sum.  A length
// outside [0, T] is recorded in the status block and taken as the nearer bound; the kernel never skips
// on the status block, since a CTA that skipped would leave its counters and slots half done.
//
// Measured (bf16, d = 128): one sequence of 262,144 tokens, 16 heads on 4: 92 us, 5.8 TB/s, of which about 8 us
// are the merge and the spread of the SMs' bandwidths; 64 sequences of 100 to 8,192 tokens, 32 heads on
// 8: 169 us, 6.35 TB/s (a plain copy 6.8).  fp32, 4 sequences up to 1,000 tokens: 10 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace ddec {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int WT = 16;            // tokens of a warp in a tile
constexpr int TILE = WARPS * WT;  // tokens of a tile
constexpr int HEADS = 8;          // query heads of a chunk; rows: map * HEADS + head
constexpr int ROWS = 2 * HEADS;
constexpr int STAGES = 3;
// Filling the ring and adding up the warps' sums at a segment's end take about as long as three tiles
// (4 us; a tile is 64 KB at d = 128, 1.45 us at the memory's rate).
constexpr int SEG_COST = 3;
constexpr int MAX_B = 4096;  // their tile counts are kept in shared memory beside the ring
constexpr int64_t MAX_T = 1 << 30;
// Units of a batch: a warp's sum of its sequences' units fits 32 bits, that of all of a CTA's threads does not.
using Units = int64_t;
static_assert(32 * (MAX_T / TILE + SEG_COST) <= std::numeric_limits<int32_t>::max());
static_assert(THREADS * (MAX_T / TILE + SEG_COST) <= std::numeric_limits<Units>::max());
constexpr float LN2 = 0.69314718055994531f;

struct Params {
  const void* q;
  const void* k;
  const void* v;
  int64_t ks[3], vs[3];  // batch, head, token strides in elements
  const int32_t* lens;
  const void* lam;
  int32_t lam_n;
  void* o;
  float* lse;
  float* part;         // [2 G][ROWS * D + 2 ROWS]
  uint32_t* counters;  // [B * Hkv * hc], zero between calls
  int32_t* status;
  int32_t B, Hq, Hkv, g, hc, T;
  float scale_log2;
};

__host__ __device__ constexpr int part_floats(int D) { return ROWS * D + 2 * ROWS; }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ int length_of(const Params& p, int b) { return min(max(p.lens[b], 0), p.T); }

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

// What a warp has of a piece: sums [rows][columns] in the engine's own register layout, and the
// running maximum (base 2) and sum of each row, written for the merge by put().

// bf16: products on the tensor cores (mma.sync: M = 16 rows are 8 heads x 2 maps, far below
// what a tcgen05 tile wants, and the kernel is bound by memory).  Each warp streams its own 16 tokens
// of every tile through its own three-stage cp.async ring, so no barrier stands in the loop.
// The first map's query has zeros in the second half of the columns and the other way round, so
// one product over all d columns gives the scores of both maps.
template <int D>
struct EngineBf16 {
  using T = __nv_bfloat16;
  static constexpr int CH = D / 8;                    // 16-byte chunks of a row
  static constexpr uint32_t HALF = WT * D * 2;        // K or V of a warp's stage
  static constexpr uint32_t STAGE = 2 * HALF;
  static constexpr uint32_t SMEM = WARPS * STAGES * STAGE;
  uint32_t qf[D / 16][2];
  float acc[D / 8][4];
  float m[2], l[2];  // of rows lane / 4 (map 1) and 8 + lane / 4 (map 2); l of this lane's columns
  uint32_t base;     // this warp's ring

  __device__ __forceinline__ void init(uint32_t smem, int warp) { base = smem + (uint32_t)(warp * STAGES) * STAGE; }

  __device__ __forceinline__ void load(const Params& p, const T* kb, const T* vb, int stage, int tok0, int len, int lane) {
    const uint32_t dst = base + (uint32_t)stage * STAGE;
#pragma unroll
    for (int i = 0; i < WT * CH / 32; ++i) {
      const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
      const uint32_t at = dst + (uint32_t)(row * D * 2) + (uint32_t)((ch ^ (row & 7)) << 4);
      const bool in = tok0 + row < len;
      const int64_t t = in ? tok0 + row : 0;  // a safe address where nothing is read
      cp_async16(at, kb + t * p.ks[2] + ch * 8, in);
      cp_async16(at + HALF, vb + t * p.vs[2] + ch * 8, in);
    }
  }

  __device__ __forceinline__ void piece(const Params& p, int b, int hk, int h0, int nh, int t0, int t1, int len, int warp,
                                        int lane) {
    const T* q = static_cast<const T*>(p.q) + ((int64_t)b * p.Hq + h0) * D;
    const T* kb = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[1];
    const T* vb = static_cast<const T*>(p.v) + b * p.vs[0] + hk * p.vs[1];
    const int head = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      if (t0 + s < t1) load(p, kb, vb, s, (t0 + s) * TILE + warp * WT, len, lane);
      cp_commit();
    }
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[s][0] = qf[s][1] = 0u;
      if (head < nh) {
        qf[s][0] = *reinterpret_cast<const uint32_t*>(q + head * D + s * 16 + c2);
        qf[s][1] = *reinterpret_cast<const uint32_t*>(q + head * D + s * 16 + c2 + 8);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    const int krow = ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;   // K: 16 tokens x 16 columns
    const int vrow = (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;  // V, transposed
    int stage = 0;
    for (int t = t0; t < t1; ++t) {
      {
        const int ahead = t + STAGES - 1;
        int s = stage + STAGES - 1;
        if (s >= STAGES) s -= STAGES;
        if (ahead < t1) load(p, kb, vb, s, ahead * TILE + warp * WT, len, lane);
        cp_commit();
      }
      cp_wait<STAGES - 1>();
      __syncwarp();
      const int tok0 = t * TILE + warp * WT;
      if (tok0 < len) {
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
          const bool first = s < D / 32;  // columns of the first map
#pragma unroll
          for (int n = 0; n < 2; ++n)
            mma16816(sc[n], first ? qf[s][0] : 0u, first ? 0u : qf[s][0], first ? qf[s][1] : 0u, first ? 0u : qf[s][1],
                     r[2 * n], r[2 * n + 1]);
        }
        if (tok0 + WT > len) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (tok0 + n * 8 + c2 + (e & 1) >= len) sc[n][e] = -INFINITY;
        }
        float f[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          float mx = fmaxf(fmaxf(sc[0][2 * w], sc[0][2 * w + 1]), fmaxf(sc[1][2 * w], sc[1][2 * w + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[w], mx * p.scale_log2);
          const float ref = mn == -INFINITY ? 0.f : mn;
          f[w] = exp2f(m[w] - ref);
          m[w] = mn;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = fast_exp2(fmaf(sc[n][2 * w + e], p.scale_log2, -ref));
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
        ms[w * HEADS + (lane >> 2)] = m[w];
        ls[w * HEADS + (lane >> 2)] = l[w];
      }
    }
  }
  // buf[row][D] = sums * 2^(m - M[row])
  __device__ __forceinline__ void put(float* buf, const float* M, int lane) const {
    const int head = lane >> 2, c2 = (lane & 3) * 2;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int row = w * HEADS + head;
      const float f = m[w] == -INFINITY ? 0.f : exp2f(m[w] - M[row]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(buf + row * D + i * 8 + c2) = make_float2(acc[i][2 * w] * f, acc[i][2 * w + 1] * f);
    }
  }
};

// fp32: CUDA cores.  A lane owns D / 32 columns, so lanes 0-15 hold the first map's columns of K and
// lanes 16-31 the second's: one reduction over 16 lanes gives both maps' scores at once.  A warp
// takes four tokens at a time from its own ring; the reduction transposes as it goes (two
// values, then one, travel), so that afterwards a lane holds one token's score and takes one
// exponential, and eight shuffles hand the weights of both maps to all lanes.
template <int D, int G>
struct EngineF32 {
  using T = float;
  static constexpr int E = D / 32;
  static constexpr int U = 4;  // tokens of a stage
  static constexpr int NS = 6;
  static constexpr uint32_t ROWB = U * D * 4;  // K or V of a stage
  static constexpr uint32_t STAGE = 2 * ROWB;
  static constexpr uint32_t SMEM = WARPS * NS * STAGE;
  float acc[2][G][E];
  float m[G], l[G];  // of this half's map; l of this lane's tokens
  uint32_t base;
  const uint8_t* ring;

  __device__ __forceinline__ void init(uint32_t smem, int warp) {
    base = smem + (uint32_t)(warp * NS) * STAGE;
    extern __shared__ __align__(128) uint8_t smem_bytes[];
    ring = smem_bytes + (size_t)(warp * NS) * STAGE;
  }

  __device__ __forceinline__ void load(const Params& p, const T* kb, const T* vb, int stage, int tok0, int len, int lane) {
    const uint32_t dst = base + (uint32_t)stage * STAGE;
    constexpr int CH = D / 4;  // 16-byte chunks of a row
#pragma unroll
    for (int i = 0; i < U * CH / 32; ++i) {
      const int idx = i * 32 + lane, row = idx / CH, ch = idx % CH;
      const bool in = tok0 + row < len;
      const int64_t t = in ? tok0 + row : 0;  // a safe address where nothing is read
      cp_async16(dst + (uint32_t)idx * 16u, kb + t * p.ks[2] + ch * 4, in);
      cp_async16(dst + ROWB + (uint32_t)idx * 16u, vb + t * p.vs[2] + ch * 4, in);
    }
  }

  __device__ __forceinline__ void piece(const Params& p, int b, int hk, int h0, int nh, int t0, int t1, int len, int warp,
                                        int lane) {
    const T* qp = static_cast<const T*>(p.q) + ((int64_t)b * p.Hq + h0) * D + lane * E;
    const T* kb = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[1];
    const T* vb = static_cast<const T*>(p.v) + b * p.vs[0] + hk * p.vs[1];
    const int n = (t1 - t0) * (WT / U);  // groups of four tokens
    auto tok_of = [&](int g) { return (t0 + g / (WT / U)) * TILE + warp * WT + g % (WT / U) * U; };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (s < n) load(p, kb, vb, s, tok_of(s), len, lane);
      cp_commit();
    }
    float q[G][E];
#pragma unroll
    for (int i = 0; i < G; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[i][e] = i < nh ? qp[i * D + e] * p.scale_log2 : 0.f;
        acc[0][i][e] = acc[1][i][e] = 0.f;
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    const bool b3 = lane & 8, b2 = lane & 4;
    const int mine = (b3 ? 2 : 0) + (b2 ? 1 : 0);  // this lane's token of a group
    int stage = 0;
    for (int g = 0; g < n; ++g) {
      {
        int s = stage + NS - 1;
        if (s >= NS) s -= NS;
        if (g + NS - 1 < n) load(p, kb, vb, s, tok_of(g + NS - 1), len, lane);
        cp_commit();
      }
      cp_wait<NS - 1>();
      __syncwarp();
      const int tok = tok_of(g);
      if (tok < len) {
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
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float s[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s[u] = fmaf(q[i][e], kx[u][e], s[u]);
          }
          float k0 = b3 ? s[2] : s[0], k1 = b3 ? s[3] : s[1];
          k0 += __shfl_xor_sync(0xffffffffu, b3 ? s[0] : s[2], 8);
          k1 += __shfl_xor_sync(0xffffffffu, b3 ? s[1] : s[3], 8);
          float x = b2 ? k1 : k0;
          x += __shfl_xor_sync(0xffffffffu, b2 ? k0 : k1, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          if (tok + mine >= len) x = -INFINITY;
          float mx = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          mx = fmaxf(m[i], fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8)));
          const float ref = mx == -INFINITY ? 0.f : mx;
          const float f = exp2f(m[i] - ref);
          m[i] = mx;
          x = exp2f(x - ref);
          l[i] = l[i] * f + x;
          if (__any_sync(0xffffffffu, f != 1.f)) {
            const float fo = __shfl_xor_sync(0xffffffffu, f, 16);
            const float f1 = lane < 16 ? f : fo, f2 = lane < 16 ? fo : f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              acc[0][i][e] *= f1;
              acc[1][i][e] *= f2;
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int src = (u >> 1) * 8 + (u & 1) * 4;
            const float p1 = __shfl_sync(0xffffffffu, x, src), p2 = __shfl_sync(0xffffffffu, x, 16 + src);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              acc[0][i][e] = fmaf(p1, vx[u][e], acc[0][i][e]);
              acc[1][i][e] = fmaf(p2, vx[u][e], acc[1][i][e]);
            }
          }
        }
      }
      __syncwarp();  // every lane is done with the stage before the next load overwrites it
      if (++stage == NS) stage = 0;
    }
    cp_wait<0>();
#pragma unroll
    for (int i = 0; i < G; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
    }
  }

  __device__ __forceinline__ void put_stats(float* ms, float* ls, int lane) const {
    if ((lane & 15) == 0) {
      const int w = lane >> 4;
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        ms[w * HEADS + i] = i < G ? m[i < G ? i : 0] : -INFINITY;
        ls[w * HEADS + i] = i < G ? l[i < G ? i : 0] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void put(float* buf, const float* M, int lane) const {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[i], 16);
      const float mw[2] = {lane < 16 ? m[i] : mo, lane < 16 ? mo : m[i]};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int row = w * HEADS + i;
        const float f = mw[w] == -INFINITY ? 0.f : exp2f(mw[w] - M[row]);
#pragma unroll
        for (int e = 0; e < E; ++e) buf[row * D + lane * E + e] = acc[w][i][e] * f;
      }
    }
  }
};

// Bytes of the engine's ring, or of the warps' sums that take its place at a piece's end.
template <typename Engine, int D>
struct Big {
  static constexpr uint32_t SUMS = (uint32_t)(WARPS * ROWS * D * 4);
  static constexpr uint32_t BYTES = Engine::SMEM > SUMS ? Engine::SMEM : SUMS;
  // the last CTA's weights, and its columns' sums by group of pieces
  static_assert(MAX_SMS * ROWS * 4 + 2 * THREADS * 16 <= SUMS, "room for the merge");
};

template <typename Engine, int D>
__global__ void __launch_bounds__(THREADS) decode_kernel(const Params p) {
  using T = typename Engine::T;
  extern __shared__ __align__(128) uint8_t smem[];
  // [ring of the engine, or the warps' sums at a piece's end | warps' maxima and sums | M, L | scan | prefix]
  constexpr uint32_t BIG = Big<Engine, D>::BYTES;
  float* sums = reinterpret_cast<float*>(smem);
  float* ms = reinterpret_cast<float*>(smem + BIG);
  float* ls = ms + WARPS * ROWS;
  float* Ms = ls + WARPS * ROWS;
  float* Ls = Ms + ROWS;
  int32_t* scan = reinterpret_cast<int32_t*>(Ls + ROWS);  // [WARPS + 2]
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + BIG + 4 * (2 * WARPS * ROWS + 2 * ROWS + 16));  // [B + 1] tiles
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_kernel_before();

  // units before each sequence
  {
    Units carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + tid;
      int n = 0;
      if (b < p.B) {
        const int raw = p.lens[b];
        if ((raw < 0 || raw > p.T) && blockIdx.x == 0) record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, 6, b);
        n = (length_of(p, b) + TILE - 1) / TILE;
        if (n > 0) n += SEG_COST;
      }
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      Units before = 0, all = 0;
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
  const int per = p.Hkv * p.hc;  // (KV head, head chunk) of a sequence
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

  // O = sums1 / l1 - lam sums2 / l2 of a head's four columns, and its two LSEs
  auto finish = [&](int b, int h, int c4, float4 x1, float4 x2, float m1, float l1, float m2, float l2) {
    const float lam = to_f(static_cast<const T*>(p.lam)[p.lam_n == 1 ? 0 : h]);
    // no cached token: O = 0 (a NaN sum stays NaN)
    const float i1 = l1 == 0.f ? 0.f : 1.f / l1, i2 = l2 == 0.f ? 0.f : lam / l2;
    const float y[4] = {x1.x * i1 - x2.x * i2, x1.y * i1 - x2.y * i2, x1.z * i1 - x2.z * i2, x1.w * i1 - x2.w * i2};
    const int64_t at = ((int64_t)b * p.Hq + h) * D + c4;
    if constexpr (sizeof(T) == 2) {
      uint2 w;
      w.x = pack_bf16x2(y[0], y[1]);
      w.y = pack_bf16x2(y[2], y[3]);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at) = w;
    } else {
      *reinterpret_cast<float4*>(static_cast<T*>(p.o) + at) = make_float4(y[0], y[1], y[2], y[3]);
    }
    if (c4 == 0) {
      float* e = p.lse + ((int64_t)b * p.Hq + h) * 2;
      e[0] = l1 == 0.f ? -INFINITY : (m1 + log2f(l1)) * LN2;
      e[1] = l2 == 0.f ? -INFINITY : (m2 + log2f(l2)) * LN2;
    }
  };

  // sequences without a cached token: O = 0, LSE = -inf
  for (int b = blockIdx.x; b < p.B; b += (int)gridDim.x)
    if (prefix[b + 1] == prefix[b])
      for (int i = tid; i < p.Hq * (D / 4); i += THREADS)
        finish(b, i / (D / 4), i % (D / 4) * 4, make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0), 0.f, 0.f, 0.f, 0.f);

  Engine eng;
  eng.init(smem_u32(smem), warp);
  int64_t x = lo;
  while (x < hi) {
    // the sequence of unit x: the last b with prefix[b] * per <= x (empty ones share its prefix)
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
    const int64_t n = prefix[b + 1] - prefix[b];  // > SEG_COST
    const int64_t seg = (x - prefix[b] * per) / n;
    const int64_t s1 = prefix[b] * per + (seg + 1) * n, s0 = s1 - n + SEG_COST;  // the segment's tiles are [s0, s1)
    const int64_t end = min(hi, s1);
    if (end <= s0) {  // nothing of it but the units before its tiles
      x = end;
      continue;
    }
    x = max(x, s0);
    const int hk = (int)(seg / p.hc), c = (int)(seg % p.hc);
    const int h0 = hk * p.g + c * HEADS, nh = min(HEADS, p.g - c * HEADS);
    eng.piece(p, b, hk, h0, nh, (int)(x - s0), (int)(end - s0), length_of(p, b), warp, lane);

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
    eng.put(sums + warp * ROWS * D, Ms, lane);
    __syncthreads();
    const int h = tid / (D / 4), c4 = tid % (D / 4) * 4;
    float4 a1 = make_float4(0, 0, 0, 0), a2 = a1;
    if (h < nh) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 y1 = *reinterpret_cast<const float4*>(sums + (w * ROWS + h) * D + c4);
        const float4 y2 = *reinterpret_cast<const float4*>(sums + (w * ROWS + HEADS + h) * D + c4);
        a1.x += y1.x, a1.y += y1.y, a1.z += y1.z, a1.w += y1.w;
        a2.x += y2.x, a2.y += y2.y, a2.z += y2.z, a2.w += y2.w;
      }
    }
    if (s0 >= lo && s1 <= hi) {
      if (h < nh) finish(b, h0 + h, c4, a1, a2, Ms[h], Ls[h], Ms[HEADS + h], Ls[HEADS + h]);
    } else {
      // a piece: slot 1 where the segment begins here and goes on, slot 0 where it began before
      float* slot = p.part + ((int64_t)blockIdx.x * 2 + (s0 >= lo ? 1 : 0)) * part_floats(D);
      if (h < nh) {
        *reinterpret_cast<float4*>(slot + h * D + c4) = a1;
        *reinterpret_cast<float4*>(slot + (HEADS + h) * D + c4) = a2;
      }
      if (tid < ROWS) {
        slot[ROWS * D + tid] = Ms[tid];
        slot[ROWS * D + ROWS + tid] = Ls[tid];
      }
      __threadfence();
      __syncthreads();
      const int64_t i0 = owner_of(s0), i1 = owner_of(s1 - 1);
      if (tid == 0) {
        uint32_t* ctr = p.counters + (int64_t)b * per + seg;
        const bool last = atomicAdd(ctr, 1u) == (uint32_t)(i1 - i0);
        if (last) *ctr = 0u;
        scan[WARPS] = last;
      }
      __syncthreads();
      if (scan[WARPS]) {
        // the last CTA adds the segment's pieces up, in order.  Row r's weights 2^(m - M) first, sixteen
        // threads a row; then every thread takes one or two 16-byte columns of the rows over all pieces, or
        // over every G-th of them where there are fewer columns than threads.  (The pieces copied to
        // shared memory with cp.async instead: 3 us slower at 38 pieces.)
        __threadfence();
        const int n_p = (int)(i1 - i0 + 1);
        float* wts = sums;                    // [n_p][ROWS]
        float* part = sums + MAX_SMS * ROWS;  // [G][2 nh][D]
        auto slot_of = [&](int k) { return p.part + ((i0 + k) * 2 + (k == 0 ? 1 : 0)) * part_floats(D); };
        {
          const int r = tid >> 4, k0 = tid & 15;
          float M = -INFINITY;
#pragma unroll 4
          for (int k = k0; k < n_p; k += 16) M = fmaxf(M, __ldcg(slot_of(k) + ROWS * D + r));
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          float L = 0.f;
#pragma unroll 4
          for (int k = k0; k < n_p; k += 16) {
            const float* st = slot_of(k) + ROWS * D + r;
            const float m = __ldcg(st), l = __ldcg(st + ROWS);
            const float f = m == -INFINITY ? 0.f : exp2f(m - M);
            wts[k * ROWS + r] = f;
            L += m == -INFINITY ? l : l * f;  // l is 0 there, or NaN
          }
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
          if (k0 == 0) {
            Ms[r] = M;
            Ls[r] = L;
          }
        }
        __syncthreads();
        const int cols = 2 * nh * (D / 4), G = cols >= THREADS ? 1 : THREADS / cols;
        for (int o = tid; o < cols * G; o += THREADS) {
          const int grp = o / cols, c = o - grp * cols, r = c / (D / 4), at = c % (D / 4) * 4;
          const int row = r < nh ? r : HEADS + r - nh;
          float4 t = make_float4(0, 0, 0, 0);
#pragma unroll 16
          for (int k = grp; k < n_p; k += G) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(slot_of(k) + row * D + at));
            const float f = wts[k * ROWS + row];
            t.x = fmaf(y.x, f, t.x), t.y = fmaf(y.y, f, t.y), t.z = fmaf(y.z, f, t.z), t.w = fmaf(y.w, f, t.w);
          }
          *reinterpret_cast<float4*>(part + (grp * 2 * nh + r) * D + at) = t;
        }
        __syncthreads();
        if (h < nh) {
          a1 = a2 = make_float4(0, 0, 0, 0);
          for (int g = 0; g < G; ++g) {
            const float4 y1 = *reinterpret_cast<const float4*>(part + (g * 2 * nh + h) * D + c4);
            const float4 y2 = *reinterpret_cast<const float4*>(part + (g * 2 * nh + nh + h) * D + c4);
            a1.x += y1.x, a1.y += y1.y, a1.z += y1.z, a1.w += y1.w;
            a2.x += y2.x, a2.y += y2.y, a2.z += y2.z, a2.w += y2.w;
          }
          finish(b, h0 + h, c4, a1, a2, Ms[h], Ls[h], Ms[HEADS + h], Ls[HEADS + h]);
        }
      }
    }
    __syncthreads();  // the sums' memory is the ring's again
    x = end;
  }
}

struct Sizes {
  int g, hc, grid;
  size_t counters_off, total;
};
static Sizes sizes_of(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int sms) {
  Sizes s{};
  s.g = Hq / Hkv;
  s.hc = (s.g + HEADS - 1) / HEADS;
  const int64_t tiles = ((int64_t)T + TILE - 1) / TILE * B * Hkv * s.hc;
  s.grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, sms));
  // the slots come first and have the same place for all sizes, so that a workspace made for larger
  // sizes serves smaller ones too without leaving anything where a counter will be
  s.counters_off = (size_t)2 * mesh::MAX_SMS * part_floats(128) * 4;
  s.total = s.counters_off + (size_t)B * Hkv * s.hc * 4;
  return s;
}

template <typename Engine, int D>
static int launch(const Params& p, int grid, cudaStream_t st, std::string* err) {
  auto kern = decode_kernel<Engine, D>;
  const size_t smem = Big<Engine, D>::BYTES + 4 * (2 * WARPS * ROWS + 2 * ROWS + 16) + 8 * ((size_t)p.B + 1);
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  cudaError_t e = cudaSuccess;
  if (once.pending(dev)) {  // the most that any batch takes
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(smem + 8 * (size_t)(MAX_B - p.B)));
    if (e == cudaSuccess) once.mark(dev);
  }
  if (e == cudaSuccess) {
    e = launch_behind(kern, dim3((unsigned)grid), THREADS, smem, st, p);
  }
  if (e != cudaSuccess) *err = std::string("diff_decode launch: ") + cudaGetErrorString(e);
  return (int)e;
}

template <int D>
static int launch_f32(const Params& p, int grid, cudaStream_t st, std::string* err) {
  const int n = std::min(p.g, HEADS);
  if (n <= 1) return launch<EngineF32<D, 1>, D>(p, grid, st, err);
  if (n <= 2) return launch<EngineF32<D, 2>, D>(p, grid, st, err);
  if (n <= 4) return launch<EngineF32<D, 4>, D>(p, grid, st, err);
  return launch<EngineF32<D, 8>, D>(p, grid, st, err);
}

}  // namespace ddec
}  // namespace mesh

using mesh::set_last_error;

static int decode_checks(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T) {
  if (B < 0 || Hq < 0 || T < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "B, Hq and T must be >= 0");
  if (Hkv < 1 || Hq % Hkv != 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need Hkv >= 1 and Hq % Hkv == 0");
  if (d != 64 && d != 128) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (B > mesh::ddec::MAX_B) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "B must be at most 4096");
  if (T > mesh::ddec::MAX_T) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "T must be at most 2^30");
  return MESH_ATTN_OK;
}

extern "C" int mesh_attn_diff_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T,
                                                    size_t* bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!bytes) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "bytes is NULL");
    const int rc = decode_checks(B, Hq, Hkv, d, T);
    if (rc) return rc;
    *bytes = mesh::ddec::sizes_of(B, Hq, Hkv, (int32_t)T, mesh::MAX_SMS).total;
    return (int)MESH_ATTN_OK;
  });
}

extern "C" int mesh_attn_diff_decode(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T,
                                     const void* q, const void* k_cache, const int64_t* k_strides, const void* v_cache,
                                     const int64_t* v_strides, const int32_t* lens, const void* lam, int32_t lam_n,
                                     float scale, void* O, float* LSE, void* workspace, size_t workspace_bytes,
                                     int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    using namespace mesh::ddec;
    if (dtype != MESH_ATTN_F32 && dtype != MESH_ATTN_BF16)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "dtype must be MESH_ATTN_F32 or MESH_ATTN_BF16");
    const int rc = decode_checks(B, Hq, Hkv, d, T);
    if (rc) return rc;
    if (lam_n != 1 && lam_n != Hq) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "lam_n must be 1 or Hq");
    if (!(scale > 0.f) || !std::isfinite(scale))
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (B == 0 || Hq == 0) return (int)MESH_ATTN_OK;
    if (!q || !lens || !lam || !O || !LSE || !workspace || !d_status || (T > 0 && (!k_cache || !v_cache)))
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor, workspace or status pointer is NULL");
    if (!k_strides || !v_strides) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "k_strides or v_strides is NULL");
    const size_t es = dtype == MESH_ATTN_BF16 ? 2 : 4;
    for (const void* x : {q, k_cache, v_cache, (const void*)O, (const void*)workspace})
      if (!mesh::is_aligned(x, 16))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "q, the caches, O and workspace must be 16-byte aligned");
    if (!mesh::is_aligned(lens, 4) || !mesh::is_aligned(LSE, 4) || !mesh::is_aligned(d_status, 4) || !mesh::is_aligned(lam, es))
      return set_last_error(MESH_ATTN_ERR_MISALIGNED, "lens, LSE, lam and status must be aligned to their element size");
    for (int i = 0; i < 3; ++i)
      if (k_strides[i] * (int64_t)es % 16 != 0 || v_strides[i] * (int64_t)es % 16 != 0)
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "cache strides must be multiples of 16 bytes");
    int sms = 0;
    const cudaError_t e = mesh::current_sms(&sms);
    if (e != cudaSuccess) return set_last_error(MESH_ATTN_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    const Sizes s = sizes_of(B, Hq, Hkv, (int32_t)T, std::min(sms, mesh::MAX_SMS));
    if (workspace_bytes < s.total)
      return set_last_error(MESH_ATTN_ERR_WORKSPACE, "workspace needs " + std::to_string(s.total) + " bytes");
    Params p{};
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    for (int i = 0; i < 3; ++i) {
      p.ks[i] = k_strides[i];
      p.vs[i] = v_strides[i];
    }
    p.lens = lens;
    p.lam = lam;
    p.lam_n = lam_n;
    p.o = O;
    p.lse = LSE;
    p.counters = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + s.counters_off);
    p.part = static_cast<float*>(workspace);
    p.status = d_status;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = s.g;
    p.hc = s.hc;
    p.T = (int32_t)T;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    std::string err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int ce;
    if (dtype == MESH_ATTN_BF16)
      ce = d == 128 ? launch<EngineBf16<128>, 128>(p, s.grid, st, &err) : launch<EngineBf16<64>, 64>(p, s.grid, st, &err);
    else
      ce = d == 128 ? launch_f32<128>(p, s.grid, st, &err) : launch_f32<64>(p, s.grid, st, &err);
    return mesh::launch_status(ce, err);
  });
}
