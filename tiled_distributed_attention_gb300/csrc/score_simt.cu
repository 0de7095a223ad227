// Attention with scores that are capped, biased and masked by ranges, fp32 inputs, on the CUDA cores: of a dense batch
// (range-masked attention, both directions) and of the new tokens of sequences in a paged cache.  The formulas are those of
// score_fwd.cuh and score_bwd.cuh; everything is fp32, sums in the order of the keys.
//
// A tile is 64 rows, the query heads of a KV head and their tokens (row = token * g + head), which stream blocks of
// 64 keys through shared memory; 256 threads hold 4 x 4 scores and 4 x D / 16 outputs each, read operands by 16-byte accesses
// and keep the row statistics in registers, 16 lanes a row.
//
// Bound by those accesses: a warp's 16 bytes a lane take four cycles of the SM's 128 bytes a cycle, whichever rows they are of, and
// eight of them stand before 64 FMAs, so that the FMA pipe is busy half of the time (measured 52 %).  In keeping with that, FMAs in
// pairs (half the instructions) and warps of 4 x 8 threads (fewer distinct rows an access) made no difference; 8 x 4 scores a
// thread have fewer accesses but half the warps, and were 5 to 15 % slower.  Measured: 777 tokens in three documents, 4 heads
// on 2, d 64, capped, slopes, both directions 66 us; 2 x 1,024, 8 heads on 2, causal, 358 (21 TFLOP/s), at d = 128 650 (23).
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "score_bwd.h"

namespace mesh {
namespace simt {

constexpr int THREADS = 256;
constexpr int TR = 64;  // rows of a tile
constexpr int TK = 64;  // keys of a block
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;
constexpr int MAX_PARTS = 16;
constexpr int ROLE_SEQ = 1, ROLE_PAGE = 2;

struct Params {
  const float* q;
  const float* k;
  const float* v;
  int64_t qs[3];          // batch, head, token strides
  int64_t ks[3], vs[3];   // batch or page, head, row strides
  const float* slopes;
  float* o;
  int64_t os[3];
  float* lse;
  int64_t ls[3];
  const int32_t* lo;
  const int32_t* hi;
  int64_t mask_bs;
  const int32_t* offsets;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_s;
  int32_t* status;
  int64_t S;
  float* part_o;  // tiles in parts: [tile of all][part][TR][D], normalised, and [tile of all][part][TR]
  float* part_lse;
  int32_t N, B, Hq, Hkv, g, n_pages, page, max_pages, max_new, window, tiles, parts;
  float scale, scale_log2, cap;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;  // 0: the 16 bytes are zero-filled and src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// A tile: rows r0 .. of the n_tok * g of sequence or batch entry b and KV head hk; keys [kmin, kmax) that some row may see.
struct Tile {
  int b, hk, r0, nr, row0, pos0, len, kmin, kmax;
};

// Tile `slot` of KV head hk (and batch entry b; paged: of all sequences) by all threads of a CTA of TR or more; false where
// there is none.  The last tokens, the longest where the mask is causal, have the first slots.  With `bounds` (shared memory)
// its keys too, and what does not fit is reported.
template <bool PAGED>
__device__ __forceinline__ bool tile_of(const Params& p, int slot, int hk, int b, Tile& t, int* bounds = nullptr) {
  const int tid = threadIdx.x;
  slot = p.tiles - 1 - slot;
  t.hk = hk;
  int n_tok;
  if (PAGED) {
    // sequence b's tiles are those from offsets[b] g / TR + b on: there is room for its own, and a few are empty
    int a = 0, z = p.B;
    while (z - a > 1) {
      const int c = (a + z) >> 1;
      if ((int64_t)max(p.offsets[c], 0) * p.g / TR + c <= slot) a = c;
      else z = c;
    }
    t.b = a;
    const Asked s = asked(p.offsets, p.lens, a, p.N, p.max_new, p.max_pages, p.page);
    if (bounds && tid == 0 && s.bad) record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_SEQ, a);
    t.row0 = s.begin;
    t.len = s.len;
    t.pos0 = s.len - s.n;
    n_tok = s.n;
    const int64_t r = ((int64_t)slot - ((int64_t)t.row0 * p.g / TR + a)) * TR;
    if (r < 0 || r >= (int64_t)n_tok * p.g) return false;
    t.r0 = (int)r;
    t.nr = min(TR, n_tok * p.g - t.r0);
    t.kmin = p.window ? max(0, t.pos0 + t.r0 / p.g + 1 - p.window) : 0;
    t.kmax = t.pos0 + (t.r0 + t.nr - 1) / p.g + 1;
  } else {
    t.b = b;
    t.row0 = t.pos0 = 0;
    t.len = (int)p.S;
    t.r0 = slot * TR;
    t.nr = (int)min((int64_t)TR, p.S * p.g - t.r0);
    if (!bounds) return true;
    if (tid == 0) {
      bounds[0] = 0x7fffffff;
      bounds[1] = 0;
    }
    __syncthreads();
    if (tid < t.nr) {
      const int tok = (t.r0 + tid) / p.g;
      const int a = max(p.lo[t.b * p.mask_bs + tok], 0), z = min(p.hi[t.b * p.mask_bs + tok], t.len);
      if (a < z) {
        atomicMin(&bounds[0], a);
        atomicMax(&bounds[1], z);
      }
    }
    __syncthreads();
    t.kmin = bounds[0];
    t.kmax = bounds[1];
  }
  return true;
}
// Of a tile's blocks [j0, j1) of TK keys those of part `part`.
__device__ __forceinline__ void part_of(const Tile& t, int parts, int part, int& j0, int& j1) {
  j0 = j1 = 0;
  if (t.kmin >= t.kmax) return;
  const int first = t.kmin / TK, n = (t.kmax + TK - 1) / TK - first, k = max(1, min(parts, n));
  j0 = first + (int)((int64_t)min(part, k) * n / k);
  j1 = first + (int)((int64_t)min(part + 1, k) * n / k);
}

template <int D>
struct Smem {
  static constexpr int LD = D + 4;   // rows of Q, K: 16-byte accesses of eight rows at once touch all banks
  static constexpr int LP = TK + 4;
  static constexpr int Q = 0, K = Q + TR * LD, V = K + TK * LD, P = V + TK * D, TOTAL = P + TR * LP;
};

// A score in base 2 from q.k: scaled, capped, biased.
__device__ __forceinline__ float score2(const Params& p, float dot, int far, float slope2) {
  float x = p.cap > 0.f ? p.cap * LOG2E * tanhf(dot * (p.scale / p.cap)) : dot * p.scale_log2;
  return slope2 != 0.f ? fmaf(-slope2, fabsf((float)far), x) : x;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(THREADS, D == 64 ? 2 : 1) fwd_kernel(const __grid_constant__ Params p) {
  using Sm = Smem<D>;
  constexpr int CW = D / 16;  // columns of a thread's outputs
  extern __shared__ __align__(16) float sm[];
  __shared__ int bounds[2];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  wait_for_kernel_before();
  if (stopped<PAGED>(p.status)) return;
  Tile t;
  const int part = PAGED ? (int)blockIdx.z : (int)blockIdx.z % p.parts;
  if (!tile_of<PAGED>(p, (int)blockIdx.x, (int)blockIdx.y, PAGED ? 0 : (int)blockIdx.z / p.parts, t, bounds)) return;
  int j_begin, j_end;
  part_of(t, p.parts, part, j_begin, j_end);
  const float* kb = p.k + (PAGED ? 0 : t.b * p.ks[0]) + t.hk * p.ks[1];
  const float* vb = p.v + (PAGED ? 0 : t.b * p.vs[0]) + t.hk * p.vs[1];
  const uint32_t sq = smem_u32(sm + Sm::Q), sk = smem_u32(sm + Sm::K), sv = smem_u32(sm + Sm::V);
  // Q: rows behind the last are zeros
  for (int i = tid; i < TR * (D / 4); i += THREADS) {
    const int r = i / (D / 4), c = i % (D / 4) * 4, row = t.r0 + r, tok = row / p.g, h = t.hk * p.g + row - tok * p.g;
    const bool in = r < t.nr;
    cp_async16(sq + (uint32_t)(r * Sm::LD + c) * 4u,
               in ? p.q + (PAGED ? 0 : t.b * p.qs[0]) + h * p.qs[1] + (int64_t)(t.row0 + tok) * p.qs[2] + c : p.q, in);
  }
  // this thread's rows
  int lo[4], hi[4], pos[4];
  float slope2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = hi[i] = pos[i] = 0;
    slope2[i] = 0.f;
    const int row = t.r0 + ty * 4 + i, tok = row / p.g;
    if (ty * 4 + i < t.nr) {
      pos[i] = t.pos0 + tok;
      if (PAGED) {
        hi[i] = pos[i] + 1;
        lo[i] = p.window ? max(0, hi[i] - p.window) : 0;
      } else {
        lo[i] = max(p.lo[t.b * p.mask_bs + tok], 0);
        hi[i] = min(p.hi[t.b * p.mask_bs + tok], t.len);
      }
      if (p.slopes) slope2[i] = p.slopes[t.hk * p.g + row - tok * p.g] * LOG2E;
    }
  }
  float m[4], l[4], o[4][CW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CW; ++c) o[i][c] = 0.f;
  }
  for (int j0 = j_begin * TK; j0 < j_end * TK; j0 += TK) {
    // K and V: keys behind the last are zeros
    for (int i = tid; i < TK * (D / 4); i += THREADS) {
      const int r = i / (D / 4), c = i % (D / 4) * 4, key = j0 + r;
      bool in = key < t.len && key >= t.kmin;  // pages before a window need not be there any more
      int64_t pg = 0, row = key;
      if (PAGED && in) {
        const int at = key / p.page;
        pg = p.table[t.b * p.table_s + at];
        row = key - at * p.page;
        if (pg < 0 || pg >= p.n_pages) {
          record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_PAGE, t.b);
          in = false;
        }
      }
      cp_async16(sk + (uint32_t)(r * Sm::LD + c) * 4u, in ? kb + pg * p.ks[0] + row * p.ks[2] + c : p.k, in);
      cp_async16(sv + (uint32_t)(r * D + c) * 4u, in ? vb + pg * p.vs[0] + row * p.vs[2] + c : p.v, in);
    }
    cp_wait_all();
    __syncthreads();
    // scores of rows ty * 4 + i and keys j0 + tx + 16 j
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sm + Sm::Q + (ty * 4 + i) * Sm::LD + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sm + Sm::K + (tx + 16 * j) * Sm::LD + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        s[i][j] = key >= lo[i] && key < hi[i] ? score2(p, s[i][j], pos[i] - key, slope2[i]) : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float ref = mx == -INFINITY ? 0.f : mx, f = exp2f(m[i] - ref);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - ref);
        sum += e;
        sm[Sm::P + (ty * 4 + i) * Sm::LP + tx + 16 * j] = e;
      }
      l[i] = l[i] * f + sum;  // of this lane's keys
#pragma unroll
      for (int c = 0; c < CW; ++c) o[i][c] *= f;
    }
    __syncwarp();  // a row's weights are its own half-warp's
#pragma unroll 4
    for (int k0 = 0; k0 < TK; k0 += 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sm + Sm::P + (ty * 4 + i) * Sm::LP + k0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          const float4 y = *reinterpret_cast<const float4*>(sm + Sm::V + (k0 + e) * D + c * 16 + tx * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
            o[i][c] = fmaf(f, y.x, o[i][c]);
            o[i][c + 1] = fmaf(f, y.y, o[i][c + 1]);
            o[i][c + 2] = fmaf(f, y.z, o[i][c + 2]);
            o[i][c + 3] = fmaf(f, y.w, o[i][c + 3]);
          }
        }
    }
    __syncthreads();  // the next block overwrites K, V and P
  }
  cp_wait_all();  // Q's copies, where no block was read
  const int64_t tile = ((int64_t)(PAGED ? 0 : t.b) * p.Hkv + t.hk) * p.tiles + blockIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (ty * 4 + i >= t.nr) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no visible key: O = 0 (a NaN sum stays NaN)
    const float lse = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * LN2;
    if (p.parts > 1) {
      const int64_t at = (tile * p.parts + part) * TR + ty * 4 + i;
      if (j_begin < j_end) {
#pragma unroll
        for (int c = 0; c < CW; c += 4)
          *reinterpret_cast<float4*>(p.part_o + at * D + c * 16 + tx * 4) =
              make_float4(o[i][c] * inv, o[i][c + 1] * inv, o[i][c + 2] * inv, o[i][c + 3] * inv);
      }
      if (tx == 0) p.part_lse[at] = lse;
      continue;
    }
    const int row = t.r0 + ty * 4 + i, tok = row / p.g, h = t.hk * p.g + row - tok * p.g;
    const int64_t bo = PAGED ? 0 : t.b, to = t.row0 + tok;
    float* dst = p.o + bo * p.os[0] + h * p.os[1] + to * p.os[2];
#pragma unroll
    for (int c = 0; c < CW; c += 4)
      *reinterpret_cast<float4*>(dst + c * 16 + tx * 4) =
          make_float4(o[i][c] * inv, o[i][c + 1] * inv, o[i][c + 2] * inv, o[i][c + 3] * inv);
    if (tx == 0) p.lse[bo * p.ls[0] + h * p.ls[1] + to * p.ls[2]] = lse;
  }
}

// O = sum_t w_t O_t over a tile's parts, w_t = exp(lse_t - lse), and the LSE, parts in order.  A thread takes a 16-byte piece of a
// row, all parts' loads in flight together; a CTA a few rows.
template <int D>
constexpr int MERGE_ROWS = THREADS / (D / 4);
template <int D, bool PAGED>
__global__ void __launch_bounds__(THREADS) merge_kernel(const __grid_constant__ Params p) {
  constexpr int PER_TILE = TR / MERGE_ROWS<D>;
  wait_for_kernel_before();
  if (stopped<PAGED>(p.status)) return;
  const int slot = (int)blockIdx.x / PER_TILE;
  const int r = (int)blockIdx.x % PER_TILE * MERGE_ROWS<D> + (int)threadIdx.x / (D / 4), c = (int)threadIdx.x % (D / 4) * 4;
  Tile t;
  if (!tile_of<PAGED>(p, slot, (int)blockIdx.y, (int)blockIdx.z, t) || r >= t.nr) return;
  const int row = t.r0 + r, tok = row / p.g, h = t.hk * p.g + row - tok * p.g;
  const int64_t at = (((int64_t)(PAGED ? 0 : t.b) * p.Hkv + t.hk) * p.tiles + slot) * p.parts * TR + r;
  float w[MAX_PARTS];
  float4 y[MAX_PARTS];
  float M = -INFINITY, W = 0.f;
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k) {
    w[k] = k < p.parts ? p.part_lse[at + (int64_t)k * TR] : -INFINITY;
    M = fmaxf(M, w[k]);
  }
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k)
    y[k] = w[k] != -INFINITY ? *reinterpret_cast<const float4*>(p.part_o + (at + (int64_t)k * TR) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float Ms = M == -INFINITY ? 0.f : M;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < MAX_PARTS; ++k) {
    const float f = expf(w[k] - Ms);
    W += f;
    o.x = fmaf(f, y[k].x, o.x), o.y = fmaf(f, y[k].y, o.y), o.z = fmaf(f, y[k].z, o.z), o.w = fmaf(f, y[k].w, o.w);
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;  // a NaN sum stays NaN
  const int64_t bo = PAGED ? 0 : t.b, to = t.row0 + tok;
  *reinterpret_cast<float4*>(p.o + bo * p.os[0] + h * p.os[1] + to * p.os[2] + c) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (c == 0) p.lse[bo * p.ls[0] + h * p.ls[1] + to * p.ls[2]] = W == 0.f ? -INFINITY : Ms + logf(W);
}

// ---------------------------------------------------------------- backward
struct BwdParams {
  const float* q;
  const float* k;
  const float* v;
  const float* go;
  const float* lse;
  const float* dsum;
  const int32_t* lo;
  const int32_t* hi;
  int64_t mask_bs;
  const float* slopes;
  float* dq;  // or the parts, [B, H, parts, S, D]
  float* dk;
  float* dv;
  int32_t* status;
  int64_t S;
  int32_t B, Hq, Hkv, g, dq_parts, kv_parts, dq_tiles, kv_tiles;
  float scale, scale_log2, cap;
};

template <int D>
struct BwdSmem {
  static constexpr int LD = D + 4, LP = TK + 4;
  static constexpr int A = 0, B = A + TR * LD, C = B + TR * LD, E = C + TK * LD, P = E + TK * LD, TOTAL = P + TR * LP;
};

// P of a score, and P (1 - t^2), which is what dS takes.
__device__ __forceinline__ void weight(const BwdParams& p, float dot, int far, float slope2, float nlse, float& P, float& W) {
  float x, f = 1.f;
  if (p.cap > 0.f) {
    const float t = tanhf(dot * (p.scale / p.cap));
    x = p.cap * LOG2E * t;
    f = 1.f - t * t;
  } else {
    x = dot * p.scale_log2;
  }
  if (slope2 != 0.f) x = fmaf(-slope2, fabsf((float)far), x);
  P = exp2f(x + nlse);
  W = P * f;
}

// acc[i][j] = sum over the columns of a's row 4 ty + i times b's row tx + 16 j
template <int D>
__device__ __forceinline__ void rows_by_rows(const float* a_s, const float* b_s, int tx, int ty, float (&acc)[4][4]) {
  constexpr int LD = D + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 8
  for (int c = 0; c < D; c += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(a_s + (ty * 4 + i) * LD + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(b_s + (tx + 16 * j) * LD + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
  }
}
// o[i][..] += sum over k of w's row 4 ty + i, column k, times x's row k
template <int D>
__device__ __forceinline__ void weights_by_rows(const float* w_s, const float* x_s, int tx, int ty, float (&o)[4][D / 16]) {
  constexpr int LD = D + 4, LP = TK + 4;
#pragma unroll 4
  for (int k0 = 0; k0 < TK; k0 += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(w_s + (ty * 4 + i) * LP + k0);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int c = 0; c < D / 16; c += 4) {
        const float4 y = *reinterpret_cast<const float4*>(x_s + (k0 + e) * LD + c * 16 + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
          o[i][c] = fmaf(f, y.x, o[i][c]);
          o[i][c + 1] = fmaf(f, y.y, o[i][c + 1]);
          o[i][c + 2] = fmaf(f, y.z, o[i][c + 2]);
          o[i][c + 3] = fmaf(f, y.w, o[i][c + 3]);
        }
      }
  }
}
// 64 rows of a dense [rows][D] tensor from row `r0` on, zeros from `n` on, into shared memory
template <int D>
__device__ __forceinline__ void load_rows(uint32_t dst, const float* src, int64_t r0, int64_t n, int tid) {
  for (int i = tid; i < 64 * (D / 4); i += THREADS) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const bool in = r0 + r < n;
    cp_async16(dst + (uint32_t)(r * (D + 4) + c) * 4u, in ? src + (r0 + r) * D + c : src, in);
  }
}

// dQ of 64 rows (token * g + head) of a batch entry and KV head, over a part of the key blocks that they see.
template <int D>
__device__ __forceinline__ void dq_tile(const BwdParams& p, float* sm, int (&bounds)[2], int tile, int hk, int b, int part) {
  using Sm = BwdSmem<D>;
  constexpr int CW = D / 16;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int r0 = (p.dq_tiles - 1 - tile) * TR, nr = (int)min((int64_t)TR, p.S * p.g - r0);
  if (tid < 2) bounds[tid] = tid ? 0 : 0x7fffffff;
  __syncthreads();
  if (tid < nr) {
    const int tok = (r0 + tid) / p.g;
    const int a = max(p.lo[b * p.mask_bs + tok], 0), z = min(p.hi[b * p.mask_bs + tok], (int)p.S);
    if (a < z) {
      atomicMin(&bounds[0], a);
      atomicMax(&bounds[1], z);
    }
  }
  __syncthreads();
  Tile t{};
  t.kmin = bounds[0], t.kmax = bounds[1];
  int j_begin, j_end;
  part_of(t, p.dq_parts, part, j_begin, j_end);
  const int64_t head0 = (int64_t)b * p.Hq + hk * p.g;
  const float* kb = p.k + ((int64_t)b * p.Hkv + hk) * p.S * D;
  const float* vb = p.v + ((int64_t)b * p.Hkv + hk) * p.S * D;
  const uint32_t base = smem_u32(sm);
  for (int i = tid; i < TR * (D / 4); i += THREADS) {  // Q and dO
    const int r = i / (D / 4), c = i % (D / 4) * 4, row = r0 + r, tok = row / p.g;
    const bool in = r < nr;
    const int64_t at = ((head0 + row - tok * p.g) * p.S + tok) * D + c;
    cp_async16(base + (uint32_t)(Sm::A + r * Sm::LD + c) * 4u, in ? p.q + at : p.q, in);
    cp_async16(base + (uint32_t)(Sm::B + r * Sm::LD + c) * 4u, in ? p.go + at : p.go, in);
  }
  int lo[4], hi[4], pos[4];
  float slope2[4], nlse[4], dsum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = r0 + ty * 4 + i, tok = row / p.g, h = row - tok * p.g;
    const bool in = ty * 4 + i < nr;
    const int64_t at = (head0 + h) * p.S + tok;
    pos[i] = tok;
    lo[i] = in ? max(p.lo[b * p.mask_bs + tok], 0) : 0;
    hi[i] = in ? min(p.hi[b * p.mask_bs + tok], (int)p.S) : 0;
    slope2[i] = in && p.slopes ? p.slopes[hk * p.g + h] * LOG2E : 0.f;
    const float l = in ? p.lse[at] : -INFINITY;
    nlse[i] = l == -INFINITY ? -INFINITY : -l * LOG2E;
    dsum[i] = in ? p.dsum[at] : 0.f;
  }
  float o[4][CW];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < CW; ++c) o[i][c] = 0.f;
  for (int jb = j_begin; jb < j_end; ++jb) {
    const int j0 = jb * TK;
    load_rows<D>(base + Sm::C * 4u, kb, j0, p.S, tid);
    load_rows<D>(base + Sm::E * 4u, vb, j0, p.S, tid);
    cp_wait_all();
    __syncthreads();
    float s[4][4], dp[4][4];
    rows_by_rows<D>(sm + Sm::A, sm + Sm::C, tx, ty, s);
    rows_by_rows<D>(sm + Sm::B, sm + Sm::E, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        float P, W;
        weight(p, s[i][j], pos[i] - key, slope2[i], nlse[i], P, W);
        sm[Sm::P + (ty * 4 + i) * Sm::LP + tx + 16 * j] = key >= lo[i] && key < hi[i] ? W * (dp[i][j] - dsum[i]) : 0.f;
      }
    __syncwarp();  // a row's weights are its own half-warp's
    weights_by_rows<D>(sm + Sm::P, sm + Sm::C, tx, ty, o);
    __syncthreads();  // the next block overwrites K, V and dS
  }
  cp_wait_all();  // Q's copies, where no block was read
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= nr) continue;
    const int row = r0 + ty * 4 + i, h = row - pos[i] * p.g;
    const int64_t at = ((head0 + h) * p.dq_parts + part) * p.S + pos[i];
#pragma unroll
    for (int c = 0; c < CW; c += 4)
      *reinterpret_cast<float4*>(p.dq + at * D + c * 16 + tx * 4) =
          make_float4(o[i][c] * p.scale, o[i][c + 1] * p.scale, o[i][c + 2] * p.scale, o[i][c + 3] * p.scale);
  }
}

// dK and dV of 64 keys of a batch entry and KV head, over a part of the blocks of 64 queries of its query heads that may see them:
// those from the first to the last query that does.
template <int D>
__device__ __forceinline__ void dkdv_tile(const BwdParams& p, float* sm, int (&bounds)[2], int tile, int hk, int b, int part) {
  using Sm = BwdSmem<D>;
  constexpr int CW = D / 16;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int k0 = tile * TK;
  if (tid < 2) bounds[tid] = tid ? 0 : 0x7fffffff;
  __syncthreads();
  {
    int first = 0x7fffffff, end = 0;
    for (int i = tid; i < (int)p.S; i += THREADS) {
      const int a = max(p.lo[b * p.mask_bs + i], 0), z = min(p.hi[b * p.mask_bs + i], (int)p.S);
      if (a < z && a < k0 + TK && z > k0) {
        first = min(first, i);
        end = i + 1;
      }
    }
    if (end) {
      atomicMin(&bounds[0], first);
      atomicMax(&bounds[1], end);
    }
  }
  __syncthreads();
  const int q_first = bounds[1] ? bounds[0] / TR : 0, per = bounds[1] ? (bounds[1] + TR - 1) / TR - q_first : 0;
  const int n = per * p.g, kp = max(1, min(p.kv_parts, n));
  const int begin = (int)((int64_t)min(part, kp) * n / kp), end = (int)((int64_t)min(part + 1, kp) * n / kp);
  const int64_t kv = (int64_t)b * p.Hkv + hk;
  const uint32_t base = smem_u32(sm);
  load_rows<D>(base + Sm::A * 4u, p.k + kv * p.S * D, k0, p.S, tid);
  load_rows<D>(base + Sm::B * 4u, p.v + kv * p.S * D, k0, p.S, tid);
  float dk[4][CW], dv[4][CW];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < CW; ++c) dk[i][c] = dv[i][c] = 0.f;
  for (int u = begin; u < end; ++u) {
    const int h = hk * p.g + u / per, q0 = (q_first + u % per) * TR;
    const int64_t head = (int64_t)b * p.Hq + h;
    load_rows<D>(base + Sm::C * 4u, p.q + head * p.S * D, q0, p.S, tid);
    load_rows<D>(base + Sm::E * 4u, p.go + head * p.S * D, q0, p.S, tid);
    const float slope2 = p.slopes ? p.slopes[h] * LOG2E : 0.f;
    float nlse[4], dsum[4];
    int lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = q0 + tx + 16 * j;
      const bool in = q < p.S;
      const float l = in ? p.lse[head * p.S + q] : -INFINITY;
      nlse[j] = l == -INFINITY ? -INFINITY : -l * LOG2E;
      dsum[j] = in ? p.dsum[head * p.S + q] : 0.f;
      lo[j] = in ? p.lo[b * p.mask_bs + q] : 0;
      hi[j] = in ? p.hi[b * p.mask_bs + q] : 0;
    }
    cp_wait_all();
    __syncthreads();
    float s[4][4], dp[4][4];
    rows_by_rows<D>(sm + Sm::A, sm + Sm::C, tx, ty, s);
    rows_by_rows<D>(sm + Sm::B, sm + Sm::E, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + ty * 4 + i;
        float P, W;
        weight(p, s[i][j], q0 + tx + 16 * j - key, slope2, nlse[j], P, W);
        const bool in = key >= lo[j] && key < hi[j];
        sm[Sm::P + (ty * 4 + i) * Sm::LP + tx + 16 * j] = in ? P : 0.f;
        dp[i][j] = in ? W * (dp[i][j] - dsum[j]) : 0.f;
      }
    __syncwarp();  // a row's weights are its own half-warp's
    weights_by_rows<D>(sm + Sm::P, sm + Sm::E, tx, ty, dv);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm[Sm::P + (ty * 4 + i) * Sm::LP + tx + 16 * j] = dp[i][j];
    __syncwarp();
    weights_by_rows<D>(sm + Sm::P, sm + Sm::C, tx, ty, dk);
    __syncthreads();  // the next block overwrites Q, dO and the weights
  }
  cp_wait_all();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t key = (int64_t)k0 + ty * 4 + i;
    if (key >= p.S) continue;
    const int64_t at = ((kv * p.kv_parts + part) * p.S + key) * D + tx * 4;
#pragma unroll
    for (int c = 0; c < CW; c += 4) {
      *reinterpret_cast<float4*>(p.dk + at + c * 16) =
          make_float4(dk[i][c] * p.scale, dk[i][c + 1] * p.scale, dk[i][c + 2] * p.scale, dk[i][c + 3] * p.scale);
      *reinterpret_cast<float4*>(p.dv + at + c * 16) = make_float4(dv[i][c], dv[i][c + 1], dv[i][c + 2], dv[i][c + 3]);
    }
  }
}

// Both in one launch, a CTA a tile and part: those of dK and dV, which take longer, first (one after the other they leave half of
// the SMs idle at each one's end: 84 us of forward and backward where this takes 69, 777 tokens of 4 heads on 2).
template <int D>
__global__ void __launch_bounds__(THREADS, D == 64 ? 2 : 1) bwd_kernel(const __grid_constant__ BwdParams p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int bounds[2];
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(p.status) != 0) return;
  const int n_kv = p.kv_tiles * p.Hkv * p.B * p.kv_parts;
  int i = (int)blockIdx.x;
  const bool kv = i < n_kv;
  if (!kv) i -= n_kv;
  const int tiles = kv ? p.kv_tiles : p.dq_tiles, parts = kv ? p.kv_parts : p.dq_parts;
  const int tile = i % tiles, hk = i / tiles % p.Hkv, z = i / tiles / p.Hkv;
  if (kv) dkdv_tile<D>(p, sm, bounds, tile, hk, z / parts, z % parts);
  else dq_tile<D>(p, sm, bounds, tile, hk, z / parts, z % parts);
}

// D = dO . O by rows, D / 4 lanes a row.
template <int D>
__global__ void __launch_bounds__(THREADS) dsum_kernel(const float4* o, const float4* go, float* dsum, int64_t rows, int32_t* status) {
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(status) != 0) return;
  constexpr int L = D / 4;
  const int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x, row = at / L;
  float s = 0.f;
  if (row < rows) {
    const float4 x = o[at], y = go[at];
    s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
  }
#pragma unroll
  for (int w = L / 2; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  if (row < rows && at % L == 0) dsum[row] = s;
}

// Sums of parts, in order: out[h] = sum over the parts of part[h, part], for up to three tensors.
struct SumParams {
  const float4* part[3];
  float4* out[3];
  int64_t n[3], per_head;
  int32_t parts[3];
  int32_t* status;
};
__global__ void __launch_bounds__(THREADS) sum_kernel(const __grid_constant__ SumParams p) {
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(p.status) != 0) return;
  int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x;
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
    p.out[w][i] = s;
    return;
  }
}

template <typename K>
static cudaError_t allow_smem(K kern, size_t bytes, OncePerDevice& once) {
  const int dev = OncePerDevice::device();
  if (!once.pending(dev)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) once.mark(dev);
  return e;
}

template <int D, bool PAGED>
static int launch_fwd(const Params& p, dim3 grid, cudaStream_t st, std::string* err) {
  auto kern = fwd_kernel<D, PAGED>;
  const size_t smem = (size_t)Smem<D>::TOTAL * 4;
  static OncePerDevice once;
  cudaError_t e = allow_smem(kern, smem, once);
  if (e == cudaSuccess) e = launch_behind(kern, dim3(grid.x, grid.y, grid.z * p.parts), THREADS, smem, st, p);
  if (e == cudaSuccess && p.parts > 1)
    e = launch_behind(merge_kernel<D, PAGED>, dim3(grid.x * (TR / MERGE_ROWS<D>), grid.y, grid.z), THREADS, 0, st, p);
  if (e != cudaSuccess) *err = std::string("score fp32 forward launch: ") + cudaGetErrorString(e);
  return (int)e;
}

template <int D>
static int launch_bwd(const RangeArgs& a, const RangeBwdShape& z, BwdParams p, cudaStream_t st, std::string* err) {
  const int64_t rows = (int64_t)a.B * a.Hq * a.S;
  const size_t smem = (size_t)BwdSmem<D>::TOTAL * 4;
  static OncePerDevice once;
  cudaError_t e = allow_smem(bwd_kernel<D>, smem, once);
  if (e == cudaSuccess)
    e = launch_behind(dsum_kernel<D>, dim3((unsigned)((rows * (D / 4) + THREADS - 1) / THREADS)), THREADS, 0, st,
                      static_cast<const float4*>(a.o), static_cast<const float4*>(a.go), const_cast<float*>(p.dsum), rows, a.status);
  if (e == cudaSuccess)
    e = launch_behind(bwd_kernel<D>, dim3((unsigned)a.Hkv * (unsigned)a.B * (unsigned)(p.kv_tiles * z.kv_parts + p.dq_tiles * z.dq_parts)),
                      THREADS, smem, st, p);
  if (e == cudaSuccess && (z.kv_parts > 1 || z.dq_parts > 1)) {
    SumParams sp{};
    const float* parts[3] = {p.dq, p.dk, p.dv};
    void* outs[3] = {a.dq, a.dk, a.dv};
    int64_t n = 0;
    for (int w = 0; w < 3; ++w) {
      sp.parts[w] = w ? z.kv_parts : z.dq_parts;
      sp.part[w] = reinterpret_cast<const float4*>(parts[w]);
      sp.out[w] = static_cast<float4*>(outs[w]);
      sp.n[w] = sp.parts[w] > 1 ? (int64_t)a.B * (w ? a.Hkv : a.Hq) * a.S * (D / 4) : 0;
      n += sp.n[w];
    }
    sp.per_head = a.S * (D / 4);
    sp.status = a.status;
    e = launch_behind(sum_kernel, dim3((unsigned)((n + THREADS - 1) / THREADS)), THREADS, 0, st, sp);
  }
  if (e != cudaSuccess) *err = std::string("score fp32 backward launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace simt

static bool grid_fits(int64_t x, int64_t y, int64_t z, std::string* err) {
  if (x <= 0x7fffffff && y <= 65535 && z <= 65535) return true;
  *err = "too many tiles, KV heads or sequences for one launch";
  return false;
}

// Tiles are cut into parts of their keys where whole ones would leave SMs idle: down to a block, and to twice the CTAs that are
// resident (two an SM), since tiles of ragged batches are of very different lengths (777 tokens of 4 heads on 2 in three
// documents: 22 us; 36 with parts of two blocks and half as many).
static int32_t fwd_parts(int64_t tiles, int64_t blocks, int sms) {
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({4 * sms / std::max<int64_t>(tiles, 1), blocks, simt::MAX_PARTS}));
}
size_t score_simt_workspace(int32_t d) { return (size_t)4 * MAX_SMS * simt::TR * (d + 1) * 4; }
static void set_parts(simt::Params& p, int64_t tiles, int64_t blocks, int sms, int32_t d, char* ws) {
  p.parts = fwd_parts(tiles, blocks, sms);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = p.part_o + (size_t)4 * MAX_SMS * simt::TR * d;
}

int launch_paged_simt(const PagedArgs& a, int sms, cudaStream_t st, std::string* err) {
  simt::Params p{};
  p.q = static_cast<const float*>(a.q);
  p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.qs[1] = a.qs[1], p.qs[2] = a.qs[0];
  for (int i = 0; i < 3; ++i) p.ks[i] = a.ks[i], p.vs[i] = a.vs[i];
  p.slopes = a.slopes;
  p.o = static_cast<float*>(a.o);
  p.os[1] = a.d, p.os[2] = (int64_t)a.Hq * a.d;
  p.lse = a.lse;
  p.ls[1] = 1, p.ls[2] = a.Hq;
  p.offsets = a.offsets;
  p.lens = a.lens;
  p.table = a.table;
  p.table_s = a.table_s;
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
  const int64_t tiles = (int64_t)a.N * p.g / simt::TR + a.B;
  if (!grid_fits(tiles, a.Hkv, 1, err)) return (int)cudaErrorInvalidConfiguration;
  p.tiles = (int32_t)tiles;
  set_parts(p, tiles * a.Hkv, (int64_t)a.max_pages * a.page / simt::TK, sms, a.d, a.ws + PAGED_WS_HEAD);
  const dim3 grid((unsigned)tiles, (unsigned)a.Hkv);
  return a.d == 128 ? simt::launch_fwd<128, true>(p, grid, st, err) : simt::launch_fwd<64, true>(p, grid, st, err);
}

int launch_range_fwd_simt(const RangeArgs& a, int sms, cudaStream_t st, std::string* err) {
  simt::Params p{};
  p.q = static_cast<const float*>(a.q);
  p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.qs[0] = (int64_t)a.Hq * a.S * a.d, p.qs[1] = a.S * a.d, p.qs[2] = a.d;
  p.ks[0] = p.vs[0] = (int64_t)a.Hkv * a.S * a.d, p.ks[1] = p.vs[1] = a.S * a.d, p.ks[2] = p.vs[2] = a.d;
  p.slopes = a.slopes;
  p.o = static_cast<float*>(a.o);
  for (int i = 0; i < 3; ++i) p.os[i] = p.qs[i];
  p.lse = a.lse;
  p.ls[0] = (int64_t)a.Hq * a.S, p.ls[1] = a.S, p.ls[2] = 1;
  p.lo = a.lo;
  p.hi = a.hi;
  p.mask_bs = a.mask_bs;
  p.status = a.status;
  p.S = a.S;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.g = a.Hq / a.Hkv;
  p.scale = a.scale;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.cap = a.cap;
  const int64_t tiles = (a.S * p.g + simt::TR - 1) / simt::TR;
  set_parts(p, tiles * a.Hkv * a.B, a.S / simt::TK, sms, a.d, a.ws);
  if (!grid_fits(tiles, a.Hkv, (int64_t)a.B * p.parts, err)) return (int)cudaErrorInvalidConfiguration;
  p.tiles = (int32_t)tiles;
  const dim3 grid((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.B);
  return a.d == 128 ? simt::launch_fwd<128, false>(p, grid, st, err) : simt::launch_fwd<64, false>(p, grid, st, err);
}

int launch_range_bwd_simt(const RangeArgs& a, const RangeBwdShape& z, cudaStream_t st, std::string* err) {
  simt::BwdParams p{};
  p.q = static_cast<const float*>(a.q);
  p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.go = static_cast<const float*>(a.go);
  p.lse = a.lse;
  p.dsum = reinterpret_cast<const float*>(a.ws + z.dsum);
  p.lo = a.lo;
  p.hi = a.hi;
  p.mask_bs = a.mask_bs;
  p.slopes = a.slopes;
  p.dq = z.dq_parts > 1 ? reinterpret_cast<float*>(a.ws + z.dq_part) : static_cast<float*>(a.dq);
  p.dk = z.kv_parts > 1 ? reinterpret_cast<float*>(a.ws + z.dk_part) : static_cast<float*>(a.dk);
  p.dv = z.kv_parts > 1 ? reinterpret_cast<float*>(a.ws + z.dv_part) : static_cast<float*>(a.dv);
  p.status = a.status;
  p.S = a.S;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.g = a.Hq / a.Hkv;
  p.dq_parts = z.dq_parts;
  p.kv_parts = z.kv_parts;
  p.scale = a.scale;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.cap = a.cap;
  const int64_t dq_tiles = (a.S * p.g + simt::TR - 1) / simt::TR, kv_tiles = (a.S + simt::TK - 1) / simt::TK;
  if (!grid_fits((int64_t)a.Hkv * a.B * (kv_tiles * z.kv_parts + dq_tiles * z.dq_parts), 1, 1, err)) return (int)cudaErrorInvalidConfiguration;
  p.dq_tiles = (int32_t)dq_tiles;
  p.kv_tiles = (int32_t)kv_tiles;
  return a.d == 128 ? simt::launch_bwd<128>(a, z, p, st, err) : simt::launch_bwd<64>(a, z, p, st, err);
}

}  // namespace mesh
