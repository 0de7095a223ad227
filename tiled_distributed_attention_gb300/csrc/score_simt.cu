// Attention with scores that are capped, biased and masked by ranges, fp32 inputs, on the CUDA cores: of a dense batch
// (range-masked attention, both directions) and of the new tokens of sequences in a paged cache.  The formulas are those of
// score_fwd.cuh and score_bwd.cu; everything is fp32, sums in the order of the keys.
//
// A tile is 64 rows, the query heads of a KV head and their tokens (row = token * g + head), which stream blocks of
// 64 keys through shared memory; 256 threads hold 4 x 4 scores and 4 x D / 16 outputs each, read operands by
// 16-byte accesses (12 shared-memory wavefronts for 64 FMAs of the scores, 20 for 128 of the outputs: the FMA pipe is the
// bound), and keep the row statistics in registers, 16 lanes a row.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace mesh {
namespace simt {

constexpr int THREADS = 256;
constexpr int TR = 64;  // rows of a tile
constexpr int TK = 64;  // keys of a block
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;
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
  int32_t N, B, Hq, Hkv, g, n_pages, page, max_pages, max_new, window, tiles;
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
__global__ void __launch_bounds__(THREADS) fwd_kernel(const __grid_constant__ Params p) {
  using Sm = Smem<D>;
  constexpr int CW = D / 16;  // columns of a thread's outputs
  extern __shared__ __align__(16) float sm[];
  __shared__ int bounds[2];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31;
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(p.status) != 0) return;
  Tile t;
  t.hk = (int)blockIdx.y;
  const int slot = p.tiles - 1 - (int)blockIdx.x;  // the last tokens, the longest where the mask is causal, first
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
    const int32_t o0 = p.offsets[a], o1 = p.offsets[a + 1], len = p.lens[a];
    t.row0 = min(max(o0, 0), p.N);
    n_tok = min(min(max(o1, t.row0), p.N) - t.row0, p.max_new);
    t.len = (int32_t)min((int64_t)max(len, n_tok), (int64_t)p.max_pages * p.page);
    if (tid == 0 && (t.row0 != o0 || n_tok != o1 - o0 || t.len != len))
      record_error(p.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_SEQ, a);
    n_tok = min(n_tok, t.len);
    t.pos0 = t.len - n_tok;
    const int64_t r = ((int64_t)slot - ((int64_t)t.row0 * p.g / TR + a)) * TR;
    if (r < 0 || r >= (int64_t)n_tok * p.g) return;
    t.r0 = (int)r;
    t.nr = min(TR, n_tok * p.g - t.r0);
    t.kmin = p.window ? max(0, t.pos0 + t.r0 / p.g + 1 - p.window) : 0;
    t.kmax = t.pos0 + (t.r0 + t.nr - 1) / p.g + 1;
  } else {
    t.b = (int)blockIdx.z;
    n_tok = (int)p.S;
    t.row0 = t.pos0 = 0;
    t.len = (int)p.S;
    t.r0 = slot * TR;
    t.nr = (int)min((int64_t)TR, p.S * p.g - t.r0);
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
  for (int j0 = t.kmin / TK * TK; j0 < t.kmax; j0 += TK) {
    // K and V: keys behind the last are zeros
    for (int i = tid; i < TK * (D / 4); i += THREADS) {
      const int r = i / (D / 4), c = i % (D / 4) * 4, key = j0 + r;
      bool in = key < t.len;
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
#pragma unroll 4
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
#pragma unroll 2
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
  (void)lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (ty * 4 + i >= t.nr) continue;
    const int row = t.r0 + ty * 4 + i, tok = row / p.g, h = t.hk * p.g + row - tok * p.g;
    const int64_t bo = PAGED ? 0 : t.b, to = t.row0 + tok;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // no visible key: O = 0 (a NaN sum stays NaN)
    float* dst = p.o + bo * p.os[0] + h * p.os[1] + to * p.os[2];
#pragma unroll
    for (int c = 0; c < CW; c += 4)
      *reinterpret_cast<float4*>(dst + c * 16 + tx * 4) =
          make_float4(o[i][c] * inv, o[i][c + 1] * inv, o[i][c + 2] * inv, o[i][c + 3] * inv);
    if (tx == 0) p.lse[bo * p.ls[0] + h * p.ls[1] + to * p.ls[2]] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * LN2;
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
  if (e == cudaSuccess) e = launch_behind(kern, grid, THREADS, smem, st, p);
  if (e != cudaSuccess) *err = std::string("score fp32 forward launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace simt

static bool grid_fits(int64_t x, int64_t y, int64_t z, std::string* err) {
  if (x <= 0x7fffffff && y <= 65535 && z <= 65535) return true;
  *err = "too many tiles, KV heads or sequences for one launch";
  return false;
}

int launch_paged_simt(const PagedArgs& a, cudaStream_t st, std::string* err) {
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
  const dim3 grid((unsigned)tiles, (unsigned)a.Hkv);
  return a.d == 128 ? simt::launch_fwd<128, true>(p, grid, st, err) : simt::launch_fwd<64, true>(p, grid, st, err);
}

int launch_range_fwd_simt(const RangeArgs& a, cudaStream_t st, std::string* err) {
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
  if (!grid_fits(tiles, a.Hkv, a.B, err)) return (int)cudaErrorInvalidConfiguration;
  p.tiles = (int32_t)tiles;
  const dim3 grid((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.B);
  return a.d == 128 ? simt::launch_fwd<128, false>(p, grid, st, err) : simt::launch_fwd<64, false>(p, grid, st, err);
}

}  // namespace mesh
