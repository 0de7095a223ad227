// Differential attention, the passes around its products: fp32 inputs split into bf16 pieces, the merge of
// the two maps' partial outputs, the row terms of the backward pass and the gradient of lam.  All are
// bound by memory and read and write whole 16-byte pieces.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace daux {

constexpr int THREADS = 256;
constexpr int MAX_PARTS = 16;  // of a tile's keys (diff_fwd32_parts)

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ float lam_of(const void* lam, int n, int h) {
  return to_f(static_cast<const T*>(lam)[n == 1 ? 0 : h]);
}

// fp32 inputs as three bf16 pieces each, x = x1 + x2 + x3 exactly (round to nearest, then the rest), in one
// launch for Q, K and V: blockIdx.y 0 is K, 1 is V, 2 is Q.  Q goes to two heads, (b, 2 h + m) holding map
// m's half of the columns and zeros in the other, so that attention of 2 Hq heads over the full d
// columns gives both maps.
__global__ void __launch_bounds__(THREADS) split_kernel(const DiffArgs a, uint2* qp, uint2* kp, uint2* vp) {
  wait_for_kernel_before();
  const TablesHeader* th = static_cast<const TablesHeader*>(a.tables);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && (th->magic != TABLES_MAGIC || th->tag != a.tag))
    record_error(a.status, MESH_ATTN_ERR_INVALID_ARG, 7, 0);  // another plan's tables: the tile kernel does nothing
  const int which = blockIdx.y, q4 = a.d / 4;
  const float* src = static_cast<const float*>(which == 0 ? a.K : which == 1 ? a.V : a.Q);
  uint2* dst = which == 0 ? kp : which == 1 ? vp : qp;
  const int64_t n = (int64_t)a.B * (which == 2 ? a.Hq : a.Hkv) * a.S * q4;
  const int64_t piece = which == 2 ? 2 * n : n;  // in groups of four
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * THREADS) {
    const float4 x = load4(src + 4 * i);
    const float e[4] = {x.x, x.y, x.z, x.w};
    uint2 w[3];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat162 p1 = __floats2bfloat162_rn(e[2 * h], e[2 * h + 1]);
      const float r0 = e[2 * h] - __low2float(p1), r1 = e[2 * h + 1] - __high2float(p1);
      const __nv_bfloat162 p2 = __floats2bfloat162_rn(r0, r1);
      const __nv_bfloat162 p3 = __floats2bfloat162_rn(r0 - __low2float(p2), r1 - __high2float(p2));
      (h ? w[0].y : w[0].x) = *reinterpret_cast<const uint32_t*>(&p1);
      (h ? w[1].y : w[1].x) = *reinterpret_cast<const uint32_t*>(&p2);
      (h ? w[2].y : w[2].x) = *reinterpret_cast<const uint32_t*>(&p3);
    }
    int64_t at = i, other = -1;
    if (which == 2) {
      const int64_t row = i / q4, bh = row / a.S, per_head = a.S * q4;
      const int64_t first = i + bh * per_head;  // head 2 h; head 2 h + 1 lies per_head behind
      const bool m1 = i - row * q4 < q4 / 2;
      at = m1 ? first : first + per_head;
      other = m1 ? first + per_head : first;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      dst[k * piece + at] = w[k];
      if (other >= 0) dst[k * piece + other] = make_uint2(0u, 0u);
    }
  }
}

// O = sum_t w1_t O1_t - lam sum_t w2_t O2_t over a row's parts, w = exp(lse_t - lse) of each map, O2 (which the
// backward pass needs) and the LSEs.  A thread takes a 16-byte piece of one map's row, all parts' loads in
// flight together (MAXP of them, 1 where nothing is cut); the maps meet in shared memory.
template <int D, int MAXP>
__global__ void __launch_bounds__(THREADS) merge_kernel(const DiffArgs a, const float* part_o, const float* part_lse, int parts,
                                                        int n_rblk) {
  constexpr int Q4 = D / 4, ROWS = THREADS / (2 * Q4);
  __shared__ float4 o2_s[ROWS * Q4];
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(a.status) != 0) return;
  const int m = (int)threadIdx.x / (ROWS * Q4), at = (int)threadIdx.x % (ROWS * Q4), c = at % Q4 * 4;
  const int64_t bh = blockIdx.x / (unsigned)n_rblk, row = (int64_t)(blockIdx.x % (unsigned)n_rblk) * ROWS + at / Q4;
  const bool in = row < a.S;
  // the parts that the row's tile of 128 has: no more than its 64-key blocks
  const int nb = (int)((a.S + 63) / 64), k = min(parts, a.causal ? min(nb, 2 * (int)(row / 128) + 2) : nb);
  const int64_t base = (2 * bh + m) * parts * a.S + row;  // row of part t: base + t S
  float w[MAXP];
  float4 v[MAXP];
#pragma unroll
  for (int t = 0; t < MAXP; ++t) {
    const bool there = in && t < k;
    w[t] = there ? part_lse[base + t * a.S] : -INFINITY;
    v[t] = there ? __ldcs(reinterpret_cast<const float4*>(part_o + (base + t * a.S) * D + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY, W = 0.f;
#pragma unroll
  for (int t = 0; t < MAXP; ++t) M = fmaxf(M, w[t]);
  const float Ms = M == -INFINITY ? 0.f : M, lse = w[0];
#pragma unroll
  for (int t = 0; t < MAXP; ++t) {
    w[t] = MAXP == 1 ? (w[t] == -INFINITY ? 0.f : 1.f) : expf(w[t] - Ms);
    W += w[t];
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int t = 0; t < MAXP; ++t) {
    const float f = t < k ? w[t] * inv : 0.f;
    o.x = fmaf(f, v[t].x, o.x);
    o.y = fmaf(f, v[t].y, o.y);
    o.z = fmaf(f, v[t].z, o.z);
    o.w = fmaf(f, v[t].w, o.w);
  }
  const int64_t dst = (bh * a.S + row) * D + c;
  if (m == 1) {
    o2_s[at] = o;
    if (in && a.O2) store4(static_cast<float*>(a.O2) + dst, o);
  }
  if (in && c == 0) a.LSE[(2 * bh + m) * a.S + row] = MAXP == 1 ? lse : W == 0.f ? -INFINITY : Ms + logf(W);
  __syncthreads();
  if (m == 0 && in) {
    const float lam = lam_of<float>(a.lam, a.lam_n, (int)(bh % a.Hq));
    const float4 y = o2_s[at];
    store4(static_cast<float*>(a.O) + dst, make_float4(fmaf(-lam, y.x, o.x), fmaf(-lam, y.y, o.y), fmaf(-lam, y.z, o.z), fmaf(-lam, y.w, o.w)));
  }
}

// Row terms of dS: D1 = dO . O1 with O1 = O + lam O2, and D2 = dO . O2, from the outputs as they were rounded: an O1
// of its own would be one more output to write and keep, for an error (3e-4 to 8e-4 of the gradients' norm in bf16) of half
// that of the rounded dS (1.7e-3) or less.  A CTA takes PREP_ROWS rows of a head, a group of lanes a row, 16 bytes of
// each of the three tensors a lane, all passes' loads in flight together.
constexpr int PREP_ROWS = 64;
template <typename T>
__device__ __forceinline__ void dot16(uint4 x, uint4 y, float& acc) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      acc = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), acc);
      acc = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), acc);
    } else {
      acc = fmaf(__uint_as_float(a[i]), __uint_as_float(b[i]), acc);
    }
  }
}
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) prep_kernel(const DiffArgs a, float* dsum, float* dlam_part, int64_t n_part) {
  constexpr int LANES = D * (int)sizeof(T) / 16, AT_ONCE = THREADS / LANES, PASSES = PREP_ROWS / AT_ONCE;
  wait_for_kernel_before();
  const TablesHeader* th = static_cast<const TablesHeader*>(a.tables);
  if (blockIdx.x == 0 && threadIdx.x == 0 && (th->magic != TABLES_MAGIC || th->tag != a.tag))
    record_error(a.status, MESH_ATTN_ERR_INVALID_ARG, 7, 0);  // another plan's tables: the launches behind do nothing
  if (*reinterpret_cast<volatile int32_t*>(a.status) != 0) return;
  const int64_t part = blockIdx.x % n_part, bh = blockIdx.x / n_part;
  const float lam = lam_of<T>(a.lam, a.lam_n, (int)(bh % a.Hq));
  const int lr = threadIdx.x / LANES, piece = threadIdx.x % LANES;
  const int64_t s0 = part * PREP_ROWS + lr;
  uint4 g[PASSES], o[PASSES], o2[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t s = s0 + i * AT_ONCE;
    g[i] = o[i] = o2[i] = make_uint4(0u, 0u, 0u, 0u);
    if (s < a.S) {
      const int64_t at = (bh * a.S + s) * LANES + piece;
      g[i] = static_cast<const uint4*>(a.dO)[at];
      o[i] = static_cast<const uint4*>(a.O)[at];
      o2[i] = static_cast<const uint4*>(a.O2)[at];
    }
  }
  double acc = 0.0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t s = s0 + i * AT_ONCE;
    float d1 = 0.f, d2 = 0.f;
    dot16<T>(g[i], o[i], d1);
    dot16<T>(g[i], o2[i], d2);
#pragma unroll
    for (int x = LANES / 2; x >= 1; x >>= 1) {
      d1 += __shfl_xor_sync(0xffffffffu, d1, x);
      d2 += __shfl_xor_sync(0xffffffffu, d2, x);
    }
    if (piece == 0 && s < a.S) {
      dsum[2 * bh * a.S + s] = fmaf(lam, d2, d1);
      dsum[(2 * bh + 1) * a.S + s] = d2;
      acc -= (double)d2;
    }
  }
  if (dlam_part) {  // dlam = -sum D2, in a fixed order
    __shared__ double sums[AT_ONCE];
    if (piece == 0) sums[lr] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
      double t = 0.0;
      for (int r = 0; r < AT_ONCE; ++r) t += sums[r];
      dlam_part[bh * n_part + part] = (float)t;
    }
  }
}

// dlam of one value (a head, or all heads where lam is shared): the sum of its partial sums, taken
// in a fixed order in fp64, since terms of both signs nearly cancel over a long batch.
template <typename T>
__global__ void __launch_bounds__(THREADS) dlam_kernel(const DiffArgs a, const float* part, int64_t n_part) {
  wait_for_kernel_before();
  if (*reinterpret_cast<volatile int32_t*>(a.status) != 0) return;
  const int h0 = a.lam_n == 1 ? 0 : (int)blockIdx.x, nh = a.lam_n == 1 ? a.Hq : 1;
  double acc = 0.0;
  const int64_t n = (int64_t)a.B * nh * n_part;
  for (int64_t i = threadIdx.x; i < n; i += THREADS) {
    const int64_t k = i % n_part, bh = i / n_part, b = bh / nh, h = h0 + bh % nh;
    acc += (double)part[(b * a.Hq + h) * n_part + k];
  }
  __shared__ double s[THREADS];
  s[threadIdx.x] = acc;
  __syncthreads();
  for (int x = THREADS / 2; x >= 1; x >>= 1) {
    if (threadIdx.x < x) s[threadIdx.x] += s[threadIdx.x + x];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    if constexpr (sizeof(T) == 2) static_cast<T*>(a.dlam)[blockIdx.x] = __float2bfloat16_rn((float)s[0]);
    else static_cast<T*>(a.dlam)[blockIdx.x] = (float)s[0];
  }
}

static int done(cudaError_t e, const char* what, std::string* err) {
  if (e != cudaSuccess) *err = std::string(what) + ": " + cudaGetErrorString(e);
  return (int)e;
}
static unsigned grid_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + THREADS - 1) / THREADS, 152 * 16)); }

}  // namespace daux

int launch_diff_split(const DiffArgs& a, const DiffWorkspace& w, void* stream, std::string* err) {
  const F32Pieces pc = f32_pieces_layout(a.B, 2 * a.Hq, a.Hkv, a.S, a.d);
  char* base = a.ws + w.pieces;
  const unsigned grid = daux::grid_for((int64_t)a.B * a.Hq * a.S * (a.d / 4));
  return daux::done(launch_behind(daux::split_kernel, dim3(grid, 3), daux::THREADS, 0, (cudaStream_t)stream, a,
                                  reinterpret_cast<uint2*>(base + pc.q_off), reinterpret_cast<uint2*>(base + pc.k_off),
                                  reinterpret_cast<uint2*>(base + pc.v_off)),
                    "diff split launch", err);
}

// Parts of every tile's keys in the fp32 forward: what fills the SMs, two 64-key blocks (2 us each) at least, where
// that saves more than the merge of more than one costs (2 to 3 us).  One head of 2,304 tokens, d = 128, causal (36
// tiles of up to 36 blocks): 84 us whole, 41 in four parts.
int32_t diff_fwd32_parts(int64_t S, int32_t B, int32_t Hq) {
  constexpr int SMS = 152;  // the whole GPU's: so the workspace's size needs no device
  const int64_t tiles = (S + 127) / 128 * B * 2 * Hq, nb = (S + 63) / 64;
  if (tiles == 0 || 2 * tiles > SMS) return 1;
  const int64_t parts = std::min<int64_t>({SMS / tiles, nb / 2, daux::MAX_PARTS});
  return (int32_t)(parts < 2 || nb - nb / parts < 2 ? 1 : parts);
}

template <int D, int MAXP>
static int merge_d(const DiffArgs& a, const DiffWorkspace& w, int32_t parts, cudaStream_t st, std::string* err) {
  constexpr int ROWS = daux::THREADS / (D / 2);
  const int64_t n_rblk = (a.S + ROWS - 1) / ROWS, blocks = n_rblk * a.B * a.Hq;
  if (blocks > 0x7fffffffLL) {
    *err = "too many rows for one merge launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  const cudaError_t e = launch_behind(daux::merge_kernel<D, MAXP>, dim3((unsigned)blocks), daux::THREADS, 0, st, a,
                                      reinterpret_cast<const float*>(a.ws + w.part_o),
                                      reinterpret_cast<const float*>(a.ws + w.part_lse), (int)parts, (int)n_rblk);
  return daux::done(e, "diff merge launch", err);
}

int launch_diff_merge(const DiffArgs& a, const DiffWorkspace& w, int32_t parts, void* stream, std::string* err) {
  cudaStream_t st = (cudaStream_t)stream;
  if (parts == 1) return a.d == 128 ? merge_d<128, 1>(a, w, parts, st, err) : merge_d<64, 1>(a, w, parts, st, err);
  return a.d == 128 ? merge_d<128, daux::MAX_PARTS>(a, w, parts, st, err) : merge_d<64, daux::MAX_PARTS>(a, w, parts, st, err);
}

int launch_diff_prep(const DiffArgs& a, const DiffWorkspace& w, mesh_attn_dtype dt, void* stream, std::string* err) {
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t n_part = (a.S + daux::PREP_ROWS - 1) / daux::PREP_ROWS, blocks = n_part * a.B * a.Hq;
  if (blocks > 0x7fffffff) {
    *err = "too many rows for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  float* dsum = reinterpret_cast<float*>(a.ws + w.dsum);
  float* dl = dt == MESH_ATTN_F32 ? reinterpret_cast<float*>(a.ws + w.dlam_part) : nullptr;
  auto go = [&](auto kern) { return launch_behind(kern, dim3((unsigned)blocks), daux::THREADS, 0, st, a, dsum, dl, n_part); };
  const cudaError_t e =
      dt == MESH_ATTN_BF16 ? go(a.d == 128 ? daux::prep_kernel<__nv_bfloat16, 128> : daux::prep_kernel<__nv_bfloat16, 64>)
                           : go(a.d == 128 ? daux::prep_kernel<float, 128> : daux::prep_kernel<float, 64>);
  return daux::done(e, "diff prep launch", err);
}

int launch_diff_dlam(const DiffArgs& a, const DiffWorkspace& w, mesh_attn_dtype dt, int64_t n_part, void* stream,
                     std::string* err) {
  cudaStream_t st = (cudaStream_t)stream;
  const float* part = reinterpret_cast<const float*>(a.ws + w.dlam_part);
  const dim3 grid((unsigned)a.lam_n);
  const cudaError_t e = dt == MESH_ATTN_BF16
                            ? launch_behind(daux::dlam_kernel<__nv_bfloat16>, grid, daux::THREADS, 0, st, a, part, n_part)
                            : launch_behind(daux::dlam_kernel<float>, grid, daux::THREADS, 0, st, a, part, n_part);
  return daux::done(e, "diff dlam launch", err);
}

}  // namespace mesh
