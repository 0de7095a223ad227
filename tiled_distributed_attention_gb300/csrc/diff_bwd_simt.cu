// Differential attention backward on the CUDA cores, fp32 throughout: the path for fp32 inputs.
//
// The formulas are those of the bf16 path (diff_bwd_tc.cu): with P_m = exp(scale q_m.k_m - LSE_m),
// dP = dO V^T and D_m = dO . O_m,
//   A = P_1 - lam P_2,  dS_1 = P_1 (dP - D_1),  dS_2 = -lam P_2 (dP - D_2),
//   dV = A^T dO,  dk_m = scale dS_m^T q_m,  dq_m = scale dS_m k_m.
// Two passes of one shape in one launch, the first CTAs along x for dK and dV, the others for dQ.  A CTA of
// 128 threads keeps 32 resident rows of one query head (keys for dK and dV, queries for dQ) and
// streams 64-row blocks of the other side through two cp.async buffers.  Per block: the 32 x 64 scores of both maps and dP, 4 x 4 a thread from 16-byte shared
// loads (12 shared-memory wavefronts to 64 FMA instructions, so the FMA pipe is the bound); the
// exponentials; then the products with the streamed rows, 4 rows x 4 columns a thread.
//
// Few rows leave SMs idle, so the streamed axis is split between CTAs (`splits`) until about two CTAs an
// SM are there; the splits, and for dK and dV the query heads of a KV head, leave partial sums that
// sum_parts adds in order.  Rows past the end are zero-filled.
//
// Measured (4 heads on 2, 777 tokens, d = 64, causal): 62 us and 6 us for the sums; 2.6 waves of short CTAs, FMA
// pipe 39 % busy.  Two launches, one CTA an SM: 85 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace dsimt {

constexpr int RB = 32;  // resident rows
constexpr int CB = 64;  // streamed rows
constexpr int THREADS = 128;
constexpr int TP = RB + 2;  // row pitch of the transposed tiles: their writes fall into all banks, and two CTAs
                            // fit an SM at d = 64
constexpr float LOG2E = 1.4426950408889634f;

struct Params {
  const float* q;
  const float* k;
  const float* v;
  const float* g;     // dO
  const float* lse;   // [B, Hq, 2, S]
  const float* dsum;  // [B, Hq, 2, S]
  const float* lam;
  float* out0;  // dQ, or dK: [B, H, n_part, S, D]
  float* out1;  // dV
  const int32_t* status;
  int64_t S;
  int32_t B, Hq, Hkv, lam_n, causal, splits, n_part;
  float scale, scale_log2;
};

template <int D>
struct Smem {
  static constexpr int P = D + 4;  // row pitch: 16-byte loads of eight rows fall into all banks
  static constexpr int RES = 2 * RB * P, STREAM = 2 * CB * P, VEC = 4 * CB;
  static constexpr int TILES = 3 * CB * TP;
  static constexpr int FLOATS = RES + 2 * (STREAM + VEC) + TILES;
};

__device__ __forceinline__ void cp16(float* dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// x[i][j] += sum over k in [k0, k1) of R[r_i][k] * C[c_j][k], r_i = ty + 8 i, c_j = tx + 16 j
template <int P>
__device__ __forceinline__ void scores(float (&x)[4][4], const float* R, const float* C, int k0, int k1, int ty, int tx) {
#pragma unroll 2
  for (int k = k0; k < k1; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(R + (ty + 8 * i) * P + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(C + (tx + 16 * j) * P + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, x[i][j]))));
  }
}

// acc[i][e] += sum over c of T[c][4 ty + i] * C[c][col + e]
template <int P>
__device__ __forceinline__ void product(float (&acc)[4][4], const float* T, const float* C, int ty, int col) {
#pragma unroll 4
  for (int c = 0; c < CB; ++c) {
    const float2 t0 = *reinterpret_cast<const float2*>(T + c * TP + 4 * ty);
    const float2 t1 = *reinterpret_cast<const float2*>(T + c * TP + 4 * ty + 2);
    const float4 x = *reinterpret_cast<const float4*>(C + c * P + col);
    const float tt[4] = {t0.x, t0.y, t1.x, t1.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][0] = fmaf(tt[i], x.x, acc[i][0]);
      acc[i][1] = fmaf(tt[i], x.y, acc[i][1]);
      acc[i][2] = fmaf(tt[i], x.z, acc[i][2]);
      acc[i][3] = fmaf(tt[i], x.w, acc[i][3]);
    }
  }
}

template <int D, bool KV>
__device__ __forceinline__ void run_pass(const Params& p, int bx, int n_blocks) {
  using Sm = Smem<D>;
  constexpr int P = Sm::P, NJ = D / 64;
  extern __shared__ float4 smem4[];
  float* res0 = reinterpret_cast<float*>(smem4);  // K, or Q rows
  float* res1 = res0 + RB * P;                    // V, or dO rows
  float* stream = res0 + Sm::RES;                 // two buffers of (Q, dO) or (K, V) rows and the query rows' values
  float* tiles = stream + 2 * (Sm::STREAM + Sm::VEC);
  float* tA = tiles;
  float* tS1 = tiles + CB * TP;
  float* tS2 = tiles + 2 * CB * TP;
  if (*reinterpret_cast<const volatile int32_t*>(p.status) != 0) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int h = blockIdx.y, b = blockIdx.z / p.splits, split = blockIdx.z % p.splits;
  const int group = p.Hq / p.Hkv, hk = h / group;
  const int64_t S = p.S;
  const int rb = !KV && p.causal ? n_blocks - 1 - bx : bx;  // the longest first
  const int64_t r0 = (int64_t)rb * RB;
  const int64_t qrow = ((int64_t)b * p.Hq + h) * S, krow = ((int64_t)b * p.Hkv + hk) * S;
  const int64_t vrow = ((int64_t)b * p.Hq + h) * 2 * S;  // of lse and dsum
  const float* R0 = (KV ? p.k + krow * D : p.q + qrow * D);
  const float* R1 = (KV ? p.v + krow * D : p.g + qrow * D);
  const float* C0 = (KV ? p.q + qrow * D : p.k + krow * D);
  const float* C1 = (KV ? p.g + qrow * D : p.v + krow * D);

  // streamed blocks of this CTA: those a row of the tile sees, shared out between the splits
  const int64_t n_all = (S + CB - 1) / CB;
  const int64_t first = KV && p.causal ? r0 / CB : 0;
  const int64_t last = !KV && p.causal ? min(n_all, (r0 + RB + CB - 1) / CB) : n_all;
  const int64_t per = (last - first + p.splits - 1) / p.splits;
  const int64_t c_begin = min(last, first + split * per), c_end = min(last, c_begin + per);

  auto load_rows = [&](float* dst, const float* src, int64_t row0, int rows) {
    for (int i = tid; i < rows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      const bool in = row0 + r < S;
      cp16(dst + r * P + c, src + (in ? row0 + r : 0) * D + c, in);
    }
  };
  // value `w` (LSE_1, LSE_2, D_1, D_2) of query row s as the kernel uses it: a row past the end, or one
  // without a visible key, gets exp2(x - inf) = 0
  auto value = [&](int w, int64_t s) -> float {
    if (s >= S) return w < 2 ? -INFINITY : 0.f;
    const float x = __ldg((w < 2 ? p.lse : p.dsum) + vrow + (w & 1) * S + s);
    return w >= 2 ? -x : x == -INFINITY ? -INFINITY : -x * LOG2E;
  };
  auto load_block = [&](int64_t cb, int buf) {
    float* d = stream + buf * (Sm::STREAM + Sm::VEC);
    load_rows(d, C0, cb * CB, CB);
    load_rows(d + CB * P, C1, cb * CB, CB);
    if (KV)
      for (int i = tid; i < 4 * CB; i += THREADS) d[Sm::STREAM + i] = value(i / CB, cb * CB + i % CB);
  };
  load_rows(res0, R0, r0, RB);
  load_rows(res1, R1, r0, RB);
  if (c_begin < c_end) load_block(c_begin, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");

  const float nlam = -p.lam[p.lam_n == 1 ? 0 : h];
  float rv[4][4];  // dq: the rows' own values
  if (!KV)
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) rv[w][i] = value(w, r0 + ty + 8 * i);
  float acc0[NJ][4][4], acc1[NJ][4][4];  // dK or dQ; dV
#pragma unroll
  for (int n = 0; n < NJ; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc0[n][i][e] = acc1[n][i][e] = 0.f;

  for (int64_t cb = c_begin; cb < c_end; ++cb) {
    const int buf = (int)((cb - c_begin) & 1);
    if (cb + 1 < c_end) load_block(cb + 1, buf ^ 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float* c0 = stream + buf * (Sm::STREAM + Sm::VEC);
    const float* c1 = c0 + CB * P;
    const float* vec = c0 + Sm::STREAM;
    float s1[4][4], s2[4][4], dp[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s1[i][j] = s2[i][j] = dp[i][j] = 0.f;
    scores<P>(s1, res0, c0, 0, D / 2, ty, tx);
    scores<P>(s2, res0, c0, D / 2, D, ty, tx);
    scores<P>(dp, res1, c1, 0, D, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ty + 8 * i, c = tx + 16 * j;
        const int64_t kq = KV ? cb * CB + c : r0 + r, kk = KV ? r0 + r : cb * CB + c;  // query, key
        const float l1 = KV ? vec[c] : rv[0][i], l2 = KV ? vec[CB + c] : rv[1][i];
        const float d1 = KV ? vec[2 * CB + c] : rv[2][i], d2 = KV ? vec[3 * CB + c] : rv[3][i];
        const bool off = kk >= S || (p.causal && kk > kq);
        const float p1 = off ? 0.f : exp2f(fmaf(s1[i][j], p.scale_log2, l1));
        const float w2 = off ? 0.f : nlam * exp2f(fmaf(s2[i][j], p.scale_log2, l2));
        if (KV) tA[c * TP + r] = p1 + w2;
        tS1[c * TP + r] = off ? 0.f : p1 * (dp[i][j] + d1);
        tS2[c * TP + r] = off ? 0.f : w2 * (dp[i][j] + d2);
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NJ; ++n) {
      const int col = 4 * tx + 64 * n;
      product<P>(acc0[n], col < D / 2 ? tS1 : tS2, c0, ty, col);
      if (KV) product<P>(acc1[n], tA, c1, ty, col);
    }
    __syncthreads();  // the tiles and this buffer are free again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the piece's sums, [b, head, part, S, D]
  const int64_t head = KV ? (int64_t)b * p.Hkv + hk : (int64_t)b * p.Hq + h;
  const int part = KV ? (h % group) * p.splits + split : split;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t s = r0 + 4 * ty + i;
    if (s >= S) continue;
    const int64_t at = ((head * p.n_part + part) * S + s) * D;
#pragma unroll
    for (int n = 0; n < NJ; ++n) {
      const int col = 4 * tx + 64 * n;
      *reinterpret_cast<float4*>(p.out0 + at + col) = make_float4(acc0[n][i][0] * p.scale, acc0[n][i][1] * p.scale,
                                                                 acc0[n][i][2] * p.scale, acc0[n][i][3] * p.scale);
      if (KV) *reinterpret_cast<float4*>(p.out1 + at + col) = make_float4(acc1[n][i][0], acc1[n][i][1], acc1[n][i][2], acc1[n][i][3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS) bwd_kernel(const Params kv, const Params dq) {
  wait_for_kernel_before();
  const int n = (int)gridDim.x / 2;  // blocks of a pass
  if ((int)blockIdx.x < n) run_pass<D, true>(kv, (int)blockIdx.x, n);
  else run_pass<D, false>(dq, (int)blockIdx.x - n, n);
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

template <int D>
static cudaError_t launch(const Params& kv, const Params& dq, cudaStream_t st) {
  static OncePerDevice once;
  const int dev = OncePerDevice::device();
  const size_t smem = sizeof(float) * Smem<D>::FLOATS;
  auto kern = bwd_kernel<D>;
  if (once.pending(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    once.mark(dev);
  }
  const dim3 grid((unsigned)(2 * ((kv.S + RB - 1) / RB)), (unsigned)kv.Hq, (unsigned)(kv.B * kv.splits));
  return launch_behind(kern, grid, THREADS, smem, st, kv, dq);
}

}  // namespace dsimt

// Parts of the streamed axis: until about two CTAs an SM are there, eight at most, none shorter than two blocks.
int diff_simt_splits(int64_t S, int32_t B, int32_t Hq, int sms) {
  const int64_t ctas = std::max<int64_t>(1, (S + dsimt::RB - 1) / dsimt::RB * B * Hq);
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(8, (S + 2 * dsimt::CB - 1) / (2 * dsimt::CB)));
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, (2LL * sms + ctas - 1) / ctas));
}

int launch_diff_bwd_simt(const DiffArgs& a, const DiffWorkspace& w, int sms, void* stream, std::string* err) {
  using namespace dsimt;
  cudaStream_t st = (cudaStream_t)stream;
  const int splits = diff_simt_splits(a.S, a.B, a.Hq, sms), group = a.Hq / a.Hkv;
  if (a.Hq > 65535 || (int64_t)a.B * splits > 65535) {
    *err = "too many heads or sequences for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  Params p{};
  p.q = static_cast<const float*>(a.Q);
  p.k = static_cast<const float*>(a.K);
  p.v = static_cast<const float*>(a.V);
  p.g = static_cast<const float*>(a.dO);
  p.lse = a.LSE;
  p.dsum = reinterpret_cast<const float*>(a.ws + w.dsum);
  p.lam = static_cast<const float*>(a.lam);
  p.status = a.status;
  p.S = a.S;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.lam_n = a.lam_n;
  p.causal = a.causal;
  p.splits = splits;
  p.scale = a.scale;
  p.scale_log2 = a.scale_log2;
  const bool q_parts = splits > 1, kv_parts = splits * group > 1;
  Params q = p;
  p.n_part = splits * group;
  p.out0 = kv_parts ? reinterpret_cast<float*>(a.ws + w.dk_part) : static_cast<float*>(a.dK);
  p.out1 = kv_parts ? reinterpret_cast<float*>(a.ws + w.dv_part) : static_cast<float*>(a.dV);
  q.n_part = splits;
  q.out0 = q_parts ? reinterpret_cast<float*>(a.ws + w.dq_part) : static_cast<float*>(a.dQ);
  cudaError_t e = a.d == 128 ? launch<128>(p, q, st) : launch<64>(p, q, st);
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
  if (e != cudaSuccess) *err = std::string("diff_bwd_simt launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace mesh
