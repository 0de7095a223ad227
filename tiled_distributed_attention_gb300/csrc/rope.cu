// Rotary positions with several axes (time, height, width) on q and k, one launch for both.
//
// A head's d columns are `groups` equal column groups rotated alike (one for plain heads, two for
// the halves of a differential head).  Pair i of a group turns by phi = pos[axis(i)] * freq(i):
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi);   backward: by -phi.
// Pairs are (i, i + n) ("half") or (2 i, 2 i + 1) ("adjacent"); columns from 2 n on are copied.
//
// Angles.  A position in a long context times a frequency in fp32 leaves no digits after the
// point (2^20 * 1.0 has an ulp of 1/8 rad), and the fp64 rate of this chip is low.  The frequency is
// held instead as a 64-bit fixed-point fraction of a turn, freq / 2 pi * 2^64: the product with an
// integer position wraps modulo one turn by itself, exactly, for any sign, with an error of |pos| *
// 2^-53 turns from the frequency's own rounding.  Its top 32 bits, as a signed number, are the angle
// in [-1/2, 1/2) turns, exact to 2^-25 of a half turn in fp32, and go to sincospi.
//
// Bound by memory: every element is read and written once.  A thread owns V pairs (16 bytes of each
// member) of one token, computes their V sines and cosines once and walks over the heads with them,
// four heads' loads in flight at a time, so the angles cost nothing per element.  With few tokens the heads
// are spread over blockIdx.y until the grid fills the GPU, each block computing the angles
// again: a decoding step is bound by latency, and one head's work a thread is the shortest path.
//
// Measured: 20 heads of 65,536 tokens, d = 128, bf16, three axes: 102 us, 6.6 TB/s (a plain copy 6.8);
// backward of 24 heads of 3 x 4,107 tokens, d = 64, fp32: 25 us; one token of 64 sequences: 3.1 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "ptx.cuh"

namespace mesh {
namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 256;
constexpr int MAX_AXES = 8;

struct Params {
  const void* x[2];
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // batch, head, token strides in elements
  int32_t H[2];
  const void* pos;
  int64_t ps[3];  // axis, batch, token strides
  int64_t tokens;  // B * S
  int64_t S;
  int32_t pos64, groups, dh, n, inverse, items, heads_per_block;
  uint64_t step[MAX_PAIRS];
  uint8_t axis[MAX_PAIRS];
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// V elements as fp32 and back (one rounding to the type); bf16 pairs go by 32-bit words.
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& x, float (&f)[V]) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f(x.v[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void narrow(const float (&f)[V], Vec<T, V>& x) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(x.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) from_f(x.v[i], f[i]);
  }
}

// V: elements of one access: 16 bytes' worth, or the half, quarter or eighth that sizes and addresses allow.
// ADJ: adjacent pairs.  A rotation item is V pairs by two accesses, one for each member, or for
// adjacent pairs one access of V / 2 pairs (two of one element at V = 1), so that neighbouring threads
// always touch neighbouring bytes; a copy item is V elements behind the rotated ones.
template <int V, bool ADJ>
struct Item {
  static constexpr int PAIRS = ADJ ? (V > 1 ? V / 2 : 1) : V;
  static constexpr bool TWO = !ADJ || V == 1;  // accesses
};

template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ Params prm) {
  const int64_t lin = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  const int item = (int)(lin % prm.items);
  const int64_t tok = lin / prm.items;
  if (tok >= prm.tokens) return;
  wait_for_kernel_before();
  const int64_t b = tok / prm.S, s = tok - b * prm.S;
  constexpr int NP = Item<V, ADJ>::PAIRS;
  constexpr bool TWO = Item<V, ADJ>::TWO;
  const int rot = prm.n / NP;                      // rotation items of a group
  const int per = rot + (prm.dh - 2 * prm.n) / V;  // items of a group
  const int grp = item / per, r = item - grp * per;
  const bool copy = r >= rot;
  // the item's two accesses
  int c0 = grp * prm.dh, c1;
  if (copy) {
    c0 += 2 * prm.n + (r - rot) * V;
    c1 = c0;
  } else if (ADJ) {
    c0 += 2 * r * NP;
    c1 = c0 + 1;
  } else {
    c0 += r * V;
    c1 = c0 + prm.n;
  }
  float cs[NP], sn[NP];
  if (!copy) {
    int have = -1;
    uint64_t p = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pr = r * NP + i;
      const int ax = prm.axis[pr];
      if (ax != have) {
        have = ax;
        const int64_t at = (int64_t)ax * prm.ps[0] + b * prm.ps[1] + s * prm.ps[2];
        p = prm.pos64 ? (uint64_t)static_cast<const int64_t*>(prm.pos)[at]
                      : (uint64_t)(int64_t)static_cast<const int32_t*>(prm.pos)[at];
      }
      const int32_t half_turns = (int32_t)((p * prm.step[pr]) >> 32);
      sincospif((float)half_turns * 0x1p-31f, &sn[i], &cs[i]);
      if (prm.inverse) sn[i] = -sn[i];
    }
  }
  using Vc = Vec<T, V>;
  constexpr int U = 4;  // heads whose loads are in flight together
  // this block's heads of q, then those of k; pointers step from head to head
  const int h_begin = (int)blockIdx.y * prm.heads_per_block, h_stop = h_begin + prm.heads_per_block;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const int before = w ? prm.H[0] : 0;
    int h = max(h_begin - before, 0);
    const int h_end = min(h_stop - before, prm.H[w]);
    if (h >= h_end) continue;
    const T* src = static_cast<const T*>(prm.x[w]) + b * prm.xs[w][0] + h * prm.xs[w][1] + s * prm.xs[w][2];
    T* dst = static_cast<T*>(prm.y[w]) + b * prm.ys[w][0] + h * prm.ys[w][1] + s * prm.ys[w][2];
    const int64_t xh = prm.xs[w][1], yh = prm.ys[w][1];
    for (; h < h_end; h += U) {
      Vc a[U], c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u < h_end) {
          a[u] = *reinterpret_cast<const Vc*>(src + c0);
          if (TWO && !copy) c[u] = *reinterpret_cast<const Vc*>(src + c1);
        }
        src += xh;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u < h_end) {
          if (!copy) {
            float xa[V], xc[V];
            widen(a[u], xa);
            if (TWO) widen(c[u], xc);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const int i0 = TWO ? i : (2 * i) % V, i1 = TWO ? i : (2 * i + 1) % V;
              const float x0 = xa[i0], x1 = TWO ? xc[i1] : xa[i1];
              xa[i0] = fmaf(x0, cs[i], -x1 * sn[i]);
              (TWO ? xc[i1] : xa[i1]) = fmaf(x1, cs[i], x0 * sn[i]);
            }
            narrow(xa, a[u]);
            if (TWO) {
              narrow(xc, c[u]);
              *reinterpret_cast<Vc*>(dst + c1) = c[u];
            }
          }
          *reinterpret_cast<Vc*>(dst + c0) = a[u];
        }
        dst += yh;
      }
    }
  }
}

template <typename T, int V>
static int launch(Params& prm, bool adjacent, int sms, cudaStream_t st, std::string* err) {
  prm.items = prm.groups * (prm.n / (adjacent ? Item<V, true>::PAIRS : V) + (prm.dh - 2 * prm.n) / V);
  const int64_t blocks = (prm.tokens * prm.items + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffLL) {
    *err = "too many tokens for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  // heads are split over blockIdx.y until about four blocks an SM are there, and no further: every
  // extra block computes the angles again
  const int H = prm.H[0] + prm.H[1];
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(H, (4LL * sms + blocks - 1) / blocks));
  prm.heads_per_block = (int)((H + want - 1) / want);
  const unsigned gy = (unsigned)((H + prm.heads_per_block - 1) / prm.heads_per_block);
  const dim3 grid((unsigned)blocks, gy);
  const cudaError_t e = adjacent ? launch_behind(rope_kernel<T, V, true>, grid, THREADS, 0, st, prm)
                                 : launch_behind(rope_kernel<T, V, false>, grid, THREADS, 0, st, prm);
  if (e != cudaSuccess) *err = std::string("rope launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace rope
}  // namespace mesh

using mesh::set_last_error;

extern "C" int mesh_attn_rope(mesh_attn_dtype dtype, int32_t B, int64_t S, int32_t d, int32_t Hq, const void* q,
                              const int64_t* q_strides, void* q_out, const int64_t* q_out_strides, int32_t Hk,
                              const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                              int32_t groups, int32_t n_pairs, int32_t n_axes, const double* freq,
                              const int32_t* pair_axis, int32_t adjacent, int32_t inverse, const void* positions,
                              int32_t pos_bits, const int64_t* pos_strides, void* stream) {
  return mesh::guarded_call([&]() -> int {
    using namespace mesh::rope;
    if (dtype != MESH_ATTN_F32 && dtype != MESH_ATTN_BF16)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "dtype must be MESH_ATTN_F32 or MESH_ATTN_BF16");
    if (B < 0 || S < 0 || Hq < 0 || Hk < 0)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "B, S, Hq and Hk must be >= 0");
    if (groups < 1 || d < 2 || d > 1024 || d % groups != 0)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need 2 <= d <= 1024, groups >= 1 and d % groups == 0");
    const int32_t dh = d / groups;
    if (n_pairs < 1 || n_pairs > MAX_PAIRS || 2 * n_pairs > dh)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need 1 <= n_pairs <= 256 and 2 * n_pairs <= d / groups");
    if (n_axes < 1 || n_axes > MAX_AXES)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "n_axes must be 1 to 8");
    if (pos_bits != 32 && pos_bits != 64)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "pos_bits must be 32 or 64");
    for (int32_t f : {adjacent, inverse})
      if (f != 0 && f != 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "adjacent and inverse must be 0 or 1");
    if (!freq || !pair_axis) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "freq or pair_axis is NULL");
    Params prm{};
    for (int i = 0; i < n_pairs; ++i) {
      if (!std::isfinite(freq[i])) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "freq must be finite");
      if (pair_axis[i] < 0 || pair_axis[i] >= n_axes)
        return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "pair_axis must be in 0 .. n_axes - 1");
      double t = freq[i] * 0.15915494309189533577;  // turns a position
      t -= std::floor(t);
      prm.step[i] = t >= 1.0 ? 0 : (uint64_t)std::ldexp(t, 64);
      prm.axis[i] = (uint8_t)pair_axis[i];
    }
    if (B == 0 || S == 0 || (Hq == 0 && Hk == 0)) return (int)MESH_ATTN_OK;
    if (!positions || !pos_strides) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "positions or pos_strides is NULL");
    struct Arg {
      int32_t H;
      const void* x;
      const int64_t* xs;
      void* y;
      const int64_t* ys;
    };
    const Arg args[2] = {{Hq, q, q_strides, q_out, q_out_strides}, {Hk, k, k_strides, k_out, k_out_strides}};
    const size_t es = dtype == MESH_ATTN_BF16 ? 2 : 4;
    int vec = (int)(16 / es);  // elements of an access: the most that divide every address and size
    auto divides = [&](int64_t elements) {
      while (elements % vec != 0) vec /= 2;
    };
    divides(adjacent ? 2 * n_pairs : n_pairs);
    divides(dh - 2 * n_pairs);
    for (int w = 0; w < 2; ++w) {
      const Arg& a = args[w];
      prm.H[w] = a.H;
      if (a.H == 0) continue;
      if (!a.x || !a.y || !a.xs || !a.ys)
        return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor or its strides are NULL");
      if (!mesh::is_aligned(a.x, es) || !mesh::is_aligned(a.y, es))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "tensors must be aligned to their element size");
      const int64_t dims[3] = {B, a.H, S};
      for (int i = 0; i < 3; ++i)
        if (a.ys[i] == 0 && dims[i] > 1)
          return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "an output must not be broadcast (stride 0)");
      prm.x[w] = a.x;
      prm.y[w] = a.y;
      divides((int64_t)(reinterpret_cast<uintptr_t>(a.x) / es));
      divides((int64_t)(reinterpret_cast<uintptr_t>(a.y) / es));
      for (int i = 0; i < 3; ++i) {
        prm.xs[w][i] = a.xs[i];
        prm.ys[w][i] = a.ys[i];
        divides(a.xs[i]);
        divides(a.ys[i]);
      }
    }
    if (!mesh::is_aligned(positions, pos_bits / 8))
      return set_last_error(MESH_ATTN_ERR_MISALIGNED, "positions must be aligned to their element size");
    prm.pos = positions;
    for (int i = 0; i < 3; ++i) prm.ps[i] = pos_strides[i];
    prm.pos64 = pos_bits == 64;
    prm.tokens = (int64_t)B * S;
    prm.S = S;
    prm.groups = groups;
    prm.dh = dh;
    prm.n = n_pairs;
    prm.inverse = inverse;
    int sms = 0;
    const cudaError_t e = mesh::current_sms(&sms);
    if (e != cudaSuccess) return set_last_error(MESH_ATTN_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
    std::string err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int ce;
    const bool adj = adjacent != 0;
    if (dtype == MESH_ATTN_BF16)
      ce = vec == 8   ? launch<__nv_bfloat16, 8>(prm, adj, sms, st, &err)
           : vec == 4 ? launch<__nv_bfloat16, 4>(prm, adj, sms, st, &err)
           : vec == 2 ? launch<__nv_bfloat16, 2>(prm, adj, sms, st, &err)
                      : launch<__nv_bfloat16, 1>(prm, adj, sms, st, &err);
    else
      ce = vec == 4   ? launch<float, 4>(prm, adj, sms, st, &err)
           : vec == 2 ? launch<float, 2>(prm, adj, sms, st, &err)
                      : launch<float, 1>(prm, adj, sms, st, &err);
    return mesh::launch_status(ce, err);
  });
}
