// New tokens' keys and values into the pages of their sequences, keys and queries rotated on the way, in one launch.
//
// The tokens of all sequences stand one after another: sequence b's are offsets[b] .. offsets[b + 1], and they are the last
// of its lens[b] cached ones, so token t of n has the place lens[b] - n + t in its sequence, row place % page of page
// table[b][place / page].  Pairs of columns turn as in mesh_attn_rope (same angles, in 64-bit fixed point), by the
// token's place or by positions of the caller's; values are copied.
//
// Bound by memory: every element is read once, where the projection wrote it, and written once, where attention reads it.
// The work of a thread is that of the rotation kernel (rope.cu): V pairs of one token, sines and cosines once, then
// all heads of q, k and v with four heads' loads in flight; a value's columns take the same accesses without the turn.
// With few tokens the heads are spread over blockIdx.y.  A warp looks its first token's sequence up 32 offsets at a time
// (one step up to 32 sequences, two up to 1,024), and a lane whose token is of a later one searches on from there.
//
// Four or five loads follow one another for that; the first heads' own are issued before them.
//
// Measured: 16,384 tokens of 8 sequences, 32 + 8 heads, d 128, bf16, 403 MB in 67.5 us, 6.0 TB/s (a plain copy: 6.8; 71 with
// the look-up first, and 500 tokens 11 us for 8); in fp32 130 us, 6.2 TB/s; one token of 64 sequences 6.2 us, most of it the host's
// call.  A second set of heads' loads beside the first's stores: 67 us, and 10 for 500 tokens; other block sizes and fewer registers
// no gain.
//
// A token whose place or page does not exist is recorded in the status block and left out; rows from offsets[B] on
// are left as they are.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope_vec.cuh"

namespace mesh {
namespace append {

using rope::Item;
using rope::Vec;

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 256;
constexpr int MAX_AXES = 8;
constexpr int ROLE_TOKEN = 1;

struct Params {
  const void* x[3];  // q, k, v [N, H, d]: token, head strides
  void* y[3];        // q_out [N, Hq, d], the pages [n_pages, Hkv, page, d]
  int64_t xs[3][2];
  int64_t qs[2];     // q_out: token, head strides
  int64_t ps[2][3];  // pages of k, v: page, head, row strides
  int32_t H[3];
  const int32_t* table;
  const int32_t* offsets;
  const int32_t* lens;
  int32_t* status;
  const void* pos;  // or NULL: the token's place
  int64_t pos_s[2];  // axis, token strides
  int64_t N, table_s;
  int32_t pos64, B, n_pages, page, max_pages, groups, dh, n, items, heads_per_block;
  uint64_t step[MAX_PAIRS];
  uint8_t axis[MAX_PAIRS];
};

template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ Params prm) {
  wait_for_kernel_before();
  const int64_t lin = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  const int item = (int)(lin % prm.items);
  const int64_t tok = lin / prm.items;
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
  // this block's heads of q, then those of k, then those of v, a few at a time: heads h .. h + n - 1 of tensor w, their loads
  // in flight together.  The first ones' are on their way before the token's page is looked up
  using Vc = Vec<T, V>;
  constexpr int U = 4;
  Vc a[U], c[U];
  int left = min(prm.heads_per_block, prm.H[0] + prm.H[1] + prm.H[2] - (int)blockIdx.y * prm.heads_per_block);
  int w = 0, h = (int)blockIdx.y * prm.heads_per_block, n = 0;
  auto next = [&]() {
    while (w < 2 && h >= prm.H[w]) h -= prm.H[w++];
    n = min(min(U, left), prm.H[w] - h);
  };
  auto load = [&]() {
    const T* src = static_cast<const T*>(prm.x[w]) + tok * prm.xs[w][0] + h * prm.xs[w][1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < n) {
        a[u] = *reinterpret_cast<const Vc*>(src + c0);
        if (TWO && !copy) c[u] = *reinterpret_cast<const Vc*>(src + c1);
      }
      src += prm.xs[w][1];
    }
  };
  next();
  if (tok < prm.N) load();
  const int b = sequence_of(prm.offsets, prm.B, __shfl_sync(0xffffffffu, tok, 0), tok);
  if (b < 0 || tok >= prm.N) return;
  const int32_t begin = prm.offsets[b], len = prm.lens[b];
  const int64_t place = (int64_t)len - prm.offsets[b + 1] + tok;  // len - n + (tok - begin)
  int32_t at = -1;
  if (tok >= begin && place >= 0 && place < (int64_t)prm.max_pages * prm.page)
    at = prm.table[b * prm.table_s + place / prm.page];
  if (at < 0 || at >= prm.n_pages) {
    if (item == 0) record_error(prm.status, MESH_ATTN_ERR_OUT_OF_RANGE, ROLE_TOKEN, (int32_t)b);
    return;
  }
  const int64_t row = place % prm.page;
  float cs[NP], sn[NP];
  if (!copy) {
    int have = -1;
    uint64_t p = (uint64_t)place;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int pr = r * NP + i;
      const int ax = prm.axis[pr];
      if (prm.pos && ax != have) {
        have = ax;
        const int64_t e = (int64_t)ax * prm.pos_s[0] + tok * prm.pos_s[1];
        p = prm.pos64 ? (uint64_t)static_cast<const int64_t*>(prm.pos)[e]
                      : (uint64_t)(int64_t)static_cast<const int32_t*>(prm.pos)[e];
      }
      const int32_t half_turns = (int32_t)((p * prm.step[pr]) >> 32);
      sincospif((float)half_turns * 0x1p-31f, &sn[i], &cs[i]);
    }
  }
#pragma unroll 1
  for (;;) {
    const int64_t yh = w == 0 ? prm.qs[1] : prm.ps[w - 1][1];
    T* dst = static_cast<T*>(prm.y[w]) + (w == 0 ? tok * prm.qs[0] : at * prm.ps[w - 1][0] + row * prm.ps[w - 1][2]) + h * yh;
    const bool turn = !copy && w < 2;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < n) {
        if (turn) {
          float xa[V], xc[V];
          rope::widen(a[u], xa);
          if (TWO) rope::widen(c[u], xc);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int i0 = TWO ? i : (2 * i) % V, i1 = TWO ? i : (2 * i + 1) % V;
            const float x0 = xa[i0], x1 = TWO ? xc[i1] : xa[i1];
            xa[i0] = fmaf(x0, cs[i], -x1 * sn[i]);
            (TWO ? xc[i1] : xa[i1]) = fmaf(x1, cs[i], x0 * sn[i]);
          }
          rope::narrow(xa, a[u]);
          if (TWO) rope::narrow(xc, c[u]);
        }
        *reinterpret_cast<Vc*>(dst + c0) = a[u];
        if (TWO && !copy) *reinterpret_cast<Vc*>(dst + c1) = c[u];
      }
      dst += yh;
    }
    left -= n;
    if (left == 0) return;
    h += n;
    next();
    load();
  }
}

template <typename T, int V>
static int launch(Params& prm, bool adjacent, int sms, cudaStream_t st, std::string* err) {
  prm.items = prm.groups * (prm.n / (adjacent ? Item<V, true>::PAIRS : V) + (prm.dh - 2 * prm.n) / V);
  const int64_t blocks = (prm.N * prm.items + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffLL) {
    *err = "too many tokens for one launch";
    return (int)cudaErrorInvalidConfiguration;
  }
  // heads are split over blockIdx.y until about four blocks an SM are there, and no further: every
  // extra block looks up the tokens and computes the angles again
  const int H = prm.H[0] + prm.H[1] + prm.H[2];
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(H, (4LL * sms + blocks - 1) / blocks));
  prm.heads_per_block = (int)((H + want - 1) / want);
  const unsigned gy = (unsigned)((H + prm.heads_per_block - 1) / prm.heads_per_block);
  const dim3 grid((unsigned)blocks, gy);
  const cudaError_t e = adjacent ? launch_behind(append_kernel<T, V, true>, grid, THREADS, 0, st, prm)
                                 : launch_behind(append_kernel<T, V, false>, grid, THREADS, 0, st, prm);
  if (e != cudaSuccess) *err = std::string("paged_append launch: ") + cudaGetErrorString(e);
  return (int)e;
}

}  // namespace append
}  // namespace mesh

using mesh::set_last_error;

extern "C" int mesh_attn_paged_append(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, const void* q,
                                      const int64_t* q_strides, void* q_out, const int64_t* q_out_strides, const void* k,
                                      const int64_t* k_strides, const void* v, const int64_t* v_strides, int32_t n_pages, int32_t page,
                                      void* k_pages, const int64_t* k_page_strides, void* v_pages, const int64_t* v_page_strides,
                                      const int32_t* table, int32_t max_pages, int64_t table_stride, const int32_t* offsets,
                                      const int32_t* lens, int32_t groups, int32_t n_pairs, int32_t n_axes, const double* freq,
                                      const int32_t* pair_axis, int32_t adjacent, const void* positions, int32_t pos_bits,
                                      const int64_t* pos_strides, int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    using namespace mesh::append;
    if (dtype != MESH_ATTN_F32 && dtype != MESH_ATTN_BF16)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "dtype must be MESH_ATTN_F32 or MESH_ATTN_BF16");
    if (N < 0 || B < 0 || Hq < 0 || Hkv < 1 || n_pages < 0 || max_pages < 0)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "N, B, Hq, n_pages and max_pages must be >= 0, Hkv >= 1");
    if (page < 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "page must be >= 1");
    if (N > 0x7fffffff) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "N must be < 2^31");
    if (groups < 1 || d < 2 || d > 1024 || d % groups != 0)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need 2 <= d <= 1024, groups >= 1 and d % groups == 0");
    const int32_t dh = d / groups;
    if (n_pairs < 0 || n_pairs > MAX_PAIRS || 2 * n_pairs > dh)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need 0 <= n_pairs <= 256 and 2 * n_pairs <= d / groups");
    if (n_axes < 1 || n_axes > MAX_AXES) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "n_axes must be 1 to 8");
    if (adjacent != 0 && adjacent != 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "adjacent must be 0 or 1");
    if (n_pairs > 0 && (!freq || !pair_axis)) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "freq or pair_axis is NULL");
    if (n_pairs > 0 && !positions && n_axes != 1)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "positions are needed where there is more than one axis");
    if (positions && ((pos_bits != 32 && pos_bits != 64) || !pos_strides))
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "pos_bits must be 32 or 64, and pos_strides be there");
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
    if (N == 0 || B == 0) return (int)MESH_ATTN_OK;
    if ((Hq > 0 && (!q || !q_out || !q_strides || !q_out_strides)) || !k || !k_strides || !v || !v_strides || !k_pages ||
        !k_page_strides || !v_pages || !v_page_strides || !table || !offsets || !lens || !d_status)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor, its strides or the status pointer is NULL");
    const size_t es = dtype == MESH_ATTN_BF16 ? 2 : 4;
    int vec = (int)(16 / es);  // elements of an access: the most that divide every address and size
    auto divides = [&](int64_t elements) {
      while (elements % vec != 0) vec /= 2;
    };
    divides(adjacent ? 2 * n_pairs : n_pairs);
    divides(dh - 2 * n_pairs);
    const void* in[3] = {q, k, v};
    const int64_t* in_s[3] = {q_strides, k_strides, v_strides};
    void* out[3] = {q_out, k_pages, v_pages};
    const int64_t* out_s[3] = {q_out_strides, k_page_strides, v_page_strides};
    const int32_t heads[3] = {Hq, Hkv, Hkv};
    for (int w = 0; w < 3; ++w) {
      prm.H[w] = heads[w];
      if (heads[w] == 0) continue;
      if (!mesh::is_aligned(in[w], es) || !mesh::is_aligned(out[w], es))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "tensors must be aligned to their element size");
      prm.x[w] = in[w];
      prm.y[w] = out[w];
      divides((int64_t)(reinterpret_cast<uintptr_t>(in[w]) / es));
      divides((int64_t)(reinterpret_cast<uintptr_t>(out[w]) / es));
      const int64_t in_dims[2] = {N, heads[w]};
      for (int i = 0; i < 2; ++i) {
        prm.xs[w][i] = in_s[w][i];
        if (in_dims[i] > 1) divides(in_s[w][i]);
      }
      const int64_t dims[3] = {w == 0 ? N : n_pages, heads[w], page};
      for (int i = 0; i < (w == 0 ? 2 : 3); ++i) {
        if (out_s[w][i] == 0 && dims[i] > 1)
          return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "an output must not be broadcast (stride 0)");
        (w == 0 ? prm.qs[i] : prm.ps[w - 1][i]) = out_s[w][i];
        if (dims[i] > 1) divides(out_s[w][i]);
      }
    }
    for (const void* p : {(const void*)table, (const void*)offsets, (const void*)lens, (const void*)d_status})
      if (!mesh::is_aligned(p, 4)) return set_last_error(MESH_ATTN_ERR_MISALIGNED, "table, offsets, lens and status must be 4-byte aligned");
    if (positions && !mesh::is_aligned(positions, pos_bits / 8))
      return set_last_error(MESH_ATTN_ERR_MISALIGNED, "positions must be aligned to their element size");
    prm.table = table;
    prm.table_s = table_stride;
    prm.offsets = offsets;
    prm.lens = lens;
    prm.status = d_status;
    prm.pos = n_pairs > 0 ? positions : nullptr;
    for (int i = 0; i < 2; ++i) prm.pos_s[i] = positions ? pos_strides[i] : 0;
    prm.pos64 = pos_bits == 64;
    prm.N = N;
    prm.B = B;
    prm.n_pages = n_pages;
    prm.page = page;
    prm.max_pages = max_pages;
    prm.groups = groups;
    prm.dh = dh;
    prm.n = n_pairs;
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
