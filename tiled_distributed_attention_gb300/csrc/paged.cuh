// What the kernels over a paged cache share: which sequence a token of the packed batch is of.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mesh_attn.h"

namespace mesh {

// Whether a kernel has nothing to do for what the status block holds.  Over a paged cache, lengths and pages that do not fit are taken
// as the nearest that do, and do not keep the other sequences, later kernels and later calls from their work.
template <bool PAGED>
__device__ __forceinline__ bool stopped(const int32_t* status) {
  const int32_t s = *reinterpret_cast<const volatile int32_t*>(status);
  return s != 0 && !(PAGED && s == MESH_ATTN_ERR_OUT_OF_RANGE);
}

// For a CTA whose wait ran out, behind the wait's own record: that takes only a block of zeros, and over pages what an earlier call
// or another sequence left there (OUT_OF_RANGE) gives way to it; words 1 and 2 stay.  (In record_error, which stands behind every
// wait of every kernel, the second exchange cost the forward 2 to 4 %: 755 -> 780 us, 1,024 new tokens over 65,536.)
__device__ __forceinline__ void timeout_takes_over(int32_t* status) {
  atomicCAS(status, MESH_ATTN_ERR_OUT_OF_RANGE, MESH_ATTN_ERR_DEVICE_TIMEOUT);
}

// The last b of [lo, B) with offsets[b] <= tok, or lo - 1 where there is none, by the calling thread alone.
__device__ __forceinline__ int last_begun(const int32_t* offsets, int lo, int B, int64_t tok) {
  int a = lo - 1, z = B;  // offsets[a] <= tok < offsets[z], as far as they are known
  while (z - a > 1) {
    const int c = (a + z) >> 1;
    if (offsets[c] <= tok) a = c;
    else z = c;
  }
  return a;
}

// The same for the whole of a converged warp and one token, 32 offsets at a time: -1 where tok is before offsets[0].
__device__ __forceinline__ int last_begun_warp(const int32_t* offsets, int B, int64_t tok) {
  const int lane = threadIdx.x & 31;
  int a = 0, n = B;  // the answer is in [a - 1, a + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = a + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < a + n && offsets[min(at, B - 1)] <= tok);
    const int c = __popc(m);  // leading lanes, where the offsets ascend
    if (c == 0) return a - 1;
    const int end = a + n;
    a += (c - 1) * step + 1;  // offsets[a - 1] <= tok
    n = min(step - 1, end - a);
  }
  return a - 1;
}

// The sequence of token `tok` of a packed batch, offsets[b] <= tok < offsets[b + 1], or -1: before the first sequence or
// behind the last.  All 32 lanes call it, `first` being the first lane's token, which none of theirs precedes.
// Offsets that do not ascend give some sequence of 0 .. B - 1 or -1.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int B, int64_t first, int64_t tok) {
  const int b0 = last_begun_warp(offsets, B, first);
  int b = b0;
  if (tok != first) b = last_begun(offsets, max(b0, 0), B, tok);
  if (b < 0 || b >= B || tok >= offsets[B]) return -1;
  return b;
}

// What a sequence asks for: n tokens, the rows of the batch from `begin` on, that are the last of `len` cached ones.  What does not fit
// is taken as the nearest that does: offsets within the batch, a length that the new tokens need and the table holds.  Of more new
// tokens than the bound the first ones are taken, at their places, and the cache as far as the last of them.
struct Asked {
  int32_t begin, n, len;
  bool bad;
};
__device__ __forceinline__ Asked asked(const int32_t* offsets, const int32_t* lens, int b, int32_t N, int32_t max_new, int32_t max_pages,
                                       int32_t page) {
  const int32_t o0 = offsets[b], o1 = offsets[b + 1], len = lens[b];
  Asked x;
  x.begin = min(max(o0, 0), N);
  const int32_t end = min(max(o1, x.begin), N);
  int32_t all = end - x.begin;
  x.len = (int32_t)min((int64_t)max(len, all), (int64_t)max_pages * page);
  x.bad = x.begin != o0 || end != o1 || x.len != len || all > x.len || all > max_new;
  all = min(all, x.len);
  x.n = min(all, max_new);
  x.len -= all - x.n;
  return x;
}

}  // namespace mesh
