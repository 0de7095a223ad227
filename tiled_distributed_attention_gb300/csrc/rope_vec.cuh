// What the kernels that rotate pairs of columns share: accesses of V elements, their widening to fp32 and back, and the
// pairs that an access holds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace mesh {
namespace rope {

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

}  // namespace rope
}  // namespace mesh
