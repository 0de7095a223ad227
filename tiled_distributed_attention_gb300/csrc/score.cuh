// What the kernels of range-masked attention and of chunks over a paged cache share: the cap of a score.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace mesh {

// tanh(z) / z for |z| <= 1 as a polynomial of z^2: least maximum of the relative error at degree 5 (iterated weighted least
// squares on 4,000 points), 5.9e-7.  A score is seldom beyond its cap, so this is the usual case: two products and five
// FMAs by pairs on the FMA pipe, where the exponential form would take two more MUFU operations beside the softmax's one.
constexpr float TANH_C0 = 0.99999941f, TANH_C1 = -0.33329042f, TANH_C2 = 0.13281434f, TANH_C3 = -0.05160567f,
                TANH_C4 = 0.01674311f, TANH_C5 = -0.00306706f;

// tanh(z) / z of a pair from u = z^2, both at most 1.
__device__ __forceinline__ uint64_t tanh_ratio2(uint64_t u) {
  uint64_t y = f2_fma(u, f2_pack(TANH_C5, TANH_C5), f2_pack(TANH_C4, TANH_C4));
  y = f2_fma(y, u, f2_pack(TANH_C3, TANH_C3));
  y = f2_fma(y, u, f2_pack(TANH_C2, TANH_C2));
  y = f2_fma(y, u, f2_pack(TANH_C1, TANH_C1));
  return f2_fma(y, u, f2_pack(TANH_C0, TANH_C0));
}

// tanh(z) for any z: 1 - 2 / (e^2z + 1), which is -1 and 1 at its ends, NaN for NaN, and off by 2^-23 or so of 1.
__device__ __forceinline__ float tanh_any(float z) {
  const float e = fast_exp2(z * 2.8853900817779268f);
  return 1.f - __fdividef(2.f, e + 1.f);
}

}  // namespace mesh
