// Tensor maps of bf16 tensors with the columns of a head consecutive, for TMA loads with 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

namespace mesh {

// dims and box from the fastest axis; strides of the axes behind it, in elements.  What a box reaches outside of an axis
// arrives as zeros.
bool encode_bf16_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const int64_t* strides, const uint32_t* box,
                     std::string* err);

}  // namespace mesh
