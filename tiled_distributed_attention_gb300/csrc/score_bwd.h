// Declarations of the tensor-core backward pass of range-masked attention.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "paged.h"

namespace mesh {

// Workspace of the backward pass (bytes from its start) and the parts that units are cut into.
struct RangeBwdShape {
  int32_t kv_parts, dq_parts;
  size_t counters, dsum, bounds, order, dq_part, dk_part, dv_part, total;
};
RangeBwdShape range_bwd_shape(bool bf16, int64_t S, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int sms);
// bf16, by head size, one translation unit each
int launch_range_bwd_64(const RangeArgs& a, const RangeBwdShape& z, int sms, cudaStream_t st, std::string* err);
int launch_range_bwd_128(const RangeArgs& a, const RangeBwdShape& z, int sms, cudaStream_t st, std::string* err);
// fp32, on the CUDA cores
int launch_range_bwd_simt(const RangeArgs& a, const RangeBwdShape& z, cudaStream_t st, std::string* err);

}  // namespace mesh
