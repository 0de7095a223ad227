// The backward pass of score_bwd.cuh for heads of 64 columns.
#include "score_bwd.cuh"

namespace mesh {

int launch_range_bwd_64(const RangeArgs& a, const RangeBwdShape& z, int sms, cudaStream_t st, std::string* err) {
  return sbw::launch<64>(a, z, sms, st, err);
}

}  // namespace mesh
