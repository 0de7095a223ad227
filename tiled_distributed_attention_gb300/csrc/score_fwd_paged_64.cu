// The forward of score_fwd.cuh for heads of 64 columns, over a paged cache.
#include "score_fwd.cuh"

namespace mesh {

int launch_score_fwd_paged_64(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err) {
  return sfw::launch<64, true>(a, z, sms, st, err);
}

}  // namespace mesh
