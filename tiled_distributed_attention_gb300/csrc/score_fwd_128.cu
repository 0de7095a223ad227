// The forward of score_fwd.cuh for heads of 128 columns, of dense batches.
#include "score_fwd.cuh"

namespace mesh {

int launch_score_fwd_128(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err) {
  return sfw::launch<128, false>(a, z, sms, st, err);
}

}  // namespace mesh
