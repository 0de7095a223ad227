// Declarations of the tensor-core forward that range-masked attention and chunks over a paged cache share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

namespace mesh {

struct ScoreFwdArgs {
  bool paged;
  const void* q;   // bf16; range: [B, Hq, S, d] dense; paged: [N, Hq, d] with token and head strides
  int64_t qs[2];
  const void* k;   // range: [B, Hkv, S, d] dense; paged: pages [n_pages, Hkv, page, d] with page, head and row strides
  const void* v;
  int64_t ks[3], vs[3];
  const float* slopes;  // [Hq] or NULL
  void* o;              // as dense q
  float* lse;           // range: [B, Hq, S]; paged: [N, Hq]
  int32_t* status;
  char* ws;
  int64_t S;            // range: tokens; paged: tokens that the table can hold
  int32_t N, B, Hq, Hkv, d;
  const int32_t* lo;    // range: keys of each query, [B, S] with a batch stride
  const int32_t* hi;
  int64_t mask_bs;
  const int32_t* offsets;  // paged
  const int32_t* lens;
  const int32_t* table;
  int64_t table_s;
  int32_t n_pages, page, max_pages, max_new, window;
  float scale, cap;
  int64_t wait_limit_ns;
};

// How the query heads of a KV head and their tokens fill a 128-row tile, and into how many parts of their keys units
// (two tiles) are cut.
struct ScoreFwdShape {
  int32_t gh, tt, hc;  // heads and tokens of a tile, chunks of heads
  int32_t tu;          // tokens of a unit
  int32_t groups;      // units of a (batch, KV head, chunk), or of a (KV head, chunk) in paged, that there may be
  int32_t lanes, parts;
  int32_t slots;  // paged: parts that there is room for, 0 where none are made
  size_t counter, plan, part_o, part_lse, total;  // workspace; plan 0 where there is none
};
constexpr int MAX_FWD_PARTS = 16, FWD_PART_WAVES = 4;
// Paged: up to so many groups of tokens of a lane are sorted and long ones cut (score_fwd.cuh); beyond there are several for each SM, and
// they are taken as they come.
constexpr int PLAN_GROUPS = 768;
constexpr size_t PLAN_BYTES = 16 + PLAN_GROUPS * (4 + 16);
ScoreFwdShape score_fwd_shape(bool paged, int64_t S, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int sms);
// Enough for any batch of these heads with at most N tokens and B sequences, on any number of SMs.
size_t score_fwd_paged_workspace(int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d);

int launch_score_fwd(const ScoreFwdArgs& a, int sms, cudaStream_t st, std::string* err);
// The kernels by head size and cache, one translation unit each.
int launch_score_fwd_128(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err);
int launch_score_fwd_64(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err);
int launch_score_fwd_paged_128(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err);
int launch_score_fwd_paged_64(const ScoreFwdArgs& a, const ScoreFwdShape& z, int sms, cudaStream_t st, std::string* err);

}  // namespace mesh
