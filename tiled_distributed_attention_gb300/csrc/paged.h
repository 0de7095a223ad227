// Declarations shared by the entry points of the paged cache's attention and its kernels' launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

namespace mesh {

// Rows of a sequence and KV head (new tokens times query heads) up to which the few-rows kernel takes a batch: one product's, and
// in fp32 what a lane's registers hold.
constexpr int PAGED_FEW_BF16 = 16, PAGED_FEW_F32 = 8;
constexpr int PAGED_MAX_B = 4096;  // the few-rows kernel keeps their unit counts in shared memory beside its ring

struct PagedArgs {
  bool bf16;
  const void* q;  // [N, Hq, d]: token, head strides in elements
  int64_t qs[2];
  const void* k;  // pages [n_pages, Hkv, page, d]: page, head, row strides
  const void* v;
  int64_t ks[3], vs[3];
  const int32_t* table;  // [B, max_pages]
  int64_t table_s;
  const int32_t* offsets;
  const int32_t* lens;
  const float* slopes;
  void* o;     // [N, Hq, d]
  float* lse;  // [N, Hq]
  char* ws;
  int32_t* status;
  int32_t N, B, Hq, Hkv, d, n_pages, page, max_pages, max_new, window;
  float scale, cap;
  int64_t wait_limit_ns;
};

// Workspace of the calls over a paged cache: [arrival counters of the few-rows kernel, zero between calls | the slots of its
// pieces, or the tensor-core kernel's counter and parts].  The counters have the same place whatever the sizes, so that a workspace
// serves calls of different sizes in turn.
constexpr size_t PAGED_WS_HEAD = 2048;  // a counter for each of its CTAs
size_t paged_rows_slots();
// Few rows a sequence and KV head, both types.
int launch_paged_rows(const PagedArgs& a, int sms, cudaStream_t st, std::string* err);

// fp32, any rows: on the CUDA cores.
int launch_paged_simt(const PagedArgs& a, int sms, cudaStream_t st, std::string* err);
size_t score_simt_workspace(int32_t d);  // of it, and of the fp32 forward of range-masked attention

struct RangeArgs {
  bool bf16;
  const void* q;  // [B, Hq, S, d]
  const void* k;  // [B, Hkv, S, d]
  const void* v;
  const int32_t* lo;  // [B, S] with a batch stride
  const int32_t* hi;
  int64_t mask_bs;
  const float* slopes;
  void* o;
  float* lse;  // [B, Hq, S]
  const void* go;
  void* dq;
  void* dk;
  void* dv;
  char* ws;
  int32_t* status;
  int64_t S;
  int32_t B, Hq, Hkv, d;
  float scale, cap;
  int64_t wait_limit_ns;
};
// fp32, on the CUDA cores.
int launch_range_fwd_simt(const RangeArgs& a, int sms, cudaStream_t st, std::string* err);

}  // namespace mesh
