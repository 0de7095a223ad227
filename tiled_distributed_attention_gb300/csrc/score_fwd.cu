// Host side of the tensor-core forward with scores that are capped, biased and masked by ranges (score_fwd.cuh): how heads and
// tokens fill its tiles, when its units are cut into parts, the workspace and the tensor maps.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "internal.h"
#include "score_fwd.h"
#include "tmap.h"

namespace mesh {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn get_encode(std::string* err) {
  static EncodeTiledFn fn = nullptr;
  if (fn) return fn;
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !ptr) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return nullptr;
  }
  fn = reinterpret_cast<EncodeTiledFn>(ptr);
  return fn;
}

bool encode_bf16_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const int64_t* strides, const uint32_t* box,
                     std::string* err) {
  EncodeTiledFn enc = get_encode(err);
  if (!enc) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    es[i] = 1;
    // the stride of an axis of one is never used, and need not be one that a map takes
    if (i > 0) s[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i - 1] * 2 : (cuuint64_t)16;
  }
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, s, b, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *err = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
    return false;
  }
  return true;
}

// Units are two tiles, whose products and softmax go on beside one another; one where that leaves an SM idle for each (2 x 1,000
// tokens of 4 heads, d 64, slopes: forward 18 us, 21 with two).
//
// Tiles.  All query heads of a KV head in one tile where they and their tokens fill it (3 heads: 42 tokens, 126 rows), else the
// heads in the fewest equal chunks that do to 7/8.
//
// Parts, of range-masked attention (over pages plan_kernel decides by the lengths, which are on the device).  The longest unit
// has to be done, and the SMs share all blocks, those of a dense batch half of the longest on average, as under a causal mask.
// A unit costs about three blocks besides its own (5 us at 1.6 us a block), and parts a merge: four blocks and the traffic of
// their fp32 rows.  The best count is taken where it saves a fifth or more: 160 units of up to 20 blocks stay whole (38 us; 67
// in 2 parts; capped, 52 and 80).
ScoreFwdShape score_fwd_shape(bool paged, int64_t S, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int sms) {
  ScoreFwdShape z{};
  const int g = Hq / Hkv;
  for (z.hc = (g + 127) / 128;; ++z.hc) {
    z.gh = (g + z.hc - 1) / z.hc;
    z.tt = 128 / z.gh;
    if (z.gh * z.tt >= 112) break;
  }
  z.hc = (g + z.gh - 1) / z.gh;
  z.tu = 2 * z.tt;
  const int64_t tu = z.tu;
  const int64_t groups = paged ? N / tu + B : (S + tu - 1) / tu;
  const int64_t lanes = (int64_t)Hkv * z.hc * (paged ? 1 : B);
  z.groups = (int32_t)std::min<int64_t>(groups, 0x7fffffff);
  z.lanes = (int32_t)std::min<int64_t>(lanes, 0x7fffffff);
  z.parts = 1;
  // units of one tile where there is an SM for each: a block of one takes less time than a block of two
  auto one_tile = [&](int64_t n) {
    z.tu = z.tt;
    z.groups = (int32_t)n;
  };
  size_t at = 256;  // the counter
  if (paged) {
    // room as for the most SMs and whether there is a plan or not, so that a workspace serves smaller batches too
    const size_t plan = at;
    at += (PLAN_BYTES + 255) / 256 * 256;
    const int64_t most = std::min<int64_t>((int64_t)FWD_PART_WAVES * MAX_SMS, lanes * std::min<int64_t>(groups, PLAN_GROUPS) * MAX_FWD_PARTS);
    z.part_o = at;
    z.part_lse = at + (size_t)most * 256 * d * 4;
    at += (size_t)most * 256 * (d + 1) * 4;
    // Parts may come of it where the longest unit there can be takes 2.5 times the SMs' share of all, half as long on average; with
    // less the merge's launch (4 us where there is nothing to merge) goes for nothing.  An order is wanted where units wait for
    // an SM, but those of a single sequence are in order as they come.
    const int64_t nb = (S + 127) / 128, units = lanes * (N / tu + 1);
    const bool cut = nb >= 8 && 2 * nb * sms > 5 * units * (nb / 2 + 3);
    if (groups <= PLAN_GROUPS && (cut || (B > 1 && lanes * groups > sms))) {
      z.plan = plan;
      if (cut) z.slots = (int32_t)most;
    } else if (lanes * (N / z.tt + B) <= sms) {
      one_tile(N / z.tt + B);
    }
    z.total = at;
    return z;
  }
  const int64_t units = lanes * groups;
  const double nb = (double)((S + 127) / 128);
  double whole = 0, best = 0;
  for (int k = 1; k <= MAX_FWD_PARTS; ++k) {
    if (k > 1 && (nb / k < 2 || units * k > FWD_PART_WAVES * sms)) break;
    const double cost = std::max(nb / k + 3, (double)units * (nb * 0.5 + 3 * k) / sms) + (k > 1 ? 4 + 0.02 * (double)units * k : 0);
    if (k == 1) whole = best = cost;
    if (cost < best && cost <= 0.8 * whole) {
      best = cost;
      z.parts = k;
    }
  }
  if (z.parts == 1 && 2 * units <= sms) one_tile((S + z.tt - 1) / z.tt);
  if (z.parts > 1) {
    const size_t rows = (size_t)z.lanes * z.groups * z.parts * 256;
    z.part_o = at;
    at += rows * d * 4;
    z.part_lse = at;
    at += rows * 4;
  }
  z.total = at;
  return z;
}

size_t score_fwd_paged_workspace(int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d) {
  return score_fwd_shape(true, 0, N, B, Hq, Hkv, d, 1).total;
}

int launch_score_fwd(const ScoreFwdArgs& a, int sms, cudaStream_t st, std::string* err) {
  const ScoreFwdShape z = score_fwd_shape(a.paged, a.S, a.N, a.B, a.Hq, a.Hkv, a.d, sms);
  if (a.paged) return a.d == 128 ? launch_score_fwd_paged_128(a, z, sms, st, err) : launch_score_fwd_paged_64(a, z, sms, st, err);
  return a.d == 128 ? launch_score_fwd_128(a, z, sms, st, err) : launch_score_fwd_64(a, z, sms, st, err);
}

}  // namespace mesh
