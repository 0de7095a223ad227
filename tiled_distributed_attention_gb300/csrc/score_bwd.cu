// Host side of range-masked attention's backward pass: the parts that its units are cut into, and the workspace.
#include <algorithm>

#include "score_bwd.h"

namespace mesh {

// Units of a pass are cut into parts of their streamed blocks where whole ones would leave slots idle: as many as fill them, of
// `least` blocks at least (halved where the mask is causal).
static int32_t parts_for(int64_t units, int64_t blocks, int64_t slots, int least) {
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>({slots / std::max<int64_t>(units, 1), blocks / least, 16}));
}

RangeBwdShape range_bwd_shape(bool bf16, int64_t S, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int sms) {
  RangeBwdShape z{};
  size_t at = 512;  // two counters
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = (at + bytes + 255) / 256 * 256;
    return o;
  };
  const int g = Hq / Hkv;
  const size_t q = (size_t)B * Hq * S, kv = (size_t)B * Hkv * S;
  if (bf16) {
    // the two passes share the SMs: dkdv units are about as long as dq units times 4 / 3 and the group's heads
    const int64_t nb = (S + 127) / 128;
    z.kv_parts = parts_for(nb * B * Hkv, nb * g, sms / 2, 4);
    z.dq_parts = parts_for(nb * B * Hq, nb, sms / 2, 4);
    z.bounds = take((size_t)B * nb * 16);
    z.order = take((size_t)B * nb * 16);
  } else {
    const int64_t nb = (S + 63) / 64, tiles = (S * g + 63) / 64;
    // of a single block, a 64 x 64 one taking some 13 us, and twice the CTAs that are resident (two an SM at d = 64), since
    // those of ragged documents are of very different lengths: 400 tokens of 4 heads on 2, both directions, 45 us; 54 with half
    // as many parts
    const int slots = (d == 64 ? 4 : 2) * sms;
    z.kv_parts = parts_for(nb * B * Hkv, nb * g, slots, 1);
    z.dq_parts = parts_for(tiles * B * Hkv, nb, slots, 1);
  }
  z.dsum = take(q * 4);
  if (z.dq_parts > 1) z.dq_part = take(z.dq_parts * q * d * 4);
  if (z.kv_parts > 1) {
    z.dk_part = take(z.kv_parts * kv * d * 4);
    z.dv_part = take(z.kv_parts * kv * d * 4);
  }
  z.total = at;
  return z;
}

}  // namespace mesh
