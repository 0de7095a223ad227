// What the kernels of range-masked attention and of chunks over a paged cache share: the cap of a score.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"

namespace mesh {

// Caps are taken by tiers, the lowest that holds for all of a warp's scores of a block (the highest z^2 says so afterwards, and
// what was too low is done again from the next): |z| <= 1/2, |z| <= 1, any.  A score is seldom near its cap, and every step of
// the polynomial costs the FMA pipe a cycle a score and sub-partition, 256 a block, beside the softmax's two.
//
// tanh(z) / z as a polynomial of z^2: least maximum of the relative error (iterated weighted least squares on 4,000
// points), 5.4e-7 at degree 3 up to 1/2 and 5.9e-7 at degree 5 up to 1.
constexpr float TANH_LOW = 0.25f, TANH_HIGH = 1.f;  // z^2
constexpr float TANH_L0 = 0.999999456f, TANH_L1 = -0.333263179f, TANH_L2 = 0.131902966f, TANH_L3 = -0.0444022256f;
constexpr float TANH_C0 = 0.99999941f, TANH_C1 = -0.33329042f, TANH_C2 = 0.13281434f, TANH_C3 = -0.05160567f,
                TANH_C4 = 0.01674311f, TANH_C5 = -0.00306706f;

// tanh(z) / z of a pair from u = z^2, both at most TANH_HIGH.
__device__ __forceinline__ uint64_t tanh_ratio2(uint64_t u) {
  uint64_t y = f2_fma(u, f2_pack(TANH_C5, TANH_C5), f2_pack(TANH_C4, TANH_C4));
  y = f2_fma(y, u, f2_pack(TANH_C3, TANH_C3));
  y = f2_fma(y, u, f2_pack(TANH_C2, TANH_C2));
  y = f2_fma(y, u, f2_pack(TANH_C1, TANH_C1));
  return f2_fma(y, u, f2_pack(TANH_C0, TANH_C0));
}

// What a call's cap comes to: y = cap log2(e) tanh(s k), k = scale / cap.
struct Cap {
  float log2;     // cap log2(e)
  float k;
  float b[4];     // the low tier's polynomial of s^2, times cap log2(e) and the powers of k
  float low;      // s^2 up to which it holds (none where the powers of k leave fp32's range)
  float inv2;     // 1 / (cap log2(e))^2
};

template <int T>
struct Tier {
  static constexpr int value = T;
};

// tanh(z) for any z: 1 - 2 / (e^2z + 1), which is -1 and 1 at its ends, NaN for NaN, and off by 2^-23 or so of 1.
__device__ __forceinline__ float tanh_any(float z) {
  const float e = fast_exp2(z * 2.8853900817779268f);
  return 1.f - __fdividef(2.f, e + 1.f);
}

inline Cap make_cap(float scale, float cap) {
  Cap c{};
  if (!(cap > 0.f)) return c;
  const double k = (double)scale / cap, l = (double)cap * 1.4426950408889634;
  const double p[4] = {TANH_L0, TANH_L1, TANH_L2, TANH_L3};
  c.log2 = (float)l;
  c.k = (float)k;
  double f = l * k;
  for (int i = 0; i < 4; ++i, f *= k * k) c.b[i] = (float)(p[i] * f);
  // the coefficients are a power of k apart each, so those between the first and the last are in range where these are
  const auto fits = [](float x) { return std::fabs(x) > 1e-30f && std::fabs(x) < 1e30f; };
  c.low = fits(c.b[0]) && fits(c.b[3]) ? (float)(TANH_LOW / (k * k)) : -1.f;
  c.inv2 = (float)(1.0 / (l * l));
  return c;
}

// A pair of scores by tier 0 or 1: r with y = s' r, s' being s (tier 0) or s k (tier 1, left in s), and the highest s'^2 so far
// in um.
template <int TIER>
__device__ __forceinline__ uint64_t cap_pair(const Cap& cap, uint64_t& s, float& um) {
  uint64_t v, r;
  if constexpr (TIER == 0) {
    v = f2_mul(s, s);
    r = f2_fma(f2_pack(cap.b[3], cap.b[3]), v, f2_pack(cap.b[2], cap.b[2]));
    r = f2_fma(r, v, f2_pack(cap.b[1], cap.b[1]));
    r = f2_fma(r, v, f2_pack(cap.b[0], cap.b[0]));
  } else {
    s = f2_mul(s, f2_pack(cap.k, cap.k));
    v = f2_mul(s, s);
    r = f2_mul(tanh_ratio2(v), f2_pack(cap.log2, cap.log2));
  }
  float v0, v1;
  f2_unpack(v, v0, v1);
  um = max3f(um, v0, v1);
  return r;
}
// Up to which um a tier holds.
__device__ __forceinline__ float cap_limit(const Cap& cap, int tier) { return tier == 0 ? cap.low : tier == 1 ? TANH_HIGH : INFINITY; }
// y of any score.
__device__ __forceinline__ float cap_any(const Cap& cap, float s) { return cap.log2 * tanh_any(s * cap.k); }

// n scores of a row of a block to y, in place; every lane of the warp calls it.  `tier` is what the last block took, `reload`
// fetches the scores again; lanes that do not count have counts = false.  An infinite score goes to +-cap, a NaN stays one.
template <int N, typename F>
__device__ __forceinline__ void cap_scores(const Cap& cap, float (&s)[N], int& tier, bool counts, F&& reload) {
  auto run = [&](auto tier_c) {
    constexpr int T = decltype(tier_c)::value;
    float um[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      uint64_t x = f2_pack(s[c], s[c + 1]);
      const uint64_t r = cap_pair<T>(cap, x, um[(c >> 1) & 3]);
      f2_unpack(f2_mul(x, r), s[c], s[c + 1]);
    }
    return fmaxf(max3f(um[0], um[1], um[2]), um[3]);
  };
#pragma unroll 1
  for (;;) {
    float most;
    if (tier == 0) {
      most = run(Tier<0>());
    } else if (tier == 1) {
      most = run(Tier<1>());
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) s[c] = cap_any(cap, s[c]);
      return;
    }
    if (__all_sync(0xffffffffu, !counts || most <= cap_limit(cap, tier))) return;
    ++tier;
    reload();
  }
}

}  // namespace mesh
