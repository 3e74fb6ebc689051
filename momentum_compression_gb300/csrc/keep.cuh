// Keep bits of the dropout operators: halfword e % 8 of Philox call e / 8,
// its lowest 15 bits compared with T = round(32768 p).  Fifteen bits give
// the probability to 1.5e-5, eight elements a call (half of what 32 bits an
// element cost), and a compare that also fits the packed half-precision
// pipe: as bit patterns, non-negative halves are ordered like whole numbers.
#pragma once

#include <cstdint>

#include "philox.cuh"

namespace ob {

struct Keep {
  PhiloxKeys keys;
  uint32_t off_lo, off_hi;
  uint32_t T;   // drop iff u < T, 0..32768
  float scale;  // 32768 / (32768 - T); 0 if T = 32768
};

// Host: the parameters of a call.
inline Keep make_keep(double p, uint64_t seed, uint64_t offset) {
  Keep k;
  k.keys = philox_keys((uint32_t)seed, (uint32_t)(seed >> 32));
  k.off_lo = (uint32_t)offset;
  k.off_hi = (uint32_t)(offset >> 32);
  k.T = (uint32_t)__builtin_nearbyint(p * 32768.0);
  k.scale = k.T < 32768u ? 32768.0f / (float)(32768u - k.T) : 0.0f;
  return k;
}

// The four words (eight halfwords) of a call.
__device__ __forceinline__ uint4 keep_words(const Keep& k, uint64_t call) {
  return philox4x32_10(make_uint4((uint32_t)call, (uint32_t)(call >> 32), k.off_lo, k.off_hi),
                       k.keys);
}

// The words of N calls, `step` calls apart: N independent chains side by side,
// so that one lane's dependent multiplies overlap.
template <int N>
__device__ __forceinline__ void keep_words_n(const Keep& k, uint64_t call, uint64_t step,
                                             uint4 (&w)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint64_t c = call + n * step;
    w[n] = make_uint4((uint32_t)c, (uint32_t)(c >> 32), k.off_lo, k.off_hi);
  }
#pragma unroll
  for (int r = 0; r < 10; ++r)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint64_t p0 = (uint64_t)0xD2511F53u * w[n].x, p1 = (uint64_t)0xCD9E8D57u * w[n].z;
      w[n] = make_uint4((uint32_t)(p1 >> 32) ^ w[n].y ^ k.keys.k0[r], (uint32_t)p1,
                        (uint32_t)(p0 >> 32) ^ w[n].w ^ k.keys.k1[r], (uint32_t)p0);
    }
}

// Whether element i (0..7) of a call's eight is kept.
__device__ __forceinline__ bool kept(const uint4& w, int i, uint32_t T) {
  const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
  return ((i & 1 ? x >> 16 : x) & 0x7fffu) >= T;
}

// The eight as a byte, bit i for element i.
__device__ __forceinline__ uint32_t keep_byte(const uint4& w, uint32_t T) {
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) b |= (uint32_t)kept(w, i, T) << i;
  return b;
}

}  // namespace ob
