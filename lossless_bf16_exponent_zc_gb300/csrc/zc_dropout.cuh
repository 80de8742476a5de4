// zc_dropout.cuh -- which values a dropout keeps: a counter-based generator, so that the mask is
// never stored and the gradient draws it again.
//
// Philox-4x32-10 of J. Salmon, M. Moraes, R. Dror and D. Shaw, "Parallel Random Numbers: As Easy as
// 1, 2, 3" (2011), with the constants printed there.  Key: the two words of the seed; counter:
// (column / 8, row, the call's number, the offset).  Its 128 bits are 16 for each of eight columns,
// and a value is kept where they are at least p in steps of 2^-16: half the rounds that 32 bits a
// value would take, for a probability that is exact to 2^-17; the factor makes up for the rounded
// probability, so that the mean stays the same.
#pragma once

#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; i++) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u, b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The generator of a call, its seed and offset read.
struct KeepRng {
  uint32_t k0, k1, call, offset, limit;
  float factor;
  __device__ __forceinline__ explicit KeepRng(const Dropout& d) : call(d.call), limit(d.limit), factor(d.factor) {
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]);
    k0 = static_cast<uint32_t>(seed);
    k1 = static_cast<uint32_t>(seed >> 32);
    offset = static_cast<uint32_t>(d.rng[1]);
  }
  // 16 bits for each of the columns 8 group .. 8 group + 7 of a row.
  __device__ __forceinline__ uint4 group(uint32_t row, uint32_t group) const {
    return philox(make_uint4(group, row, call, offset), k0, k1);
  }
  __device__ __forceinline__ bool keeps(uint32_t bits) const { return bits >= limit; }
  // Column j (0 .. 7) of a group.
  __device__ __forceinline__ bool keeps(uint4 g, uint32_t j) const {
    const uint32_t w = j & 4 ? (j & 2 ? g.w : g.z) : (j & 2 ? g.y : g.x);
    return keeps(j & 1 ? w >> 16 : w & 0xFFFFu);
  }
  // Drops out N values, N even, by their 16 bits each.
  template <int N>
  __device__ __forceinline__ void apply(float (&v)[N], const uint32_t (&bits)[N / 2]) const {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const uint32_t b = j & 1 ? bits[j / 2] >> 16 : bits[j / 2] & 0xFFFFu;
      v[j] = keeps(b) ? v[j] * factor : 0.f;
    }
  }
  // Drops out the V values of a row from column `col` on, a multiple of V.
  template <int V>
  __device__ __forceinline__ void apply(float (&v)[V], uint32_t row, uint32_t col) const {
    static_assert(V == 1 || V == 4 || V == 8, "a part of a group");
    const uint4 g = group(row, col / 8);
    if constexpr (V == 8) {
      const uint32_t w[4] = {g.x, g.y, g.z, g.w};
      apply<8>(v, w);
    } else if constexpr (V == 4) {
      const uint32_t w[2] = {col & 4 ? g.z : g.x, col & 4 ? g.w : g.y};
      apply<4>(v, w);
    } else {
      v[0] = keeps(g, col & 7) ? v[0] * factor : 0.f;
    }
  }
};

}  // namespace zc
