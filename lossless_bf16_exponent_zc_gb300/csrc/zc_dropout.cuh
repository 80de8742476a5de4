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

// N counters at once: they share the rounds' keys.
template <int N>
__device__ __forceinline__ void philox(uint4 (&c)[N], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; i++) {
#pragma unroll
    for (int n = 0; n < N; n++) {
      const uint64_t a = static_cast<uint64_t>(c[n].x) * 0xD2511F53u, b = static_cast<uint64_t>(c[n].z) * 0xCD9E8D57u;
      c[n] = make_uint4(static_cast<uint32_t>(b >> 32) ^ c[n].y ^ k0, static_cast<uint32_t>(b),
                        static_cast<uint32_t>(a >> 32) ^ c[n].w ^ k1, static_cast<uint32_t>(a));
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// The generator of a call, its seed and offset read.  A value's bits, at the top of a word with
// anything behind them, are at least the limit if the word is above `below` (a limit of zero drops
// nothing and needs no generator; one of 2^16 keeps nothing, nothing being above 2^32 - 1).
struct KeepRng {
  uint32_t k0, k1, call, offset, below;
  float factor;
  __device__ __forceinline__ explicit KeepRng(const Dropout& d)
      : call(d.call), below((d.limit << 16) - 1u), factor(d.factor) {
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]);
    k0 = static_cast<uint32_t>(seed);
    k1 = static_cast<uint32_t>(seed >> 32);
    offset = static_cast<uint32_t>(d.rng[1]);
  }
  // 16 bits for each of the columns 8 group .. 8 group + 7 of a row.
  __device__ __forceinline__ uint4 group(uint32_t row, uint32_t group) const {
    uint4 c[1] = {make_uint4(group, row, call, offset)};
    philox<1>(c, k0, k1);
    return c[0];
  }
  // The same for N groups.
  template <int N>
  __device__ __forceinline__ void groups(const uint32_t (&row)[N], const uint32_t (&group)[N], uint4 (&g)[N]) const {
#pragma unroll
    for (int n = 0; n < N; n++) g[n] = make_uint4(group[n], row[n], call, offset);
    philox<N>(g, k0, k1);
  }
  // The first and the second of the two values that share a word.
  __device__ __forceinline__ bool keeps_low(uint32_t w) const { return w << 16 > below; }
  __device__ __forceinline__ bool keeps_high(uint32_t w) const { return w > below; }
  // Column j (0 .. 7) of a group.
  __device__ __forceinline__ bool keeps(uint4 g, uint32_t j) const {
    const uint32_t w = j & 4 ? (j & 2 ? g.w : g.z) : (j & 2 ? g.y : g.x);
    return j & 1 ? keeps_high(w) : keeps_low(w);
  }
  // Drops out N values, N even, by their 16 bits each.
  template <int N>
  __device__ __forceinline__ void apply(float (&v)[N], const uint32_t (&bits)[N / 2]) const {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float2 f = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(factor, factor));
      v[j] = keeps_low(bits[j / 2]) ? f.x : 0.f;
      v[j + 1] = keeps_high(bits[j / 2]) ? f.y : 0.f;
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

// The same for a thread's columns of a ring of rows (RowRing, zc_norm.cuh): NV pieces of V, piece me +
// i threads, each starting `lead` columns early, V / 2 words of bits a piece; `threads` is a multiple
// of 32.  No group is drawn twice where that can be helped: a piece of four columns is half a group,
// so of two neighbouring lanes each draws for one of two pieces and they trade halves; and a piece
// that starts early takes the bits of the piece before it from the lane below.  What lane 0 needs
// from the warp below it draws itself, the 32 lanes for the next 32 rows at once.
template <int V, int NV, bool SHIFT>
struct KeepColumns {
  static constexpr int W = V / 2;
  KeepRng rng;
  uint32_t me, threads, first_group, lead;
  uint32_t edge[SHIFT ? NV : 1][W];  // of the piece before lane 0's, of the lane's row of 32
  uint32_t turn = 0;
  __device__ __forceinline__ KeepColumns(const Dropout& d, uint32_t me_, uint32_t threads_, uint32_t first,
                                         uint32_t lead_)
      : rng(d), me(me_), threads(threads_), first_group(first / 8), lead(lead_) {}

  // Draws the bits of row `row`, to be followed by row + step.
  __device__ __forceinline__ void draw(uint32_t row, uint32_t step, uint32_t (&bits)[NV][W]) {
    const uint32_t lane = lane_id();
    uint32_t own[NV][W];
    if constexpr (V == 8) {
      uint4 g[NV];
      uint32_t rows[NV], at[NV];
#pragma unroll
      for (int i = 0; i < NV; i++) rows[i] = row, at[i] = first_group + me + i * threads;
      rng.template groups<NV>(rows, at, g);
#pragma unroll
      for (int i = 0; i < NV; i++) own[i][0] = g[i].x, own[i][1] = g[i].y, own[i][2] = g[i].z, own[i][3] = g[i].w;
    } else {
      static_assert(V == 4 && NV % 2 == 0, "pairs of pieces");
      const bool odd = lane & 1;
#pragma unroll
      for (int i = 0; i < NV; i += 2) {
        const uint4 g = rng.group(row, first_group + (me + (odd ? i + 1 : i) * threads) / 2);
        const uint32_t a = __shfl_xor_sync(kFull, odd ? g.x : g.z, 1), b = __shfl_xor_sync(kFull, odd ? g.y : g.w, 1);
        own[i][0] = odd ? a : g.x, own[i][1] = odd ? b : g.y;
        own[i + 1][0] = odd ? g.z : a, own[i + 1][1] = odd ? g.w : b;
      }
    }
    if constexpr (!SHIFT) {
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < W; j++) bits[i][j] = own[i][j];
    } else {
      if (turn == 0) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const uint32_t piece = me - lane + i * threads - 1;  // of 8 or 4 columns; it may lie before the row
          const uint4 g = rng.group(row + lane * step, V == 8 ? piece : piece / 2);
          edge[i][0] = V == 8 ? g.x : g.z;  // a half before an even piece is a second one
          edge[i][1] = V == 8 ? g.y : g.w;
          if constexpr (V == 8) edge[i][2] = g.z, edge[i][3] = g.w;
        }
      }
#pragma unroll
      for (int i = 0; i < NV; i++) {
        uint32_t before[W];
#pragma unroll
        for (int j = 0; j < W; j++) {
          before[j] = __shfl_up_sync(kFull, own[i][j], 1);
          const uint32_t e = __shfl_sync(kFull, edge[i][j], turn);
          before[j] = lane ? before[j] : e;
        }
        uint4 w;
        if constexpr (V == 8)  // 0 .. 7 columns early
          w = lead ? shift_pieces<__half>(make_uint4(before[0], before[1], before[2], before[3]),
                                          make_uint4(own[i][0], own[i][1], own[i][2], own[i][3]), 16 - 2 * lead)
                   : make_uint4(own[i][0], own[i][1], own[i][2], own[i][3]);
        else
          w = shift_pieces<__half>(make_uint4(before[0], before[1], own[i][0], own[i][1]), make_uint4(0u, 0u, 0u, 0u),
                                   8 - 2 * lead);
        bits[i][0] = w.x, bits[i][1] = w.y;
        if constexpr (V == 8) bits[i][2] = w.z, bits[i][3] = w.w;
      }
      turn = (turn + 1) & 31;
    }
  }
  // Drops out the thread's columns of a row.
  __device__ __forceinline__ void apply(float2 (&v)[NV * V / 2], const uint32_t (&bits)[NV][W]) const {
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int j = 0; j < W; j++) {
        const float2 f = __fmul2_rn(v[i * W + j], make_float2(rng.factor, rng.factor));
        v[i * W + j] = make_float2(rng.keeps_low(bits[i][j]) ? f.x : 0.f, rng.keeps_high(bits[i][j]) ? f.y : 0.f);
      }
  }
};

}  // namespace zc
