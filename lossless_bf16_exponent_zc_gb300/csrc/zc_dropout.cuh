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

#include <type_traits>

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
    static_assert(V == 4 || V == 8, "a part of a group");
    const uint4 g = group(row, col / 8);
    if constexpr (V == 8) {
      const uint32_t w[4] = {g.x, g.y, g.z, g.w};
      apply<8>(v, w);
    } else {
      const uint32_t w[2] = {col & 4 ? g.z : g.x, col & 4 ? g.w : g.y};
      apply<4>(v, w);
    }
  }
  // Values taken one by one: the bits of a row of `width` columns into shared memory (16-byte aligned,
  // `width` rounded up to whole groups), by the threads `me` of `step`; and one value by them.
  __device__ __forceinline__ void bits_of_row(uint16_t* bits, uint32_t row, uint32_t width, uint32_t me,
                                              uint32_t step) const {
    for (uint32_t c = me; c * 8 < width; c += step) *reinterpret_cast<uint4*>(bits + c * 8) = group(row, c);
  }
  __device__ __forceinline__ float apply(float v, uint16_t bits) const {
    return keeps_low(bits) ? v * factor : 0.f;
  }
};

// 2 W 16-bit values: from value `first` (below 2 W) on of those in `low`, and behind them `high`.
// (Read at their place in shared memory they are 4 words apart from lane to lane, four lanes to a bank:
// 11181 x 3001 bf16 61 us forward and 91 back, this way 58 and 89.)
template <int W>
__device__ __forceinline__ void join_bits(const uint32_t (&low)[W], const uint32_t (&high)[W], uint32_t first,
                                          uint32_t (&bits)[W]) {
  static_assert(W == 2 || W == 4, "first / 2 has log2(W) bits");
  uint32_t w[2 * W];
#pragma unroll
  for (int j = 0; j < W; j++) w[j] = low[j], w[W + j] = high[j];
  if constexpr (W == 4) {
#pragma unroll
    for (int j = 0; j < 6; j++) w[j] = first & 4 ? w[j + 2] : w[j];
  }
#pragma unroll
  for (int j = 0; j <= W; j++) w[j] = first & 2 ? w[j + 1] : w[j];
#pragma unroll
  for (int j = 0; j < W; j++) bits[j] = __funnelshift_r(w[j], w[j + 1], (first & 1) * 16);
}

// The same for a thread's columns of a ring of rows (RowRing, zc_norm.cuh): NV pieces of V, piece me +
// i threads, each starting `lead` columns early, V / 2 words of bits a piece; `threads` is a multiple
// of 32.  No group is drawn twice where that can be helped: a piece of four columns is half a group,
// so of two neighbouring lanes each draws for one of two pieces and they trade halves; and a piece
// that starts early takes the bits of the piece before it from the lane below, through shared memory.
// What lane 0 needs from the warp below it draws itself, the 32 lanes for the next 32 rows at once.
// `smem`: keep_bytes(threads) with SHIFT, 16-byte aligned; a barrier of the warp or the CTA has to lie
// between two rows.
template <int V, int NV, bool SHIFT>
struct KeepColumns {
  static constexpr int W = V / 2;
  using Words = typename std::conditional<V == 8, uint4, uint2>::type;
  KeepRng rng;
  uint32_t me, threads, lead;
  uint32_t turn = 0;
  // Of this warp, for every piece: the lanes' own, and what lies before lane 0's in 32 rows.
  static constexpr int kSlots = 64;
  Words* slots;
  __host__ __device__ static constexpr int keep_bytes(int threads) {
    return SHIFT ? threads / 32 * kSlots * NV * static_cast<int>(sizeof(Words)) : 0;
  }
  __device__ __forceinline__ KeepColumns(const Dropout& d, uint32_t me_, uint32_t threads_, uint32_t lead_, void* smem)
      : rng(d), me(me_), threads(threads_), lead(lead_), slots(static_cast<Words*>(smem) + (me_ / 32) * (kSlots * NV)) {}

  // What lies before lane 0's pieces, for 32 rows.  Inlined it would take the registers that the rounds'
  // keys stay in.
  __device__ __noinline__ static void draw_before(KeepRng rng, uint32_t row, uint32_t step, uint32_t me,
                                                  uint32_t threads, Words* slots) {
    const uint32_t lane = lane_id();
    for (int i = 0; i < NV; i++) {
      const uint32_t piece = me - lane + i * threads - 1;  // of 8 or 4 columns; it may lie before the row
      const uint4 g = rng.group(row + lane * step, V == 8 ? piece : piece / 2);
      if constexpr (V == 8)
        slots[i * kSlots + 32 + lane] = g;
      else
        slots[i * kSlots + 32 + lane] = make_uint2(g.z, g.w);  // a half before an even piece is a second one
    }
  }

  // Draws the bits of row `row`, to be followed by row + step.
  __device__ __forceinline__ void draw(uint32_t row, uint32_t step, uint32_t (&bits)[NV][W]) {
    const uint32_t lane = lane_id();
    if constexpr (V == 8) {
      uint4 g[NV];
      uint32_t rows[NV], at[NV];
#pragma unroll
      for (int i = 0; i < NV; i++) rows[i] = row, at[i] = me + i * threads;
      rng.template groups<NV>(rows, at, g);
#pragma unroll
      for (int i = 0; i < NV; i++) bits[i][0] = g[i].x, bits[i][1] = g[i].y, bits[i][2] = g[i].z, bits[i][3] = g[i].w;
    } else {
      static_assert(V == 4 && NV % 2 == 0, "pairs of pieces");
      const bool odd = lane & 1;
      uint4 g[NV / 2];
      uint32_t rows[NV / 2], at[NV / 2];
#pragma unroll
      for (int i = 0; i < NV; i += 2) rows[i / 2] = row, at[i / 2] = (me + (odd ? i + 1 : i) * threads) / 2;
      rng.template groups<NV / 2>(rows, at, g);
#pragma unroll
      for (int i = 0; i < NV; i += 2) {
        const uint4 w = g[i / 2];
        const uint32_t a = __shfl_xor_sync(kFull, odd ? w.x : w.z, 1), b = __shfl_xor_sync(kFull, odd ? w.y : w.w, 1);
        bits[i][0] = odd ? a : w.x, bits[i][1] = odd ? b : w.y;
        bits[i + 1][0] = odd ? w.z : a, bits[i + 1][1] = odd ? w.w : b;
      }
    }
    if constexpr (SHIFT) {
      if (lead == 0) return;
      if (turn == 0) {
        draw_before(rng, row, step, me, threads, slots);
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < NV; i++) {
        if constexpr (V == 8)
          slots[i * kSlots + lane] = make_uint4(bits[i][0], bits[i][1], bits[i][2], bits[i][3]);
        else
          slots[i * kSlots + lane] = make_uint2(bits[i][0], bits[i][1]);
      }
      __syncwarp();
      const Words* before = slots + (lane ? lane - 1 : 32 + turn);
      turn = (turn + 1) & 31;
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const Words low = before[i * kSlots];
        if constexpr (V == 8) {
          const uint32_t w[4] = {low.x, low.y, low.z, low.w};
          join_bits<4>(w, bits[i], V - lead, bits[i]);
        } else {
          const uint32_t w[2] = {low.x, low.y};
          join_bits<2>(w, bits[i], V - lead, bits[i]);
        }
      }
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
