// zc_layer.cuh -- device building blocks of the operators around an expert-parallel layer
// (zc_moe.cu, zc_norm.cu) and next to it: values of three types moved in 16-byte pieces or one at a time, computed
// in fp32, and sums over a warp or a CTA whose order is fixed (the same inputs give the same bits).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "zc_device.cuh"

namespace zc {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// fp32 -> T, round to nearest even: the one rounding of a result.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V values of T as they lie in memory: one 16-byte piece (V = 16 / sizeof(T)) or a single value (V
// = 1, for widths, strides and addresses that 16 bytes do not divide).
template <typename T, int V>
struct Piece;

template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ static Piece load(const T* p) { return Piece{*p}; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ static Piece zero() { return Piece{from_f32<T>(0.f)}; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32<T>(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
};

template <>
struct Piece<float, 4> {
  uint4 v;
  __device__ __forceinline__ static Piece load(const float* p) { return Piece{*reinterpret_cast<const uint4*>(p)}; }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ static Piece zero() { return Piece{make_uint4(0u, 0u, 0u, 0u)}; }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ __forceinline__ void set(const float (&f)[4]) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
struct Piece<T, 8> {
  uint4 v;
  __device__ __forceinline__ static Piece load(const T* p) { return Piece{*reinterpret_cast<const uint4*>(p)}; }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ static Piece zero() { return Piece{make_uint4(0u, 0u, 0u, 0u)}; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    unpack2(v.x, f[0], f[1], T());
    unpack2(v.y, f[2], f[3], T());
    unpack2(v.z, f[4], f[5], T());
    unpack2(v.w, f[6], f[7], T());
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    v = make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
  }
};

// Values of T in a 16-byte piece.
template <typename T>
constexpr int kPieceOf = 16 / static_cast<int>(sizeof(T));

// The 16 bytes from byte `off` (0 .. 15, a multiple of T's size) of two neighbouring pieces on: values
// at any address are read as the aligned pieces that hold them, shifted together.  A piece that holds
// at least one value of the caller's is never where its memory cannot be; neighbouring threads ask
// for the same pieces, so the second comes from the L1 cache.
template <typename T>
__device__ __forceinline__ uint4 shift_pieces(uint4 lo, uint4 hi, uint32_t off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; i++) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; i++) w[i] = w[i + 1];
  }
  if (sizeof(T) == 2 && (off & 2)) {
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stores those of a piece's values, the first of them number `first` of the row, that lie in it.
template <typename T>
__device__ __forceinline__ void store_part(T* p, Piece<T, kPieceOf<T>> v, uint32_t first, uint32_t width) {
  const uint32_t w[4] = {v.v.x, v.v.y, v.v.z, v.v.w};
#pragma unroll
  for (uint32_t j = 0; j < kPieceOf<T>; j++) {
    if (first + j >= width) continue;
    if (sizeof(T) == 4)
      reinterpret_cast<uint32_t*>(p)[j] = w[j & 3];
    else
      reinterpret_cast<uint16_t*>(p)[j] = static_cast<uint16_t>(w[j / 2 & 3] >> (j & 1) * 16);
  }
}

// Pairs of neighbouring pieces that a row of `width` values can touch wherever it starts, the first
// with nothing before its second.
template <typename T>
__host__ __device__ constexpr uint32_t any_pairs(uint32_t width) {
  return (width + 2 * (kPieceOf<T> - 1)) / kPieceOf<T> + 1;
}

// True if the kPieceOf<T> values from `first` (taken modulo 2^32) on all lie in a row of `width`.
template <typename T>
__device__ __forceinline__ bool whole_piece(uint32_t first, uint32_t width) {
  return width >= kPieceOf<T> && first <= width - kPieceOf<T>;
}

// How a row of `width` values that is written at p falls into aligned 16-byte pieces: `head` values
// before the first piece, `body` pieces, and the rest.  Work on the row is cut into units: the
// pieces, then the values outside them one by one, so that no thread has several of those to take
// in turn; at most any_units(width) of them.
template <typename T>
struct RowCut {
  uint32_t head, body;
  __device__ __forceinline__ RowCut(const T* p, uint32_t width) {
    constexpr uint32_t kV = kPieceOf<T>;
    head = static_cast<uint32_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
    head = head < width ? head : width;
    body = (width - head) / kV;
  }
  // Unit u's first value, and how many it has: a piece's, 1, or 0 where the row has no such unit.
  __device__ __forceinline__ uint32_t unit(uint32_t u, uint32_t width, uint32_t* first) const {
    constexpr uint32_t kV = kPieceOf<T>;
    if (u < body) {
      *first = head + u * kV;
      return kV;
    }
    const uint32_t e = u - body;
    *first = e < head ? e : body * kV + e;
    return *first < width ? 1 : 0;
  }
};
template <typename T>
__host__ __device__ constexpr uint32_t any_units(uint32_t width) { return width / kPieceOf<T> + 2 * (kPieceOf<T> - 1); }

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ float warp_max_f32(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

// 1 / (1 + exp(-l)), each step rounded as the plain expression's (a correctly rounded reciprocal is
// the quotient).
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(__fadd_rn(1.f, expf(-l))); }

// Lane l's N values of a row, N l .. N l + N - 1; minus infinity beyond the width.  VEC: they are
// whole 4-, 8- or 16-byte pieces.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_row(const T* row, uint32_t width, float (&v)[N]) {
  const uint32_t first = lane_id() * N;
  if (VEC && N * sizeof(T) >= 4) {
    constexpr int kBytes = N * static_cast<int>(sizeof(T));
    constexpr int kPart = kBytes >= 16 ? 16 : kBytes;  // bytes of a piece
    constexpr int kOf = kPart / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < N; i += kOf) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (first + i < width) {
        const T* src = row + first + i;
        if (kPart == 16) {
          const uint4 q = *reinterpret_cast<const uint4*>(src);
          w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else if (kPart == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(src);
          w[0] = q.x, w[1] = q.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
#pragma unroll
      for (int j = 0; j < kOf; j++) {
        float f;
        if constexpr (sizeof(T) == 4) {
          f = __uint_as_float(w[j & 3]);
        } else {
          float lo, hi;
          unpack2(w[(j / 2) & 3], lo, hi, T());
          f = j & 1 ? hi : lo;
        }
        v[i + j] = first + i < width ? f : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) v[j] = first + j < width ? to_f32<T>(row[first + j]) : -INFINITY;
  }
}

// Division of 32-bit numbers below 2^31 by a divisor that the host knows: the quotient is the upper
// half of n * ceil(2^(31 + bits) / d), shifted, bits = ceil(log2 d) (Granlund and Montgomery, 1994).
struct Divisor {
  uint32_t d, mul, shift;
  __host__ explicit Divisor(uint32_t divisor) : d(divisor) {
    uint32_t bits = 0;
    while (bits < 31 && (1u << bits) < d) bits++;
    shift = bits ? bits - 1 : 0;
    mul = bits ? static_cast<uint32_t>(((1ull << (31 + bits)) + d - 1) / d) : 0;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
};

// The largest of the warp's values that are not NaN.
__device__ __forceinline__ float warp_max_of(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Thread-block clusters: the barrier of all threads of the cluster in its two halves (release,
// acquire), and a store to the same variable in the shared memory of the cluster's CTA `cta`.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void st_shared_of_cta(uint32_t* var, uint32_t cta, uint32_t v) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(
          smem_u32(var)),
      "r"(cta), "r"(v)
      : "memory");
}

// The same variable of the cluster's CTA `cta`.
__device__ __forceinline__ uint32_t ld_shared_of_cta(const uint32_t* var, uint32_t cta) {
  uint32_t v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(smem_u32(var)), "r"(cta)
               : "memory");
  return v;
}

// Sums of N values over a CTA of whole warps, every thread getting all of them.  `red` holds N x 32
// floats; a caller that sums again before a __syncthreads of its own passes another buffer.
template <int N>
__device__ __forceinline__ void block_sum_f32(float (&v)[N], float* red) {
  const uint32_t warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = lane_id();
#pragma unroll
  for (int i = 0; i < N; i++) v[i] = warp_sum_f32(v[i]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; i++) red[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; i++) v[i] = warp_sum_f32(lane < warps ? red[i * 32 + lane] : 0.f);
}

// As block_sum_f32 for 2 or 4 values with fewer shuffles.  Halving the lanes' groups, every lane
// keeps half of the values and gives the others to its partner, until the lanes of group g (of 32 /
// N lanes) hold value g; the rest is a tree inside the group.  The CTA's partial sums are added the
// same way.  `red`: N x kSumSlots floats, 16-byte aligned, those of absent warps zero (the caller
// clears them all before the first use, with a barrier of the CTA or the cluster in between,
// whatever the instance: the slots of a warp are cleared by others); as above, two sums in a row
// need two buffers.  CLUSTER: over all `ctas` CTAs of the cluster, this one being `rank`; every CTA
// leaves its partial sums in all of them (a sum of two barriers, the CTA's and the cluster's, would
// wait twice).  kSumSlots: 16 warps each of up to 4 CTAs, or 32 of one.
constexpr int kSumSlots = 64;
template <int N, bool CLUSTER = false>
__device__ __forceinline__ void block_sum_shared(float (&v)[N], float* red, uint32_t rank = 0, uint32_t ctas = 1) {
  static_assert(N == 2 || N == 4, "lane groups of 16 or 8");
  constexpr uint32_t kGroup = 32 / N;
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  float s[N];
#pragma unroll
  for (int i = 0; i < N; i++) s[i] = v[i];
  int d = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < n; i++) {
      const float give = up ? s[i] : s[i + n];
      s[i] = (up ? s[i + n] : s[i]) + __shfl_xor_sync(kFull, give, d);
    }
  }
#pragma unroll
  for (; d >= 1; d /= 2) s[0] += __shfl_xor_sync(kFull, s[0], d);
  float* slot = red + (lane / kGroup) * kSumSlots + warp;
  if constexpr (CLUSTER) {
    if ((lane & (kGroup - 1)) == 0)
      for (uint32_t c = 0; c < ctas; c++)
        st_shared_of_cta(reinterpret_cast<uint32_t*>(slot + 16 * rank), c, __float_as_uint(s[0]));
    cluster_arrive();
    cluster_wait();
  } else {
    if ((lane & (kGroup - 1)) == 0) *slot = s[0];
    __syncthreads();
  }
  // slots of a lane: all 64 of a cluster, or the first 32
  constexpr uint32_t kOf = (CLUSTER ? kSumSlots : 32) / kGroup;
  const float* part = red + (lane / kGroup) * kSumSlots + (lane & (kGroup - 1)) * kOf;
  float sum = 0.f;
  if constexpr (kOf == 2) {
    const float2 a = *reinterpret_cast<const float2*>(part);
    sum = a.x + a.y;
  } else {
#pragma unroll
    for (uint32_t i = 0; i < kOf; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(part + i);
      sum += (a.x + a.y) + (a.z + a.w);
    }
  }
#pragma unroll
  for (int i = kGroup / 2; i >= 1; i /= 2) sum += __shfl_xor_sync(kFull, sum, i);
#pragma unroll
  for (int i = 0; i < N; i++) v[i] = __shfl_sync(kFull, sum, i * kGroup);
}

// 4-byte asynchronous copy, both addresses 4-byte aligned.
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace zc
