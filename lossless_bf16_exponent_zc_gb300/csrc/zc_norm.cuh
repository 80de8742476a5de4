// zc_norm.cuh -- what the block norms' forward and backward kernels share.
#pragma once

#include <atomic>

#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

// V parameters (norm weights or a gate row) from column `col` on: in the values' type, or in fp32
// next to 16-bit values.
template <typename T, int V>
__device__ __forceinline__ void load_params(const void* base, int is_f32, uint64_t col, float (&f)[V]) {
  if (sizeof(T) == 4 || !is_f32) {
    Piece<T, V>::load(static_cast<const T*>(base) + col).get(f);
  } else {
    const float* src = static_cast<const float*>(base) + col;
    if constexpr (V == 8) {
      const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < V; j++) f[j] = src[j];
    }
  }
}

template <typename T>
__device__ __forceinline__ float load_param(const void* base, int is_f32, uint64_t i) {
  float f[1];
  load_params<T, 1>(base, is_f32, i, f);
  return f[0];
}

// V fp32 values at p, 16-byte aligned where V is a multiple of 4.
template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = p[i];
  }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = f[i];
  }
}

// Launch shapes.  A narrow row is held by a warp.  Wider rows stream through a CTA's shared memory,
// one thread for every 8 or 16 columns, the widest through a cluster's or, in the forward pass, a
// CTA's registers.
constexpr int kNormWarps = 8;  // rows of a CTA in the warp shape
constexpr int kNormRingThreads = 512;
constexpr int kNormRingSmem = 225 * 1024;  // what the ring may take of the 227 KB a CTA can have

// The ring: the next STAGES rows of ARRAYS matrices, copied asynchronously (16 bytes at a time; 4
// where the rows are not so aligned) by the threads of the CTA.  Every thread keeps the same COLS
// columns in every row, in NV pieces of V values: its pieces lie in slots of its own, so shared
// memory is read without bank conflicts and a thread waits for nobody's copies but its own.  Rows
// of 16-bit values at odd addresses (kWords) are copied as the 4-byte words that cover them and
// read value by value, by other threads than copied them; their first and last word may hold a
// neighbour's value, which is not used.
// SHIFT: rows off 16 bytes, but all of a walker's rows in all matrices equally so, by `lead` values.
// They are then copied as the aligned pieces that cover them: a thread's columns start `lead` before
// those of its pieces, and what the first and the last piece hold of other rows becomes zero.
template <typename T, int V, int COLS, int ARRAYS, int STAGES, bool SHIFT = false>
struct RowRing {
  static constexpr int NV = COLS / V;
  static constexpr bool kWords = V == 1 && sizeof(T) == 2;
  uint8_t* smem;
  uint32_t me, threads, pieces;  // this thread among those that share a row (or its part of a cluster's), and its pieces
  uint32_t first = 0;            // column that the part starts at
  uint32_t lead = 0, width = 0;  // SHIFT: values before a row in its first piece, and of the row

  __host__ __device__ static uint32_t region(uint32_t threads) {  // bytes of one row of one matrix
    return kWords ? (threads * NV * 2 + 4 + 15) / 16 * 16 : threads * NV * V * static_cast<uint32_t>(sizeof(T));
  }
  __host__ __device__ static uint32_t bytes(uint32_t threads) { return STAGES * ARRAYS * region(threads); }

  __device__ __forceinline__ uint8_t* at(int stage, int array) const {
    return smem + (stage * ARRAYS + array) * region(threads);
  }
  // Where a thread's walk through a matrix starts: its first column of row t.
  template <typename U>
  __device__ __forceinline__ U* start(U* base, uint64_t t, uint64_t stride) const {
    if (SHIFT) return base + t * stride + me * V - lead;
    return base + t * stride + first + (kWords ? 0 : me * V);
  }
  __device__ __forceinline__ void copy(int stage, int array, const T* row) const {
    uint8_t* to = at(stage, array);
    if (kWords) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(row);
      const uint32_t words = (static_cast<uint32_t>(a & 2) + 2 * pieces + 3) / 4;
      const uint32_t* from = reinterpret_cast<const uint32_t*>(a & ~static_cast<uintptr_t>(3));
      for (uint32_t w = me; w < words; w += threads) cp_async_4(to + 4 * w, from + w);
    } else {
      to += me * V * sizeof(T);
#pragma unroll
      for (int i = 0; i < NV; i++) {
        if (me + i * threads >= pieces) continue;
        if (V == 1)
          cp_async_4(to + i * threads * 4, row + i * threads);
        else if (SHIFT)  // zeros after the row's end
          cp_async_16(to + i * threads * 16, row + i * threads * V,
                      min(16u, (lead + width - (me + i * threads) * V) * static_cast<uint32_t>(sizeof(T))));
        else
          cp_async_16(to + i * threads * 16, row + i * threads * V, 16);
      }
    }
  }
  // Zeroes this thread's slots that no copy ever fills (its columns beyond the width, and all of a
  // matrix that is not there), so that reading them needs no test.
  __device__ __forceinline__ void clear(int array, bool all) const {
    if constexpr (!kWords) {
      for (int stage = 0; stage < STAGES; stage++)
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const uint32_t c = me + i * threads;
          if (all || c >= pieces) Piece<T, V>::zero().store(reinterpret_cast<T*>(at(stage, array)) + c * V);
        }
    }
  }
  // Zeroes what the first piece of a row that has landed holds of the row before.
  __device__ __forceinline__ void cut(int stage) const {
    if constexpr (SHIFT) {
      if (me || !lead) return;
      uint4 head[ARRAYS];
#pragma unroll
      for (int a = 0; a < ARRAYS; a++) head[a] = *reinterpret_cast<const uint4*>(at(stage, a));
      const uint32_t bits = lead * 8 * static_cast<uint32_t>(sizeof(T));  // to clear, in front
      auto mask = [&](uint32_t word) { return bits >= 32 * word + 32 ? 0u : bits > 32 * word ? 0xFFFF0000u : kFull; };
      const uint4 m = make_uint4(mask(0), mask(1), mask(2), mask(3));
#pragma unroll
      for (int a = 0; a < ARRAYS; a++)
        *reinterpret_cast<uint4*>(at(stage, a)) =
            make_uint4(head[a].x & m.x, head[a].y & m.y, head[a].z & m.z, head[a].w & m.w);
    }
  }
  // This thread's columns of a row (its address as given to copy()) as they lie in memory; zeros
  // beyond the width.
  __device__ __forceinline__ void get(int stage, int array, const T* row, Piece<T, V> (&v)[NV]) const {
    const uint8_t* from = at(stage, array) + (kWords ? reinterpret_cast<uintptr_t>(row) & 2 : 0);
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * threads;
      v[i] = Piece<T, V>::zero();
      if (!kWords || c < pieces) v[i] = Piece<T, V>::load(reinterpret_cast<const T*>(from) + c * V);
    }
  }
  // The same straight from the matrix.
  __device__ __forceinline__ void load(const T* row, Piece<T, V> (&v)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; i++) {
      v[i] = Piece<T, V>::zero();
      if (me + i * threads < pieces) v[i] = Piece<T, V>::load(row + (me + i * threads) * V);
    }
  }
  __device__ __forceinline__ static void unpack(const Piece<T, V> (&v)[NV], float2 (&f)[COLS / 2]) {
    float* flat = reinterpret_cast<float*>(f);
#pragma unroll
    for (int i = 0; i < NV; i++) {
      float u[V];
      v[i].get(u);
#pragma unroll
      for (int j = 0; j < V; j++) flat[i * V + j] = u[j];
    }
  }
  __device__ __forceinline__ void get(int stage, int array, const T* row, float2 (&f)[COLS / 2]) const {
    Piece<T, V> v[NV];
    get(stage, array, row, v);
    unpack(v, f);
  }
  // Writes this thread's columns of an output row, from its address by start().
  __device__ __forceinline__ void put(T* row, const float2 (&f)[COLS / 2]) const {
    const float* flat = reinterpret_cast<const float*>(f);
    if (kWords) row += me;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      float v[V];
#pragma unroll
      for (int j = 0; j < V; j++) v[j] = flat[i * V + j];
      Piece<T, V> o;
      o.set(v);
      if constexpr (SHIFT) {
        const uint32_t c = me + i * threads, col = c * V - lead;
        if (whole_piece<T>(col, width)) {
          o.store(row + i * threads * V);
        } else if (c < pieces) {
          store_part<T>(row + i * threads * V, o, col, width);
        }
      } else {
        if (me + i * threads < pieces) o.store(row + i * threads * V);
      }
    }
  }
  // This thread's columns of a parameter row.
  __device__ __forceinline__ void params(const void* base, int is_f32, uint64_t row, float2 (&f)[COLS / 2]) const {
    float* flat = reinterpret_cast<float*>(f);
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * threads;
      float v[V];
#pragma unroll
      for (int j = 0; j < V; j++) v[j] = 0.f;
      if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < V; j++)
          if (c * V + j - lead < width) v[j] = load_param<T>(base, is_f32, row + (c * V + j - lead));
      } else {
        if (c < pieces) load_params<T, V>(base, is_f32, row + first + static_cast<uint64_t>(c) * V, v);
      }
#pragma unroll
      for (int j = 0; j < V; j++) flat[i * V + j] = v[j];
    }
  }
};

// Two fp32 operations of one instruction each.
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// How the rows of a call's matrices lie relative to 16 bytes: alike if they start equally far into a
// piece in all of them, and then rows `period` apart do.
struct RowPlaces {
  bool any = false, alike = true;
  uint64_t base = 0, step = 0;
  void add(const void* p, uint64_t stride_bytes) {
    if (!p) return;
    const uint64_t b = reinterpret_cast<uintptr_t>(p) & 15, s = stride_bytes & 15;
    if (any && (b != base || s != step)) alike = false;
    any = true, base = b, step = s;
  }
  uint64_t period() const { return step ? 16 / (step & (~step + 1)) : 1; }
};

// CTAs of a ring kernel (clusters of them) that the GPU holds, by CTA size (the ring's size follows
// from it); looked up once per device, size and cluster.
struct RingPrep {
  std::atomic<int> fit[kMaxDevices][kNormRingThreads / 32 + 1];
};
cudaError_t prepare_ring(RingPrep& rp, const void* fn, int threads, int smem_bytes, const DeviceInfo& dev, int cluster,
                         int* fit);

}  // namespace zc
