// zc_norm.cuh -- what the block norms' forward and backward kernels share.
#pragma once

#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

// V parameters (norm weights or a gate row) from column `col` on: in the
// values' type, or in fp32 next to 16-bit values.
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

// Launch shapes.  A row is held by a warp (up to kNormWarpWidth values) or by a CTA, each
// thread keeping 8 or 16 of its values in registers.
constexpr uint32_t kNormWarpWidth = 512;
constexpr int kNormWarps = 8;  // rows of a CTA in the warp shape

}  // namespace zc
