// zc_layer_norm.cuh -- what the layer norms' forward and backward kernels share.
#pragma once

#include "zc_dropout.cuh"
#include "zc_norm.cuh"

namespace zc {

// The ring's shapes.  A thread has 16 columns of a row of 16-bit values (16384 x 4096 bf16 with dropout
// 92.5 us forward and 111 back, 8 in twice the threads 6 to 7% more), or 8 where the launches' rules find
// them faster.
constexpr int kLayerWideCols = 16;
// Stages, forward and back: more of them move no more bytes a second, for reads and writes share the
// memory's bus (forward, 16 columns: 4 stages 96 us, 3 95, 2 91 to 94; without a branch 48, 48, 49.5;
// fp32 4 stages 168 us, 3 192; back 4 stages 111 us, 3 110, 5 126).
template <int C, bool BRANCH>
constexpr int kLayerStages = C == 8 ? 4 : BRANCH ? 2 : 3;
template <typename T, int C>
constexpr int kLayerBwdStages = sizeof(T) == 4 && C == 16 ? 2 : 3;

// Which of a thread's columns lie in the row; a warp whose columns all do skips the test.
template <int V, int C, bool SHIFT, typename Ring>
struct InRow {
  uint32_t bits = 0;
  __device__ __forceinline__ explicit InRow(const Ring& r) {
#pragma unroll
    for (int i = 0; i < C / V; i++)
#pragma unroll
      for (int j = 0; j < V; j++) {
        const uint32_t c = r.me + i * r.threads;
        if (SHIFT ? c * V + j - r.lead < r.width : c < r.pieces) bits |= 1u << (i * V + j);
      }
  }
  __device__ __forceinline__ void keep(float2 (&v)[C / 2]) const {
    if (bits == (C == 32 ? kFull : (1u << (C & 31)) - 1u)) return;
#pragma unroll
    for (int i = 0; i < C / 2; i++) {
      if (!(bits >> (2 * i) & 1)) v[i].x = 0.f;
      if (!(bits >> (2 * i + 1) & 1)) v[i].y = 0.f;
    }
  }
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// The sum over 16 lanes, the same 16 values lying in both halves of the warp.
__device__ __forceinline__ float half_warp_sum_f32(float v) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// Sums of two values over a CTA of up to 16 warps: half of each warp takes one of them.  `red` holds 32
// floats, those of absent warps zero; two sums in a row need two.
__device__ __forceinline__ void cta_sum_pair(float& a, float& b, float* red) {
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const bool up = lane & 16;
  float v = (up ? b : a) + __shfl_xor_sync(kFull, up ? a : b, 16);
  v = half_warp_sum_f32(v);
  if ((lane & 15) == 0) red[lane + warp] = v;
  __syncthreads();
  v = half_warp_sum_f32(red[lane]);
  const float other = __shfl_xor_sync(kFull, v, 16);
  a = up ? other : v;
  b = up ? v : other;
}

// In place of a dropout's columns where there is none.
struct NoColumns {
  __host__ __device__ static constexpr int keep_bytes(int) { return 0; }
  __device__ __forceinline__ NoColumns(const Dropout&, uint32_t, uint32_t, uint32_t, void*) {}
};
template <int V, int NV, bool SHIFT, bool DROP>
using ColumnsOf = typename std::conditional<DROP, KeepColumns<V, NV, SHIFT>, NoColumns>::type;

}  // namespace zc
