// zc_norm.cu -- the norms before and after a block, with the block's gate and residual scale,
// forward (the gradient is in zc_norm_bwd.cu).
//
//   x' = a x + g * (y r(y) w),   h = x' r(x') w2,   r(z) = 1 / sqrt(mean(z^2) + eps)
//
// One pass: a row of y and x is read once, both sums of squares are taken on chip, and x' and the
// next block's input h are written.  h is the norm of x' before its rounding to the stored type, so
// each output is rounded once.  Bound by memory, 4 values moved per 11 operations: 16384 x 4096
// bf16, 0.54 GB, 87 us, 93% of the measured copy's rate (with a CTA per row and no copies ahead of
// it 133; with one barrier a row instead of two, as in the gradient, 93).  Rows off 16 bytes, 4081
// wide, 100 us as the pieces that cover them, 168 value by value.
#include "zc_norm.cuh"

namespace zc {

namespace {

// Rows held in registers, NV pieces a thread: by a warp (WARP), or the widest by a CTA.
template <typename T, int V, int NV, bool WARP, bool BRANCH, bool NEXT, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(NormParams p) {
  __shared__ float red[2][32];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const uint32_t pieces = p.hidden / V;
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const uint64_t rows_a_turn = WARP ? static_cast<uint64_t>(gridDim.x) * kNormWarps : gridDim.x;
  int turn = 0;
  auto row_sum = [&](float v) {
    if (WARP) return warp_sum_f32(v);
    float s[1] = {v};
    block_sum_f32<1>(s, red[turn]);
    turn ^= 1;
    return s[0];
  };
  for (uint64_t t = WARP ? static_cast<uint64_t>(blockIdx.x) * kNormWarps + warp : blockIdx.x; t < p.tokens;
       t += rows_a_turn) {
    Piece<T, V> y[NV], x[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * step;
      const uint64_t at = static_cast<uint64_t>(c) * V;
      y[i] = x[i] = Piece<T, V>::zero();
      if (c < pieces) {
        if (BRANCH) y[i] = Piece<T, V>::load(static_cast<const T*>(p.y) + t * p.y_stride + at);
        x[i] = Piece<T, V>::load(static_cast<const T*>(p.x) + t * p.x_stride + at);
      }
    }
    float n[NV][V];  // the new x
    if (BRANCH) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; i++) {
        float f[V];
        y[i].get(f);
#pragma unroll
        for (int j = 0; j < V; j++) sum = fmaf(f[j], f[j], sum);
      }
      const float r = rsqrtf(row_sum(sum) * inv_d + p.eps);
      const uint64_t gate_row = p.gate ? t / p.gate_tokens : 0;
      const float gate_one = p.gate && !p.gate_wide ? load_param<T>(p.gate, p.params_f32, gate_row) : 1.f;
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t c = me + i * step;
        const uint64_t at = static_cast<uint64_t>(c) * V;
        float f[V], w[V], g[V], o[V];
        y[i].get(f);
        x[i].get(o);
#pragma unroll
        for (int j = 0; j < V; j++) w[j] = 0.f, g[j] = gate_one;
        if (c < pieces) {
          load_params<T, V>(p.weight, p.params_f32, at, w);
          if (p.gate && p.gate_wide) load_params<T, V>(p.gate, p.params_f32, gate_row * p.hidden + at, g);
        }
#pragma unroll
        for (int j = 0; j < V; j++) n[i][j] = fmaf(g[j], f[j] * r * w[j], p.residual_scale * o[j]);
        if (c < pieces) {
          Piece<T, V> out;
          out.set(n[i]);
          out.store(static_cast<T*>(p.x_new) + t * p.hidden + at);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; i++) x[i].get(n[i]);
    }
    if (NEXT) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) sum = fmaf(n[i][j], n[i][j], sum);
      const float r = rsqrtf(row_sum(sum) * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t c = me + i * step;
        const uint64_t at = static_cast<uint64_t>(c) * V;
        if (c >= pieces) continue;
        float w[V], h[V];
        load_params<T, V>(p.next_weight, p.params_f32, at, w);
#pragma unroll
        for (int j = 0; j < V; j++) h[j] = n[i][j] * r * w[j];
        Piece<T, V> out;
        out.set(h);
        out.store(static_cast<T*>(p.h) + t * p.hidden + at);
      }
    }
  }
}

// Columns of a thread and stages of the ring: 8 columns, and 16 for rows that 8 of each of 512
// threads do not hold.
constexpr int kFwdCols = 8, kFwdWideCols = 16;
template <int C>
constexpr int kFwdStages = C == kFwdCols ? 4 : 3;

// The ring shape: rows walker, walker + walkers, ... stream through the shared memory of a CTA or a
// cluster of two.
template <typename T, int V, int C, int CTAS, bool SHIFT, bool BRANCH, bool NEXT>
__global__ void __launch_bounds__(kNormRingThreads, C == kFwdCols ? 2 : 1) norm_ring_kernel(NormParams p) {
  constexpr int P = C / 2, kStages = kFwdStages<C>;
  using Ring = RowRing<T, V, C, BRANCH ? 2 : 1, kStages, SHIFT>;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ __align__(16) float red[2][2 * kSumSlots];
  pdl_allow_dependents();
  for (uint32_t i = threadIdx.x; i < 4 * kSumSlots; i += blockDim.x) red[0][i] = 0.f;
  if (CTAS > 1) {  // every CTA's sums are cleared before another writes there
    cluster_arrive();
    cluster_wait();
  }
  pdl_wait();
  const uint32_t rank = CTAS > 1 ? cluster_rank() : 0, part = blockDim.x * C;
  const uint32_t width = CTAS > 1 ? min(part, p.hidden - rank * part) : p.hidden;
  const uint64_t walker = blockIdx.x / CTAS, walkers = gridDim.x / CTAS;
  const T* row0 = static_cast<const T*>(p.x) + walker * p.x_stride;
  const uint32_t lead = SHIFT ? (reinterpret_cast<uintptr_t>(row0) & 15) / static_cast<uint32_t>(sizeof(T)) : 0;
  const Ring ring{ring_smem, threadIdx.x, blockDim.x, SHIFT ? (lead + width + V - 1) / V : width / V, rank * part, lead,
                  width};
#pragma unroll
  for (int i = 0; i < (BRANCH ? 2 : 1); i++) ring.clear(i, false);
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const bool wide = BRANCH && p.gate && p.gate_wide, narrow = BRANCH && p.gate && !p.gate_wide;
  const T *x_at = static_cast<const T*>(p.x), *y_at = static_cast<const T*>(p.y);
  uint64_t ahead = walker;
  auto issue = [&](int stage) {
    if (ahead < p.tokens) {
      ring.copy(stage, 0, ring.start(x_at, ahead, p.x_stride));
      if (BRANCH) ring.copy(stage, 1, ring.start(y_at, ahead, p.y_stride));
      ahead += walkers;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; s++) issue(s);
  float2 w[P], w2[P], k[P];
  if (BRANCH) ring.params(p.weight, p.params_f32, 0, w);
  if (NEXT) ring.params(p.next_weight, p.params_f32, 0, w2);
#pragma unroll
  for (int i = 0; i < P; i++) k[i] = splat(1.f);
  uint64_t gate_row = ~0ull;  // the gate row that k holds
  cp_async_wait<kStages - 1>();
  __syncthreads();
  int stage = 0, turn = 0;
  for (uint64_t t = walker; t < p.tokens; t += walkers) {
    float2 x[P];
    float sums[2];
    ring.cut(stage);
    ring.get(stage, 0, x_at + t * p.x_stride + ring.first, x);
    if (BRANCH) {
      float2 y[P], yy = splat(0.f);
      ring.get(stage, 1, y_at + t * p.y_stride + ring.first, y);
#pragma unroll
      for (int i = 0; i < P; i++) yy = fma2(y[i], y[i], yy);
      sums[0] = yy.x + yy.y;
      sums[1] = 0.f;
      cp_async_wait<kStages - 2>();  // the next row, which the barrier below shows to all
      block_sum_shared<2, (CTAS > 1)>(sums, red[turn], rank, CTAS);
      turn ^= 1;
      issue(stage);
      const float2 r = splat(rsqrtf(sums[0] * inv_d + p.eps)), a = splat(p.residual_scale);
      if (wide && t / p.gate_tokens != gate_row) {
        gate_row = t / p.gate_tokens;
        ring.params(p.gate, p.params_f32, gate_row * p.hidden, k);
      } else if (narrow) {
        const float one = load_param<T>(p.gate, p.params_f32, t / p.gate_tokens);
#pragma unroll
        for (int i = 0; i < P; i++) k[i] = splat(one);
      }
#pragma unroll
      for (int i = 0; i < P; i++) x[i] = fma2(k[i], mul2(mul2(y[i], r), w[i]), mul2(a, x[i]));
      ring.put(ring.start(static_cast<T*>(p.x_new), t, p.hidden), x);
    }
    if (NEXT) {
      float2 xx = splat(0.f);
#pragma unroll
      for (int i = 0; i < P; i++) xx = fma2(x[i], x[i], xx);
      sums[0] = xx.x + xx.y;
      sums[1] = 0.f;
      if (!BRANCH) cp_async_wait<kStages - 2>();
      block_sum_shared<2, (CTAS > 1)>(sums, red[turn], rank, CTAS);
      turn ^= 1;
      if (!BRANCH) issue(stage);
      const float2 r = splat(rsqrtf(sums[0] * inv_d + p.eps));
#pragma unroll
      for (int i = 0; i < P; i++) x[i] = mul2(mul2(x[i], r), w2[i]);
      ring.put(ring.start(static_cast<T*>(p.h), t, p.hidden), x);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

template <typename T, int V, int NV, bool WARP, int THREADS>
cudaError_t run_shape(NormParams& p, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const void* fn = nullptr;
  if (p.y && p.next_weight)
    fn = reinterpret_cast<const void*>(norm_kernel<T, V, NV, WARP, true, true, THREADS>);
  else if (p.y)
    fn = reinterpret_cast<const void*>(norm_kernel<T, V, NV, WARP, true, false, THREADS>);
  else
    fn = reinterpret_cast<const void*>(norm_kernel<T, V, NV, WARP, false, true, THREADS>);
  const uint64_t units = WARP ? (p.tokens + kNormWarps - 1) / kNormWarps : p.tokens;
  const uint64_t most = static_cast<uint64_t>(dev.sm_count) * 2048 / static_cast<uint64_t>(threads);
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(units < most ? units : most)), dim3(threads), 0, stream, args,
                       false);
}

template <typename T, int V, int C, int CTAS, bool SHIFT, bool BRANCH, bool NEXT>
cudaError_t run_ring(NormParams& p, int threads, uint64_t period, cudaStream_t stream, const DeviceInfo& dev) {
  static RingPrep prep;
  const int smem = static_cast<int>(RowRing<T, V, C, BRANCH ? 2 : 1, kFwdStages<C>>::bytes(threads));
  const void* fn = reinterpret_cast<const void*>(norm_ring_kernel<T, V, C, CTAS, SHIFT, BRANCH, NEXT>);
  int fit = 0;
  cudaError_t e = prepare_ring(prep, fn, threads, smem, dev, CTAS, &fit);
  if (e != cudaSuccess) return e;
  uint64_t walkers = static_cast<uint64_t>(fit);
  if (walkers > period) walkers -= walkers % period;
  if (p.tokens < walkers) walkers = p.tokens;
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(walkers) * CTAS), dim3(threads), smem, stream, args, false, CTAS);
}

// Runs the ring with C columns a thread and CTAS CTAs a row if it holds such rows.
template <typename T, int V, int C, int CTAS, bool SHIFT = false>
bool run_ring(NormParams& p, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e, uint64_t period = 1) {
  constexpr uint32_t kAll = CTAS * C * 32;
  const int threads = static_cast<int>((p.hidden + (SHIFT ? V - 1 : 0) + kAll - 1) / kAll * 32);
  if (threads > kNormRingThreads || RowRing<T, V, C, 2, kFwdStages<C>>::bytes(threads) > kNormRingSmem) return false;
  if (p.y && p.next_weight)
    *e = run_ring<T, V, C, CTAS, SHIFT, true, true>(p, threads, period, stream, dev);
  else if (p.y)
    *e = run_ring<T, V, C, CTAS, SHIFT, true, false>(p, threads, period, stream, dev);
  else
    *e = run_ring<T, V, C, CTAS, SHIFT, false, true>(p, threads, period, stream, dev);
  return true;
}

template <typename T, int V>
cudaError_t run_width(NormParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint32_t d = p.hidden;
  // A warp holds up to 512 values, in 16-byte pieces 1024 if the rows keep all SMs busy: then it
  // beats the ring's four warps a row (65536 x 1024 bf16 93 us against 100), with few rows it is
  // slower (8 x 1024 3.5 us against 2.2).
  constexpr int kWarp = kNormWarps * 32;
  if constexpr (V > 1) {
    if (d <= 256) return run_shape<T, V, 8 / V, true, kWarp>(p, kWarp, stream, dev);
    if (d <= 512) return run_shape<T, V, 16 / V, true, kWarp>(p, kWarp, stream, dev);
    if (d <= 1024 && p.tokens >= 16ull * static_cast<uint64_t>(dev.sm_count))
      return run_shape<T, V, 32 / V, true, kWarp>(p, kWarp, stream, dev);
  } else {
    if (d <= 256) return run_shape<T, V, 8, true, kWarp>(p, kWarp, stream, dev);
    if (d <= 512) return run_shape<T, V, 16, true, kWarp>(p, kWarp, stream, dev);
  }
  cudaError_t e;
  if constexpr (V == 1) {
    RowPlaces rows;
    rows.add(p.x, p.x_stride * sizeof(T));
    rows.add(p.y, p.y_stride * sizeof(T));
    rows.add(p.x_new, static_cast<uint64_t>(d) * sizeof(T));
    rows.add(p.h, static_cast<uint64_t>(d) * sizeof(T));
    if (rows.alike) {
      if (run_ring<T, kPieceOf<T>, kFwdCols, 1, true>(p, stream, dev, &e, rows.period())) return e;
      if (run_ring<T, kPieceOf<T>, kFwdWideCols, 1, true>(p, stream, dev, &e, rows.period())) return e;
    }
  }
  if (run_ring<T, V, kFwdCols, 1>(p, stream, dev, &e)) return e;
  if (run_ring<T, V, kFwdWideCols, 1>(p, stream, dev, &e)) return e;
  // Wider still: in 16-byte pieces a CTA holds a row in registers (4096 x 16384 bf16 114 us; a
  // cluster of two through the ring 152, its two cluster barriers a row wait too long), otherwise
  // the cluster takes it.
  if constexpr (V > 1) {
    return run_shape<T, V, 16 / V, false, 1024>(p, static_cast<int>((d + 511) / 512 * 32), stream, dev);
  } else {
    if (run_ring<T, V, kFwdWideCols, 2>(p, stream, dev, &e)) return e;
    return cudaErrorInvalidValue;  // wider than ZC_NORM_MAX_HIDDEN
  }
}

template <typename T>
cudaError_t run_typed(NormParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? run_width<T, kPieceOf<T>>(p, stream, dev) : run_width<T, 1>(p, stream, dev);
}

}  // namespace

cudaError_t launch_norm(const NormParams& params, int dtype, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  if (params.tokens == 0) return cudaSuccess;
  NormParams p = params;
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return run_typed<__half>(p, vec, stream, dev);
    default: return run_typed<float>(p, vec, stream, dev);
  }
}

}  // namespace zc
