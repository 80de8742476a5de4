// zc_layer_norm.cu -- layer norm, by itself and behind a block whose output is dropped out and added
// to the residual stream in the same pass (the gradient is in zc_layer_norm_bwd.cu).
//
//   x' = a x + D(y),   m = mean(x'),  r = 1 / sqrt(mean((x' - m)^2) + eps),   h = (x' - m) r w + b
//
// One pass: a row is read once and everything else happens on chip.  h is taken from x' before its
// rounding to the stored type, so each output is rounded once.  The mean is taken before the squares
// of what differs from it, so that a large mean costs no bits.
//
// Bound by memory where rows are whole 16-byte pieces: 16384 x 4096 bf16 behind a dropped-out branch 92.5 us
// (86% of the copy's rate), fp32 162 (98%), 8192 x 8192 bf16 85 (94%), the norm alone 48 (83%).  Off 16 bytes
// by instructions: 21916 x 1531 bf16 with dropout 70 us (56%), without 52; fp32 10958 x 1531 50 (80%).  8 rows
// of 4096: 2.1 us.
#include "zc_layer_norm.cuh"

namespace zc {

namespace {

// Rows held in registers, NV pieces a thread: by a warp (WARP), or by a CTA.  The CTA's form has no row on
// its way while it computes (4096 x 16384 bf16 with dropout 141 us, 56% of the copy's rate) and off 16 bytes
// takes values one by one (4096 x 8191 223 us): it is for what the ring does not hold.
template <typename T, int V, int NV, bool WARP, bool BRANCH, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(LayerNormParams p) {
  constexpr bool kBits = DROP && V == 1;  // values one by one: a row's bits lie in shared memory
  __shared__ float red[2][32];
  __shared__ __align__(16) uint16_t bits_of[kBits ? NV * THREADS : 8];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  uint16_t* bits = bits_of + (kBits && WARP ? warp * (NV * 32) : 0);
  const uint32_t pieces = p.hidden / V;
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const uint64_t rows_a_turn = WARP ? static_cast<uint64_t>(gridDim.x) * kNormWarps : gridDim.x;
  auto row_sum = [&](float v, int turn) {
    if (WARP) return warp_sum_f32(v);
    float s[1] = {v};
    block_sum_f32<1>(s, red[turn]);
    return s[0];
  };
  for (uint64_t t = WARP ? static_cast<uint64_t>(blockIdx.x) * kNormWarps + warp : blockIdx.x; t < p.tokens;
       t += rows_a_turn) {
    float n[NV][V], sum = 0.f;
    if constexpr (kBits) {
      if (WARP) __syncwarp();  // the row before has been read (a CTA's sums lie in between)
      KeepRng(p.drop).bits_of_row(bits, static_cast<uint32_t>(t), p.hidden, me, step);
      if (WARP)
        __syncwarp();
      else
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * step;
      const uint64_t at = static_cast<uint64_t>(c) * V;
#pragma unroll
      for (int j = 0; j < V; j++) n[i][j] = 0.f;
      if (c >= pieces) continue;
      Piece<T, V>::load(static_cast<const T*>(p.x) + t * p.x_stride + at).get(n[i]);
      if (BRANCH) {
        float y[V];
        Piece<T, V>::load(static_cast<const T*>(p.y) + t * p.y_stride + at).get(y);
        if constexpr (kBits)
          y[0] = KeepRng(p.drop).apply(y[0], bits[c]);
        else if constexpr (DROP)
          KeepRng(p.drop).template apply<V>(y, static_cast<uint32_t>(t), c * V);
#pragma unroll
        for (int j = 0; j < V; j++) n[i][j] = fmaf(p.residual_scale, n[i][j], y[j]);
        Piece<T, V> out;
        out.set(n[i]);
        out.store(static_cast<T*>(p.x_new) + t * p.hidden + at);
      }
#pragma unroll
      for (int j = 0; j < V; j++) sum += n[i][j];
    }
    const float mean = row_sum(sum, 0) * inv_d;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int j = 0; j < V; j++) {
        n[i][j] -= mean;
        if (me + i * step < pieces) sum = fmaf(n[i][j], n[i][j], sum);
      }
    const float root = rsqrtf(row_sum(sum, 1) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * step;
      const uint64_t at = static_cast<uint64_t>(c) * V;
      if (c >= pieces) continue;
      float w[V], b[V], h[V];
      load_params<T, V>(p.weight, p.params_f32, at, w);
#pragma unroll
      for (int j = 0; j < V; j++) b[j] = 0.f;
      if (p.bias) load_params<T, V>(p.bias, p.params_f32, at, b);
#pragma unroll
      for (int j = 0; j < V; j++) h[j] = fmaf(n[i][j] * root, w[j], b[j]);
      Piece<T, V> out;
      out.set(h);
      out.store(static_cast<T*>(p.h) + t * p.hidden + at);
    }
    if (p.stats && me == 0) *reinterpret_cast<float2*>(p.stats + 2 * t) = make_float2(mean, root);
  }
}

// The ring shape: rows walker, walker + walkers, ... stream through the shared memory of a CTA.  A
// warp takes its columns' sum and their squares about their own mean; between warps, squares about
// the row's mean are those plus (columns) (the warp's mean - the row's)^2.  So no squares of a mean
// are ever subtracted, and a row costs one barrier.  4096 columns of 16 bits take two CTAs an SM of 256
// threads, which wait for shared memory (55% of the issue slots busy).
template <typename T, int V, int C, bool SHIFT, bool BRANCH, bool DROP>
__global__ void __launch_bounds__(kNormRingThreads, C == 8 ? 2 : 1) layer_norm_ring_kernel(LayerNormParams p) {
  constexpr int P = C / 2, kStages = kLayerStages<C, BRANCH>;
  using Ring = RowRing<T, V, C, BRANCH ? 2 : 1, kStages, SHIFT>;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float2 red[2][16];
  pdl_begin();
  const uint64_t walker = blockIdx.x, walkers = gridDim.x;
  const T *x_at = static_cast<const T*>(p.x), *y_at = static_cast<const T*>(p.y);
  const uint32_t lead =
      SHIFT ? (reinterpret_cast<uintptr_t>(x_at + walker * p.x_stride) & 15) / static_cast<uint32_t>(sizeof(T)) : 0;
  const Ring ring{ring_smem, threadIdx.x, blockDim.x, SHIFT ? (lead + p.hidden + V - 1) / V : p.hidden / V, 0, lead,
                  p.hidden};
#pragma unroll
  for (int i = 0; i < (BRANCH ? 2 : 1); i++) ring.clear(i, false);
  const float inv_d = 1.f / static_cast<float>(p.hidden);
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
  float2 w[P], b[P];
  ring.params(p.weight, p.params_f32, 0, w);
#pragma unroll
  for (int i = 0; i < P; i++) b[i] = splat(0.f);
  if (p.bias) ring.params(p.bias, p.params_f32, 0, b);
  const InRow<V, C, SHIFT, Ring> in_row(ring);
  // This warp's columns of the row, and those of warp lane & 15.
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const float own = static_cast<float>(__reduce_add_sync(kFull, __popc(in_row.bits)));
  if (threadIdx.x < 16) red[0][threadIdx.x] = red[1][threadIdx.x] = make_float2(0.f, 0.f);
  __syncthreads();
  if (lane == 0) red[0][warp].x = own;
  __syncthreads();
  const float columns = red[0][lane & 15].x;
  const float inv_own = own > 0.f ? 1.f / own : 0.f, inv_columns = columns > 0.f ? 1.f / columns : 0.f;
  __syncthreads();
  if (threadIdx.x < 16) red[0][threadIdx.x] = make_float2(0.f, 0.f);
  __syncthreads();
  ColumnsOf<V, C / V, SHIFT, DROP> keep(p.drop, threadIdx.x, blockDim.x, lead, ring_smem + Ring::bytes(blockDim.x));
  int stage = 0, turn = 0;
  for (uint64_t t = walker; t < p.tokens; t += walkers) {
    float2 x[P];
    cp_async_wait<kStages - 1>();  // a thread reads what it has copied itself
    ring.cut(stage);
    ring.get(stage, 0, x_at, x);
    if (BRANCH) {
      float2 y[P];
      ring.get(stage, 1, y_at, y);
      issue(stage);
      if constexpr (DROP) {
        uint32_t bits[C / V][V / 2];
        keep.draw(static_cast<uint32_t>(t), static_cast<uint32_t>(walkers), bits);
        keep.apply(y, bits);
      }
      const float2 a = splat(p.residual_scale);
#pragma unroll
      for (int i = 0; i < P; i++) x[i] = fma2(a, x[i], y[i]);
      ring.put(ring.start(static_cast<T*>(p.x_new), t, p.hidden), x);
    } else {
      issue(stage);
    }
    float2 s = splat(0.f), c[P];
#pragma unroll
    for (int i = 0; i < P; i++) s = add2(s, x[i]);
    const float sum = warp_sum_f32(s.x + s.y);
#pragma unroll
    for (int i = 0; i < P; i++) c[i] = add2(x[i], splat(-sum * inv_own));
    in_row.keep(c);
    s = splat(0.f);
#pragma unroll
    for (int i = 0; i < P; i++) s = fma2(c[i], c[i], s);
    const float squares = warp_sum_f32(s.x + s.y);
    if (lane == 0) red[turn][warp] = make_float2(sum, squares);
    __syncthreads();
    const float2 of_warp = red[turn][lane & 15];
    turn ^= 1;
    const float mean = half_warp_sum_f32(of_warp.x) * inv_d, off = of_warp.x * inv_columns - mean;
    const float root = rsqrtf(half_warp_sum_f32(fmaf(columns * off, off, of_warp.y)) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < P; i++) x[i] = fma2(mul2(add2(x[i], splat(-mean)), splat(root)), w[i], b[i]);
    ring.put(ring.start(static_cast<T*>(p.h), t, p.hidden), x);
    if (p.stats && threadIdx.x == 0) *reinterpret_cast<float2*>(p.stats + 2 * t) = make_float2(mean, root);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

template <typename T, int V, int NV, bool WARP, int THREADS>
cudaError_t run_shape(LayerNormParams& p, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const void* fn = nullptr;
  if (p.drop.rng)
    fn = reinterpret_cast<const void*>(layer_norm_kernel<T, V, NV, WARP, true, true, THREADS>);
  else if (p.y)
    fn = reinterpret_cast<const void*>(layer_norm_kernel<T, V, NV, WARP, true, false, THREADS>);
  else
    fn = reinterpret_cast<const void*>(layer_norm_kernel<T, V, NV, WARP, false, false, THREADS>);
  const uint64_t units = WARP ? (p.tokens + kNormWarps - 1) / kNormWarps : p.tokens;
  const uint64_t most = static_cast<uint64_t>(dev.sm_count) * 2048 / static_cast<uint64_t>(threads);
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(units < most ? units : most)), dim3(threads), 0, stream, args,
                       false);
}

template <typename T, int C, bool SHIFT, bool BRANCH, bool DROP>
cudaError_t run_ring(LayerNormParams& p, int threads, uint64_t period, cudaStream_t stream, const DeviceInfo& dev) {
  static RingPrep prep;
  constexpr int V = kPieceOf<T>;
  const int smem = static_cast<int>(RowRing<T, V, C, BRANCH ? 2 : 1, kLayerStages<C, BRANCH>>::bytes(threads)) +
                   ColumnsOf<V, C / V, SHIFT, DROP>::keep_bytes(threads);
  const void* fn = reinterpret_cast<const void*>(layer_norm_ring_kernel<T, V, C, SHIFT, BRANCH, DROP>);
  static_assert(kLayerStages<C, BRANCH> * (BRANCH ? 2 : 1) * kNormRingThreads * C * sizeof(T) +
                        ColumnsOf<V, C / V, SHIFT, DROP>::keep_bytes(kNormRingThreads) <=
                    kNormRingSmem,
                "a CTA's shared memory");
  int fit = 0;
  cudaError_t e = prepare_ring(prep, fn, threads, smem, dev, 1, &fit);
  if (e != cudaSuccess) return e;
  uint64_t walkers = static_cast<uint64_t>(fit);
  if (walkers > period) walkers -= walkers % period;
  if (p.tokens < walkers) walkers = p.tokens;
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(walkers)), dim3(threads), smem, stream, args, false);
}

// Runs the ring with C columns a thread if it holds such rows.
template <typename T, int C, bool SHIFT>
bool run_ring(LayerNormParams& p, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e, uint64_t period = 1) {
  const int threads = static_cast<int>((p.hidden + (SHIFT ? kPieceOf<T> - 1 : 0) + C * 32 - 1) / (C * 32) * 32);
  if (threads > kNormRingThreads) return false;
  if (!p.y) {
    *e = run_ring<T, C, SHIFT, false, false>(p, threads, period, stream, dev);
    return true;
  }
  if constexpr (C == 8 && SHIFT) {
    return false;  // never asked for (below)
  } else {
    *e = p.drop.rng ? run_ring<T, C, SHIFT, true, true>(p, threads, period, stream, dev)
                    : run_ring<T, C, SHIFT, true, false>(p, threads, period, stream, dev);
    return true;
  }
}

template <typename T, bool SHIFT>
bool run_ring(LayerNormParams& p, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e, uint64_t period = 1) {
  if constexpr (sizeof(T) == 4) {
    // 8 columns a thread of wide fp32 rows, where a CTA of them is large enough to draw beside its copies (4096 x
    // 4096 with dropout 45 us, with 16 columns 48; 2331 x 1531 alone 8.2, 8.8), but 16 otherwise (16384 x 1024 with
    // dropout 47 us, with 8 51; off 16 bytes 43577 x 385 50, 76; 8188 x 2049 48, 64; 4111 x 4081 50, 61).
    if (p.y ? !SHIFT && p.hidden > 2048 : p.hidden > 1024)
      if (run_ring<T, 8, SHIFT>(p, stream, dev, e, period)) return true;
  }
  return run_ring<T, kLayerWideCols, SHIFT>(p, stream, dev, e, period);
}

template <typename T, int V>
cudaError_t run_width(LayerNormParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint32_t d = p.hidden;
  constexpr int kWarp = kNormWarps * 32;
  // A warp holds up to 256 values (65536 x 256 bf16 with dropout 29 us, by the ring 37; from 512 on the
  // ring's 49 us beat a warp's 51, and 16384 x 1024 24 beat 36).
  if (d <= 256) return run_shape<T, V, 8 / V, true, kWarp>(p, kWarp, stream, dev);
  cudaError_t e;
  if constexpr (V > 1) {
    if (run_ring<T, false>(p, stream, dev, &e)) return e;
  } else {
    RowPlaces rows;
    rows.add(p.x, p.x_stride * sizeof(T));
    rows.add(p.y, p.y_stride * sizeof(T));
    rows.add(p.x_new, static_cast<uint64_t>(d) * sizeof(T));
    rows.add(p.h, static_cast<uint64_t>(d) * sizeof(T));
    if (rows.alike && run_ring<T, true>(p, stream, dev, &e, rows.period())) return e;
  }
  // Wider still, or rows that start elsewhere in one matrix than in another: a CTA holds a row in
  // registers.
  if constexpr (V == 1) {
    if (d <= 4096) return run_shape<T, V, 8, false, 512>(p, static_cast<int>((d + 255) / 256 * 32), stream, dev);
  }
  return run_shape<T, V, 16 / V, false, 1024>(p, static_cast<int>((d + 511) / 512 * 32), stream, dev);
}

template <typename T>
cudaError_t run_typed(LayerNormParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? run_width<T, kPieceOf<T>>(p, stream, dev) : run_width<T, 1>(p, stream, dev);
}
}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& params, int dtype, bool vec, cudaStream_t stream,
                              const DeviceInfo& dev) {
  if (params.tokens == 0) return cudaSuccess;
  LayerNormParams p = params;
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return run_typed<__half>(p, vec, stream, dev);
    default: return run_typed<float>(p, vec, stream, dev);
  }
}

}  // namespace zc
