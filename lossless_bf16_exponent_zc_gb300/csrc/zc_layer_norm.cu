// zc_layer_norm.cu -- layer norm, by itself and behind a block whose output is dropped out and added
// to the residual stream in the same pass, and its gradient.
//
//   x' = a x + D(y),   m = mean(x'),  r = 1 / sqrt(mean((x' - m)^2) + eps),   h = (x' - m) r w + b
//
// With n = (x' - m) r and u = dh w the gradient is, per row,
//   G  = dx' + r (u - mean(u) - n mean(u n)),   dx = a G,   dy = D(G)
// and over the rows  dw = sum dh n,  db = sum dh.  D keeps the same values both times, drawn again
// from the counters (zc_dropout.cuh).  The mean is taken before the squares of what differs from
// it, so that a large mean costs no bits; the backward pass gets both from the forward one.
#include "zc_dropout.cuh"
#include "zc_norm.cuh"

namespace zc {

namespace {

// Rows held in registers, NV pieces a thread: by a warp (WARP), or by a CTA.
template <typename T, int V, int NV, bool WARP, bool BRANCH, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(LayerNormParams p) {
  __shared__ float red[2][32];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
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
        if (DROP) KeepRng(p.drop).template apply<V>(y, static_cast<uint32_t>(t), c * V);
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

// Columns of a thread in NV pieces, over all rows of its CTA; the sums of its columns stay in
// registers until the end.
template <typename T, int V, int NV, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_bwd_kernel(LayerNormBwdParams p) {
  __shared__ float red[2][2 * 32];
  pdl_begin();
  const uint32_t me = threadIdx.x, step = blockDim.x, pieces = p.hidden / V;
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < V; j++) dw[i][j] = db[i][j] = 0.f;
  int turn = 0;
  for (uint64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const float2 stats = *reinterpret_cast<const float2*>(p.stats + 2 * t);
    float u[NV][V], n[NV][V], sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * step;
      const uint64_t at = static_cast<uint64_t>(c) * V;
      if (c >= pieces) continue;
      float w[V];
      Piece<T, V>::load(static_cast<const T*>(p.dh) + t * p.dh_stride + at).get(u[i]);
      Piece<T, V>::load(static_cast<const T*>(p.x_new) + t * p.x_new_stride + at).get(n[i]);
      load_params<T, V>(p.weight, p.params_f32, at, w);
#pragma unroll
      for (int j = 0; j < V; j++) {
        n[i][j] = (n[i][j] - stats.x) * stats.y;
        dw[i][j] = fmaf(u[i][j], n[i][j], dw[i][j]);
        db[i][j] += u[i][j];
        u[i][j] *= w[j];
        sums[0] += u[i][j];
        sums[1] = fmaf(u[i][j], n[i][j], sums[1]);
      }
    }
    block_sum_f32<2>(sums, red[turn]);
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = me + i * step;
      const uint64_t at = static_cast<uint64_t>(c) * V;
      if (c >= pieces) continue;
      float g[V], o[V];
#pragma unroll
      for (int j = 0; j < V; j++) g[j] = 0.f;
      if (p.dx_new) Piece<T, V>::load(static_cast<const T*>(p.dx_new) + t * p.dx_new_stride + at).get(g);
#pragma unroll
      for (int j = 0; j < V; j++) {
        g[j] = fmaf(stats.y, u[i][j] - sums[0] * inv_d - n[i][j] * (sums[1] * inv_d), g[j]);
        o[j] = p.residual_scale * g[j];
      }
      Piece<T, V> out;
      out.set(o);
      out.store(static_cast<T*>(p.dx) + t * p.hidden + at);
      if (p.dy) {
        if (DROP) KeepRng(p.drop).template apply<V>(g, static_cast<uint32_t>(t), c * V);
        out.set(g);
        out.store(static_cast<T*>(p.dy) + t * p.hidden + at);
      }
    }
  }
  float* mine = p.parts + static_cast<uint64_t>(blockIdx.x) * 2 * p.hidden;
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < V; j++) {
      const uint32_t c = (me + i * step) * V + j;
      if (c >= pieces * V) continue;
      mine[c] = dw[i][j];
      mine[p.hidden + c] = db[i][j];
    }
}

// Adds the CTAs' sums, in order: the warps take a share of the parts each, a lane a column.
// blockIdx.y: 0 the weight's gradient, 1 the bias's.
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_parts_kernel(LayerNormBwdParams p) {
  __shared__ float sums[32][33];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  void* dst = blockIdx.y ? p.dbias : p.dweight;
  if (!dst) return;
  float s = 0.f;
  const uint32_t first = p.ctas * warp / 32, last = p.ctas * (warp + 1) / 32;
  if (col < p.hidden) {
#pragma unroll 8
    for (uint32_t i = first; i < last; i++) s += p.parts[(2ull * i + blockIdx.y) * p.hidden + col];
  }
  sums[warp][lane] = s;
  __syncthreads();
  s = warp_sum_f32(sums[lane][warp]);
  const uint32_t mine = blockIdx.x * 32 + warp;
  if (lane || mine >= p.hidden) return;
  if (p.params_f32)
    static_cast<float*>(dst)[mine] = s;
  else
    static_cast<T*>(dst)[mine] = from_f32<T>(s);
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

template <typename T, int V>
cudaError_t run_width(LayerNormParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint32_t d = p.hidden;
  constexpr int kWarp = kNormWarps * 32;
  if (d <= 256) return run_shape<T, V, 8 / V, true, kWarp>(p, kWarp, stream, dev);
  if (d <= 512) return run_shape<T, V, 16 / V, true, kWarp>(p, kWarp, stream, dev);
  if (d <= 4096) return run_shape<T, V, 8 / V, false, 512>(p, static_cast<int>((d + 255) / 256 * 32), stream, dev);
  return run_shape<T, V, 16 / V, false, 1024>(p, static_cast<int>((d + 511) / 512 * 32), stream, dev);
}

template <typename T, int V, int NV, int THREADS>
cudaError_t run_shape(LayerNormBwdParams& p, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const void* fn = p.drop.rng ? reinterpret_cast<const void*>(layer_norm_bwd_kernel<T, V, NV, true, THREADS>)
                              : reinterpret_cast<const void*>(layer_norm_bwd_kernel<T, V, NV, false, THREADS>);
  uint64_t ctas = static_cast<uint64_t>(dev.sm_count) * (1024u / static_cast<unsigned>(threads));
  if (ctas > 4ull * static_cast<uint64_t>(dev.sm_count)) ctas = 4ull * static_cast<uint64_t>(dev.sm_count);
  if (ctas > norm_max_walkers(p.hidden)) ctas = norm_max_walkers(p.hidden);
  if (ctas > p.tokens) ctas = p.tokens;
  p.ctas = static_cast<uint32_t>(ctas);
  void* args[] = {&p};
  cudaError_t e = launch_kernel(fn, dim3(p.ctas), dim3(threads), 0, stream, args, false);
  if (e != cudaSuccess) return e;
  return launch_kernel(reinterpret_cast<const void*>(layer_norm_parts_kernel<T>), dim3((p.hidden + 31) / 32, p.dbias ? 2 : 1),
                       dim3(1024), 0, stream, args, false);
}

template <typename T, int V>
cudaError_t run_width(LayerNormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint32_t d = p.hidden;
  if (d <= 4096) return run_shape<T, V, 8 / V, 512>(p, static_cast<int>((d + 255) / 256 * 32), stream, dev);
  return run_shape<T, V, 16 / V, 1024>(p, static_cast<int>((d + 511) / 512 * 32), stream, dev);
}

template <typename T, typename P>
cudaError_t run_typed(P& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? run_width<T, kPieceOf<T>>(p, stream, dev) : run_width<T, 1>(p, stream, dev);
}
template <typename P>
cudaError_t run_dtype(P& p, int dtype, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return run_typed<__half>(p, vec, stream, dev);
    default: return run_typed<float>(p, vec, stream, dev);
  }
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& params, int dtype, bool vec, cudaStream_t stream,
                              const DeviceInfo& dev) {
  if (params.tokens == 0) return cudaSuccess;
  LayerNormParams p = params;
  return run_dtype(p, dtype, vec, stream, dev);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& params, int dtype, bool vec, cudaStream_t stream,
                                  const DeviceInfo& dev) {
  LayerNormBwdParams p = params;
  return run_dtype(p, dtype, vec, stream, dev);
}

}  // namespace zc
