// zc_norm_bwd.cu -- gradient of the norms around a block (zc_norm.cu).
//
// With n = y r(y), n2 = x' r(x') and the incoming gradients dx' and dh, per row
//   u   = dh w2                     G = dx' + r(x') (u - n2 mean(u n2))
//   dx  = a G                       v = G g w
//   dy  = r(y) (v - n mean(v n))
// and over the rows  dw2 = sum dh n2,  dw = sum G g n,  dg = sum G n w.
//
// One pass over the data: a row's four inputs are read once, r(y) and r(x')
// are taken again from them instead of being saved, and a thread adds up the
// parameters' gradients of its own columns in registers over all rows of its
// CTA.  Every CTA then writes its sums to the workspace and a second, small
// kernel adds them in CTA order, so no result depends on timing.
#include "zc_norm.cuh"

namespace zc {

namespace {

constexpr uint32_t kNormMaxCtas = 512;

template <typename T, int V, int NV, bool WARP, bool BRANCH, bool NEXT, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(NormBwdParams p) {
  __shared__ float red[2][3 * 32];
  __shared__ float cols[WARP ? kNormWarpWidth : 1];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const uint32_t pieces = p.hidden / V;
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const bool wide = p.gate && p.gate_wide;
  float* gate_parts = p.parts + static_cast<uint64_t>(p.ctas) * 2 * p.hidden;  // one row per unit, or one value per token
  int turn = 0;
  float sum_w[NV][V], sum_n[NV][V], sum_g[NV][V];
#pragma unroll
  for (int i = 0; i < NV; i++)
#pragma unroll
    for (int j = 0; j < V; j++) sum_w[i][j] = sum_n[i][j] = sum_g[i][j] = 0.f;

  // The CTA's sum of one column array to dst[0 .. hidden), fp32 or, `last`, a
  // finished gradient row in the parameters' type.  In the warp shape the
  // warps add theirs in turn.
  auto flush = [&](float (&s)[NV][V], void* dst, bool last) {
    if (WARP) {
      for (uint32_t w = 0; w < kNormWarps; w++) {
        if (warp == w) {
#pragma unroll
          for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < V; j++) {
              const uint32_t col = (me + i * step) * V + j;
              if (col < p.hidden) cols[col] = (w ? cols[col] : 0.f) + s[i][j];
            }
        }
        __syncthreads();
      }
      for (uint32_t col = threadIdx.x; col < p.hidden; col += kNormWarps * 32) {
        if (last && !p.params_f32)
          static_cast<T*>(dst)[col] = from_f32<T>(cols[col]);
        else
          static_cast<float*>(dst)[col] = cols[col];
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
          const uint32_t col = (me + i * step) * V + j;
          if (col >= p.hidden) continue;
          if (last && !p.params_f32)
            static_cast<T*>(dst)[col] = from_f32<T>(s[i][j]);
          else
            static_cast<float*>(dst)[col] = s[i][j];
        }
    }
  };

  for (uint32_t u = blockIdx.x; u < p.units; u += p.ctas) {
    const uint64_t group = u / p.splits, split = u - static_cast<uint32_t>(group) * p.splits;
    const uint64_t size = wide ? p.gate_tokens : p.tokens;
    const uint64_t first = group * size + size * split / p.splits, last = group * size + size * (split + 1) / p.splits;
    for (uint64_t t = first + (WARP ? warp : 0); t < last; t += WARP ? kNormWarps : 1) {
      Piece<T, V> gx[NV], gh[NV], y[NV], x[NV];
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t c = me + i * step;
        const uint64_t at = static_cast<uint64_t>(c) * V;
        gx[i] = gh[i] = y[i] = x[i] = Piece<T, V>::zero();
        if (c < pieces) {
          if (NEXT) {
            x[i] = Piece<T, V>::load(static_cast<const T*>(p.x_new) + t * p.x_new_stride + at);
            gh[i] = Piece<T, V>::load(static_cast<const T*>(p.dh) + t * p.dh_stride + at);
          }
          if (BRANCH) y[i] = Piece<T, V>::load(static_cast<const T*>(p.y) + t * p.y_stride + at);
          if (p.dx_new) gx[i] = Piece<T, V>::load(static_cast<const T*>(p.dx_new) + t * p.dx_new_stride + at);
        }
      }
      float s[3] = {0.f, 0.f, 0.f};  // sums of x'^2, u x', y^2
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t c = me + i * step;
        float f[V];
        if (NEXT) {
          float h[V], w[V];
          x[i].get(f);
          gh[i].get(h);
#pragma unroll
          for (int j = 0; j < V; j++) w[j] = 0.f;
          if (c < pieces) load_params<T, V>(p.next_weight, p.params_f32, static_cast<uint64_t>(c) * V, w);
#pragma unroll
          for (int j = 0; j < V; j++) {
            s[0] = fmaf(f[j], f[j], s[0]);
            s[1] = fmaf(h[j] * w[j], f[j], s[1]);
          }
        }
        if (BRANCH) {
          y[i].get(f);
#pragma unroll
          for (int j = 0; j < V; j++) s[2] = fmaf(f[j], f[j], s[2]);
        }
      }
      if (WARP) {
#pragma unroll
        for (int i = 0; i < 3; i++) s[i] = warp_sum_f32(s[i]);
      } else {
        block_sum_f32<3>(s, red[turn]);
        turn ^= 1;
      }
      const float r2 = rsqrtf(s[0] * inv_d + p.eps), mean2 = s[1] * r2 * inv_d;  // mean(u n2)
      const float r = rsqrtf(s[2] * inv_d + p.eps);
      const uint64_t gate_row = p.gate ? t / p.gate_tokens : 0;
      const float gate_one = p.gate && !p.gate_wide ? load_param<T>(p.gate, p.params_f32, gate_row) : 1.f;
      float v[NV][V];  // G g w
      float dots[2] = {0.f, 0.f};  // sums of v n and of G n w
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const uint32_t c = me + i * step;
        const uint64_t at = static_cast<uint64_t>(c) * V;
        float g[V];
        gx[i].get(g);
        if (NEXT) {
          float f[V], h[V], w[V];
          x[i].get(f);
          gh[i].get(h);
#pragma unroll
          for (int j = 0; j < V; j++) w[j] = 0.f;
          if (c < pieces) load_params<T, V>(p.next_weight, p.params_f32, at, w);
#pragma unroll
          for (int j = 0; j < V; j++) {
            const float n2 = f[j] * r2;
            g[j] += r2 * (h[j] * w[j] - n2 * mean2);
            sum_n[i][j] = fmaf(h[j], n2, sum_n[i][j]);
          }
        }
        if (c < pieces) {
          float o[V];
#pragma unroll
          for (int j = 0; j < V; j++) o[j] = p.residual_scale * g[j];
          Piece<T, V> out;
          out.set(o);
          out.store(static_cast<T*>(p.dx) + t * p.hidden + at);
        }
        if (BRANCH) {
          float f[V], w[V], k[V];
          y[i].get(f);
#pragma unroll
          for (int j = 0; j < V; j++) w[j] = 0.f, k[j] = gate_one;
          if (c < pieces) {
            load_params<T, V>(p.weight, p.params_f32, at, w);
            if (wide) load_params<T, V>(p.gate, p.params_f32, gate_row * p.hidden + at, k);
          }
#pragma unroll
          for (int j = 0; j < V; j++) {
            const float n = f[j] * r, e = g[j] * n;  // e w: the gate's gradient; e k: the weight's
            sum_w[i][j] = fmaf(e, k[j], sum_w[i][j]);
            if (wide) sum_g[i][j] = fmaf(e, w[j], sum_g[i][j]);
            v[i][j] = g[j] * k[j] * w[j];
            dots[0] = fmaf(v[i][j], n, dots[0]);
            dots[1] = fmaf(e, w[j], dots[1]);
          }
        }
      }
      if (BRANCH) {
        if (WARP) {
          dots[0] = warp_sum_f32(dots[0]);
          dots[1] = warp_sum_f32(dots[1]);
        } else {
          block_sum_f32<2>(dots, red[turn]);
          turn ^= 1;
        }
        const float mean = dots[0] * inv_d;
        if (p.gate && !wide && me == 0) {
          if (p.gate_tokens > 1)
            gate_parts[t] = dots[1];
          else if (p.params_f32)
            static_cast<float*>(p.dgate)[t] = dots[1];
          else
            static_cast<T*>(p.dgate)[t] = from_f32<T>(dots[1]);
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const uint32_t c = me + i * step;
          if (c >= pieces) continue;
          float f[V], o[V];
          y[i].get(f);
#pragma unroll
          for (int j = 0; j < V; j++) o[j] = r * (v[i][j] - f[j] * r * mean);
          Piece<T, V> out;
          out.set(o);
          out.store(static_cast<T*>(p.dy) + t * p.hidden + static_cast<uint64_t>(c) * V);
        }
      }
    }
    if (BRANCH && wide) {
      if (p.splits > 1)
        flush(sum_g, gate_parts + static_cast<uint64_t>(u) * p.hidden, false);
      else
        flush(sum_g, static_cast<uint8_t*>(p.dgate) + group * p.hidden * (p.params_f32 ? 4 : sizeof(T)), true);
#pragma unroll
      for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < V; j++) sum_g[i][j] = 0.f;
    }
  }
  float* mine = p.parts + static_cast<uint64_t>(blockIdx.x) * 2 * p.hidden;
  if (BRANCH) flush(sum_w, mine, false);
  if (NEXT) flush(sum_n, mine + p.hidden, false);
}

// Adds the CTAs' sums, in order: 8 threads per column take an eighth of the
// parts each and thread 0 of the 8 adds theirs.  blockIdx.y: 0 the branch
// weight's gradient, 1 the next weight's, 2 + g gate row g's.
template <typename T>
__global__ void __launch_bounds__(256) norm_parts_kernel(NormBwdParams p) {
  __shared__ float sums[8][32];
  pdl_begin();
  const uint32_t lane = lane_id(), slice = threadIdx.x >> 5, job = blockIdx.y;
  const uint32_t col = blockIdx.x * 32 + lane;
  const float* src;
  uint64_t stride;
  uint32_t count;
  void* dst;
  if (job < 2) {
    src = p.parts + job * p.hidden;
    stride = 2ull * p.hidden;
    count = p.ctas;
    dst = job ? p.dnext_weight : p.dweight;
  } else {
    src = p.parts + (static_cast<uint64_t>(p.ctas) * 2 + static_cast<uint64_t>(job - 2) * p.splits) * p.hidden;
    stride = p.hidden;
    count = p.splits;
    dst = static_cast<uint8_t*>(p.dgate) + static_cast<uint64_t>(job - 2) * p.hidden * (p.params_f32 ? 4 : sizeof(T));
  }
  if (!dst) return;
  float s = 0.f;
  const uint32_t first = count * slice / 8, last = count * (slice + 1) / 8;
  if (col < p.hidden) {
#pragma unroll 8
    for (uint32_t i = first; i < last; i++) s += src[i * stride + col];
  }
  sums[slice][lane] = s;
  __syncthreads();
  if (slice || col >= p.hidden) return;
#pragma unroll
  for (int i = 1; i < 8; i++) s += sums[i][lane];
  if (p.params_f32)
    static_cast<float*>(dst)[col] = s;
  else
    static_cast<T*>(dst)[col] = from_f32<T>(s);
}

// A one-column gate's gradient where several tokens share a gate value: one
// CTA per value.
template <typename T>
__global__ void __launch_bounds__(256) norm_narrow_gate_kernel(NormBwdParams p) {
  __shared__ float red[32];
  pdl_begin();
  const float* src =
      p.parts + static_cast<uint64_t>(p.ctas) * 2 * p.hidden + static_cast<uint64_t>(blockIdx.x) * p.gate_tokens;
  float s[1] = {0.f};
  for (uint64_t i = threadIdx.x; i < p.gate_tokens; i += 256) s[0] += src[i];
  block_sum_f32<1>(s, red);
  if (threadIdx.x) return;
  if (p.params_f32)
    static_cast<float*>(p.dgate)[blockIdx.x] = s[0];
  else
    static_cast<T*>(p.dgate)[blockIdx.x] = from_f32<T>(s[0]);
}

template <typename T, int V, int NV, bool WARP, int THREADS>
cudaError_t run_shape(NormBwdParams& p, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const void* fn = nullptr;
  if (p.y && p.next_weight)
    fn = reinterpret_cast<const void*>(norm_bwd_kernel<T, V, NV, WARP, true, true, THREADS>);
  else if (p.y)
    fn = reinterpret_cast<const void*>(norm_bwd_kernel<T, V, NV, WARP, true, false, THREADS>);
  else
    fn = reinterpret_cast<const void*>(norm_bwd_kernel<T, V, NV, WARP, false, true, THREADS>);
  const bool wide = p.gate && p.gate_wide;
  uint64_t most = 2ull * static_cast<uint64_t>(dev.sm_count);
  if (most > kNormMaxCtas) most = kNormMaxCtas;
  const uint64_t groups = wide ? p.gate_rows : 1, size = wide ? p.gate_tokens : p.tokens;
  const uint64_t turns = WARP ? (size + kNormWarps - 1) / kNormWarps : size;  // most ranges worth making of a group
  uint64_t splits = groups >= most ? 1 : most / groups;
  if (splits > turns) splits = turns;  // no tokens: no ranges, and the sums over none of them are zero
  p.splits = static_cast<uint32_t>(splits);
  const uint64_t units = groups * splits;
  if (units > 0xFFFFFFFFull) return cudaErrorInvalidConfiguration;
  p.units = static_cast<uint32_t>(units);
  p.ctas = static_cast<uint32_t>(units < most ? units : most);
  void* args[] = {&p};
  cudaError_t e = cudaSuccess;
  if (p.ctas) e = launch_kernel(fn, dim3(p.ctas), dim3(threads), 0, stream, args, false);
  if (e != cudaSuccess) return e;
  const uint32_t jobs = 2 + (wide && splits != 1 ? static_cast<uint32_t>(groups) : 0u);
  e = launch_kernel(reinterpret_cast<const void*>(norm_parts_kernel<T>), dim3((p.hidden + 31) / 32, jobs), dim3(256), 0,
                    stream, args, false);
  if (e != cudaSuccess || !p.gate || wide || p.gate_tokens == 1) return e;
  return launch_kernel(reinterpret_cast<const void*>(norm_narrow_gate_kernel<T>),
                       dim3(static_cast<unsigned>(p.gate_rows)), dim3(256), 0, stream, args, false);
}

template <typename T>
cudaError_t run_typed(NormBwdParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  constexpr int V = kPieceOf<T>;
  const uint32_t d = p.hidden;
  auto cta = [&](uint32_t per_thread) { return static_cast<int>((d + per_thread * 32 - 1) / (per_thread * 32) * 32); };
  if (!vec) {
    if (d <= kNormWarpWidth) return run_shape<T, 1, 16, true, kNormWarps * 32>(p, kNormWarps * 32, stream, dev);
    return run_shape<T, 1, 16, false, 1024>(p, cta(16), stream, dev);
  }
  if (d <= 256) return run_shape<T, V, 8 / V, true, kNormWarps * 32>(p, kNormWarps * 32, stream, dev);
  if (d <= kNormWarpWidth) return run_shape<T, V, 16 / V, true, kNormWarps * 32>(p, kNormWarps * 32, stream, dev);
  if (d <= 4096) return run_shape<T, V, 8 / V, false, 512>(p, cta(8), stream, dev);
  return run_shape<T, V, 16 / V, false, 1024>(p, cta(16), stream, dev);
}

}  // namespace

uint64_t norm_workspace_bytes(uint64_t tokens, uint32_t hidden) {
  const uint64_t ctas = tokens < kNormMaxCtas ? tokens : kNormMaxCtas;
  return 4 * (3 * ctas * hidden + tokens);
}

cudaError_t launch_norm_bwd(const NormBwdParams& params, int dtype, bool vec, cudaStream_t stream,
                            const DeviceInfo& dev) {
  NormBwdParams p = params;
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return run_typed<__half>(p, vec, stream, dev);
    default: return run_typed<float>(p, vec, stream, dev);
  }
}

}  // namespace zc
