// zc_layer_norm_bwd.cu -- gradient of the layer norms (zc_layer_norm.cu).
//
// With n = (x' - m) r and u = dh w, per row
//   G  = dx' + r (u - mean(u) - n mean(u n)),   dx = a G,   dy = D(G)
// and over the rows  dw = sum dh n,  db = sum dh.  The forward pass has left m and r, so a row takes
// two sums and one barrier.  D keeps what it kept before, drawn again from the counters
// (zc_dropout.cuh).
//
// Bound by memory where rows are whole 16-byte pieces: 16384 x 4096 bf16 with dropout 111 us (90% of the
// copy's rate), without 85 (93%), fp32 with dropout 230 (86%).  Off 16 bytes by the instructions that shift
// pieces and trade the dropout's bits: 21916 x 1531 bf16 with dropout 110 us (45%), without 67 (59%), fp32 10958
// x 1531 61 and 50 (82, 80%).  With few rows the second launch, which adds the CTAs' sums, weighs as much as
// the first: 2331 x 1531 fp32 16 us, 64 x 4096 bf16 6.0.
#include "zc_layer_norm.cuh"

namespace zc {

namespace {

// Columns of a thread in NV pieces, over all rows of its CTA; the sums of its columns stay in
// registers until the end.  For what the ring does not hold (4096 x 16384 bf16 with dropout 211 us, 47% of
// the copy's rate; off 16 bytes, value by value, 4096 x 8191 410).
template <typename T, int V, int NV, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_bwd_kernel(LayerNormBwdParams p) {
  constexpr bool kBits = DROP && V == 1;  // values one by one: a row's bits lie in shared memory
  __shared__ float red[2][2 * 32];
  __shared__ __align__(16) uint16_t bits[kBits ? NV * THREADS : 8];
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
    if constexpr (kBits) {  // read before the next row's sums
      KeepRng(p.drop).bits_of_row(bits, static_cast<uint32_t>(t), p.hidden, me, step);
      __syncthreads();
    }
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
        if constexpr (kBits)
          g[0] = KeepRng(p.drop).apply(g[0], bits[c]);
        else if constexpr (DROP)
          KeepRng(p.drop).template apply<V>(g, static_cast<uint32_t>(t), c * V);
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

// The gradient's ring: three matrices, or two where nothing reaches x' but through h.  4096 columns of 16
// bits take two CTAs an SM of 256 threads, whose 122 registers hold 16 columns' sums, weights and a row.
// PAIR: 80 registers a thread, so that an SM holds two CTAs of up to kLayerPairThreads.
constexpr int kLayerPairThreads = 384;
template <typename T, int V, int C, bool SHIFT, bool DROP, bool PAIR>
__global__ void __launch_bounds__(PAIR ? kLayerPairThreads : kNormRingThreads, PAIR ? 2 : 1)
    layer_norm_bwd_ring_kernel(LayerNormBwdParams p) {
  constexpr int P = C / 2, kStages = kLayerBwdStages<T, C>;
  constexpr int kH = 0, kX = 1, kPast = 2;
  using Ring = RowRing<T, V, C, 3, kStages, SHIFT>;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float red[2][32];
  pdl_begin();
  if (threadIdx.x < 32) red[0][threadIdx.x] = red[1][threadIdx.x] = 0.f;
  __syncthreads();  // a warp's slots are cleared by others
  const uint64_t walker = blockIdx.x, walkers = gridDim.x;
  const T *h_at = static_cast<const T*>(p.dh), *x_at = static_cast<const T*>(p.x_new),
          *past_at = static_cast<const T*>(p.dx_new);
  const uint32_t lead =
      SHIFT ? (reinterpret_cast<uintptr_t>(x_at + walker * p.x_new_stride) & 15) / static_cast<uint32_t>(sizeof(T)) : 0;
  const Ring ring{ring_smem, threadIdx.x, blockDim.x, SHIFT ? (lead + p.hidden + V - 1) / V : p.hidden / V, 0, lead,
                  p.hidden};
#pragma unroll
  for (int i = 0; i < 3; i++) ring.clear(i, i == kPast && !p.dx_new);
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  uint64_t ahead = walker;
  auto issue = [&](int stage) {
    if (ahead < p.tokens) {
      ring.copy(stage, kH, ring.start(h_at, ahead, p.dh_stride));
      ring.copy(stage, kX, ring.start(x_at, ahead, p.x_new_stride));
      if (p.dx_new) ring.copy(stage, kPast, ring.start(past_at, ahead, p.dx_new_stride));
      ahead += walkers;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages; s++) issue(s);
  float2 w[P], dw[P], db[P];
  ring.params(p.weight, p.params_f32, 0, w);
#pragma unroll
  for (int i = 0; i < P; i++) dw[i] = db[i] = splat(0.f);
  const InRow<V, C, SHIFT, Ring> in_row(ring);
  ColumnsOf<V, C / V, SHIFT, DROP> keep(p.drop, threadIdx.x, blockDim.x, lead, ring_smem + Ring::bytes(blockDim.x));
  const float2* stats = reinterpret_cast<const float2*>(p.stats);
  float2 of_row = stats[walker];
  int stage = 0, turn = 0;
  for (uint64_t t = walker; t < p.tokens; t += walkers) {
    const float2 mine = of_row;
    if (t + walkers < p.tokens) of_row = stats[t + walkers];
    float2 u[P], n[P], g[P], a = splat(0.f), b = splat(0.f);
    cp_async_wait<kStages - 1>();
    ring.cut(stage);
    ring.get(stage, kH, h_at, u);
    ring.get(stage, kX, x_at, n);
#pragma unroll
    for (int i = 0; i < P; i++) n[i] = mul2(add2(n[i], splat(-mine.x)), splat(mine.y));
    in_row.keep(n);
#pragma unroll
    for (int i = 0; i < P; i++) {
      dw[i] = fma2(u[i], n[i], dw[i]);
      db[i] = add2(db[i], u[i]);
      u[i] = mul2(u[i], w[i]);
      a = add2(a, u[i]);
      b = fma2(u[i], n[i], b);
    }
    float sum_u = a.x + a.y, sum_un = b.x + b.y;
    ring.get(stage, kPast, past_at, g);
    issue(stage);
    uint32_t bits[C / V][V / 2];
    if constexpr (DROP) keep.draw(static_cast<uint32_t>(t), static_cast<uint32_t>(walkers), bits);
    cta_sum_pair(sum_u, sum_un, red[turn]);
    turn ^= 1;
    const float2 ma = splat(-sum_u * inv_d), mb = splat(-sum_un * inv_d), root = splat(mine.y);
#pragma unroll
    for (int i = 0; i < P; i++)
      g[i] = fma2(root, fma2(n[i], mb, add2(u[i], ma)), g[i]);
    {
      const float2 scale = splat(p.residual_scale);
#pragma unroll
      for (int i = 0; i < P; i++) u[i] = mul2(scale, g[i]);
      ring.put(ring.start(static_cast<T*>(p.dx), t, p.hidden), u);
    }
    if (p.dy) {
      if constexpr (DROP) keep.apply(g, bits);
      ring.put(ring.start(static_cast<T*>(p.dy), t, p.hidden), g);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  float* mine = p.parts + walker * 2 * p.hidden;
  const float *fw = reinterpret_cast<const float*>(dw), *fb = reinterpret_cast<const float*>(db);
#pragma unroll
  for (int i = 0; i < Ring::NV; i++) {
    const uint32_t c = threadIdx.x + i * blockDim.x;
    float ow[V], ob[V];
#pragma unroll
    for (int j = 0; j < V; j++) ow[j] = fw[i * V + j], ob[j] = fb[i * V + j];
    if constexpr (SHIFT) {
#pragma unroll
      for (int j = 0; j < V; j++) {
        const uint32_t col = c * V + j - lead;
        if (col >= p.hidden) continue;
        mine[col] = ow[j];
        mine[p.hidden + col] = ob[j];
      }
    } else if (c < ring.pieces) {
      store_f32<V>(mine + c * V, ow);
      store_f32<V>(mine + p.hidden + c * V, ob);
    }
  }
}

// Narrow rows: every warp walks rows of its own, the next one's loads under way while it computes; a
// CTA adds its warps' sums at the end (65536 x 256 bf16 with dropout 38.6 us, 64% of the copy's rate).
constexpr uint32_t kLayerWarpWidth = 256;
template <typename T, int V, bool DROP>
__global__ void __launch_bounds__(kNormWarps * 32) layer_norm_bwd_warp_kernel(LayerNormBwdParams p) {
  constexpr int NV = 8 / V;
  constexpr bool kBits = DROP && V == 1;  // values one by one: a row's bits lie in shared memory
  __shared__ float tile[kNormWarps][kLayerWarpWidth];
  __shared__ __align__(16) uint16_t bits_of[kNormWarps][kBits ? kLayerWarpWidth : 8];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, pieces = p.hidden / V;
  uint16_t* bits = bits_of[warp];
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const uint64_t walkers = static_cast<uint64_t>(gridDim.x) * kNormWarps;
  float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; i++) {
#pragma unroll
    for (int j = 0; j < V; j++) w[i][j] = dw[i][j] = db[i][j] = 0.f;
    if (lane + i * 32 < pieces) load_params<T, V>(p.weight, p.params_f32, (lane + i * 32) * V, w[i]);
  }
  struct Row {
    Piece<T, V> h[NV], x[NV], past[NV];
    float2 stats;
  };
  auto load = [&](Row& r, uint64_t t) {
    r.stats = reinterpret_cast<const float2*>(p.stats)[t];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = lane + i * 32;
      r.h[i] = r.x[i] = r.past[i] = Piece<T, V>::zero();
      if (c >= pieces) continue;
      r.h[i] = Piece<T, V>::load(static_cast<const T*>(p.dh) + t * p.dh_stride + c * V);
      r.x[i] = Piece<T, V>::load(static_cast<const T*>(p.x_new) + t * p.x_new_stride + c * V);
      if (p.dx_new) r.past[i] = Piece<T, V>::load(static_cast<const T*>(p.dx_new) + t * p.dx_new_stride + c * V);
    }
  };
  uint64_t t = static_cast<uint64_t>(blockIdx.x) * kNormWarps + warp;
  Row row, next;
  if (t < p.tokens) load(row, t);
  for (; t < p.tokens; t += walkers) {
    if (t + walkers < p.tokens) load(next, t + walkers);
    float u[NV][V], n[NV][V], a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      row.h[i].get(u[i]);
      row.x[i].get(n[i]);
#pragma unroll
      for (int j = 0; j < V; j++) {
        n[i][j] = (n[i][j] - row.stats.x) * row.stats.y;  // beyond the width u is zero
        dw[i][j] = fmaf(u[i][j], n[i][j], dw[i][j]);
        db[i][j] += u[i][j];
        u[i][j] *= w[i][j];
        a += u[i][j];
        b = fmaf(u[i][j], n[i][j], b);
      }
    }
    if constexpr (kBits) {
      __syncwarp();  // the row before has been read
      KeepRng(p.drop).bits_of_row(bits, static_cast<uint32_t>(t), p.hidden, lane, 32);
      __syncwarp();
    }
    a = warp_sum_f32(a) * inv_d;
    b = warp_sum_f32(b) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t c = lane + i * 32;
      const uint64_t at = t * p.hidden + c * V;
      float g[V], o[V];
      row.past[i].get(g);
#pragma unroll
      for (int j = 0; j < V; j++) {
        g[j] = fmaf(row.stats.y, u[i][j] - a - n[i][j] * b, g[j]);
        o[j] = p.residual_scale * g[j];
      }
      if (c >= pieces) continue;
      Piece<T, V> out;
      out.set(o);
      out.store(static_cast<T*>(p.dx) + at);
      if (!p.dy) continue;
      if constexpr (kBits)
        g[0] = KeepRng(p.drop).apply(g[0], bits[c]);
      else if constexpr (DROP)
        KeepRng(p.drop).template apply<V>(g, static_cast<uint32_t>(t), c * V);
      out.set(g);
      out.store(static_cast<T*>(p.dy) + at);
    }
    row = next;
  }
  float* mine = p.parts + static_cast<uint64_t>(blockIdx.x) * 2 * p.hidden;
  auto flush = [&](const float (&s)[NV][V], float* dst) {
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int j = 0; j < V; j++)
        if (lane + i * 32 < pieces) tile[warp][(lane + i * 32) * V + j] = s[i][j];
    __syncthreads();
    if (threadIdx.x < p.hidden) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kNormWarps; q++) sum += tile[q][threadIdx.x];
      dst[threadIdx.x] = sum;
    }
    __syncthreads();
  };
  flush(dw, mine);
  flush(db, mine + p.hidden);
}

// Adds the CTAs' sums, in order: COLS columns a CTA, whose warps take a share of the parts each, 32 / COLS
// of them at a time.  blockIdx.y: 0 the weight's gradient, 1 the bias's.
template <typename T, int COLS>
__global__ void __launch_bounds__(1024) layer_norm_parts_kernel(LayerNormBwdParams p) {
  constexpr uint32_t kShares = 1024 / COLS;
  __shared__ float sums[kShares][COLS + 1];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, share = threadIdx.x / COLS, in = threadIdx.x % COLS;
  const uint32_t col = blockIdx.x * COLS + in;
  void* dst = blockIdx.y ? p.dbias : p.dweight;
  if (!dst) return;
  float s = 0.f;
  const uint32_t first = p.ctas * share / kShares, last = p.ctas * (share + 1) / kShares;
  if (col < p.hidden) {
#pragma unroll 8
    for (uint32_t i = first; i < last; i++) s += p.parts[(2ull * i + blockIdx.y) * p.hidden + col];
  }
  sums[share][in] = s;
  __syncthreads();
  const uint32_t mine = blockIdx.x * COLS + warp;
  if (warp >= COLS) return;
  s = 0.f;
#pragma unroll
  for (uint32_t q = 0; q < kShares; q += 32) s += sums[q + lane][warp];
  s = warp_sum_f32(s);
  if (lane || mine >= p.hidden) return;
  if (p.params_f32)
    static_cast<float*>(dst)[mine] = s;
  else
    static_cast<T*>(dst)[mine] = from_f32<T>(s);
}

template <typename T>
cudaError_t add_parts(LayerNormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  void* args[] = {&p};
  // 8 columns a CTA where that makes no more than two of them an SM: with 32 the narrow rows, which have
  // the most parts, leave most SMs idle (4096 x 512 bf16 takes 2.1 us longer, 1024 x 1024 2.8).  Wider rows are
  // as fast with 16 and 32.
  const uint32_t sums = p.dbias ? 2 : 1, eights = (p.hidden + 7) / 8;
  const bool narrow = eights * sums <= 2 * static_cast<uint32_t>(dev.sm_count);
  return launch_kernel(narrow ? reinterpret_cast<const void*>(layer_norm_parts_kernel<T, 8>)
                              : reinterpret_cast<const void*>(layer_norm_parts_kernel<T, 32>),
                       dim3(narrow ? eights : (p.hidden + 31) / 32, sums), dim3(1024), 0, stream, args, false);
}

template <typename T>
cudaError_t run_walkers(LayerNormBwdParams& p, const void* fn, uint64_t most, uint64_t rows_a_cta, int threads, int smem,
                        cudaStream_t stream, const DeviceInfo& dev, uint64_t period = 1) {
  if (most > norm_max_walkers(p.hidden)) most = norm_max_walkers(p.hidden);
  const uint64_t ctas = (p.tokens + rows_a_cta - 1) / rows_a_cta;
  // Of few turns none is for a part of the CTAs alone: fewer sums to add up (1024 x 4096 bf16 with dropout,
  // 256 CTAs instead of 304, 0.9 us less).  Of many that costs more warps than it saves (65536 x 256, 14 turns,
  // 40.4 us, not 38.6).
  const uint64_t turns = (ctas + most - 1) / most;
  if (turns <= 8) most = ((ctas + turns - 1) / turns + period - 1) / period * period;
  p.ctas = static_cast<uint32_t>(ctas < most ? ctas : most);
  void* args[] = {&p};
  cudaError_t e = launch_kernel(fn, dim3(p.ctas), dim3(threads), smem, stream, args, false);
  return e == cudaSuccess ? add_parts<T>(p, stream, dev) : e;
}

template <typename T, int V, int NV, int THREADS>
cudaError_t run_shape(LayerNormBwdParams& p, int threads, cudaStream_t stream, const DeviceInfo& dev) {
  const void* fn = p.drop.rng ? reinterpret_cast<const void*>(layer_norm_bwd_kernel<T, V, NV, true, THREADS>)
                              : reinterpret_cast<const void*>(layer_norm_bwd_kernel<T, V, NV, false, THREADS>);
  const uint64_t most = static_cast<uint64_t>(dev.sm_count) * (threads > 256 ? 1024u / static_cast<unsigned>(threads) : 4u);
  return run_walkers<T>(p, fn, most, 1, threads, 0, stream, dev);
}

template <typename T, int C, bool SHIFT>
bool run_ring(LayerNormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e, uint64_t period = 1) {
  constexpr int V = kPieceOf<T>;
  const int threads = static_cast<int>((p.hidden + (SHIFT ? V - 1 : 0) + C * 32 - 1) / (C * 32) * 32);
  if (threads > kNormRingThreads) return false;
  static RingPrep prep[2];
  const bool drop = p.drop.rng != nullptr;
  const int smem = static_cast<int>(RowRing<T, V, C, 3, kLayerBwdStages<T, C>>::bytes(threads)) +
                   (drop ? KeepColumns<V, C / V, SHIFT>::keep_bytes(threads) : 0);
  const void* fn = drop ? reinterpret_cast<const void*>(layer_norm_bwd_ring_kernel<T, V, C, SHIFT, true, false>)
                        : reinterpret_cast<const void*>(layer_norm_bwd_ring_kernel<T, V, C, SHIFT, false, false>);
  // 8 16-bit columns of more than 256 threads: with more registers an SM holds one such CTA (13102 x 2561 bf16
  // 63 us, one CTA 73, 16 columns a thread 80; with dropout 98, 119, 110).  Smaller CTAs lose by it (87154 x 385
  // 98 us instead of 73, 43633 x 769 72 and 69, with dropout 162 and 125, 115 and 115), and of fp32 shared
  // memory holds no more.
  if constexpr (C == 8 && sizeof(T) == 2) {
    if (threads > 256 && threads <= kLayerPairThreads)
      fn = drop ? reinterpret_cast<const void*>(layer_norm_bwd_ring_kernel<T, V, C, SHIFT, true, true>)
                : reinterpret_cast<const void*>(layer_norm_bwd_ring_kernel<T, V, C, SHIFT, false, true>);
  }
  static_assert(kLayerBwdStages<T, C> * 3 * kNormRingThreads * C * sizeof(T) +
                        KeepColumns<V, C / V, SHIFT>::keep_bytes(kNormRingThreads) <=
                    kNormRingSmem,
                "a CTA's shared memory");
  int fit = 0;
  *e = prepare_ring(prep[drop], fn, threads, smem, dev, 1, &fit);
  if (*e != cudaSuccess) return true;
  uint64_t most = static_cast<uint64_t>(fit);
  if (most > norm_max_walkers(p.hidden)) most = norm_max_walkers(p.hidden);
  if (most > period) most -= most % period;
  *e = run_walkers<T>(p, fn, most, 1, threads, smem, stream, dev, period);
  return true;
}

template <typename T, int V>
cudaError_t run_width(LayerNormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint32_t d = p.hidden;
  cudaError_t e;
  if (d <= kLayerWarpWidth) {
    const void* fn = p.drop.rng ? reinterpret_cast<const void*>(layer_norm_bwd_warp_kernel<T, V, true>)
                                : reinterpret_cast<const void*>(layer_norm_bwd_warp_kernel<T, V, false>);
    return run_walkers<T>(p, fn, 4ull * static_cast<uint64_t>(dev.sm_count), kNormWarps, kNormWarps * 32, 0, stream, dev);
  }
  if constexpr (V > 1) {
    // 8 columns a thread of fp32 rows (10922 x 1536 with dropout 58 us, with 16 67), of narrow 16-bit ones and of
    // few: with dropout 65536 x 512 bf16 59 us, with 16 columns 83, 32768 x 1024 61 and 61, 2331 x 1536 12.6 and
    // 14.8, 64 x 4096 6.0 and 7.4.  16 of the others, which have room for more on their way: 21845 x 1536 61 us,
    // with 8 columns 66, 8192 x 4096 58 and 63.
    if (sizeof(T) == 4 || d <= 1024 || p.tokens <= 16ull * static_cast<uint64_t>(dev.sm_count))
      if (run_ring<T, 8, false>(p, stream, dev, &e)) return e;
    if (run_ring<T, kLayerWideCols, false>(p, stream, dev, &e)) return e;
  } else {
    RowPlaces rows;
    rows.add(p.dh, p.dh_stride * sizeof(T));
    rows.add(p.x_new, p.x_new_stride * sizeof(T));
    rows.add(p.dx_new, p.dx_new_stride * sizeof(T));
    rows.add(p.dx, static_cast<uint64_t>(d) * sizeof(T));
    rows.add(p.dy, static_cast<uint64_t>(d) * sizeof(T));
    if (rows.alike) {
      // 8 columns a thread (21916 x 1531 bf16 67 us, with 16 89; with dropout 113, 127)
      if (run_ring<T, 8, true>(p, stream, dev, &e, rows.period())) return e;
      if (run_ring<T, kLayerWideCols, true>(p, stream, dev, &e, rows.period())) return e;
    }
  }
  if constexpr (V == 1) {
    if (d <= 4096) return run_shape<T, V, 8, 512>(p, static_cast<int>((d + 255) / 256 * 32), stream, dev);
  }
  return run_shape<T, V, 16 / V, 1024>(p, static_cast<int>((d + 511) / 512 * 32), stream, dev);
}

template <typename T>
cudaError_t run_typed(LayerNormBwdParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? run_width<T, kPieceOf<T>>(p, stream, dev) : run_width<T, 1>(p, stream, dev);
}
}  // namespace

cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& params, int dtype, bool vec, cudaStream_t stream,
                                  const DeviceInfo& dev) {
  LayerNormBwdParams p = params;
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return run_typed<__half>(p, vec, stream, dev);
    default: return run_typed<float>(p, vec, stream, dev);
  }
}

}  // namespace zc
