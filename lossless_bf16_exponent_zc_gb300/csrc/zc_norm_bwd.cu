// zc_norm_bwd.cu -- gradient of the norms around a block (zc_norm.cu).
//
// With n = y r(y), n2 = x' r(x') and the incoming gradients dx' and dh, per row
//   u   = dh w2                     G = dx' + r(x') (u - n2 mean(u n2))
//   dx  = a G                       v = G g w
//   dy  = r(y) (v - n mean(v n))
// and over the rows  dw2 = sum dh n2,  dw = sum G g n,  dg = sum G n w.
//
// One pass over the data: a row's four inputs are read once, r(y) and r(x') are taken again from
// them instead of being saved, and a thread adds up the column sums of its own columns in registers
// over all rows of its walker. (The weight's and the gate's gradient share the sum of G n while the
// gate row stays the same.)  Every walker then writes its sums to the workspace and a second, small
// kernel adds them in order, so no result depends on timing.  Bound by memory: 16384 x 4096 bf16,
// 0.81 GB, 124 us, 97% of the measured copy's rate; off 16 bytes it waits a row for the two warps
// that cut its first and last piece (16384 x 4081 bf16 155 us, 173 with a slower cut; with every
// row taken value by value 284).
#include "zc_norm.cuh"

namespace zc {

namespace {

constexpr uint32_t kNormWarpWidth = 256;  // widest row that a warp holds
// Most ranges of rows, and CTAs, whose sums the workspace holds.
__host__ __device__ constexpr uint32_t norm_max_units(uint32_t hidden) {
  return hidden > 2048 ? 608 : hidden > kNormWarpWidth ? 1216 : 4864;
}
constexpr int kBwdStages = 3;

// Columns of a thread in the ring shape: 8, and 16 for 16-bit rows that 8 of each of 512 threads do
// not hold; still wider rows are shared by a cluster of 2 or 4 CTAs.  With 8 the column sums, the
// weights and a row fit the 128 registers of a 512-thread CTA; 16 columns in 256 threads, two CTAs
// an SM, spill registers and take 170 us instead of 130 (16384 x 4096 bf16), and 8 in 64 registers,
// again for two CTAs, 238 us: the ring leaves the L1 cache too small for spilled registers.
constexpr int kBwdCols = 8, kBwdWideCols = 16;

// Rows of a walker (a CTA; a warp in the warp shape), unit after unit: u = its number, number +
// walkers, ...  A unit takes every splits-th row of a gate row's tokens, so that neighbouring
// walkers read neighbouring rows at about the same time.
struct BwdWalk {
  uint32_t u;
  uint64_t t, last;
  __device__ __forceinline__ void open(const NormBwdParams& p) {
    const uint64_t size = p.gate && p.gate_wide ? p.gate_tokens : p.tokens;
    const uint32_t group = u / p.splits;
    t = group * size + (u - group * p.splits);
    last = group * size + size;
  }
  __device__ __forceinline__ bool valid(const NormBwdParams& p) const { return u < p.units; }
  // Moves on by a row; true if that ended the unit.  No unit is empty.
  __device__ __forceinline__ bool next(const NormBwdParams& p) {
    t += p.splits;
    if (t < last) return false;
    u += p.walkers;
    if (u < p.units) open(p);
    return true;
  }
};

// The ring shape.  A row takes two sums over the CTA, of x'^2, u x' and y^2 and then, once G is
// known, of v y.  The second is taken together with the next row's first, so that a row costs one
// barrier: between two barriers the CTA writes the last row's dy, takes this row's G, dx, column
// sums and v y, and the next row's first sums.  The inputs are read from the stage twice rather
// than held, so that the column sums and the weights stay in registers.
template <typename T, int V, int C, bool CLUSTER, bool SHIFT, bool BRANCH, bool NEXT>
__global__ void __launch_bounds__(kNormRingThreads, 1) norm_bwd_ring_kernel(NormBwdParams p) {
  constexpr int P = C / 2;
  constexpr int kGx = 0, kGh = 1, kX = 2, kY = NEXT ? 3 : 1, kArrays = BRANCH && NEXT ? 4 : NEXT ? 3 : 2;
  using Ring = RowRing<T, V, C, kArrays, kBwdStages, SHIFT>;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ __align__(16) float red[2][4 * kSumSlots];
  pdl_allow_dependents();
  for (uint32_t i = threadIdx.x; i < 8 * kSumSlots; i += blockDim.x) red[0][i] = 0.f;
  __syncthreads();  // a warp's slots are cleared by others, and the first sum may be next
  if (CLUSTER) {  // every CTA's sums are cleared before another writes there
    cluster_arrive();
    cluster_wait();
  }
  pdl_wait();
  // this CTA's part of the rows, and who walks them: the CTA or its cluster
  const uint32_t rank = CLUSTER ? cluster_rank() : 0, walker = CLUSTER ? blockIdx.x / p.cluster : blockIdx.x;
  const uint32_t part = blockDim.x * C;
  const uint32_t width = CLUSTER ? min(part, p.hidden - rank * part) : p.hidden;
  BwdWalk ahead{walker, 0, 0}, now{walker, 0, 0};
  ahead.open(p);
  now.open(p);
  const T* row0 = static_cast<const T*>(p.dx) + now.t * p.hidden;
  const uint32_t lead = SHIFT ? (reinterpret_cast<uintptr_t>(row0) & 15) / static_cast<uint32_t>(sizeof(T)) : 0;
  const Ring ring{ring_smem, threadIdx.x, blockDim.x, SHIFT ? (lead + width + V - 1) / V : width / V, rank * part, lead,
                  width};
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const bool wide = BRANCH && p.gate && p.gate_wide, narrow = BRANCH && p.gate && !p.gate_wide;
  const bool past = p.dx_new != nullptr;
  float* gate_parts = p.parts + static_cast<uint64_t>(p.ctas) * 2 * p.hidden;
#pragma unroll
  for (int i = 0; i < kArrays; i++) ring.clear(i, i == kGx && !past);

  // Addresses of the row to copy next and, for rows at odd addresses, of the row being computed.
  const T *gx = nullptr, *gh = nullptr, *x = nullptr, *y = nullptr;
  auto aim = [&](uint64_t t) {
    if (past) gx = ring.start(static_cast<const T*>(p.dx_new), t, p.dx_new_stride);
    if (NEXT) {
      gh = ring.start(static_cast<const T*>(p.dh), t, p.dh_stride);
      x = ring.start(static_cast<const T*>(p.x_new), t, p.x_new_stride);
    }
    if (BRANCH) y = ring.start(static_cast<const T*>(p.y), t, p.y_stride);
  };
  aim(ahead.t);
  auto issue = [&](int stage) {
    if (ahead.valid(p)) {
      if (NEXT) {
        ring.copy(stage, kGh, gh);
        ring.copy(stage, kX, x);
        gh += p.dh_stride * p.splits;
        x += p.x_new_stride * p.splits;
      }
      if (BRANCH) {
        ring.copy(stage, kY, y);
        y += p.y_stride * p.splits;
      }
      if (past) {
        ring.copy(stage, kGx, gx);
        gx += p.dx_new_stride * p.splits;
      }
      if (ahead.next(p) && ahead.valid(p)) aim(ahead.t);
    }
    cp_async_commit();
  };
  // The address of the row at hand, of which only rows at odd addresses need to know.
  auto row_of = [&](const void* base, uint64_t t, uint64_t stride) {
    return Ring::kWords ? static_cast<const T*>(base) + t * stride + ring.first : nullptr;
  };
#pragma unroll
  for (int s = 0; s < kBwdStages; s++) issue(s);

  // w2, and g w of the unit's gate row (w alone under a one-column gate); the sums of dh n2, and of
  // G n over the unit, which give the weight's gradient times g and the gate's times w when the
  // unit ends.
  float2 w2[P], gw[P], sum_n[P], sum_b[P];
  if (NEXT) ring.params(p.next_weight, p.params_f32, 0, w2);
  auto open_unit = [&](uint32_t u) {
    ring.params(p.weight, p.params_f32, 0, gw);
    if (wide) {
      float2 k[P];
      ring.params(p.gate, p.params_f32, (u / p.splits) * static_cast<uint64_t>(p.hidden), k);
#pragma unroll
      for (int i = 0; i < P; i++) gw[i] = mul2(gw[i], k[i]);
    }
#pragma unroll
    for (int i = 0; i < P; i++) sum_b[i] = splat(0.f);
  };
  float* mine = p.parts + static_cast<uint64_t>(walker) * 2 * p.hidden + ring.first;
  auto close_unit = [&](uint32_t u) {
    const float* fb = reinterpret_cast<const float*>(sum_b);
#pragma unroll
    for (int i = 0; i < Ring::NV; i++) {
      const uint32_t c = threadIdx.x + i * blockDim.x;
      if (c >= ring.pieces) continue;
      if constexpr (SHIFT) {  // a walker has one unit only
#pragma unroll
        for (int j = 0; j < V; j++) {
          const uint32_t col = c * V + j - lead;
          if (col >= width) continue;
          const uint64_t at = static_cast<uint64_t>(u) * p.hidden + col;
          float dw = fb[i * V + j];
          if (wide) {
            const float dg = dw * load_param<T>(p.weight, p.params_f32, col);
            dw *= load_param<T>(p.gate, p.params_f32, (u / p.splits) * static_cast<uint64_t>(p.hidden) + col);
            if (p.splits > 1)
              gate_parts[at] = dg;
            else if (p.params_f32)
              static_cast<float*>(p.dgate)[at] = dg;
            else
              static_cast<T*>(p.dgate)[at] = from_f32<T>(dg);
          }
          mine[col] = dw;
        }
        continue;
      }
      float k[V], w[V];
      if (wide) {
        load_params<T, V>(p.gate, p.params_f32, (u / p.splits) * static_cast<uint64_t>(p.hidden) + ring.first + c * V, k);
        load_params<T, V>(p.weight, p.params_f32, ring.first + c * V, w);
      }
      float dw[V], dg[V];
#pragma unroll
      for (int j = 0; j < V; j++) {
        dw[j] = wide ? fb[i * V + j] * k[j] : fb[i * V + j];
        dg[j] = wide ? fb[i * V + j] * w[j] : 0.f;
      }
      if (u != walker) {  // a walker's first unit has its number
        float sum[V];
        load_f32<V>(mine + c * V, sum);
#pragma unroll
        for (int j = 0; j < V; j++) dw[j] += sum[j];
      }
      store_f32<V>(mine + c * V, dw);
      if (!wide) continue;
      const uint64_t at = static_cast<uint64_t>(u) * p.hidden + ring.first + c * V;
      if (p.splits > 1) {
        store_f32<V>(gate_parts + at, dg);
      } else if (p.params_f32) {
#pragma unroll
        for (int j = 0; j < V; j++) static_cast<float*>(p.dgate)[at + j] = dg[j];
      } else {
#pragma unroll
        for (int j = 0; j < V; j++) static_cast<T*>(p.dgate)[at + j] = from_f32<T>(dg[j]);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < P; i++) sum_n[i] = splat(0.f);
  if (BRANCH) open_unit(now.u);

  // Partial sums of row t's x'^2, u x' and y^2.
  auto first_sums = [&](int stage, uint64_t t, float (&sums)[4]) {
    if (NEXT) {
      float2 h[P], v[P], xx = splat(0.f), ux = splat(0.f);
      ring.get(stage, kGh, row_of(p.dh, t, p.dh_stride), h);
      ring.get(stage, kX, row_of(p.x_new, t, p.x_new_stride), v);
#pragma unroll
      for (int i = 0; i < P; i++) {
        xx = fma2(v[i], v[i], xx);
        ux = fma2(mul2(h[i], w2[i]), v[i], ux);
      }
      sums[0] = xx.x + xx.y;
      sums[1] = ux.x + ux.y;
    }
    if (BRANCH) {
      float2 v[P], yy = splat(0.f);
      ring.get(stage, kY, row_of(p.y, t, p.y_stride), v);
#pragma unroll
      for (int i = 0; i < P; i++) yy = fma2(v[i], v[i], yy);
      sums[2] = yy.x + yy.y;
    }
  };

  // Between barriers: `t` is the row whose first sums are known; v (in g), y and the scalars of the
  // row before wait for their last sum.
  float2 g[P];
  // With few columns a thread holds the row's y and refills the stage at once; with many the
  // registers do not allow it, y is read again from its stage, and that is refilled after it.
  constexpr bool kHold = C <= kBwdCols;
  Piece<T, V> y_row[kHold ? Ring::NV : 1];
  int y_stage = 0;
  uint64_t before = ~0ull;
  float root = 0.f, one = 1.f;
  float sums[4] = {0.f, 0.f, 0.f, 0.f};
  auto finish = [&](float vy) {  // dy of the row before
    const float2 m = splat(-(vy * root * inv_d) * root), rr = splat(root * one);
    float2 v[P];
    if constexpr (kHold)
      Ring::unpack(y_row, v);
    else
      ring.get(y_stage, kY, row_of(p.y, before, p.y_stride), v);
#pragma unroll
    for (int i = 0; i < P; i++) v[i] = mul2(rr, fma2(v[i], m, g[i]));
    ring.put(ring.start(static_cast<T*>(p.dy), before, p.hidden), v);
    if (narrow && threadIdx.x == 0 && rank == 0) {
      const float dg = root * vy;  // sum of G n w
      if (p.gate_tokens > 1)
        gate_parts[before] = dg;
      else if (p.params_f32)
        static_cast<float*>(p.dgate)[before] = dg;
      else
        static_cast<T*>(p.dgate)[before] = from_f32<T>(dg);
    }
  };

  int stage = 0, turn = 0;
  cp_async_wait<kBwdStages - 1>();
  if (Ring::kWords) __syncthreads();
  ring.cut(0);
  first_sums(0, now.t, sums);
  block_sum_shared<4, CLUSTER>(sums, red[1], rank, p.cluster);
  while (now.valid(p)) {
    const uint64_t t = now.t;
    if (BRANCH && before != ~0ull) {
      finish(sums[3]);
      if (!kHold) issue(y_stage);
    }
    if (!Ring::kWords || past) {
      ring.get(stage, kGx, row_of(p.dx_new, t, p.dx_new_stride), g);
    } else {
#pragma unroll
      for (int i = 0; i < P; i++) g[i] = splat(0.f);
    }
    if (NEXT) {
      const float r2 = rsqrtf(sums[0] * inv_d + p.eps);
      const float2 rr = splat(r2), m = splat(-(sums[1] * r2 * inv_d) * r2 * r2);  // -r2^2 mean(u n2)
      float2 h[P], v[P];
      ring.get(stage, kGh, row_of(p.dh, t, p.dh_stride), h);
      ring.get(stage, kX, row_of(p.x_new, t, p.x_new_stride), v);
#pragma unroll
      for (int i = 0; i < P; i++) {
        g[i] = fma2(rr, mul2(h[i], w2[i]), fma2(v[i], m, g[i]));
        sum_n[i] = fma2(h[i], mul2(v[i], rr), sum_n[i]);
      }
    }
    {
      float2 o[P];
      const float2 a = splat(p.residual_scale);
#pragma unroll
      for (int i = 0; i < P; i++) o[i] = mul2(a, g[i]);
      ring.put(ring.start(static_cast<T*>(p.dx), t, p.hidden), o);
    }
    sums[3] = 0.f;
    if (BRANCH) {
      root = rsqrtf(sums[2] * inv_d + p.eps);
      one = narrow ? load_param<T>(p.gate, p.params_f32, t / p.gate_tokens) : 1.f;
      const float2 rr = splat(root * one);
      float2 v[P], vy = splat(0.f);
      if constexpr (kHold) {
        ring.get(stage, kY, row_of(p.y, t, p.y_stride), y_row);
        Ring::unpack(y_row, v);
      } else {
        ring.get(stage, kY, row_of(p.y, t, p.y_stride), v);
        y_stage = stage;
      }
#pragma unroll
      for (int i = 0; i < P; i++) {
        sum_b[i] = fma2(g[i], mul2(v[i], rr), sum_b[i]);
        g[i] = mul2(g[i], gw[i]);  // v, but for a one-column gate
        vy = fma2(g[i], v[i], vy);
      }
      sums[3] = vy.x + vy.y;
    }
    const int done = stage;
    if (!Ring::kWords && (kHold || !BRANCH)) issue(done);
    before = t;
    const uint32_t unit = now.u;
    if (now.next(p) && BRANCH) {
      close_unit(unit);
      if (now.valid(p)) open_unit(now.u);
    }
    stage = stage + 1 == kBwdStages ? 0 : stage + 1;
    sums[0] = sums[1] = sums[2] = 0.f;
    if (now.valid(p)) {
      // the next row: all but the copies issued after its own
      cp_async_wait<Ring::kWords || (!kHold && BRANCH) ? kBwdStages - 2 : kBwdStages - 1>();
      if (Ring::kWords) __syncthreads();
      ring.cut(stage);
      first_sums(stage, now.t, sums);
    }
    block_sum_shared<4, CLUSTER>(sums, red[turn], rank, p.cluster);
    turn ^= 1;
    if (Ring::kWords) issue(done);  // now every thread is past its last reading of the row
  }
  if (BRANCH) finish(sums[3]);
  cp_async_wait<0>();
  if (NEXT) {
    const float* fn = reinterpret_cast<const float*>(sum_n);
#pragma unroll
    for (int i = 0; i < Ring::NV; i++) {
      const uint32_t c = threadIdx.x + i * blockDim.x;
      float dn[V];
#pragma unroll
      for (int j = 0; j < V; j++) dn[j] = fn[i * V + j];
      if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < V; j++)
          if (c * V + j - lead < width) mine[p.hidden + (c * V + j - lead)] = dn[j];
      } else {
        if (c < ring.pieces) store_f32<V>(mine + p.hidden + c * V, dn);
      }
    }
  }
}

// The warp shape: every warp walks rows of its own, the next one's loads under way while it
// computes; a CTA adds its warps' sums of the weights' gradients at the end.
template <typename T, int V, bool BRANCH, bool NEXT>
__global__ void __launch_bounds__(kNormWarps * 32, 2) norm_bwd_warp_kernel(NormBwdParams p) {
  constexpr int C = 8, P = C / 2;
  using Cols = RowRing<T, V, C, 1, 1>;
  __shared__ float tile[kNormWarps][kNormWarpWidth];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const Cols cols{nullptr, lane, 32, p.hidden / V};
  const float inv_d = 1.f / static_cast<float>(p.hidden);
  const bool wide = BRANCH && p.gate && p.gate_wide, narrow = BRANCH && p.gate && !p.gate_wide;
  float* gate_parts = p.parts + static_cast<uint64_t>(p.ctas) * 2 * p.hidden;
  float2 w2[P], gw[P], sum_n[P], sum_w[P], sum_b[P];  // as in the ring shape; sum_w over the units
#pragma unroll
  for (int i = 0; i < P; i++) w2[i] = gw[i] = sum_n[i] = sum_w[i] = sum_b[i] = splat(0.f);
  if (NEXT) cols.params(p.next_weight, p.params_f32, 0, w2);
  auto gate_of = [&](uint32_t u, float2(&k)[P]) {
    cols.params(p.gate, p.params_f32, (u / p.splits) * static_cast<uint64_t>(p.hidden), k);
  };
  auto open_unit = [&](uint32_t u) {
    cols.params(p.weight, p.params_f32, 0, gw);
    if (!wide) return;
    float2 k[P];
    gate_of(u, k);
#pragma unroll
    for (int i = 0; i < P; i++) gw[i] = mul2(gw[i], k[i]);
  };
  auto close_unit = [&](uint32_t u) {
    float2 dg[P];
    if (wide) {
      gate_of(u, dg);
#pragma unroll
      for (int i = 0; i < P; i++) sum_w[i] = fma2(sum_b[i], dg[i], sum_w[i]);
      cols.params(p.weight, p.params_f32, 0, dg);
    }
#pragma unroll
    for (int i = 0; i < P; i++) {
      if (wide)
        dg[i] = mul2(sum_b[i], dg[i]);
      else
        sum_w[i] = fma2(sum_b[i], splat(1.f), sum_w[i]);
      sum_b[i] = splat(0.f);
    }
    if (!wide) return;
    const float* f = reinterpret_cast<const float*>(dg);
#pragma unroll
    for (int i = 0; i < Cols::NV; i++) {
      const uint32_t c = lane + i * 32;
      if (c >= cols.pieces) continue;
      const uint64_t at = static_cast<uint64_t>(u) * p.hidden + c * V;
#pragma unroll
      for (int j = 0; j < V; j++) {
        if (p.splits > 1)
          gate_parts[at + j] = f[i * V + j];
        else if (p.params_f32)
          static_cast<float*>(p.dgate)[at + j] = f[i * V + j];
        else
          static_cast<T*>(p.dgate)[at + j] = from_f32<T>(f[i * V + j]);
      }
    }
  };
  struct Row {
    Piece<T, V> gx[Cols::NV], gh[Cols::NV], x[Cols::NV], y[Cols::NV];
  };
  auto load = [&](Row& r, uint64_t t) {
    if (NEXT) {
      cols.load(static_cast<const T*>(p.dh) + t * p.dh_stride, r.gh);
      cols.load(static_cast<const T*>(p.x_new) + t * p.x_new_stride, r.x);
    }
    if (BRANCH) cols.load(static_cast<const T*>(p.y) + t * p.y_stride, r.y);
    if (p.dx_new) {
      cols.load(static_cast<const T*>(p.dx_new) + t * p.dx_new_stride, r.gx);
    } else {
#pragma unroll
      for (int i = 0; i < Cols::NV; i++) r.gx[i] = Piece<T, V>::zero();
    }
  };
  BwdWalk now{blockIdx.x * kNormWarps + warp, 0, 0};
  Row row, next;
  if (now.valid(p)) {
    now.open(p);
    if (BRANCH) open_unit(now.u);
    load(row, now.t);
  }
  while (now.valid(p)) {
    const uint64_t t = now.t;
    const uint32_t unit = now.u;
    const bool ended = now.next(p);
    if (now.valid(p)) load(next, now.t);
    float2 g[P], h[P], x[P], y[P];
    float sums[3] = {0.f, 0.f, 0.f};
    Cols::unpack(row.gx, g);
    if (NEXT) {
      float2 xx = splat(0.f), ux = splat(0.f);
      Cols::unpack(row.gh, h);
      Cols::unpack(row.x, x);
#pragma unroll
      for (int i = 0; i < P; i++) {
        xx = fma2(x[i], x[i], xx);
        ux = fma2(mul2(h[i], w2[i]), x[i], ux);
      }
      sums[0] = warp_sum_f32(xx.x + xx.y);
      sums[1] = warp_sum_f32(ux.x + ux.y);
    }
    if (BRANCH) {
      float2 yy = splat(0.f);
      Cols::unpack(row.y, y);
#pragma unroll
      for (int i = 0; i < P; i++) yy = fma2(y[i], y[i], yy);
      sums[2] = warp_sum_f32(yy.x + yy.y);
    }
    if (NEXT) {
      const float r2 = rsqrtf(sums[0] * inv_d + p.eps);
      const float2 rr = splat(r2), m = splat(-(sums[1] * r2 * inv_d) * r2 * r2);  // -r2^2 mean(u n2)
#pragma unroll
      for (int i = 0; i < P; i++) {
        g[i] = fma2(rr, mul2(h[i], w2[i]), fma2(x[i], m, g[i]));
        sum_n[i] = fma2(h[i], mul2(x[i], rr), sum_n[i]);
      }
    }
    float2 o[P];
    const float2 a = splat(p.residual_scale);
#pragma unroll
    for (int i = 0; i < P; i++) o[i] = mul2(a, g[i]);
    cols.put(cols.start(static_cast<T*>(p.dx), t, p.hidden), o);
    if (BRANCH) {
      const float root = rsqrtf(sums[2] * inv_d + p.eps);
      const float one = narrow ? load_param<T>(p.gate, p.params_f32, t / p.gate_tokens) : 1.f;
      const float2 rr = splat(root * one);
      float2 vy = splat(0.f);
#pragma unroll
      for (int i = 0; i < P; i++) {
        sum_b[i] = fma2(g[i], mul2(y[i], rr), sum_b[i]);
        g[i] = mul2(g[i], gw[i]);  // v, but for a one-column gate
        vy = fma2(g[i], y[i], vy);
      }
      const float dot = warp_sum_f32(vy.x + vy.y);
      const float2 m = splat(-(dot * root * inv_d) * root);
#pragma unroll
      for (int i = 0; i < P; i++) g[i] = mul2(rr, fma2(y[i], m, g[i]));
      cols.put(cols.start(static_cast<T*>(p.dy), t, p.hidden), g);
      if (narrow && lane == 0) {
        const float dg = root * dot;  // sum of G n w
        if (p.gate_tokens > 1)
          gate_parts[t] = dg;
        else if (p.params_f32)
          static_cast<float*>(p.dgate)[t] = dg;
        else
          static_cast<T*>(p.dgate)[t] = from_f32<T>(dg);
      }
    }
    if (ended && BRANCH) {
      close_unit(unit);
      if (now.valid(p)) open_unit(now.u);
    }
    row = next;
  }
  float* mine = p.parts + static_cast<uint64_t>(blockIdx.x) * 2 * p.hidden;
  auto flush = [&](const float2(&s)[P], float* dst) {
    const float* f = reinterpret_cast<const float*>(s);
#pragma unroll
    for (int i = 0; i < Cols::NV; i++)
#pragma unroll
      for (int j = 0; j < V; j++)
        if (lane + i * 32 < cols.pieces) tile[warp][(lane + i * 32) * V + j] = f[i * V + j];
    __syncthreads();
    if (threadIdx.x < p.hidden) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kNormWarps; q++) sum += tile[q][threadIdx.x];
      dst[threadIdx.x] = sum;
    }
    __syncthreads();
  };
  if (BRANCH) flush(sum_w, mine);
  if (NEXT) flush(sum_n, mine + p.hidden);
}

// Adds the CTAs' sums, in order: the warps take a share of the parts each, a lane a column, and
// then half a warp, or a warp, adds a column's shares.  blockIdx.y: 0 the branch weight's gradient,
// 1 the next weight's, 2 + g gate row g's.
template <typename T, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) norm_parts_kernel(NormBwdParams p) {
  __shared__ float sums[WARPS][33];
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
  const uint32_t first = count * slice / WARPS, last = count * (slice + 1) / WARPS;
  if (col < p.hidden) {
#pragma unroll 8
    for (uint32_t i = first; i < last; i++) s += src[i * stride + col];
  }
  sums[slice][lane] = s;
  __syncthreads();
  constexpr uint32_t kEach = 32 / WARPS;  // columns of a warp
  const uint32_t mine = slice * kEach + lane / WARPS;
  s = sums[lane % WARPS][mine];
#pragma unroll
  for (int d = WARPS / 2; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
  if (lane % WARPS || blockIdx.x * 32 + mine >= p.hidden) return;
  if (p.params_f32)
    static_cast<float*>(dst)[blockIdx.x * 32 + mine] = s;
  else
    static_cast<T*>(dst)[blockIdx.x * 32 + mine] = from_f32<T>(s);
}

// A one-column gate's gradient where several tokens share a gate value: one CTA per value.
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

// Ranges of a gate row's `size` tokens, of `groups` gate rows for `most` walkers.
uint64_t row_splits(uint64_t groups, uint64_t size, uint64_t most, uint64_t period) {
  uint64_t splits = groups >= most ? 1 : most / groups;
  if (splits >= size) return size;
  return splits > period ? splits - splits % period : splits;
}

// Cuts the rows into ranges for at most `most` walkers, `per_cta` of them in a CTA or each a
// cluster of p.cluster CTAs (a range lies in one gate row's tokens), launches `fn` and adds up what
// it left.  With a period, a range's rows are a multiple of it apart, and there is one a walker.
template <typename T>
cudaError_t launch_ranges(NormBwdParams& p, const void* fn, uint64_t most, uint32_t per_cta, int threads, int smem,
                          cudaStream_t stream, const DeviceInfo& dev, uint64_t period = 1) {
  const bool wide = p.gate && p.gate_wide;
  if (most > norm_max_units(p.hidden)) most = norm_max_units(p.hidden);
  const uint64_t groups = wide ? p.gate_rows : 1, size = wide ? p.gate_tokens : p.tokens;
  const uint64_t splits = row_splits(groups, size, most, period);
  p.splits = static_cast<uint32_t>(splits);
  const uint64_t units = groups * splits;
  if (units > 0xFFFFFFFFull) return cudaErrorInvalidConfiguration;
  p.units = static_cast<uint32_t>(units);
  p.walkers = static_cast<uint32_t>(units < most ? units : most);
  p.ctas = (p.walkers + per_cta - 1) / per_cta;
  p.walkers = p.ctas * per_cta;
  void* args[] = {&p};
  cudaError_t e = launch_kernel(fn, dim3(p.ctas * p.cluster), dim3(threads), smem, stream, args, false, p.cluster);
  if (e != cudaSuccess) return e;
  const uint32_t jobs = 2 + (wide && splits > 1 ? static_cast<uint32_t>(groups) : 0u);
  // 32 warps a CTA while the GPU holds all such CTAs at once, two an SM (4452 x 704 fp32 18.1 us in
  // all against 22.9 with 16); beyond that 16, four an SM (512 x 4096 bf16 10.8 against 13.0).
  const dim3 parts((p.hidden + 31) / 32, jobs);
  if (static_cast<uint64_t>(parts.x) * parts.y <= 2ull * static_cast<uint64_t>(dev.sm_count))
    e = launch_kernel(reinterpret_cast<const void*>(norm_parts_kernel<T, 32>), parts, dim3(1024), 0, stream, args, false);
  else
    e = launch_kernel(reinterpret_cast<const void*>(norm_parts_kernel<T, 16>), parts, dim3(512), 0, stream, args, false);
  if (e != cudaSuccess || !p.gate || wide || p.gate_tokens == 1) return e;
  return launch_kernel(reinterpret_cast<const void*>(norm_narrow_gate_kernel<T>),
                       dim3(static_cast<unsigned>(p.gate_rows)), dim3(256), 0, stream, args, false);
}

// fn<BRANCH, NEXT> of a kernel template by what the call has.
#define ZC_NORM_MODE(KERNEL, ...)                                                                       \
  (p.y && p.next_weight ? reinterpret_cast<const void*>(KERNEL<__VA_ARGS__, true, true>)                \
   : p.y                ? reinterpret_cast<const void*>(KERNEL<__VA_ARGS__, true, false>)               \
                        : reinterpret_cast<const void*>(KERNEL<__VA_ARGS__, false, true>))

template <typename T, int V, int C, bool CLUSTER, bool SHIFT, bool BRANCH, bool NEXT>
cudaError_t run_ring(NormBwdParams& p, int threads, uint64_t period, cudaStream_t stream, const DeviceInfo& dev) {
  static RingPrep prep[2];  // for clusters of 2 and 4
  constexpr int kArrays = BRANCH && NEXT ? 4 : NEXT ? 3 : 2;
  const int smem = static_cast<int>(RowRing<T, V, C, kArrays, kBwdStages>::bytes(threads));
  const void* fn = reinterpret_cast<const void*>(norm_bwd_ring_kernel<T, V, C, CLUSTER, SHIFT, BRANCH, NEXT>);
  int fit = 0;
  cudaError_t e = prepare_ring(prep[p.cluster == 4], fn, threads, smem, dev, static_cast<int>(p.cluster), &fit);
  if (e != cudaSuccess) return e;
  return launch_ranges<T>(p, fn, static_cast<uint64_t>(fit), 1, threads, smem, stream, dev, period);
}

// Runs the ring with C columns a thread and so many CTAs a row if it holds such rows.
template <typename T, int V, int C, bool CLUSTER, bool SHIFT = false>
bool run_ring(NormBwdParams& p, uint32_t cluster, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e,
              uint64_t period = 1) {
  const uint32_t all = cluster * C * 32;
  const int threads = static_cast<int>((p.hidden + (SHIFT ? V - 1 : 0) + all - 1) / all * 32);
  if (threads > kNormRingThreads || RowRing<T, V, C, 4, kBwdStages>::bytes(threads) > kNormRingSmem) return false;
  p.cluster = cluster;
  if (p.y && p.next_weight)
    *e = run_ring<T, V, C, CLUSTER, SHIFT, true, true>(p, threads, period, stream, dev);
  else if (p.y)
    *e = run_ring<T, V, C, CLUSTER, SHIFT, true, false>(p, threads, period, stream, dev);
  else
    *e = run_ring<T, V, C, CLUSTER, SHIFT, false, true>(p, threads, period, stream, dev);
  return true;
}

// The ring on rows off 16 bytes, but alike in all matrices, if its walkers can keep to rows that
// lie alike and hold them.
template <typename T>
bool run_shifted(NormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev, cudaError_t* e) {
  RowPlaces rows;
  rows.add(p.y, p.y_stride * sizeof(T));
  if (p.next_weight) rows.add(p.x_new, p.x_new_stride * sizeof(T));
  rows.add(p.dh, p.dh_stride * sizeof(T));
  rows.add(p.dx_new, p.dx_new_stride * sizeof(T));
  rows.add(p.dx, static_cast<uint64_t>(p.hidden) * sizeof(T));
  rows.add(p.dy, static_cast<uint64_t>(p.hidden) * sizeof(T));
  if (!rows.alike) return false;
  const bool wide = p.gate && p.gate_wide;
  const uint64_t groups = wide ? p.gate_rows : 1, size = wide ? p.gate_tokens : p.tokens, period = rows.period();
  const uint64_t most = static_cast<uint64_t>(dev.sm_count), splits = row_splits(groups, size, most, period);
  // at least a walker an SM; a few fewer where the period wants it, but not many
  if (groups * splits > most || (splits < size && (splits % period || 2 * groups * splits < most))) return false;
  constexpr int V = kPieceOf<T>;
  if (run_ring<T, V, kBwdCols, false, true>(p, 1, stream, dev, e, period)) return true;
  if constexpr (sizeof(T) == 2) return run_ring<T, V, kBwdWideCols, false, true>(p, 1, stream, dev, e, period);
  return false;
}

template <typename T, int V>
cudaError_t run_width(NormBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  p.cluster = 1;
  cudaError_t e;
  // Off 16 bytes the ring copies whole pieces where the warp shape loads values, which pays once its
  // many small CTAs have some rows each to add up: 16384 x 129 bf16 23.4 us against 28.0, 131072 87
  // against 150; 2000 x 201 17.0 against 12.4.
  if constexpr (V == 1) {
    if ((p.hidden > kNormWarpWidth || p.tokens >= 32ull * static_cast<uint64_t>(dev.sm_count)) &&
        run_shifted<T>(p, stream, dev, &e))
      return e;
  }
  if (p.hidden <= kNormWarpWidth)
    return launch_ranges<T>(p, ZC_NORM_MODE(norm_bwd_warp_kernel, T, V),
                            4ull * kNormWarps * static_cast<uint64_t>(dev.sm_count), kNormWarps, kNormWarps * 32, 0,
                            stream, dev);
  constexpr int kWide = sizeof(T) == 2 && V > 1 ? kBwdWideCols : kBwdCols;
  if (run_ring<T, V, kBwdCols, false>(p, 1, stream, dev, &e)) return e;
  if constexpr (kWide != kBwdCols) {
    if (run_ring<T, V, kWide, false>(p, 1, stream, dev, &e)) return e;
  }
  if (run_ring<T, V, kWide, true>(p, 2, stream, dev, &e)) return e;
  if (run_ring<T, V, kWide, true>(p, 4, stream, dev, &e)) return e;
  return cudaErrorInvalidValue;  // wider than ZC_NORM_MAX_HIDDEN
}
#undef ZC_NORM_MODE

template <typename T>
cudaError_t run_typed(NormBwdParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? run_width<T, kPieceOf<T>>(p, stream, dev) : run_width<T, 1>(p, stream, dev);
}

}  // namespace

cudaError_t prepare_ring(RingPrep& rp, const void* fn, int threads, int smem_bytes, const DeviceInfo& dev, int cluster,
                         int* fit) {
  const bool cached = dev.device >= 0 && dev.device < kMaxDevices;
  std::atomic<int>* known = cached ? &rp.fit[dev.device][threads / 32] : nullptr;
  if (known) {
    *fit = known->load(std::memory_order_acquire);
    if (*fit > 0) return cudaSuccess;
  }
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingSmem);
  if (e != cudaSuccess) return e;
  if (cluster == 1) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(fit, fn, threads, static_cast<size_t>(smem_bytes));
    *fit *= dev.sm_count;
  } else {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / cluster * cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(fit, fn, &cfg);
  }
  if (e != cudaSuccess) return e;
  if (*fit < 1) return cudaErrorInvalidConfiguration;
  if (known) known->store(*fit, std::memory_order_release);
  return cudaSuccess;
}

uint64_t norm_max_walkers(uint32_t hidden) { return norm_max_units(hidden); }

uint64_t norm_workspace_bytes(uint64_t tokens, uint32_t hidden) {
  // two sums a CTA, and one a range or a value a token for the gate
  const uint64_t units = tokens < norm_max_units(hidden) ? tokens : norm_max_units(hidden);
  return 4 * (3 * units * hidden + tokens);
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
