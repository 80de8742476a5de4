// zc_moe.cu -- the operators on both sides of an expert-parallel exchange:
// choosing experts for every token, sorting tokens by expert into contiguous
// pieces, bringing the experts' outputs back weighted, and their gradients.
// Definitions in include/zc.h.
//
// Everything here is bound by memory: each value is read or written once and
// takes a few operations.  No kernel uses atomics on global memory and every
// sum has a fixed order, so the same inputs give the same bits.
#include <type_traits>

#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

namespace {

// ------------------------------------------------------------------ routing
constexpr int kRouteWarps = 4;  // tokens per CTA, one warp each

// Order-preserving image of a score: larger score, larger key.  0 stands for
// "cannot be chosen" (minus infinity); NaN is above everything, as a sort has
// it, so that it shows in the weights; both zeros are equal.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xFFFFFFFFu;
  if (f == -INFINITY) return 0u;
  const uint32_t b = f == 0.f ? 0u : __float_as_uint(f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l))); }

// One warp per token, lane l holding experts l, l + 32, ...: K times the
// largest key (ties: the lowest expert) is found and cleared.  Pick k ends in
// lane k, which then reads its logit again (an L1 hit) for the weight.
template <typename T, int NPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteParams p) {
  pdl_begin();
  const uint32_t lane = lane_id();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride;
  float l[NPL];
  uint32_t key[NPL];
#pragma unroll
  for (int j = 0; j < NPL; j++) {
    const uint32_t e = j * 32 + lane;
    l[j] = e < p.experts ? to_f32<T>(row[e]) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < NPL; j++) {
    const uint32_t e = j * 32 + lane;
    float s = l[j];
    if (p.sigmoid) s = __fadd_rn(sigmoid(l[j]), p.bias && e < p.experts ? p.bias[e] : 0.f);
    key[j] = l[j] == -INFINITY ? 0u : order_key(s);
  }
  uint32_t mine = kFull;
  for (uint32_t k = 0; k < p.k; k++) {
    uint32_t best = key[0], at = 0;
#pragma unroll
    for (int j = 1; j < NPL; j++)
      if (key[j] > best) best = key[j], at = j;
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;
    const uint32_t e = __reduce_min_sync(kFull, best == top ? at * 32 + lane : kFull);
    if (lane == k) mine = e;
#pragma unroll
    for (int j = 0; j < NPL; j++)
      if (e == j * 32 + lane) key[j] = 0;
  }
  const bool have = mine != kFull;
  const float lm = have ? to_f32<T>(row[mine]) : -INFINITY;
  float w;
  if (p.sigmoid) {
    w = have ? sigmoid(lm) : 0.f;
    if (p.renormalize) w = w / (warp_sum_f32(w) + 1e-20f);
  } else {
    const float top = __shfl_sync(kFull, lm, 0);  // the first pick is the row's largest logit
    w = have ? expf(lm - top) : 0.f;
    float sum;
    if (p.renormalize) {
      sum = warp_sum_f32(w);
    } else {
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < NPL; j++) sum += l[j] == -INFINITY ? 0.f : expf(l[j] - top);
      sum = warp_sum_f32(sum);
    }
    w = have ? w / sum : 0.f;
  }
  if (lane < p.k) {
    p.weights[t * p.k + lane] = p.scale * w;
    p.ids[t * p.k + lane] = have ? static_cast<int32_t>(mine) : -1;
  }
}

// Gradient of the logits: G_k = scale dw_k for the chosen experts.  A
// renormalised softmax and both sigmoid forms depend on the chosen logits
// alone, so only those are read and every other gradient is zero; the plain
// softmax needs the whole row.
template <typename T, int NPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(RouteBwdParams p) {
  pdl_begin();
  const uint32_t lane = lane_id();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride;
  T* out = static_cast<T*>(p.dlogits) + t * p.experts;
  int32_t id = -1;
  float g = 0.f, lm = -INFINITY;
  if (lane < p.k) {
    id = p.ids[t * p.k + lane];
    if (static_cast<uint32_t>(id) >= p.experts) id = -1;
    if (id >= 0) {
      g = p.scale * p.dweights[t * p.k + lane];
      lm = to_f32<T>(row[id]);
    }
  }
  const bool have = id >= 0;
  const bool whole = !p.sigmoid && !p.renormalize;
  float prob[NPL];
  float d = 0.f, mean = 0.f;  // this lane's chosen logit's gradient; sum of G p over the row
  if (whole) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; j++) {
      const uint32_t e = j * 32 + lane;
      prob[j] = e < p.experts ? to_f32<T>(row[e]) : -INFINITY;
      top = fmaxf(top, prob[j]);
    }
    top = warp_max_f32(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; j++) {
      prob[j] = prob[j] == -INFINITY ? 0.f : expf(prob[j] - top);
      sum += prob[j];
    }
    sum = warp_sum_f32(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row with every expert masked has no gradient
#pragma unroll
    for (int j = 0; j < NPL; j++) prob[j] *= inv;
    mean = warp_sum_f32(have ? g * (expf(lm - top) * inv) : 0.f);
    d = g;
  } else if (p.sigmoid) {
    const float s = have ? sigmoid(lm) : 0.f;
    if (p.renormalize) {
      const float total = warp_sum_f32(s) + 1e-20f;
      g = (g - warp_sum_f32(g * s) / total) / total;
    }
    d = have ? g * s * (1.f - s) : 0.f;
  } else {
    const float top = warp_max_f32(lm);
    float f = have ? expf(lm - top) : 0.f;
    const float sum = warp_sum_f32(f);
    f = have ? f / sum : 0.f;
    d = f * (g - warp_sum_f32(g * f));
  }
  float acc[NPL];
#pragma unroll
  for (int j = 0; j < NPL; j++) acc[j] = 0.f;
  for (uint32_t k = 0; k < p.k; k++) {
    const int32_t e = __shfl_sync(kFull, id, k);
    const float dk = __shfl_sync(kFull, d, k);
    if (e < 0) continue;
#pragma unroll
    for (int j = 0; j < NPL; j++)
      if (static_cast<uint32_t>(e) == j * 32 + lane) acc[j] += dk;
  }
#pragma unroll
  for (int j = 0; j < NPL; j++) {
    const uint32_t e = j * 32 + lane;
    if (whole) acc[j] = prob[j] * (acc[j] - mean);
    if (e < p.experts) out[e] = from_f32<T>(acc[j]);
  }
}

// ------------------------------------------------------------------ dispatch
constexpr int kSortThreads = 256;

// The expert of slot i, or `experts` for a slot that is not routed.
__device__ __forceinline__ uint32_t slot_key(const DispatchParams& p, uint64_t i) {
  const int64_t v = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
  return v >= 0 && v < static_cast<int64_t>(p.experts) ? static_cast<uint32_t>(v) : p.experts;
}

// Exclusive prefix sums of a[0 .. count), in place; count <= 8 * kSortThreads.
__device__ __forceinline__ void block_exclusive_scan(uint32_t* a, uint32_t count, uint32_t* warp_totals) {
  const uint32_t per = (count + kSortThreads - 1) / kSortThreads, first = threadIdx.x * per;
  uint32_t sum = 0;
  for (uint32_t i = first; i < first + per && i < count; i++) sum += a[i];
  const uint32_t upto = warp_inclusive_scan(sum);
  if (lane_id() == 31) warp_totals[threadIdx.x >> 5] = upto;
  __syncthreads();
  uint32_t base = upto - sum;
  for (uint32_t w = 0; w < threadIdx.x >> 5; w++) base += warp_totals[w];
  for (uint32_t i = first; i < first + per && i < count; i++) {
    const uint32_t v = a[i];
    a[i] = base;
    base += v;
  }
  __syncthreads();
}

// First of two passes of the stable counting sort: how many slots of each
// expert a chunk of tokens holds, counts[expert][chunk].
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(DispatchParams p) {
  __shared__ uint32_t hist[kMoeMaxExperts + 1];
  pdl_allow_dependents();
  for (uint32_t e = threadIdx.x; e <= kMoeMaxExperts; e += kSortThreads) hist[e] = 0;
  pdl_wait();
  __syncthreads();
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * p.chunk_tokens * p.k;
  const uint64_t all = p.tokens * p.k, last = min(all, first + static_cast<uint64_t>(p.chunk_tokens) * p.k);
  for (uint64_t i = first + threadIdx.x; i < last; i += kSortThreads) atomicAdd(&hist[slot_key(p, i)], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads)
    p.counts[static_cast<uint64_t>(e) * p.chunks + blockIdx.x] = hist[e];
}

// Exclusive prefix over the chunks of every expert, in place, one warp per
// expert; the total goes behind the table.
__global__ void __launch_bounds__(128) moe_prefix_kernel(DispatchParams p) {
  pdl_begin();
  const uint32_t e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = lane_id();
  if (e > p.experts) return;
  uint32_t* c = p.counts + static_cast<uint64_t>(e) * p.chunks;
  uint32_t base = 0;
  for (uint32_t i = 0; i < p.chunks; i += 32) {
    const uint32_t v = i + lane < p.chunks ? c[i + lane] : 0;
    const uint32_t upto = warp_inclusive_scan(v);
    if (i + lane < p.chunks) c[i + lane] = base + upto - v;
    base += __shfl_sync(kFull, upto, 31);
  }
  if (lane == 0) p.counts[static_cast<uint64_t>(p.experts + 1) * p.chunks + e] = base;
}

// Row of every slot, and the rows themselves.  A CTA places the slots of a
// few tokens: row = first row of the expert + the expert's slots in earlier
// chunks + those earlier in this chunk + those earlier among its own.  With
// one chunk in all (`single`) the CTA counts all slots itself, so small calls are one
// launch.  Then it reads each token once and writes its K rows.
template <typename T, int V>
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(DispatchParams p) {
  __shared__ uint32_t start[kMoeMaxExperts + 1];   // first row of each expert
  __shared__ uint32_t before[kMoeMaxExperts + 1];  // its slots in this chunk before this CTA's
  __shared__ uint32_t warp_totals[kSortThreads / 32];
  __shared__ uint32_t own_key[kMoePlaceTokens * kMoeMaxK];
  __shared__ int32_t own_pos[kMoePlaceTokens * kMoeMaxK];
  pdl_allow_dependents();
  for (uint32_t e = threadIdx.x; e <= kMoeMaxExperts; e += kSortThreads) start[e] = before[e] = 0;
  pdl_wait();
  __syncthreads();
  const uint64_t t0 = static_cast<uint64_t>(blockIdx.x) * p.cta_tokens;
  const uint32_t nt = static_cast<uint32_t>(min(static_cast<uint64_t>(p.cta_tokens), p.tokens - min(p.tokens, t0)));
  const uint64_t s0 = t0 * p.k, all = p.tokens * p.k;
  const uint32_t own = nt * p.k;
  const uint32_t chunk = p.single ? 0 : static_cast<uint32_t>(t0 / p.chunk_tokens);
  const uint64_t c0 = static_cast<uint64_t>(chunk) * p.chunk_tokens * p.k;
  for (uint32_t i = threadIdx.x; i < own; i += kSortThreads) own_key[i] = slot_key(p, s0 + i);
  if (p.single) {
    for (uint64_t i = threadIdx.x; i < all; i += kSortThreads) {
      const uint32_t e = slot_key(p, i);
      atomicAdd(&start[e], 1u);
      if (i < s0) atomicAdd(&before[e], 1u);
    }
  } else {
    for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads)
      start[e] = p.counts[static_cast<uint64_t>(p.experts + 1) * p.chunks + e];
    for (uint64_t i = c0 + threadIdx.x; i < s0; i += kSortThreads) atomicAdd(&before[slot_key(p, i)], 1u);
  }
  __syncthreads();
  block_exclusive_scan(start, p.experts + 1, warp_totals);
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) p.offsets[e] = static_cast<int32_t>(start[e]);
  for (uint32_t i = threadIdx.x; i < own; i += kSortThreads) {
    const uint32_t e = own_key[i];
    uint32_t r = start[e] + before[e];
    if (!p.single) r += p.counts[static_cast<uint64_t>(e) * p.chunks + chunk];
    for (uint32_t j = 0; j < i; j++) r += own_key[j] == e;
    const int32_t pos = e < p.experts ? static_cast<int32_t>(r) : ~static_cast<int32_t>(r);
    own_pos[i] = pos;
    if (blockIdx.y == 0) {
      p.positions[s0 + i] = pos;
      p.slots[r] = static_cast<int32_t>(s0 + i);
    }
  }
  __syncthreads();
  const uint32_t pieces = p.hidden / V;
  for (uint32_t t = 0; t < nt; t++) {
    const T* src = static_cast<const T*>(p.x) + (t0 + t) * p.stride;
    for (uint32_t c = blockIdx.y * kSortThreads + threadIdx.x; c < pieces; c += gridDim.y * kSortThreads) {
      const Piece<T, V> v = Piece<T, V>::load(src + static_cast<uint64_t>(c) * V);
      for (uint32_t k = 0; k < p.k; k++) {
        const int32_t pos = own_pos[t * p.k + k];
        const uint64_t row = static_cast<uint64_t>(pos < 0 ? ~pos : pos);
        T* dst = static_cast<T*>(p.rows) + row * p.hidden + static_cast<uint64_t>(c) * V;
        if (pos < 0)
          Piece<T, V>::zero().store(dst);
        else
          v.store(dst);
      }
    }
  }
}

// ------------------------------------------------------------------ combine
constexpr int kCombineThreads = 256;
constexpr int kCombineK = 8;  // rows of one token in flight together

// The row of a slot: true if it is routed.  `row` is the row to read (or,
// unrouted, the one to clear, which the buffer need not hold); a routed row
// outside the buffer is reported and skipped.
__device__ __forceinline__ bool slot_row(int32_t pos, uint64_t n_rows, int32_t* status, uint64_t* row, bool* inside) {
  *row = static_cast<uint64_t>(pos < 0 ? ~pos : pos);
  *inside = *row < n_rows;
  if (!*inside && pos >= 0) set_status(status, ZC_ERR_BAD_INDEX);
  return *inside && pos >= 0;
}

// out[t] = sum over k, in order, of w[t][k] rows[pos[t][k]], in fp32.  One
// thread per 16-byte piece of a token: the rows of up to eight slots are
// loaded before the first is added.
template <typename T, int V>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(CombineParams p) {
  pdl_begin();
  const uint32_t pieces = p.hidden / V;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kCombineThreads + threadIdx.x;
  const uint64_t t = i / pieces;
  if (t >= p.tokens) return;
  const uint64_t c = (i - t * pieces) * V;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; j++) acc[j] = 0.f;
  for (uint32_t k0 = 0; k0 < p.k; k0 += kCombineK) {
    Piece<T, V> v[kCombineK];
    float w[kCombineK];
#pragma unroll
    for (int k = 0; k < kCombineK; k++) {
      w[k] = 0.f;
      v[k] = Piece<T, V>::zero();
      if (k0 + k < p.k) {
        uint64_t row;
        bool inside;
        if (slot_row(p.positions[t * p.k + k0 + k], p.n_rows, p.status, &row, &inside)) {
          w[k] = p.weights ? p.weights[t * p.k + k0 + k] : 1.f;
          v[k] = Piece<T, V>::load(static_cast<const T*>(p.rows) + row * p.row_stride + c);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kCombineK; k++) {
      float f[V];
      v[k].get(f);
#pragma unroll
      for (int j = 0; j < V; j++) acc[j] = fmaf(w[k], f[j], acc[j]);
    }
  }
  Piece<T, V> o;
  o.set(acc);
  o.store(static_cast<T*>(p.out) + t * p.hidden + c);
}

// drows[pos] = w dout and dw = <dout, rows[pos]>: dout's row is read once for
// four slots, each row once; the products are summed in registers over a
// thread's pieces, then over the CTA (or the warp, for narrow rows).
constexpr int kCombineBwdK = 4;

template <typename T, int V, bool WARP>
__global__ void __launch_bounds__(512) moe_combine_bwd_kernel(CombineBwdParams p) {
  __shared__ float red[2][kCombineBwdK * 32];
  pdl_begin();
  const uint32_t lane = lane_id(), warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const uint64_t t = WARP ? static_cast<uint64_t>(blockIdx.x) * warps + warp : blockIdx.x;
  if (t >= p.tokens) return;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const uint32_t pieces = p.hidden / V;
  const T* dout = static_cast<const T*>(p.dout) + t * p.dout_stride;
  for (uint32_t k0 = 0, turn = 0; k0 < p.k; k0 += kCombineBwdK, turn ^= 1) {
    float dot[kCombineBwdK], w[kCombineBwdK];
    uint64_t row[kCombineBwdK];
    bool routed[kCombineBwdK], inside[kCombineBwdK];
#pragma unroll
    for (int k = 0; k < kCombineBwdK; k++) {
      dot[k] = 0.f;
      w[k] = 0.f;
      routed[k] = inside[k] = false;
      if (k0 + k < p.k) {
        routed[k] = slot_row(p.positions[t * p.k + k0 + k], p.n_rows, p.status, &row[k], &inside[k]);
        if (routed[k]) w[k] = p.weights[t * p.k + k0 + k];
      }
    }
    for (uint32_t c = me; c < pieces; c += step) {
      const uint64_t at = static_cast<uint64_t>(c) * V;
      float g[V];
      Piece<T, V> v[kCombineBwdK];
#pragma unroll
      for (int k = 0; k < kCombineBwdK; k++)
        v[k] = routed[k] ? Piece<T, V>::load(static_cast<const T*>(p.rows) + row[k] * p.row_stride + at)
                         : Piece<T, V>::zero();
      Piece<T, V>::load(dout + at).get(g);
#pragma unroll
      for (int k = 0; k < kCombineBwdK; k++) {
        if (!inside[k]) continue;
        float f[V], d[V];
        v[k].get(f);
#pragma unroll
        for (int j = 0; j < V; j++) {
          dot[k] = routed[k] ? fmaf(g[j], f[j], dot[k]) : 0.f;
          d[j] = routed[k] ? w[k] * g[j] : 0.f;
        }
        Piece<T, V> o;
        o.set(d);
        o.store(static_cast<T*>(p.drows) + row[k] * p.hidden + at);
      }
    }
    if (WARP) {
#pragma unroll
      for (int k = 0; k < kCombineBwdK; k++) dot[k] = warp_sum_f32(dot[k]);
    } else {
      block_sum_f32<kCombineBwdK>(dot, red[turn]);
    }
    if (me == 0) {
#pragma unroll
      for (int k = 0; k < kCombineBwdK; k++)
        if (k0 + k < p.k) p.dweights[t * p.k + k0 + k] = dot[k];
    }
  }
}

// ------------------------------------------------------------------ launches
template <typename F>
cudaError_t run(F* kernel, uint64_t grid_x, uint32_t grid_y, int threads, cudaStream_t stream, void* params) {
  if (grid_x == 0) return cudaSuccess;
  if (grid_x > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  void* args[] = {params};
  return launch_kernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<unsigned>(grid_x), grid_y),
                       dim3(threads), 0, stream, args, false);
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

template <typename T, typename P>
cudaError_t route_of(const P& params, cudaStream_t stream) {
  P p = params;
  const uint64_t grid = ceil_div(p.tokens, kRouteWarps);
#define ZC_ROUTE(NPL)                                                                      \
  if (p.experts <= 32 * NPL) {                                                             \
    if constexpr (std::is_same<P, RouteParams>::value)                                     \
      return run(route_kernel<T, NPL>, grid, 1, kRouteWarps * 32, stream, &p);             \
    else                                                                                   \
      return run(route_bwd_kernel<T, NPL>, grid, 1, kRouteWarps * 32, stream, &p);         \
  }
  ZC_ROUTE(2)
  ZC_ROUTE(4)
  ZC_ROUTE(8)
  ZC_ROUTE(16)
  ZC_ROUTE(32)
#undef ZC_ROUTE
  return cudaErrorInvalidValue;
}

template <typename P>
cudaError_t route_typed(const P& p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case ZC_BF16: return route_of<__nv_bfloat16>(p, stream);
    case ZC_F16: return route_of<__half>(p, stream);
    default: return route_of<float>(p, stream);
  }
}

template <typename T>
cudaError_t place(DispatchParams& p, bool vec, uint64_t grid, uint32_t split, cudaStream_t stream) {
  if (vec) return run(moe_place_kernel<T, kPieceOf<T>>, grid, split, kSortThreads, stream, &p);
  return run(moe_place_kernel<T, 1>, grid, split, kSortThreads, stream, &p);
}

template <typename T>
cudaError_t combine(CombineParams& p, bool vec, cudaStream_t stream) {
  const uint64_t pieces = p.hidden / (vec ? kPieceOf<T> : 1);
  const uint64_t grid = ceil_div(p.tokens * pieces, kCombineThreads);
  if (vec) return run(moe_combine_kernel<T, kPieceOf<T>>, grid, 1, kCombineThreads, stream, &p);
  return run(moe_combine_kernel<T, 1>, grid, 1, kCombineThreads, stream, &p);
}

template <typename T, int V>
cudaError_t combine_bwd(CombineBwdParams& p, cudaStream_t stream) {
  const uint64_t pieces = p.hidden / V;
  if (pieces <= 64) return run(moe_combine_bwd_kernel<T, V, true>, ceil_div(p.tokens, 4), 1, 128, stream, &p);
  const int threads = pieces >= 512 ? 256 : static_cast<int>(ceil_div(pieces, 64) * 32);
  return run(moe_combine_bwd_kernel<T, V, false>, p.tokens, 1, threads, stream, &p);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t stream) {
  return route_typed(p, dtype, stream);
}

cudaError_t launch_route_bwd(const RouteBwdParams& p, int dtype, cudaStream_t stream) {
  return route_typed(p, dtype, stream);
}

uint64_t moe_chunks(uint64_t tokens, uint32_t k) {
  const uint64_t chunk_tokens = kMoeChunkSlots / (k * kMoePlaceTokens) * kMoePlaceTokens;
  return ceil_div(tokens, chunk_tokens);
}

uint64_t moe_workspace_bytes(uint64_t tokens, uint32_t k, uint32_t experts) {
  return 4 * (static_cast<uint64_t>(experts) + 1) * (moe_chunks(tokens, k) + 1);
}

cudaError_t launch_dispatch(const DispatchParams& params, int dtype, bool vec, cudaStream_t stream,
                            const DeviceInfo& dev) {
  DispatchParams p = params;
  p.chunk_tokens = kMoeChunkSlots / (p.k * kMoePlaceTokens) * kMoePlaceTokens;
  p.chunks = static_cast<uint32_t>(moe_chunks(p.tokens, p.k));
  p.single = p.tokens * p.k <= kMoeSingleSlots;
  if (!p.single) {
    cudaError_t e = run(moe_count_kernel, p.chunks, 1, kSortThreads, stream, &p);
    if (e != cudaSuccess) return e;
    e = run(moe_prefix_kernel, ceil_div(p.experts + 1, 4), 1, 128, stream, &p);
    if (e != cudaSuccess) return e;
  }
  // Tokens per CTA: few while the grid does not fill the GPU, up to
  // kMoePlaceTokens once it does (the ranking is then shared by more rows).
  const uint64_t fill = 4ull * static_cast<uint64_t>(dev.sm_count);
  p.cta_tokens = static_cast<uint32_t>(p.tokens / fill);
  if (p.cta_tokens < 1) p.cta_tokens = 1;
  if (p.cta_tokens > kMoePlaceTokens) p.cta_tokens = kMoePlaceTokens;
  while (kMoePlaceTokens % p.cta_tokens) p.cta_tokens--;  // a CTA's tokens lie in one chunk
  const uint64_t grid = p.tokens ? ceil_div(p.tokens, p.cta_tokens) : 1;  // no tokens: the offsets are still written
  switch (dtype) {
    case ZC_BF16: return place<__nv_bfloat16>(p, vec, grid, 1, stream);
    case ZC_F16: return place<__half>(p, vec, grid, 1, stream);
    default: return place<float>(p, vec, grid, 1, stream);
  }
}

cudaError_t launch_combine(const CombineParams& params, int dtype, bool vec, cudaStream_t stream) {
  CombineParams p = params;
  switch (dtype) {
    case ZC_BF16: return combine<__nv_bfloat16>(p, vec, stream);
    case ZC_F16: return combine<__half>(p, vec, stream);
    default: return combine<float>(p, vec, stream);
  }
}

cudaError_t launch_combine_bwd(const CombineBwdParams& params, int dtype, bool vec, cudaStream_t stream) {
  CombineBwdParams p = params;
  switch (dtype) {
    case ZC_BF16:
      return vec ? combine_bwd<__nv_bfloat16, 8>(p, stream) : combine_bwd<__nv_bfloat16, 1>(p, stream);
    case ZC_F16: return vec ? combine_bwd<__half, 8>(p, stream) : combine_bwd<__half, 1>(p, stream);
    default: return vec ? combine_bwd<float, 4>(p, stream) : combine_bwd<float, 1>(p, stream);
  }
}

}  // namespace zc
