// zc_moe.cu -- the operators on both sides of an expert-parallel exchange: choosing experts for
// every token, sorting tokens by expert into contiguous pieces, bringing the experts' outputs back
// weighted, and their gradients.  Definitions in include/zc.h.
//
// All but the router are bound by memory: each value is read or written once and takes a few
// operations.  No result depends on the order of atomics (counts are whole numbers) and every sum
// has a fixed order, so the same inputs give the same bits.
#include <cfloat>

#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

namespace {

// ------------------------------------------------------------------ routing
constexpr int kRouteWarps = 4;  // tokens per CTA, one warp each

__device__ __forceinline__ uint32_t lanes_below() { return (1u << lane_id()) - 1u; }

// Order-preserving image of a score: larger score, larger key.  NaN is above everything, as a sort
// has it, so that it shows in the weights; both zeros are equal.  Up to kClosed (minus infinity) an
// expert cannot be chosen.
constexpr uint32_t kClosed = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float f) {
  const int32_t b = __float_as_int(f + 0.f);
  const uint32_t key = static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
  return f != f ? 0xFFFFFFFFu : key;
}

// The hyperbolic tangent, good to 2^-11 of it (the instruction's stated error).
__device__ __forceinline__ float tanh_estimate(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// An expert's choice: its logit, or its sigmoid plus its bias; minus infinity if it is closed.
__device__ __forceinline__ float choice_of(const RouteParams& p, float l, uint32_t e, float* prob) {
  if (!p.sigmoid || l == -INFINITY) return l;
  *prob = sigmoid(l);
  return p.bias ? __fadd_rn(*prob, p.bias[e]) : *prob;
}

// One warp per token, every lane holding N experts next to one another.  The K-th largest of the
// lanes' best choices is a bound that at least K experts reach and few more do: those are gathered
// in shared memory, a lane each, and every lane counts the ones before its own.  Where more than 32
// reach it (equal logits, or too few lanes left open) the largest is taken K times instead, the
// lowest expert on ties.  For the bound a sigmoid (1 + tanh(l / 2)) / 2 by the tanh instruction will
// do, at most 2^-12 off: with the bound lowered by four times that and the sums' rounding, no expert
// that belongs among the K stays out, and the exact sigmoid is taken of those gathered alone, one a
// lane.  Bound by instructions, 560 a warp at 70% of the issue slots: 16384 x 256 fp32, 8 taken with
// a bias, 10.8 us (softmax 9.5), its bytes 2.7.  With sigmoids good to 2^-20 for the bound and
// choices compared as whole numbers it took 12.6, with exact sigmoids of all experts 15.0; sorting
// each lane's experts and taking the largest 8 times 16.5 (512 experts: 41 against 15); warps that
// stay and load the next token ahead 18.3, for fewer of them fit an SM.
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteParams p) {
  __shared__ __align__(16) unsigned long long found[kRouteWarps][32];
  __shared__ float2 order[kRouteWarps][32];  // by rank: the expert, and its logit or its sigmoid
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride;
  float l[N], v[N];  // logits; choices, the sigmoid's estimated, NaN as infinity
  load_row<T, N, VEC>(row, p.experts, l);
  if (p.sigmoid) {
    float bias[N];
#pragma unroll
    for (int j = 0; j < N; j++) bias[j] = 0.f;
    if (p.bias) {
      if (VEC && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0 && p.experts % 4 == 0)
        load_row<float, N, true>(p.bias, p.experts, bias);
      else
        load_row<float, N, false>(p.bias, p.experts, bias);
    }
#pragma unroll
    for (int j = 0; j < N; j++)
      v[j] = l[j] == -INFINITY ? l[j] : fminf(fmaf(0.5f, tanh_estimate(0.5f * l[j]), 0.5f + bias[j]), INFINITY);
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) v[j] = fminf(l[j], INFINITY);
  }
  float bound;
  {
    float best = v[0];
#pragma unroll
    for (int j = 1; j < N; j++) best = fmaxf(best, v[j]);
    uint32_t lanes = 0;
    while (true) {
      bound = warp_max_of(best);
      if (bound == -INFINITY) break;
      lanes += __popc(__ballot_sync(kFull, best == bound));
      if (lanes >= p.k) break;
      best = best == bound ? -INFINITY : best;
    }
    if (p.sigmoid && bound < INFINITY) bound -= 0x1p-10f + fabsf(bound) * 0x1p-20f;
    bound = fmaxf(bound, -FLT_MAX);
  }
  uint32_t reach = 0;  // this lane's experts that reach it
#pragma unroll
  for (int j = 0; j < N; j++) reach |= v[j] >= bound ? 1u << j : 0u;
  uint32_t n = 0, at = 0;  // of the warp, and of the lanes below
#pragma unroll
  for (int b = 1; b <= N; b *= 2) {
    const uint32_t lanes = __ballot_sync(kFull, __popc(reach) & b);
    n += b * __popc(lanes);
    at += b * __popc(lanes & lanes_below());
  }
  if (n <= 32) {
    for (; reach; reach &= reach - 1) found[warp][at++] = lane * N + __ffs(reach) - 1;
  }
  uint32_t mine = kFull;
  float value = -INFINITY;  // of expert `mine`: its logit, or its sigmoid
  __syncwarp();
  if (n <= 32) {
    const uint32_t e = lane < n ? static_cast<uint32_t>(found[warp][lane]) : 0;
    float mid = lane < n ? to_f32<T>(row[e]) : -INFINITY, prob = 0.f;
    const uint32_t exact = order_key(choice_of(p, mid, e, &prob));
    if (p.sigmoid) mid = prob;
    const unsigned long long own = lane < n ? static_cast<unsigned long long>(exact) << 32 | (kFull - e) : 0;
    __syncwarp();
    found[warp][lane] = own;
    __syncwarp();
    uint32_t before = 0;
    for (uint32_t i = 0; i < n; i += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&found[warp][i]);
      before += (two.x > own) + (two.y > own);
    }
    if (lane < n) order[warp][before] = make_float2(__uint_as_float(e), mid);
    __syncwarp();
    if (lane < n && lane < p.k) {
      mine = __float_as_uint(order[warp][lane].x);
      value = order[warp][lane].y;
    }
  } else {
    uint32_t key[N];
#pragma unroll
    for (int j = 0; j < N; j++) {
      float prob;
      const uint32_t e = lane * N + j;
      key[j] = e < p.experts ? order_key(choice_of(p, l[j], e, &prob)) : 0;
    }
    for (uint32_t k = 0; k < p.k; k++) {
      uint32_t best = key[0], at = 0;
#pragma unroll
      for (int j = 1; j < N; j++)
        if (key[j] > best) best = key[j], at = j;
      const uint32_t top = __reduce_max_sync(kFull, best);
      if (top <= kClosed) break;
      const uint32_t winner = __ffs(__ballot_sync(kFull, best == top)) - 1;
      const uint32_t e = __shfl_sync(kFull, lane * N + at, winner);
      if (lane == k) mine = e;
#pragma unroll
      for (int j = 0; j < N; j++)
        if (lane == winner && at == j) key[j] = 0;
    }
    if (mine != kFull) {
      value = to_f32<T>(row[mine]);
      if (p.sigmoid) value = sigmoid(value);
    }
  }
  const bool have = mine != kFull;
  float w;
  if (p.sigmoid) {
    w = have ? value : 0.f;
    if (p.renormalize) w = w / (warp_sum_f32(w) + 1e-20f);
  } else {
    const float top = __shfl_sync(kFull, value, 0);  // the first pick is the row's largest logit
    w = have ? expf(value - top) : 0.f;
    float sum;
    if (p.renormalize) {
      sum = warp_sum_f32(w);
    } else {
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < N; j++) sum += l[j] == -INFINITY ? 0.f : expf(l[j] - top);
      sum = warp_sum_f32(sum);
    }
    w = have ? w / sum : 0.f;
  }
  if (lane < p.k) {
    p.weights[t * p.k + lane] = p.scale * w;
    p.ids[t * p.k + lane] = have ? static_cast<int32_t>(mine) : -1;
  }
}

// Gradient of the logits: G_k = scale dw_k for the chosen experts.  A renormalised softmax and both
// sigmoid forms depend on the chosen logits alone, so only those are read and every other gradient
// is zero; the plain softmax needs the whole row.  The chosen experts' values meet the lanes that
// hold those experts in a row of shared memory.
template <typename T, int N>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(RouteBwdParams p) {
  __shared__ float rows[kRouteWarps][32 * N];
  pdl_begin();
  const uint32_t lane = lane_id();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.stride;
  T* out = static_cast<T*>(p.dlogits) + t * p.experts;
  float* mid = rows[threadIdx.x >> 5];
#pragma unroll
  for (int j = 0; j < N; j++) mid[j * 32 + lane] = 0.f;
  int32_t id = -1;
  float g = 0.f, lm = -INFINITY;
  if (lane < p.k) {
    id = p.ids[t * p.k + lane];
    if (static_cast<uint32_t>(id) >= p.experts) id = -1;
    if (id >= 0) {
      g = p.scale * p.dweights[t * p.k + lane];
      lm = to_f32<T>(row[id]);
      if (lm == -INFINITY) id = -1, g = 0.f;  // the router cannot have chosen it
    }
  }
  const bool have = id >= 0;
  const bool whole = !p.sigmoid && !p.renormalize;
  float prob[N];
  float d = 0.f, mean = 0.f;  // this lane's chosen logit's gradient; sum of G p over the row
  if (whole) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; j++) {  // lane l's experts: l, l + 32, ...
      const uint32_t e = j * 32 + lane;
      prob[j] = e < p.experts ? to_f32<T>(row[e]) : -INFINITY;
      top = fmaxf(top, prob[j]);
    }
    top = warp_max_f32(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) {
      prob[j] = prob[j] == -INFINITY ? 0.f : expf(prob[j] - top);
      sum += prob[j];
    }
    sum = warp_sum_f32(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row with every expert masked has no gradient
#pragma unroll
    for (int j = 0; j < N; j++) prob[j] *= inv;
    mean = warp_sum_f32(have ? g * (expf(lm - top) * inv) : 0.f);
    d = g;
  } else if (p.sigmoid) {
    const float s = have ? sigmoid(lm) : 0.f;
    if (p.renormalize) {
      const float total = warp_sum_f32(s) + 1e-20f;
      g = (g - warp_sum_f32(g * s) / total) / total;
    }
    // 1 - s: as a difference it keeps no bits from a logit of 17 on (at 10 it is off by 2^-11)
    d = have ? g * s * (lm > 0.f ? expf(-lm) * s : 1.f - s) : 0.f;
  } else {
    const float top = warp_max_f32(lm);
    float f = have ? expf(lm - top) : 0.f;
    const float sum = warp_sum_f32(f);
    f = have ? f / sum : 0.f;
    d = f * (g - warp_sum_f32(g * f));
  }
  __syncwarp();
  // An expert named more than once (never by the router) gets its gradients one after the other.
  if (have) mid[id] = __uint_as_float(lane);
  __syncwarp();
  const bool alone = !have || __float_as_uint(mid[id]) == lane;
  if (__all_sync(kFull, alone)) {
    if (have) mid[id] = d;
  } else {
    if (have) mid[id] = 0.f;
    __syncwarp();
    for (uint32_t k = 0; k < p.k; k++) {
      if (lane == k && have) mid[id] += d;
      __syncwarp();
    }
  }
  __syncwarp();
  if (!whole) {
    for (uint32_t e = lane; e < p.experts; e += 32) out[e] = from_f32<T>(mid[e]);
    return;
  }
#pragma unroll
  for (int j = 0; j < N; j++) {
    const uint32_t e = j * 32 + lane;
    if (e < p.experts) out[e] = from_f32<T>(prob[j] * (mid[e] - mean));
  }
}

// ------------------------------------------------------------------ dispatch
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;

// The expert of slot i, or `experts` for a slot that is not routed.
__device__ __forceinline__ uint32_t slot_key(const DispatchParams& p, uint64_t i) {
  const int64_t v = p.ids64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
  return v >= 0 && v < static_cast<int64_t>(p.experts) ? static_cast<uint32_t>(v) : p.experts;
}

// The lanes whose key equals this one's, by a vote on each of the low `bits` bits.
__device__ __forceinline__ uint32_t equal_lanes(uint32_t key, int bits) {
  uint32_t equal = kFull;
  for (int b = 0; b < bits; b++) {
    const bool one = (key >> b) & 1u;
    const uint32_t ones = __ballot_sync(kFull, one);
    equal &= one ? ones : ~ones;
  }
  return equal;
}
// Bits that tell 0 .. experts and "no slot" (all ones) apart.
__device__ __forceinline__ int key_bits(uint32_t experts) { return 32 - __clz(experts + 1); }

// Exclusive prefix sums of a[0 .. count), in place, over a CTA of whole warps.
__device__ __forceinline__ void block_exclusive_scan(uint32_t* a, uint32_t count, uint32_t* warp_totals) {
  const uint32_t per = (count + blockDim.x - 1) / blockDim.x, first = threadIdx.x * per;
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

// The stable counting sort of a call with many slots, first of three launches.  A CTA takes a chunk
// of 1024 slots, each warp an eighth of it in order: counts per warp and expert, their prefix over
// the warps, and then every slot's place among its expert's in the chunk, 32 at a time (its equals
// among the lanes below it).  positions[] holds that place until the rows are placed.
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(DispatchParams p) {
  extern __shared__ uint32_t hist[];  // [kSortWarps][experts + 1]
  pdl_allow_dependents();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  pdl_wait();
  const uint32_t e1 = p.experts + 1;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kMoeChunkSlots;
  const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kMoeChunkSlots), p.tokens * p.k - first));
  constexpr uint32_t kTurns = kMoeChunkSlots / kSortThreads;
  const uint32_t base = warp * (kTurns * 32) + lane;
  uint32_t key[kTurns];
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) key[i] = base + i * 32 < n ? slot_key(p, first + base + i * 32) : kFull;
  uint32_t* own = hist + warp * e1;
  for (uint32_t e = lane; e < e1; e += 32) own[e] = 0;
  const int bits = key_bits(p.experts);
  uint32_t equal[kTurns];
  __syncwarp();
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) {
    equal[i] = equal_lanes(key[i], bits);
    if (key[i] != kFull && (equal[i] & lanes_below()) == 0) own[key[i]] += __popc(equal[i]);
    __syncwarp();
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < e1; e += kSortThreads) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; w++) {
      const uint32_t c = hist[w * e1 + e];
      hist[w * e1 + e] = sum;
      sum += c;
    }
    p.counts[static_cast<uint64_t>(e) * p.chunks + blockIdx.x] = sum;
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) {
    const uint32_t below = equal[i] & lanes_below();
    if (key[i] != kFull) p.positions[first + base + i * 32] = static_cast<int32_t>(own[key[i]] + __popc(below));
    __syncwarp();
    if (key[i] != kFull && below == 0) own[key[i]] += __popc(equal[i]);
    __syncwarp();
  }
}

// With many counts: the exclusive prefix over the chunks of every expert, in place, a warp per expert, and
// from the totals the experts' first rows.  One cluster: its CTAs leave their totals in the first
// one's shared memory, which adds them up (256 experts, 64 chunks: 5.5 us by itself, in one CTA
// 13.5).  Letting every CTA of the last launch add up what its slots need instead took longer:
// 131072 slots of 512 values 58 us against 41, and sorting in one cluster of 8 CTAs 55.
constexpr uint32_t kPrefixCtas = 8;
constexpr int kPrefixThreads = 1024;
__global__ void __launch_bounds__(kPrefixThreads) __cluster_dims__(kPrefixCtas, 1, 1)
    moe_prefix_kernel(DispatchParams p) {
  __shared__ uint32_t total[kMoeMaxExperts + 1];
  __shared__ uint32_t warp_totals[32];
  pdl_allow_dependents();
  const uint32_t lane = lane_id(), warps = kPrefixCtas * (kPrefixThreads / 32);
  cluster_arrive();  // shared memory of the first CTA may be written once it has started, that is after this barrier
  pdl_wait();
  cluster_wait();
  for (uint32_t e = (threadIdx.x >> 5) * kPrefixCtas + blockIdx.x; e <= p.experts; e += warps) {
    uint32_t* c = p.counts + static_cast<uint64_t>(e) * p.chunks;
    uint32_t base = 0;
    for (uint32_t i = 0; i < p.chunks; i += 128) {  // four pieces on their way at once
      uint32_t v[4];
#pragma unroll
      for (uint32_t q = 0; q < 4; q++) v[q] = i + q * 32 + lane < p.chunks ? c[i + q * 32 + lane] : 0;
#pragma unroll
      for (uint32_t q = 0; q < 4; q++) {
        if (i + q * 32 >= p.chunks) break;
        const uint32_t upto = warp_inclusive_scan(v[q]);
        if (i + q * 32 + lane < p.chunks) c[i + q * 32 + lane] = base + upto - v[q];
        base += __shfl_sync(kFull, upto, 31);
      }
    }
    if (lane == 0) st_shared_of_cta(&total[e], 0, base);
  }
  cluster_arrive();
  cluster_wait();
  if (blockIdx.x) return;
  block_exclusive_scan(total, p.experts + 1, warp_totals);
  for (uint32_t e = threadIdx.x; e <= p.experts; e += kPrefixThreads) p.offsets[e] = static_cast<int32_t>(total[e]);
}

// Where a slot's row goes.  A token's row is read in its own aligned pieces; off bytes into every
// pair of neighbours lie the 16 bytes of an aligned piece of the row to write.
struct PlaceRow {
  uint64_t at;   // address of the piece that pair 0 holds
  uint32_t off;  // 0 .. 15
  uint32_t routed;
};

// Last: the row of every slot, and the rows themselves.  A CTA places the slots of a few tokens,
// then reads each token once and writes its K rows.  A slot's row is its expert's first + those in
// earlier chunks + its place in the chunk.  Where there are few counts (`few_counts`) the CTA adds
// them up itself and the launch of the prefix falls away: 4096 slots of 128 experts 6.7 us against
// 7.8, 12288 8.3 against 9.4; 16384 of 128, 2064 counts, 12.4 against 10.5.  With few slots
// (`single`) it counts all of them itself, those before its own apart (two counts in a word), and
// ranks its own by ballots, so that the call is one launch: 1024 slots 3.2 us against 5.2 in two,
// 2048 4.2 against 5.6, 4096 7.3 against 6.6.  Slots of the same token never meet in a bin of this
// count, with fewer than four a token more lanes may: 2048 skewed slots, one a token, 10.4 against
// 7.6.  (Clusters of 8 CTAs that share this count: 4096 slots 8.2, 8192 9.8.)  Bound by memory,
// mostly writes: 16384 x 4096 bf16 to 4 experts each, 0.67 GB, 115 us in all, of which the sort
// about 7.  Rows off 16 bytes are read once, in pairs of pieces, and shifted for every slot: 16384 x
// 4095 131 us; with a read for every slot, cut at that row's own pieces, 174.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(DispatchParams p) {
  __shared__ uint32_t start[kMoeMaxExperts + 1];
  __shared__ uint32_t before[kMoeMaxExperts + 1];
  __shared__ uint32_t warp_totals[kSortWarps];
  __shared__ PlaceRow own_row[kMoePlaceTokens * kMoeMaxK];
  pdl_allow_dependents();
  const uint32_t lane = lane_id();
  pdl_wait();
  const uint64_t t0 = static_cast<uint64_t>(blockIdx.x) * p.cta_tokens;
  const uint32_t nt = static_cast<uint32_t>(min(static_cast<uint64_t>(p.cta_tokens), p.tokens - min(p.tokens, t0)));
  const uint64_t s0 = t0 * p.k;
  const uint32_t own = nt * p.k;
  auto token = [&](uint32_t t) { return static_cast<const T*>(p.x) + (t0 + t) * p.stride; };
  // Row r is that of the CTA's slot i.
  auto place = [&](uint32_t i, uint32_t r, bool routed) {
    const int32_t pos = routed ? static_cast<int32_t>(r) : ~static_cast<int32_t>(r);
    const uint64_t dst = reinterpret_cast<uint64_t>(static_cast<T*>(p.rows) + static_cast<uint64_t>(r) * p.hidden);
    const uint32_t lead = VEC ? 0 : reinterpret_cast<uintptr_t>(token(i / p.k)) & 15;
    const uint32_t off = VEC ? 0 : (lead - static_cast<uint32_t>(dst)) & 15;
    own_row[i] = PlaceRow{dst - lead + off, off, routed};
    p.positions[s0 + i] = pos;
    p.slots[r] = static_cast<int32_t>(s0 + i);
  };
  if (p.single) {
    const uint32_t all = static_cast<uint32_t>(p.tokens) * p.k, mine = static_cast<uint32_t>(s0);
    for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) start[e] = 0;
    __syncthreads();
    constexpr uint32_t kTurns = 8;  // keys on their way at once
    for (uint32_t i = threadIdx.x; i < all; i += kTurns * kSortThreads) {
      uint32_t key[kTurns];
#pragma unroll
      for (uint32_t q = 0; q < kTurns; q++)
        key[q] = i + q * kSortThreads < all ? slot_key(p, i + q * kSortThreads) : kFull;
#pragma unroll
      for (uint32_t q = 0; q < kTurns; q++)
        if (key[q] != kFull) atomicAdd(&start[key[q]], i + q * kSortThreads < mine ? 0x10001u : 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) {
      before[e] = start[e] >> 16;
      start[e] &= 0xFFFFu;
    }
    __syncthreads();
    block_exclusive_scan(start, p.experts + 1, warp_totals);
    if (blockIdx.x == 0)
      for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) p.offsets[e] = static_cast<int32_t>(start[e]);
    if (threadIdx.x < 32) {
      const int bits = key_bits(p.experts);
      for (uint32_t i = lane; i < (own + 31) / 32 * 32; i += 32) {
        const uint32_t e = i < own ? slot_key(p, s0 + i) : kFull;
        const uint32_t equal = equal_lanes(e, bits);
        uint32_t r = 0;
        if (e != kFull) r = start[e] + before[e] + __popc(equal & lanes_below());
        __syncwarp();
        if (e != kFull && (equal & lanes_below()) == 0) before[e] += __popc(equal);
        __syncwarp();
        if (e == kFull) continue;
        place(i, r, e < p.experts);
      }
    }
  } else {
    if (p.few_counts) {
      for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) {
        uint32_t sum = 0;
#pragma unroll 8
        for (uint32_t c = 0; c < p.chunks; c++) sum += p.counts[e * p.chunks + c];
        start[e] = sum;
      }
      __syncthreads();
      block_exclusive_scan(start, p.experts + 1, warp_totals);
      if (blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e <= p.experts; e += kSortThreads) p.offsets[e] = static_cast<int32_t>(start[e]);
    }
    for (uint32_t i = threadIdx.x; i < own; i += kSortThreads) {
      const uint32_t e = slot_key(p, s0 + i), chunk = static_cast<uint32_t>((s0 + i) / kMoeChunkSlots);
      const uint32_t* counts = p.counts + static_cast<uint64_t>(e) * p.chunks;
      uint32_t r = static_cast<uint32_t>(p.positions[s0 + i]);
      if (p.few_counts) {
        r += start[e];
#pragma unroll 8
        for (uint32_t c = 0; c < chunk; c++) r += counts[c];
      } else {
        r += static_cast<uint32_t>(p.offsets[e]) + counts[chunk];
      }
      place(i, r, e < p.experts);
    }
  }
  __syncthreads();
  constexpr uint32_t V = kPieceOf<T>;
  const uint32_t pieces = VEC ? p.hidden / V : any_pairs<T>(p.hidden);
  const uint64_t all = static_cast<uint64_t>(nt) * pieces;
#pragma unroll 2
  for (uint64_t i = threadIdx.x; i < all; i += kSortThreads) {
    const uint32_t t = all >> 32 ? static_cast<uint32_t>(i / pieces) : static_cast<uint32_t>(i) / pieces;
    const uint32_t u = static_cast<uint32_t>(i) - t * pieces - (VEC ? 0 : 1);  // -1: the pair before the row's pieces
    const uint64_t src = reinterpret_cast<uint64_t>(token(t));
    const PlaceRow* rows = own_row + t * p.k;
    const uint32_t lead = VEC ? 0 : src & 15, held = (lead / static_cast<uint32_t>(sizeof(T)) + p.hidden + V - 1) / V;
    const uint4* from = reinterpret_cast<const uint4*>(src - lead) + static_cast<int32_t>(u);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 lo = zero, hi = zero;
    if (VEC || u < held) lo = from[0];
    if (!VEC && u + 1 < held) hi = from[1];
    for (uint32_t k = 0; k < p.k; k++) {
      const PlaceRow row = rows[k];
      uint4* to = reinterpret_cast<uint4*>(row.at) + static_cast<int32_t>(u);
      const uint4 v = !row.routed ? zero : VEC ? lo : shift_pieces<T>(lo, hi, row.off);
      // the piece's first value; it wraps below 0
      const uint32_t first = u * V + static_cast<uint32_t>((static_cast<int32_t>(row.off) - static_cast<int32_t>(lead)) /
                                                             static_cast<int32_t>(sizeof(T)));
      if (VEC || whole_piece<T>(first, p.hidden)) {
        *to = v;
      } else {
        store_part<T>(reinterpret_cast<T*>(to), Piece<T, V>{v}, first, p.hidden);
      }
    }
  }
}

// ------------------------------------------------------------------ combine
constexpr int kCombineThreads = 256;
constexpr int kCombineLoads = 8;  // pieces a thread has in flight

// The row of a slot: true if it is routed.  `row` is the row to read (or, unrouted, the one to
// clear, which the buffer need not hold); a routed row outside the buffer is reported and skipped.
__device__ __forceinline__ bool slot_row(int32_t pos, uint64_t n_rows, int32_t* status, uint64_t* row, bool* inside) {
  *row = static_cast<uint64_t>(pos < 0 ? ~pos : pos);
  *inside = *row < n_rows;
  if (!*inside && pos >= 0) set_status(status, ZC_ERR_BAD_INDEX);
  return *inside && pos >= 0;
}

// out[t] = sum over k, in order, of w[t][k] rows[pos[t][k]], in fp32.  A thread has 8 16-byte
// pieces in flight before it adds the first: those of KU slots of 8 / KU pieces of the output,
// kCombineThreads pieces apart.  More than 8 slots (LOOP) are added KU at a time.  Bound by memory:
// 16384 x 4096 bf16 from 4 slots each, 0.67 GB, 101 us, the measured copy's rate; one piece of 4
// slots at a time 132.
template <typename T, int KU, bool LOOP>
__global__ void __launch_bounds__(kCombineThreads, KU <= 2 ? 3 : 4) moe_combine_kernel(CombineParams p) {
  constexpr int V = kPieceOf<T>, kPieces = kCombineLoads / KU;
  pdl_begin();
  const uint32_t pieces = p.hidden / V;
  // the CTA's first piece: token t0, piece c0 of it
  const uint64_t i0 = static_cast<uint64_t>(blockIdx.x) * (kCombineThreads * kPieces);
  const uint64_t t0 = i0 / pieces;
  const uint32_t c0 = static_cast<uint32_t>(i0 - t0 * pieces) + threadIdx.x;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; j++) acc[j] = 0.f;
  for (uint32_t k0 = 0; k0 < (LOOP ? p.k : 1u); k0 += KU) {
    Piece<T, V> v[kPieces][KU];
    float w[kPieces][KU];
    T* to[kPieces];
#pragma unroll
    for (int q = 0; q < kPieces; q++) {
      const uint32_t i = c0 + q * kCombineThreads, dt = i / pieces, first = (i - dt * pieces) * V;
      const uint64_t t = t0 + dt;
      to[q] = t < p.tokens ? static_cast<T*>(p.out) + t * p.hidden + first : nullptr;
#pragma unroll
      for (int k = 0; k < KU; k++) {
        w[q][k] = 0.f;
        v[q][k] = Piece<T, V>::zero();
        if (to[q] && k0 + k < p.k) {
          uint64_t row;
          bool inside;
          if (slot_row(p.positions[t * p.k + k0 + k], p.n_rows, p.status, &row, &inside)) {
            w[q][k] = p.weights ? p.weights[t * p.k + k0 + k] : 1.f;
            v[q][k] = Piece<T, V>::load(static_cast<const T*>(p.rows) + row * p.row_stride + first);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kPieces; q++) {
#pragma unroll
      for (int k = 0; k < KU; k++) {
        float f[V];
        v[q][k].get(f);
#pragma unroll
        for (int j = 0; j < V; j++) acc[j] = fmaf(w[q][k], f[j], acc[j]);
      }
      if ((!LOOP || k0 + KU >= p.k) && to[q]) {
        Piece<T, V> o;
        o.set(acc);
        o.store(to[q]);
      }
      if (!LOOP) {
#pragma unroll
        for (int j = 0; j < V; j++) acc[j] = 0.f;
      }
    }
  }
}

// The same for rows that lie off 16 bytes: a warp takes some of the units of a token's output
// (RowCut).  Each slot's row has its own place relative to those pieces, found once by a lane and
// kept in shared memory: the piece that output piece 0 starts in, and at which byte.  Bound by the
// instructions that shift the pieces: 16384 x 4095 bf16 from 4 slots each 138 us in 32 registers,
// 154 in 40; fp32, with half the values a piece, 208, the copy's rate; with all of this found by
// every thread for itself 225 and 436.
constexpr uint32_t kAnySlots = 4;  // slots read at once
constexpr uint32_t kAnyTurns = 4;  // units of a lane, where there are many (8: 164 us against 152)
struct AnyRow {
  uint64_t at;  // 0: nothing to add
  uint32_t off;
  float w;
};

template <typename T>
__global__ void __launch_bounds__(kCombineThreads, 8) moe_combine_any_kernel(CombineParams p, uint32_t turns) {
  constexpr int V = kPieceOf<T>;
  __shared__ AnyRow rows_of[kCombineThreads / 32][kMoeMaxK];
  pdl_begin();
  const uint32_t lane = lane_id(), units = any_units<T>(p.hidden), shares = (units + 32 * turns - 1) / (32 * turns);
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * (kCombineThreads / 32) + (threadIdx.x >> 5), t = i / shares;
  if (t >= p.tokens) return;
  const uint32_t share = static_cast<uint32_t>(i - t * shares);
  AnyRow* rows = rows_of[threadIdx.x >> 5];
  T* out = static_cast<T*>(p.out) + t * p.hidden;
  const RowCut<T> cut(out, p.hidden);
  if (lane < p.k) {
    AnyRow r{0, 0, 0.f};
    uint64_t row;
    bool inside;
    if (slot_row(p.positions[t * p.k + lane], p.n_rows, p.status, &row, &inside)) {
      const uint64_t at =
          reinterpret_cast<uint64_t>(static_cast<const T*>(p.rows) + row * p.row_stride + cut.head);
      r = AnyRow{at & ~15ull, static_cast<uint32_t>(at & 15), p.weights ? p.weights[t * p.k + lane] : 1.f};
    }
    rows[lane] = r;
  }
  __syncwarp();
  for (uint32_t turn = 0; turn < turns; turn++) {
    const uint32_t u = (share * turns + turn) * 32 + lane;
    uint32_t first;
    const uint32_t values = cut.unit(u, p.hidden, &first);
    if (values == V) {
      float acc[V];
#pragma unroll
      for (int j = 0; j < V; j++) acc[j] = 0.f;
      for (uint32_t k0 = 0; k0 < p.k; k0 += kAnySlots) {
        uint4 lo[kAnySlots], hi[kAnySlots];
        AnyRow r[kAnySlots];
#pragma unroll
        for (uint32_t k = 0; k < kAnySlots; k++) {
          r[k] = k0 + k < p.k ? rows[k0 + k] : AnyRow{0, 0, 0.f};
          lo[k] = hi[k] = make_uint4(0u, 0u, 0u, 0u);
          const uint4* from = reinterpret_cast<const uint4*>(r[k].at) + u;
          if (r[k].at) lo[k] = from[0];
          if (r[k].off) hi[k] = from[1];
        }
#pragma unroll
        for (uint32_t k = 0; k < kAnySlots; k++) {
          float f[V];
          Piece<T, V>{shift_pieces<T>(lo[k], hi[k], r[k].off)}.get(f);
#pragma unroll
          for (int j = 0; j < V; j++) acc[j] = fmaf(r[k].w, f[j], acc[j]);
        }
      }
      Piece<T, V> o;
      o.set(acc);
      o.store(out + first);
    } else if (values) {  // a value outside the pieces
      float sum = 0.f;
#pragma unroll 4
      for (uint32_t k = 0; k < p.k; k++) {
        const AnyRow r = rows[k];
        if (!r.at) continue;
        const T* from = reinterpret_cast<const T*>(r.at + r.off) + (static_cast<int64_t>(first) - cut.head);
        sum = fmaf(r.w, to_f32<T>(*from), sum);
      }
      out[first] = from_f32<T>(sum);
    }
  }
}

// drows[pos] = w dout and dw = <dout, rows[pos]>: dout's row is read once for four slots, each row
// once; the products are summed in registers over a thread's pieces, then over the CTA (or the
// warp, for narrow rows).  Bound by memory: 16384 x 4096 bf16, 4 slots each, 1.21 GB, 181 us, the
// measured copy's rate; off 16 bytes by the instructions that shift the pieces, 4095 wide 254 us (two
// slots at once in 64 registers; four in 124 423).
template <bool VEC>
constexpr int kCombineBwdK = VEC ? 4 : 2;  // slots at once; off 16 bytes four take twice the registers

template <typename T, bool VEC, bool WARP>
__global__ void __launch_bounds__(512, 2) moe_combine_bwd_kernel(CombineBwdParams p) {
  constexpr int V = kPieceOf<T>, KU = kCombineBwdK<VEC>;
  __shared__ float red[2][KU * 32];
  pdl_begin();
  const uint32_t lane = lane_id(), warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  const uint64_t t = WARP ? static_cast<uint64_t>(blockIdx.x) * warps + warp : blockIdx.x;
  if (t >= p.tokens) return;
  const uint32_t me = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const uint32_t pieces = VEC ? p.hidden / V : any_pairs<T>(p.hidden);
  const T* dout = static_cast<const T*>(p.dout) + t * p.dout_stride;
  for (uint32_t k0 = blockIdx.y * KU, turn = 0; k0 < p.k; k0 += gridDim.y * KU, turn ^= 1) {
    float dot[KU], w[KU];
    const T* from[KU];
    T* to[KU];
    bool routed[KU], inside[KU];
#pragma unroll
    for (int k = 0; k < KU; k++) {
      dot[k] = 0.f;
      w[k] = 0.f;
      routed[k] = inside[k] = false;
      from[k] = nullptr;
      to[k] = nullptr;
      if (k0 + k < p.k) {
        uint64_t row;
        routed[k] = slot_row(p.positions[t * p.k + k0 + k], p.n_rows, p.status, &row, &inside[k]);
        if (routed[k]) w[k] = p.weights[t * p.k + k0 + k];
        from[k] = static_cast<const T*>(p.rows) + row * p.row_stride;
        to[k] = static_cast<T*>(p.drows) + row * p.hidden;
      }
    }
    // Off 16 bytes: dout is read in pairs of its own pieces; `off` bytes into each lies a piece of the
    // gradient's row k to write, which takes the values of the row itself that start at byte `foff`
    // of a piece (none, where both rows lie alike).
    uint32_t off[KU], foff[KU];
    const uint32_t lead = VEC ? 0 : reinterpret_cast<uintptr_t>(dout) & 15;
    const uint32_t held = (lead / static_cast<uint32_t>(sizeof(T)) + p.hidden + V - 1) / V;
    if (!VEC) {
#pragma unroll
      for (int k = 0; k < KU; k++) {
        off[k] = (lead - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to[k]))) & 15;
        const int64_t move = static_cast<int64_t>(off[k]) - lead;
        to[k] = reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(to[k]) + move);
        const uintptr_t at = reinterpret_cast<uintptr_t>(from[k]) + move;
        foff[k] = at & 15;
        from[k] = reinterpret_cast<const T*>(at - foff[k]);
      }
    }
    for (uint32_t i = me; i < pieces; i += step) {
      if (VEC) {
        const uint64_t at = static_cast<uint64_t>(i) * V;
        float g[V];
        Piece<T, V> v[KU];
#pragma unroll
        for (int k = 0; k < KU; k++)
          v[k] = routed[k] ? Piece<T, V>::load(from[k] + at) : Piece<T, V>::zero();
        Piece<T, V>::load(dout + at).get(g);
#pragma unroll
        for (int k = 0; k < KU; k++) {
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
          o.store(to[k] + at);
        }
      } else {
        const uint32_t u = i - 1;  // -1: the pair before dout's pieces
        const int64_t at = static_cast<int64_t>(static_cast<int32_t>(u)) * V;
        const uint4* g_at = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(dout) - lead) +
                            static_cast<int32_t>(u);
        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo, vlo[KU], vhi[KU];
        uint32_t first[KU];
        if (u < held) lo = g_at[0];
        if (u + 1 < held) hi = g_at[1];
#pragma unroll
        for (int k = 0; k < KU; k++) {
          first[k] = u * V + static_cast<uint32_t>((static_cast<int32_t>(off[k]) - static_cast<int32_t>(lead)) /
                                                   static_cast<int32_t>(sizeof(T)));
          vlo[k] = vhi[k] = make_uint4(0u, 0u, 0u, 0u);
          if (routed[k] && whole_piece<T>(first[k], p.hidden)) {
            const uint4* v_at = reinterpret_cast<const uint4*>(from[k] + at);
            vlo[k] = v_at[0];
            if (foff[k]) vhi[k] = v_at[1];
          }
        }
#pragma unroll
        for (int k = 0; k < KU; k++) {
          if (!inside[k]) continue;
          float f[V], d[V];
          Piece<T, V>{shift_pieces<T>(lo, hi, off[k])}.get(d);
          if (whole_piece<T>(first[k], p.hidden)) {
            if (foff[k]) vlo[k] = shift_pieces<T>(vlo[k], vhi[k], foff[k]);
            Piece<T, V>{vlo[k]}.get(f);
#pragma unroll
            for (int j = 0; j < V; j++) {
              dot[k] = routed[k] ? fmaf(d[j], f[j], dot[k]) : 0.f;
              d[j] = routed[k] ? w[k] * d[j] : 0.f;
            }
            Piece<T, V> o;
            o.set(d);
            o.store(to[k] + at);
          } else {  // a piece that the row does not fill
            const T* v_at =
                reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(from[k]) + foff[k]) + at;
#pragma unroll
            for (int j = 0; j < V; j++) {
              if (routed[k] && first[k] + j < p.hidden) dot[k] = fmaf(d[j], to_f32<T>(v_at[j]), dot[k]);
              d[j] = routed[k] ? w[k] * d[j] : 0.f;
            }
            Piece<T, V> o;
            o.set(d);
            store_part<T>(to[k] + at, o, first[k], p.hidden);
          }
        }
      }
    }
    if (WARP) {
#pragma unroll
      for (int k = 0; k < KU; k++) dot[k] = warp_sum_f32(dot[k]);
    } else {
      block_sum_f32<KU>(dot, red[turn]);
    }
    if (me == 0) {
#pragma unroll
      for (int k = 0; k < KU; k++)
        if (k0 + k < p.k) p.dweights[t * p.k + k0 + k] = dot[k];
    }
  }
}

// ------------------------------------------------------------------ launches
template <typename F>
cudaError_t run(F* kernel, uint64_t grid_x, uint32_t grid_y, int threads, cudaStream_t stream, void* params,
                int smem = 0) {
  if (grid_x == 0) return cudaSuccess;
  if (grid_x > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  void* args[] = {params};
  return launch_kernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<unsigned>(grid_x), grid_y),
                       dim3(threads), smem, stream, args, false);
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

template <typename T, int N>
cudaError_t route_width(RouteParams& p, cudaStream_t stream) {
  // a lane's values as whole pieces: of 16 bytes, or of all its values where those are fewer
  constexpr uint64_t kPart = N * sizeof(T) < 16 ? N * sizeof(T) : 16;
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % kPart == 0 && p.stride * sizeof(T) % kPart == 0 &&
                   p.experts * sizeof(T) % kPart == 0;
  const uint64_t grid = ceil_div(p.tokens, kRouteWarps);
  if (vec) return run(route_kernel<T, N, true>, grid, 1, kRouteWarps * 32, stream, &p);
  return run(route_kernel<T, N, false>, grid, 1, kRouteWarps * 32, stream, &p);
}
template <typename T, int N>
cudaError_t route_width(RouteBwdParams& p, cudaStream_t stream) {
  return run(route_bwd_kernel<T, N>, ceil_div(p.tokens, kRouteWarps), 1, kRouteWarps * 32, stream, &p);
}

template <typename T, typename P>
cudaError_t route_of(const P& params, cudaStream_t stream) {
  P p = params;
  if (p.experts <= 32) return route_width<T, 1>(p, stream);
  if (p.experts <= 64) return route_width<T, 2>(p, stream);
  if (p.experts <= 128) return route_width<T, 4>(p, stream);
  if (p.experts <= 256) return route_width<T, 8>(p, stream);
  if (p.experts <= 512) return route_width<T, 16>(p, stream);
  return route_width<T, 32>(p, stream);
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
cudaError_t place(DispatchParams& p, bool vec, uint64_t grid, cudaStream_t stream) {
  if (vec) return run(moe_place_kernel<T, true>, grid, 1, kSortThreads, stream, &p);
  return run(moe_place_kernel<T, false>, grid, 1, kSortThreads, stream, &p);
}

template <typename T>
cudaError_t combine(CombineParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  if (!vec) {
    // one unit a lane until the warps fill the GPU
    const uint64_t turns_all = ceil_div(any_units<T>(p.hidden), 32);
    uint64_t turns = p.tokens * turns_all / (64ull * static_cast<uint64_t>(dev.sm_count));
    turns = turns < 1 ? 1 : turns > kAnyTurns ? kAnyTurns : turns;
    turns = ceil_div(turns_all, ceil_div(turns_all, turns));  // evenly over a token's warps
    uint32_t each = static_cast<uint32_t>(turns);
    const uint64_t grid = ceil_div(p.tokens * ceil_div(turns_all, turns), kCombineThreads / 32);
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    void* args[] = {&p, &each};
    return launch_kernel(reinterpret_cast<const void*>(moe_combine_any_kernel<T>), dim3(static_cast<unsigned>(grid)),
                         dim3(kCombineThreads), 0, stream, args, false);
  }
  const uint64_t all = p.tokens * (p.hidden / kPieceOf<T>);
  const int ku = p.k <= 1 ? 1 : p.k <= 2 ? 2 : p.k <= 4 ? 4 : 8;
  const uint64_t grid = ceil_div(all, kCombineThreads * (kCombineLoads / ku));
  if (p.k > 8) return run(moe_combine_kernel<T, 8, true>, grid, 1, kCombineThreads, stream, &p);
  switch (ku) {
    case 1: return run(moe_combine_kernel<T, 1, false>, grid, 1, kCombineThreads, stream, &p);
    case 2: return run(moe_combine_kernel<T, 2, false>, grid, 1, kCombineThreads, stream, &p);
    case 4: return run(moe_combine_kernel<T, 4, false>, grid, 1, kCombineThreads, stream, &p);
    default: return run(moe_combine_kernel<T, 8, false>, grid, 1, kCombineThreads, stream, &p);
  }
}

template <typename T, bool VEC>
cudaError_t combine_bwd(CombineBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  const uint64_t pieces = VEC ? p.hidden / kPieceOf<T> : any_pairs<T>(p.hidden);
  // Few tokens leave SMs idle: their slots, a few at a time, then go to CTAs of their own, which
  // hold a piece a thread.
  const bool few = p.tokens < 2ull * static_cast<uint64_t>(dev.sm_count);
  const uint32_t split = few ? static_cast<uint32_t>(ceil_div(p.k, kCombineBwdK<VEC>)) : 1;
  // a warp a token while that is a few turns: 16384 x 640 bf16 32.8 us against 38.1 by two warps, 2048 92.4
  // against 90.8 by four
  if (pieces <= (few ? 64 : 128))
    return run(moe_combine_bwd_kernel<T, VEC, true>, ceil_div(p.tokens, 4), split, 128, stream, &p);
  // a piece a thread up to 16 warps, or 8 warps in whole turns; off 16 bytes 4 (16384 x 4095 bf16 254 us
  // against 303)
  const uint64_t turns = few ? ceil_div(pieces, 512) : pieces < 512 ? 2 : pieces / (VEC ? 256 : 128);
  return run(moe_combine_bwd_kernel<T, VEC, false>, p.tokens, split, static_cast<int>(32 * ceil_div(pieces, 32 * turns)),
             stream, &p);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t stream) {
  return route_typed(p, dtype, stream);
}

cudaError_t launch_route_bwd(const RouteBwdParams& p, int dtype, cudaStream_t stream) {
  return route_typed(p, dtype, stream);
}

uint64_t moe_workspace_bytes(uint64_t tokens, uint32_t k, uint32_t experts) {
  return 4 * (static_cast<uint64_t>(experts) + 1) * (ceil_div(tokens * k, kMoeChunkSlots) + 1);
}

cudaError_t launch_dispatch(const DispatchParams& params, int dtype, bool vec, cudaStream_t stream,
                            const DeviceInfo& dev) {
  DispatchParams p = params;
  const uint64_t slots = p.tokens * p.k;
  p.chunks = static_cast<uint32_t>(ceil_div(slots, kMoeChunkSlots));
  p.single = slots <= (p.k < 4 ? kMoeSingleSlots / 2 : kMoeSingleSlots);
  if (!p.single) {
    static KernelPrep prep;
    constexpr int kMostSmem = kSortWarps * (kMoeMaxExperts + 1) * 4;
    int per_sm = 0;
    cudaError_t e = prepare_kernel(prep, reinterpret_cast<const void*>(moe_count_kernel), kSortThreads, kMostSmem, dev,
                                   &per_sm);
    if (e != cudaSuccess) return e;
    e = run(moe_count_kernel, p.chunks, 1, kSortThreads, stream, &p,
            kSortWarps * (static_cast<int>(p.experts) + 1) * 4);
    if (e != cudaSuccess) return e;
    p.few_counts = p.chunks <= 16 && (p.experts + 1) * p.chunks <= 1600;
    if (!p.few_counts) e = run(moe_prefix_kernel, kPrefixCtas, 1, kPrefixThreads, stream, &p);
    if (e != cudaSuccess) return e;
  }
  // Tokens per CTA: few while the grid does not fill the GPU, up to kMoePlaceTokens once it does
  // (the ranking is then shared by more rows).
  const uint64_t fill = 4ull * static_cast<uint64_t>(dev.sm_count);
  p.cta_tokens = static_cast<uint32_t>(p.tokens / fill);
  if (p.cta_tokens < 1) p.cta_tokens = 1;
  if (p.cta_tokens > kMoePlaceTokens) p.cta_tokens = kMoePlaceTokens;
  const uint64_t grid = p.tokens ? ceil_div(p.tokens, p.cta_tokens) : 1;  // no tokens: the offsets are still written
  switch (dtype) {
    case ZC_BF16: return place<__nv_bfloat16>(p, vec, grid, stream);
    case ZC_F16: return place<__half>(p, vec, grid, stream);
    default: return place<float>(p, vec, grid, stream);
  }
}

cudaError_t launch_combine(const CombineParams& params, int dtype, bool vec, cudaStream_t stream,
                           const DeviceInfo& dev) {
  CombineParams p = params;
  switch (dtype) {
    case ZC_BF16: return combine<__nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return combine<__half>(p, vec, stream, dev);
    default: return combine<float>(p, vec, stream, dev);
  }
}

cudaError_t launch_combine_bwd(const CombineBwdParams& params, int dtype, bool vec, cudaStream_t stream,
                               const DeviceInfo& dev) {
  CombineBwdParams p = params;
  switch (dtype) {
    case ZC_BF16:
      return vec ? combine_bwd<__nv_bfloat16, true>(p, stream, dev) : combine_bwd<__nv_bfloat16, false>(p, stream, dev);
    case ZC_F16: return vec ? combine_bwd<__half, true>(p, stream, dev) : combine_bwd<__half, false>(p, stream, dev);
    default: return vec ? combine_bwd<float, true>(p, stream, dev) : combine_bwd<float, false>(p, stream, dev);
  }
}

}  // namespace zc
