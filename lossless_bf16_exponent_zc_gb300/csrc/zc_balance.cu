// zc_balance.cu -- the loss that keeps a router's load even, the experts' counts it is made from,
// and its gradient.  Definitions in include/zc.h.
//
// With c[s][e] = E count[s][e] / (S k T_s^2) for each of S sequences, T_s its counted tokens,
//   loss = sum over s, e of c[s][e] sum over the sequence's tokens of p[t][e],
// p the softmax of the logits or their sigmoids over the sigmoids' sum.  The counts have no
// gradient, so for a token's row
//   softmax   dl = g p (c - sum p c)
//   sigmoid   dl = g s (1 - s) (c - sum p c) / Z.
// A warp takes a token's row in registers.  Forward, a CTA adds up its tokens' p and counts, and a
// second launch the CTAs' sums in order: no result depends on timing.
//
// Nothing here is near the memory's rate.  16384 x 256 fp32 (17 MB, 2.5 us at the copy's rate), sigmoid, 8
// sequences: forward 11.6 us in two launches, the first bound by its exponentials and divisions (66% of the
// issue slots), the second by a chain of dependent loads, shuffles and barriers; gradient 8.7 us (78% of the
// issue slots).  5003 x 61 bf16 8.8 and 2.6 us.
//
// Sigmoids are taken by the fast quotient, within two units of the last place (zero from logits of -87.3 down,
// where they are below 2^-126), not rounded as the router's, and p is the exponential or the sigmoid times
// the rounded reciprocal of their sum.  The errors against 64 bits stay those of plain fp32; the router's
// sigmoid took 13.3 us forward instead of 12.1 and 10.5 back instead of 9.6 (16384 x 256 fp32, other tensors).
#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

namespace {

// Warps of a CTA: 16, whose sums are half as much to add up as twice 8 warps' (16384 x 256 fp32 11.7 us, with
// 8 warps 13.2; 16384 x 64 bf16, 16 sequences, 9.1 and 11.6; 4096 x 64 8.3 and 8.1), while shared memory has
// room for them.  A warp takes 4 tokens where there are not too many.
template <int N>
constexpr int kBalanceWarps = N <= 16 ? 16 : 8;
constexpr int kBackWarps = 8;

// A row's p, from its logits in l; false, and p all zero, where no logit is above minus infinity.
// `raw` gets the exponentials or the sigmoids s, `inv` the reciprocal of their sum.  SLOPE: in place of s
// the smaller of s and 1 - s, negative where that is s: s (1 - s) = m (1 - m) by it, and 1 - s = e s with
// e = exp(-logit) where the logit is above zero.  A difference from 1 would keep no bits of it from a logit
// of 17 on (at 10 it is off by 2^-11).
template <int N, bool SLOPE>
__device__ __forceinline__ bool probabilities(float (&l)[N], bool sigmoid_score, float (&raw)[N], float* inv) {
  float best = l[0];
#pragma unroll
  for (int j = 1; j < N; j++) best = fmaxf(best, l[j]);  // of those that are not NaN
  const float top = warp_max_of(best);
  float sum = 0.f;
  if (sigmoid_score) {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const float e = expf(-l[j]), s = __fdividef(1.f, 1.f + e);  // 1 / infinity: zero
      raw[j] = !SLOPE ? s : l[j] > 0.f ? e * s : -s;
      sum += s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) {
      raw[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - top);
      sum += raw[j];
    }
  }
  sum = warp_sum_f32(sum) + (sigmoid_score ? 1e-20f : 0.f);
  const bool any = top > -INFINITY || sum != sum;
  *inv = any ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    float v = raw[j];
    if (SLOPE && sigmoid_score) v = signbit(v) ? -v : 1.f - v;
    l[j] = any ? v * *inv : 0.f;
  }
  return any;
}

// A warp's tokens first, first + step, ... below last: adds their p to acc and their slots to the CTA's
// counts, and returns how many count.  The next token's row is on its way meanwhile, if there is room for it.
template <typename T, int N, bool VEC>
__device__ __forceinline__ uint32_t add_tokens(const BalanceParams& p, uint64_t first, uint64_t last, uint32_t step,
                                               float (&acc)[N], int32_t* counts) {
  const uint32_t lane = lane_id();
  float next[N];
  int32_t next_id = -1;
  bool next_in = false;
  constexpr bool kAhead = N <= 8;  // more experts a lane leave no registers for it
  auto load = [&](uint64_t t) {
    next_in = t < last && (!p.mask || p.mask[t]);
    if (!next_in) return;
    load_row<T, N, VEC>(static_cast<const T*>(p.logits) + t * p.stride, p.experts, next);
    next_id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  };
#pragma unroll
  for (int j = 0; j < N; j++) acc[j] = next[j] = 0.f;
  if (kAhead) load(first);
  uint32_t counted = 0;
  for (uint64_t t = first; t < last; t += step) {
    float l[N], raw[N], inv;
    if (!kAhead) load(t);
#pragma unroll
    for (int j = 0; j < N; j++) l[j] = next[j];
    const int32_t id = next_id;
    const bool in = next_in;
    if (kAhead) load(t + step);
    if (!in || !probabilities<N, false>(l, p.sigmoid, raw, &inv)) continue;
    counted++;
#pragma unroll
    for (int j = 0; j < N; j++) acc[j] += l[j];
    if (static_cast<uint32_t>(id) < p.experts) atomicAdd(&counts[id], 1);
  }
  return counted;
}

__device__ __forceinline__ float slope_of(const BalanceParams& p, int32_t count, uint32_t counted) {
  const float tokens = static_cast<float>(counted);
  return counted ? static_cast<float>(count) * static_cast<float>(p.experts) /
                       (static_cast<float>(p.sequences) * static_cast<float>(p.k) * tokens * tokens)
                 : 0.f;
}

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kBalanceWarps<N> * 32) balance_kernel(BalanceParams p) {
  constexpr int kWarps = kBalanceWarps<N>;
  __shared__ float sums[kWarps][N * 32];
  __shared__ int32_t counts[N * 32];
  __shared__ uint32_t counted;
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  for (uint32_t e = threadIdx.x; e < N * 32; e += kWarps * 32) counts[e] = 0;
  if (threadIdx.x == 0) counted = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  __syncthreads();
  const uint64_t n = p.tokens / p.sequences, seq = blockIdx.x / p.chunks, chunk = blockIdx.x - seq * p.chunks;
  float acc[N];
  const uint32_t mine = add_tokens<T, N, VEC>(p, seq * n + chunk * p.chunk_tokens + warp,
                                              seq * n + min(n, (chunk + 1) * p.chunk_tokens), kWarps, acc, counts);
  if (lane == 0) atomicAdd(&counted, mine);
#pragma unroll
  for (int j = 0; j < N; j++) sums[warp][lane * N + j] = acc[j];
  __syncthreads();
  const uint64_t at = static_cast<uint64_t>(blockIdx.x) * p.experts;
  for (uint32_t e = threadIdx.x; e < p.experts; e += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) s += sums[w][e];
    p.part_sums[at + e] = s;
    p.part_counts[at + e] = counts[e];
  }
  if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = counted;
}

// Adds the CTAs' sums of a sequence, 32 experts a CTA (blockIdx.y): a lane an expert, the warps a
// share of the CTAs each, and then a warp an expert.  The last CTA to finish adds up the parts of
// the loss in order.  Bound by latency; by one cluster of 8 CTAs the whole took 14.8 us instead of 13.2.
__global__ void __launch_bounds__(1024) balance_sum_kernel(BalanceParams p) {
  __shared__ float sums[32][33];
  __shared__ int32_t counts[32][33];
  __shared__ uint32_t tokens_of[32];
  __shared__ bool is_last;
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, e = blockIdx.y * 32 + lane;
  const uint64_t seq = blockIdx.x, first = seq * p.chunks;
  const uint32_t from = static_cast<uint32_t>(static_cast<uint64_t>(p.chunks) * warp / 32),
                 to = static_cast<uint32_t>(static_cast<uint64_t>(p.chunks) * (warp + 1) / 32);
  uint32_t n = 0;
  for (uint32_t i = threadIdx.x; i < p.chunks; i += 1024) n += p.part_tokens[first + i];
  float s = 0.f;
  int32_t c = 0;
  if (e < p.experts) {
#pragma unroll 8
    for (uint32_t i = from; i < to; i++) {
      s += p.part_sums[(first + i) * p.experts + e];
      c += p.part_counts[(first + i) * p.experts + e];
    }
  }
  n = __reduce_add_sync(kFull, n);
  sums[warp][lane] = s;
  counts[warp][lane] = c;
  if (lane == 0) tokens_of[warp] = n;
  __syncthreads();
  // from here on warp w has expert w
  const uint32_t mine = blockIdx.y * 32 + warp;
  s = warp_sum_f32(sums[lane][warp]);
  c = __reduce_add_sync(kFull, counts[lane][warp]);
  n = __reduce_add_sync(kFull, tokens_of[lane]);
  const float slope = slope_of(p, c, n);
  if (lane == 0 && mine < p.experts) {
    p.counts[seq * p.experts + mine] = c;
    p.slope[seq * p.experts + mine] = slope;
  }
  __syncthreads();
  if (lane == 0) sums[0][warp] = mine < p.experts ? slope * s : 0.f;
  __syncthreads();
  if (warp == 0) {
    const float part = warp_sum_f32(sums[0][lane]);
    if (lane == 0) {
      p.part_loss[seq * gridDim.y + blockIdx.y] = part;
      __threadfence();
      is_last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!is_last) return;
  float loss[1] = {0.f};
  const uint64_t parts = static_cast<uint64_t>(gridDim.x) * gridDim.y;
  for (uint64_t i = threadIdx.x; i < parts; i += 1024) loss[0] += __ldcg(p.part_loss + i);
  block_sum_f32<1>(loss, sums[0]);
  if (threadIdx.x == 0) *p.loss = loss[0];
}

// Few tokens in 1, 2, 4 or 8 sequences: one cluster, so one launch, 8 / sequences CTAs a sequence.  The
// first of those adds up what the others have in shared memory.  512 x 64 fp32 5.0 us, most of it barriers
// and a token's chain of shuffles (30% of the issue slots).
constexpr uint32_t kBalanceCtas = 8;
constexpr int kClusterWarps = 32;
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kClusterWarps * 32) balance_cluster_kernel(BalanceParams p) {
  extern __shared__ float warp_sums[];  // [warps][32 N], of which the first row takes the CTA's sums
  __shared__ int32_t counts[N * 32];
  __shared__ uint32_t counted;
  __shared__ float red[32];
  __shared__ float losses[kBalanceCtas];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, rank = blockIdx.x;
  for (uint32_t e = threadIdx.x; e < N * 32; e += kClusterWarps * 32) counts[e] = 0;
  if (threadIdx.x == 0) counted = 0;
  __syncthreads();
  const uint32_t group = kBalanceCtas / static_cast<uint32_t>(p.sequences), seq = rank / group, share = rank - seq * group;
  const uint64_t n = p.tokens / p.sequences;
  float acc[N];
  const uint32_t mine = add_tokens<T, N, VEC>(p, seq * n + share * kClusterWarps + warp, (seq + 1) * n,
                                              group * kClusterWarps, acc, counts);
  if (lane == 0) atomicAdd(&counted, mine);
#pragma unroll
  for (int j = 0; j < N; j++) warp_sums[warp * (N * 32) + lane * N + j] = acc[j];
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < p.experts; e += kClusterWarps * 32) {
    float s = 0.f;
#pragma unroll 8
    for (int w = 0; w < kClusterWarps; w++) s += warp_sums[w * (N * 32) + e];
    warp_sums[e] = s;  // read by this thread alone so far
  }
  cluster_arrive();
  cluster_wait();
  if (share == 0) {
    uint32_t all = 0;
    for (uint32_t r = 0; r < group; r++) all += ld_shared_of_cta(&counted, rank + r);
    float loss[1] = {0.f};
    for (uint32_t e = threadIdx.x; e < p.experts; e += kClusterWarps * 32) {
      float s = 0.f;
      int32_t c = 0;
      for (uint32_t r = 0; r < group; r++) {
        s += __uint_as_float(ld_shared_of_cta(reinterpret_cast<const uint32_t*>(warp_sums + e), rank + r));
        c += static_cast<int32_t>(ld_shared_of_cta(reinterpret_cast<const uint32_t*>(counts + e), rank + r));
      }
      const float slope = slope_of(p, c, all);
      p.counts[seq * p.experts + e] = c;
      p.slope[seq * p.experts + e] = slope;
      loss[0] = fmaf(slope, s, loss[0]);
    }
    block_sum_f32<1>(loss, red);
    if (threadIdx.x == 0) st_shared_of_cta(reinterpret_cast<uint32_t*>(&losses[seq]), 0, __float_as_uint(loss[0]));
  }
  cluster_arrive();
  cluster_wait();
  if (rank || threadIdx.x) return;
  float loss = 0.f;
  for (uint32_t q = 0; q < p.sequences; q++) loss += losses[q];
  *p.loss = loss;
}

// Lane l's N values of a row of the output.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_row(T* row, uint32_t width, const float (&v)[N]) {
  constexpr int V = kPieceOf<T>;
  const uint32_t first = lane_id() * N;
  if constexpr (VEC && N % V == 0) {
#pragma unroll
    for (int i = 0; i < N; i += V) {
      if (first + i >= width) continue;
      float f[V];
#pragma unroll
      for (int j = 0; j < V; j++) f[j] = v[i + j];
      Piece<T, V> o;
      o.set(f);
      o.store(row + first + i);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j++)
      if (first + j < width) row[first + j] = from_f32<T>(v[j]);
  }
}

// A warp a token, read and written once: 16384 x 256 fp32 8.7 us with sigmoids (57% of the copy's rate; its
// exponentials keep 78% of the issue slots busy), 8.2 by softmax.  Persistent warps with the next row on its way took 8.0 to 8.6 us, but
// 5.6 instead of 4.5 for 16384 x 64 bf16; two tokens a warp 8.5.
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kBackWarps * 32) balance_bwd_kernel(BalanceBwdParams p) {
  pdl_begin();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kBackWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  T* out = static_cast<T*>(p.dlogits) + t * p.experts;
  float l[N], c[N], raw[N], inv = 0.f;
  if (p.mask && !p.mask[t]) {
#pragma unroll
    for (int j = 0; j < N; j++) l[j] = 0.f;
    store_row<T, N, VEC>(out, p.experts, l);
    return;
  }
  load_row<T, N, VEC>(static_cast<const T*>(p.logits) + t * p.stride, p.experts, l);
  load_row<float, N, VEC>(p.slope + t / p.seq_tokens * p.experts, p.experts, c);
  const float g = *p.dloss;
  const bool any = probabilities<N, true>(l, p.sigmoid, raw, &inv);
  float mean = 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    c[j] = c[j] == -INFINITY ? 0.f : c[j];  // beyond the width
    mean = fmaf(l[j], c[j], mean);
  }
  mean = warp_sum_f32(mean);
#pragma unroll
  for (int j = 0; j < N; j++) {
    const float m = fabsf(raw[j]), d = p.sigmoid ? m * (1.f - m) * inv : l[j];
    l[j] = any ? d * (g * (c[j] - mean)) : 0.f;
  }
  store_row<T, N, VEC>(out, p.experts, l);
}

// Tokens that one cluster takes, of up to 256 experts (more spill its registers): 512 x 64 fp32 5.0 us, in two
// launches 7.0; 1500 x 64 7.3 and 7.1, 2048 x 256 12.7 and 10.3.
constexpr uint64_t kBalanceFew = 1024;

template <typename T, int N>
cudaError_t run_width(BalanceParams& p, cudaStream_t stream) {
  constexpr uint64_t kPart = N * sizeof(T) < 16 ? N * sizeof(T) : 16;
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % kPart == 0 && p.stride * sizeof(T) % kPart == 0 &&
                   p.experts * sizeof(T) % kPart == 0;
  void* args[] = {&p};
  if constexpr (N <= 8) {
    if (p.tokens <= kBalanceFew && kBalanceCtas % p.sequences == 0) {
      static KernelPrep prep[2];
      const void* fn = vec ? reinterpret_cast<const void*>(balance_cluster_kernel<T, N, true>)
                           : reinterpret_cast<const void*>(balance_cluster_kernel<T, N, false>);
      constexpr int kSmem = kClusterWarps * N * 32 * 4;
      DeviceInfo dev;
      int per_sm = 0;
      cudaError_t e = device_info(&dev);
      if (e == cudaSuccess) e = prepare_kernel(prep[vec], fn, kClusterWarps * 32, kSmem, dev, &per_sm);
      if (e != cudaSuccess) return e;
      return launch_kernel(fn, dim3(kBalanceCtas), dim3(kClusterWarps * 32), kSmem, stream, args, false, kBalanceCtas);
    }
  }
  const void* fn = vec ? reinterpret_cast<const void*>(balance_kernel<T, N, true>)
                       : reinterpret_cast<const void*>(balance_kernel<T, N, false>);
  cudaError_t e = launch_kernel(fn, dim3(static_cast<unsigned>(p.sequences * p.chunks)),
                                dim3(kBalanceWarps<N> * 32), 0,
                                stream, args, false);
  if (e != cudaSuccess) return e;
  return launch_kernel(reinterpret_cast<const void*>(balance_sum_kernel),
                       dim3(static_cast<unsigned>(p.sequences), (p.experts + 31) / 32), dim3(1024), 0, stream, args,
                       false);
}
template <typename T, int N>
cudaError_t run_width(BalanceBwdParams& p, cudaStream_t stream) {
  // 16-byte pieces of the logits, the slopes and the gradient
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.stride * sizeof(T) % 16 == 0 &&
                   p.experts * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(p.slope) % 16 == 0;
  const void* fn = vec ? reinterpret_cast<const void*>(balance_bwd_kernel<T, N, true>)
                       : reinterpret_cast<const void*>(balance_bwd_kernel<T, N, false>);
  const uint64_t grid = (p.tokens + kBackWarps - 1) / kBackWarps;
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kBackWarps * 32), 0, stream, args, false);
}

template <typename T, typename P>
cudaError_t run_experts(P& p, cudaStream_t stream) {
  if (p.experts <= 32) return run_width<T, 1>(p, stream);
  if (p.experts <= 64) return run_width<T, 2>(p, stream);
  if (p.experts <= 128) return run_width<T, 4>(p, stream);
  if (p.experts <= 256) return run_width<T, 8>(p, stream);
  if (p.experts <= 512) return run_width<T, 16>(p, stream);
  return run_width<T, 32>(p, stream);
}

template <typename P>
cudaError_t run_typed(P& p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case ZC_BF16: return run_experts<__nv_bfloat16>(p, stream);
    case ZC_F16: return run_experts<__half>(p, stream);
    default: return run_experts<float>(p, stream);
  }
}

// Chunks of a sequence's tokens, a CTA each: a few tokens a warp, and not so many chunks that their
// sums weigh as much as the logits.
struct BalanceCut {
  uint32_t chunks;
  uint64_t chunk_tokens;
};
constexpr uint64_t kBalanceMost = 1216;  // chunks of all sequences, if these are not more themselves
uint64_t least_chunk(uint32_t experts) {
  return 4 * static_cast<uint64_t>(experts <= 512 ? kBalanceWarps<16> : kBalanceWarps<32>);
}
BalanceCut balance_cut(uint64_t tokens, uint32_t experts, uint64_t sequences) {
  const uint64_t n = tokens / sequences, most = sequences < kBalanceMost ? kBalanceMost / sequences : 1;
  uint64_t each = (n + most - 1) / most;
  each = each < least_chunk(experts) ? least_chunk(experts) : each;
  const uint64_t chunks = n ? (n + each - 1) / each : 1;
  return {static_cast<uint32_t>(chunks), each};
}

}  // namespace

// Room for any batch of up to so many tokens in up to so many sequences.  The chunks themselves become fewer
// where more tokens lengthen each of them: s sequences of n tokens have at most s n / least + s of them, least
// being the shortest, and at most kBalanceMost or s.
uint64_t balance_workspace_bytes(uint64_t tokens, uint32_t experts, uint64_t sequences) {
  const uint64_t shortest = tokens / least_chunk(experts) + sequences;
  const uint64_t most = sequences > kBalanceMost ? sequences : kBalanceMost;
  const uint64_t units = shortest < most ? shortest : most;
  return 16 + 4 * (2 * units * experts + units + sequences * ((experts + 31) / 32));
}

cudaError_t launch_balance(const BalanceParams& params, int dtype, void* ws, cudaStream_t stream) {
  BalanceParams p = params;
  const BalanceCut cut = balance_cut(p.tokens, p.experts, p.sequences);
  p.chunks = cut.chunks;
  p.chunk_tokens = cut.chunk_tokens;
  const uint64_t units = p.sequences * p.chunks;
  if (units > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  p.ticket = static_cast<uint32_t*>(ws);
  p.part_sums = reinterpret_cast<float*>(p.ticket + 4);
  p.part_counts = reinterpret_cast<int32_t*>(p.part_sums + units * p.experts);
  p.part_tokens = reinterpret_cast<uint32_t*>(p.part_counts + units * p.experts);
  p.part_loss = reinterpret_cast<float*>(p.part_tokens + units);
  return run_typed(p, dtype, stream);
}

cudaError_t launch_balance_bwd(const BalanceBwdParams& params, int dtype, cudaStream_t stream) {
  if (params.tokens == 0) return cudaSuccess;
  BalanceBwdParams p = params;
  return run_typed(p, dtype, stream);
}

}  // namespace zc
