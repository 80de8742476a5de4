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
#include "zc_internal.h"
#include "zc_layer.cuh"

namespace zc {

namespace {

constexpr int kBalanceWarps = 8;

// A row's p, from its logits in l; false, and p all zero, where no logit is above minus infinity.
// `raw` gets the sigmoids, `inv` the reciprocal of their sum.
template <int N>
__device__ __forceinline__ bool probabilities(float (&l)[N], bool sigmoid_score, float (&raw)[N], float* inv) {
  bool open = false;
#pragma unroll
  for (int j = 0; j < N; j++) open |= l[j] != -INFINITY;
  const bool any = __any_sync(kFull, open);
  float sum = 0.f;
  if (sigmoid_score) {
#pragma unroll
    for (int j = 0; j < N; j++) raw[j] = l[j] == -INFINITY ? 0.f : sigmoid(l[j]);
  } else {
    float top = l[0];
#pragma unroll
    for (int j = 1; j < N; j++) top = fmaxf(top, l[j]);
    top = warp_max_f32(top);
#pragma unroll
    for (int j = 0; j < N; j++) raw[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - top);
  }
#pragma unroll
  for (int j = 0; j < N; j++) sum += raw[j];
  sum = warp_sum_f32(sum) + (sigmoid_score ? 1e-20f : 0.f);
  *inv = any ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) l[j] = any ? raw[j] * *inv : 0.f;
  return any;
}

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kBalanceWarps * 32) balance_kernel(BalanceParams p) {
  __shared__ float sums[kBalanceWarps][N * 32];
  __shared__ int32_t counts[N * 32];
  __shared__ uint32_t counted;
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  for (uint32_t e = threadIdx.x; e < N * 32; e += kBalanceWarps * 32) counts[e] = 0;
  if (threadIdx.x == 0) counted = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  __syncthreads();
  const uint64_t n = p.tokens / p.sequences, seq = blockIdx.x / p.chunks, chunk = blockIdx.x - seq * p.chunks;
  const uint64_t last = min(n, (chunk + 1) * p.chunk_tokens);
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; j++) acc[j] = 0.f;
  uint32_t mine = 0;
  for (uint64_t i = chunk * p.chunk_tokens + warp; i < last; i += kBalanceWarps) {
    const uint64_t t = seq * n + i;
    if (p.mask && !p.mask[t]) continue;
    float l[N], raw[N], inv;
    load_row<T, N, VEC>(static_cast<const T*>(p.logits) + t * p.stride, p.experts, l);
    const int32_t id = lane < p.k ? p.ids[t * p.k + lane] : -1;
    if (!probabilities<N>(l, p.sigmoid, raw, &inv)) continue;
    mine++;
#pragma unroll
    for (int j = 0; j < N; j++) acc[j] += l[j];
    if (static_cast<uint32_t>(id) < p.experts) atomicAdd(&counts[id], 1);
  }
  if (lane == 0) atomicAdd(&counted, mine);
#pragma unroll
  for (int j = 0; j < N; j++) sums[warp][lane * N + j] = acc[j];
  __syncthreads();
  const uint64_t at = static_cast<uint64_t>(blockIdx.x) * p.experts;
  for (uint32_t e = threadIdx.x; e < p.experts; e += kBalanceWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBalanceWarps; w++) s += sums[w][e];
    p.part_sums[at + e] = s;
    p.part_counts[at + e] = counts[e];
  }
  if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = counted;
}

// Adds the CTAs' sums of a sequence, 32 experts a CTA (blockIdx.y): a lane an expert, the warps a
// share of the CTAs each.  The last CTA to finish adds up the parts of the loss in order.
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
  float s = 0.f;
  int32_t c = 0;
  if (e < p.experts) {
#pragma unroll 8
    for (uint32_t i = from; i < to; i++) {
      s += p.part_sums[(first + i) * p.experts + e];
      c += p.part_counts[(first + i) * p.experts + e];
    }
  }
  uint32_t n = 0;
  for (uint32_t i = threadIdx.x; i < p.chunks; i += 1024) n += p.part_tokens[first + i];
  n = __reduce_add_sync(kFull, n);
  sums[warp][lane] = s;
  counts[warp][lane] = c;
  if (lane == 0) tokens_of[warp] = n;
  __syncthreads();
  if (warp == 0) {
    s = 0.f, c = 0;
#pragma unroll 8
    for (int w = 0; w < 32; w++) s += sums[w][lane], c += counts[w][lane];
    n = __reduce_add_sync(kFull, tokens_of[lane]);
    const float tokens = static_cast<float>(n);
    const float slope = n ? static_cast<float>(c) * static_cast<float>(p.experts) /
                                (static_cast<float>(p.sequences) * static_cast<float>(p.k) * tokens * tokens)
                          : 0.f;
    if (e < p.experts) {
      p.counts[seq * p.experts + e] = c;
      p.slope[seq * p.experts + e] = slope;
    }
    const float part = warp_sum_f32(e < p.experts ? slope * s : 0.f);
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

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kBalanceWarps * 32) balance_bwd_kernel(BalanceBwdParams p) {
  pdl_begin();
  const uint64_t t = static_cast<uint64_t>(blockIdx.x) * kBalanceWarps + (threadIdx.x >> 5);
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
  const bool any = probabilities<N>(l, p.sigmoid, raw, &inv);
  float mean = 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) {
    c[j] = c[j] == -INFINITY ? 0.f : c[j];  // beyond the width
    mean = fmaf(l[j], c[j], mean);
  }
  mean = warp_sum_f32(mean);
#pragma unroll
  for (int j = 0; j < N; j++) {
    const float d = p.sigmoid ? raw[j] * (1.f - raw[j]) * inv : l[j];
    l[j] = any ? d * (g * (c[j] - mean)) : 0.f;
  }
  store_row<T, N, VEC>(out, p.experts, l);
}

template <typename T, int N>
cudaError_t run_width(BalanceParams& p, cudaStream_t stream) {
  constexpr uint64_t kPart = N * sizeof(T) < 16 ? N * sizeof(T) : 16;
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % kPart == 0 && p.stride * sizeof(T) % kPart == 0 &&
                   p.experts * sizeof(T) % kPart == 0;
  const void* fn = vec ? reinterpret_cast<const void*>(balance_kernel<T, N, true>)
                       : reinterpret_cast<const void*>(balance_kernel<T, N, false>);
  void* args[] = {&p};
  cudaError_t e = launch_kernel(fn, dim3(static_cast<unsigned>(p.sequences * p.chunks)), dim3(kBalanceWarps * 32), 0,
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
  const uint64_t grid = (p.tokens + kBalanceWarps - 1) / kBalanceWarps;
  void* args[] = {&p};
  return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kBalanceWarps * 32), 0, stream, args, false);
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
BalanceCut balance_cut(uint64_t tokens, uint64_t sequences) {
  constexpr uint64_t kTokens = 4 * kBalanceWarps, kMost = 1216;
  const uint64_t n = tokens / sequences, most = sequences < kMost ? kMost / sequences : 1;
  uint64_t each = (n + most - 1) / most;
  each = each < kTokens ? kTokens : each;
  const uint64_t chunks = n ? (n + each - 1) / each : 1;
  return {static_cast<uint32_t>(chunks), each};
}

}  // namespace

uint64_t balance_workspace_bytes(uint64_t tokens, uint32_t experts, uint64_t sequences) {
  const uint64_t units = sequences * balance_cut(tokens, sequences).chunks;
  return 16 + 4 * (2 * units * experts + units + sequences * ((experts + 31) / 32));
}

cudaError_t launch_balance(const BalanceParams& params, int dtype, void* ws, cudaStream_t stream) {
  BalanceParams p = params;
  const BalanceCut cut = balance_cut(p.tokens, p.sequences);
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
