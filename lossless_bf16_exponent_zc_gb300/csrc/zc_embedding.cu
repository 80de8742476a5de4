// zc_embedding.cu -- rows of an embedding table for a run of token ids, scaled, and the table's
// gradient.  Definitions in include/zc.h.
//
//   out[t] = scale table[id_t],    dtable[v] = scale (sum over t with id_t = v, in order, of dout[t])
//
// The gradient sorts the tokens by id (a stable radix sort), cuts them into runs of up to 32, sums a row's
// tokens in fp32 in their order within a run, then its runs in theirs, and writes every row of the table
// once: no sum depends on timing.  (The runs' length follows from the sizes and the number of SMs: the same
// bits on one kind of GPU, not on any.)  Both directions are bound by memory where there is much of it: 16384 tokens of 131072 x 4096 bf16, ids by 1 / rank, 33 us
// forward (85% of the copy's rate) and 206 back (87%, most of it zeros for rows without a token), 68 added
// to what the table holds.
#include "zc_internal.h"
#include "zc_layer.cuh"
#include "zc_norm.cuh"

namespace zc {

namespace {

constexpr int kEmbedThreads = 256;

__device__ __forceinline__ int64_t id_at(const void* ids, int ids64, uint64_t t) {
  return ids64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
}

// True if a token has a row: its id is reported if it is beyond the table.
__device__ __forceinline__ bool has_row(int64_t id, uint64_t vocab, int32_t* status) {
  if (id >= static_cast<int64_t>(vocab)) set_status(status, ZC_ERR_BAD_INDEX);
  return id >= 0 && id < static_cast<int64_t>(vocab);
}

// N values of TT at p, which lies anywhere, as the 16-byte pieces that hold them (ALIGNED: it lies
// on one), read now and taken apart later.
template <typename TT, int N, bool ALIGNED>
struct AnyValues {
  static constexpr int V = kPieceOf<TT>, NP = N / V;
  uint4 w[ALIGNED ? NP : NP + 1];
  uint32_t off;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < (ALIGNED ? NP : NP + 1); k++) w[k] = make_uint4(0u, 0u, 0u, 0u);
    off = 0;
  }
  __device__ __forceinline__ void load(const TT* p) {
    off = ALIGNED ? 0 : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
#pragma unroll
    for (int k = 0; k < NP; k++) w[k] = from[k];
    if constexpr (!ALIGNED) w[NP] = off ? from[NP] : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
    for (int k = 0; k < NP; k++) {
      float v[V];
      if constexpr (ALIGNED)
        Piece<TT, V>{w[k]}.get(v);
      else
        Piece<TT, V>{shift_pieces<TT>(w[k], w[k + 1], off)}.get(v);
#pragma unroll
      for (int j = 0; j < V; j++) f[k * V + j] = v[j];
    }
  }
};

// ------------------------------------------------------------------ lookup
// A thread takes UNITS 16-byte pieces of the output, kEmbedThreads apart, all loads before the first
// store.
template <typename T, typename TT, int UNITS>
__global__ void __launch_bounds__(kEmbedThreads, 8) embed_kernel(EmbedParams p, Divisor pieces) {
  constexpr int V = kPieceOf<T>;
  pdl_begin();
  const uint64_t i0 = static_cast<uint64_t>(blockIdx.x) * (kEmbedThreads * UNITS);
  const uint64_t t0 = i0 >> 31 ? i0 / pieces.d : pieces(static_cast<uint32_t>(i0));
  const uint32_t c0 = static_cast<uint32_t>(i0 - t0 * pieces.d) + threadIdx.x;
  AnyValues<TT, V, true> v[UNITS];
  float scale[UNITS];  // zero for no token, whose row stays positive zeros whatever the call's scale
  T* to[UNITS];
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    const uint32_t i = c0 + q * kEmbedThreads, dt = pieces(i), first = (i - dt * pieces.d) * V;
    const uint64_t t = t0 + dt;
    to[q] = t < p.tokens ? static_cast<T*>(p.out) + t * p.hidden + first : nullptr;
    v[q].clear();
    scale[q] = 0.f;
    if (!to[q]) continue;
    const int64_t id = id_at(p.ids, p.ids64, t);
    if (!has_row(id, p.vocab, p.status)) continue;
    scale[q] = p.scale;
    v[q].load(static_cast<const TT*>(p.table) + static_cast<uint64_t>(id) * p.table_stride + first);
  }
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    if (!to[q]) continue;
    float f[V];
    v[q].get(f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] *= scale[q];
    Piece<T, V> o;
    o.set(f);
    o.store(to[q]);
  }
}

// Rows of many pieces: a warp takes 32 UNITS of a token's, so that it looks up one id (16384 x 4096 bf16
// 32.3 us, by the kernel above 34.6; 65536 x 1024 28.1 and 32.0).
template <typename T, typename TT, int UNITS>
__global__ void __launch_bounds__(kEmbedThreads) embed_wide_kernel(EmbedParams p, Divisor shares) {
  constexpr int V = kPieceOf<T>;
  pdl_begin();
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * (kEmbedThreads / 32) + (threadIdx.x >> 5);
  const uint64_t t = i >> 31 ? i / shares.d : shares(static_cast<uint32_t>(i));
  if (t >= p.tokens) return;
  const uint32_t c0 = static_cast<uint32_t>(i - t * shares.d) * (32 * UNITS) + lane_id(), pieces = p.hidden / V;
  const int64_t id = id_at(p.ids, p.ids64, t);
  const bool there = has_row(id, p.vocab, p.status);
  const float scale = there ? p.scale : 0.f;
  const TT* row = static_cast<const TT*>(p.table) + (there ? static_cast<uint64_t>(id) * p.table_stride : 0);
  T* out = static_cast<T*>(p.out) + t * p.hidden;
  AnyValues<TT, V, true> v[UNITS];
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    v[q].clear();
    if (there && c0 + q * 32 < pieces) v[q].load(row + static_cast<uint64_t>(c0 + q * 32) * V);
  }
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    if (c0 + q * 32 >= pieces) continue;
    float f[V];
    v[q].get(f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] *= scale;
    Piece<T, V> o;
    o.set(f);
    o.store(out + static_cast<uint64_t>(c0 + q * 32) * V);
  }
}

// The same off 16 bytes: a lane takes a unit of a token's output (RowCut).
template <typename T, typename TT>
__global__ void __launch_bounds__(kEmbedThreads) embed_any_kernel(EmbedParams p, uint32_t shares) {
  constexpr int V = kPieceOf<T>;
  pdl_begin();
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * (kEmbedThreads / 32) + (threadIdx.x >> 5), t = i / shares;
  if (t >= p.tokens) return;
  T* out = static_cast<T*>(p.out) + t * p.hidden;
  const RowCut<T> cut(out, p.hidden);
  uint32_t first;
  const uint32_t values = cut.unit(static_cast<uint32_t>(i - t * shares) * 32 + lane_id(), p.hidden, &first);
  const int64_t id = id_at(p.ids, p.ids64, t);
  const bool there = has_row(id, p.vocab, p.status);
  const float scale = there ? p.scale : 0.f;
  const TT* row = static_cast<const TT*>(p.table) + (there ? static_cast<uint64_t>(id) * p.table_stride : 0);
  if (values == V) {
    AnyValues<TT, V, false> v;
    v.clear();
    if (there) v.load(row + first);
    float f[V];
    v.get(f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] *= scale;
    Piece<T, V> o;
    o.set(f);
    o.store(out + first);
  } else if (values) {
    out[first] = from_f32<T>(there ? scale * to_f32<TT>(row[first]) : 0.f);
  }
}

// ------------------------------------------------------------------ the tokens sorted by id
// A stable radix sort, a digit of up to 10 bits a pass: counts of every chunk's digits, their prefix
// over the chunks, then the places.  Tokens without a row have key `vocab` and come last.  Three launches a
// pass, each bound by its latency (65536 tokens: 5 to 9 us each when profiled alone).
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr uint32_t kSortBins = 1u << kEmbedDigitBits;

__device__ __forceinline__ uint32_t sort_key(const EmbedBwdParams& p, uint64_t i) {
  if (p.keys_in) return p.keys_in[i];
  const int64_t id = id_at(p.ids, p.ids64, i);
  return static_cast<uint32_t>(has_row(id, p.vocab, p.status) ? id : static_cast<int64_t>(p.vocab));
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(EmbedBwdParams p) {
  __shared__ uint32_t hist[kSortBins];
  pdl_allow_dependents();
  for (uint32_t e = threadIdx.x; e < kSortBins; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kEmbedSortChunk;
  const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kEmbedSortChunk), p.tokens - first));
  const uint32_t bins = 1u << p.digit_bits;
  for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
    const uint32_t key = sort_key(p, first + i);
    atomicAdd(&hist[(key >> p.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < bins; e += kSortThreads)
    p.counts[static_cast<uint64_t>(e) * p.sort_chunks + blockIdx.x] = hist[e];
}

// The exclusive prefix over the chunks of a digit's counts, in place, and their total: a warp a digit.
__global__ void __launch_bounds__(kSortThreads) embed_prefix_kernel(EmbedBwdParams p) {
  pdl_begin();
  const uint32_t digit = blockIdx.x * kSortWarps + (threadIdx.x >> 5), lane = lane_id();
  if (digit >= 1u << p.digit_bits) return;
  uint32_t* c = p.counts + static_cast<uint64_t>(digit) * p.sort_chunks;
  uint32_t base = 0;
  for (uint32_t i = 0; i < p.sort_chunks; i += 128) {  // four pieces on their way at once
    uint32_t v[4];
#pragma unroll
    for (uint32_t q = 0; q < 4; q++) v[q] = i + q * 32 + lane < p.sort_chunks ? c[i + q * 32 + lane] : 0;
#pragma unroll
    for (uint32_t q = 0; q < 4; q++) {
      const uint32_t upto = warp_inclusive_scan(v[q]);
      if (i + q * 32 + lane < p.sort_chunks) c[i + q * 32 + lane] = base + upto - v[q];
      base += __shfl_sync(kFull, upto, 31);
    }
  }
  if (lane == 0) p.totals[digit] = base;
}

__device__ __forceinline__ uint32_t lanes_below_mask() { return (1u << lane_id()) - 1u; }

// The lanes whose digit equals this one's.
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, uint32_t bits) {
  uint32_t equal = kFull;
  for (uint32_t b = 0; b < bits; b++) {
    const bool one = (digit >> b) & 1u;
    const uint32_t ones = __ballot_sync(kFull, one);
    equal &= one ? ones : ~ones;
  }
  return equal;
}

// Places a chunk's keys: each warp an eighth of it in order, 32 keys at a time.
__global__ void __launch_bounds__(kSortThreads) embed_place_kernel(EmbedBwdParams p) {
  extern __shared__ uint32_t sort_smem[];  // [kSortWarps][bins], then the digits' first places [bins]
  __shared__ uint32_t warp_totals[kSortWarps];
  pdl_begin();
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, bins = 1u << p.digit_bits;
  uint32_t* start = sort_smem + kSortWarps * bins;
  uint32_t* own = sort_smem + warp * bins;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * kEmbedSortChunk;
  const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kEmbedSortChunk), p.tokens - first));
  constexpr uint32_t kTurns = kEmbedSortChunk / kSortThreads;
  const uint32_t base = warp * (kTurns * 32) + lane;
  uint32_t key[kTurns], token[kTurns], equal[kTurns];
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) {
    const bool there = base + i * 32 < n;
    key[i] = there ? sort_key(p, first + base + i * 32) : 0xFFFFFFFFu;
    token[i] = static_cast<uint32_t>(first + base + i * 32);
    if (there && p.keys_in) token[i] = p.tokens_in[first + base + i * 32];
  }
  // where each digit starts: the totals' exclusive prefix
  const uint32_t per = (bins + kSortThreads - 1) / kSortThreads;
  uint32_t sum = 0;
  for (uint32_t i = 0; i < per; i++)
    if (threadIdx.x * per + i < bins) sum += p.totals[threadIdx.x * per + i];
  const uint32_t upto = warp_inclusive_scan(sum);
  if (lane == 31) warp_totals[warp] = upto;
  for (uint32_t e = lane; e < bins; e += 32) own[e] = 0;
  __syncthreads();
  uint32_t at = upto - sum;
  for (uint32_t w = 0; w < warp; w++) at += warp_totals[w];
  for (uint32_t i = 0; i < per; i++) {
    const uint32_t e = threadIdx.x * per + i;
    if (e >= bins) break;
    start[e] = at + p.counts[static_cast<uint64_t>(e) * p.sort_chunks + blockIdx.x];
    at += p.totals[e];
  }
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) {
    const bool there = base + i * 32 < n;
    const uint32_t digit = there ? (key[i] >> p.shift) & (bins - 1) : bins;  // its own class beyond the end
    equal[i] = same_digit(digit, p.digit_bits + 1);
    if (there && (equal[i] & lanes_below_mask()) == 0) own[digit] += __popc(equal[i]);
    __syncwarp();
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < bins; e += kSortThreads) {
    uint32_t before = start[e];
#pragma unroll
    for (int w = 0; w < kSortWarps; w++) {
      const uint32_t c = sort_smem[w * bins + e];
      sort_smem[w * bins + e] = before;
      before += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < kTurns; i++) {
    const bool there = base + i * 32 < n;
    const uint32_t below = equal[i] & lanes_below_mask();
    const uint32_t digit = (key[i] >> p.shift) & (bins - 1);
    if (there) {
      const uint32_t to = own[digit] + __popc(below);
      p.keys_out[to] = key[i];
      p.tokens_out[to] = token[i];
    }
    __syncwarp();
    if (there && below == 0) own[digit] += __popc(equal[i]);
    __syncwarp();
  }
}

// Up to kEmbedClusterTokens tokens are sorted in the shared memory of one cluster, and the other
// clusters of the same launch zero the table's rows that no token asks for meanwhile: each looks
// through all ids for those of its own rows, which takes less time than the sort.  A warp of the
// sort holds 32 `items` keys in order; a pass counts its digits warp by warp, the CTAs tell one
// another their counts, and every key goes to its place in the shared memory of the CTA that it
// falls to, in the last pass to the workspace.  Profiled alone the sort of 8 tokens takes 8 us, of 16384 17,
// of 32768 27; zeros of 131072 x 4096 bf16 take 165, so there it is free.  Leaving a part of the zeros to the
// SMs that the joins do not use made the whole slower (206 us -> 220): memory still writes back what the
// earlier launch left in L2.
constexpr int kClusterThreads = 512, kClusterWarps = kClusterThreads / 32;
constexpr uint32_t kMostItems = kEmbedClusterTokens / (kEmbedClusterCtas * kClusterThreads);
constexpr uint32_t kClusterBins = 512;
constexpr uint32_t kFillRows = 32768;  // rows whose presence a CTA keeps at once

struct ClusterSort {
  uint32_t items, ctas, bits, passes;
  uint32_t fill, late;           // CTAs that zero rows: those beside the sort, and those that follow it on its SMs
  uint64_t fill_rows, late_rows;  // rows of each of them
};

__device__ __forceinline__ void zero_row(uint8_t* row, uint64_t bytes) {
  const uint32_t lane = lane_id();
  const uint64_t head = min(bytes, static_cast<uint64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15));
  const uint64_t body = (bytes - head) / 16, rest = bytes - body * 16;  // rest: bytes outside the pieces
  uint4* pieces = reinterpret_cast<uint4*>(row + head);
  for (uint64_t i = lane; i < body; i += 32) pieces[i] = make_uint4(0u, 0u, 0u, 0u);
  if (lane * 2 < rest) {
    const uint64_t at = lane * 2 < head ? lane * 2 : body * 16 + lane * 2;
    *reinterpret_cast<uint16_t*>(row + at) = 0;
  }
}

// Zeroes the rows of `first` .. `last` that no token asks for; `present` holds a bit for kFillRows.
__device__ __forceinline__ void fill_rows(const EmbedBwdParams& p, uint64_t first, uint64_t last,
                                          uint32_t* present) {
  const uint64_t bytes = static_cast<uint64_t>(p.hidden) * p.size;
  for (uint64_t v0 = first; v0 < last; v0 += kFillRows) {
    const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kFillRows), last - v0));
    for (uint32_t i = threadIdx.x; i < (n + 31) / 32; i += kClusterThreads) present[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (uint64_t i = threadIdx.x; i < p.tokens; i += kClusterThreads) {
      const uint64_t at = static_cast<uint64_t>(id_at(p.ids, p.ids64, i)) - v0;  // wraps below the first row
      if (at < n) atomicOr(&present[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    for (uint32_t r = threadIdx.x >> 5; r < n; r += kClusterWarps)
      if (!(present[r >> 5] >> (r & 31) & 1)) zero_row(static_cast<uint8_t*>(p.dtable) + (v0 + r) * bytes, bytes);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kClusterThreads, 2) embed_cluster_kernel(EmbedBwdParams p, ClusterSort c, Divisor cap) {
  extern __shared__ __align__(16) uint8_t cluster_smem[];
  __shared__ uint32_t warp_totals[kClusterWarps];
  pdl_begin();
  if (blockIdx.x >= c.ctas) {
    const uint32_t i = blockIdx.x - c.ctas;
    if (i >= c.fill + c.late) return;
    const uint64_t rows = i < c.fill ? c.fill_rows : c.late_rows;
    const uint64_t first = i < c.fill ? i * rows : c.fill * c.fill_rows + (i - c.fill) * rows;
    if (first < p.vocab)
      fill_rows(p, first, min(p.vocab, first + rows), reinterpret_cast<uint32_t*>(cluster_smem));
    return;
  }
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5, rank = blockIdx.x;
  uint16_t* hist = reinterpret_cast<uint16_t*>(cluster_smem);            // [warps][bins]
  uint32_t* totals = reinterpret_cast<uint32_t*>(hist + kClusterWarps * kClusterBins);  // [ctas][bins]
  uint32_t* start = totals + kEmbedClusterCtas * kClusterBins;           // [bins]
  uint32_t* buffers = start + kClusterBins;                              // keys and tokens, once or twice
  cluster_arrive();  // shared memory of another CTA may be written once it has started
  cluster_wait();
  const uint32_t base = warp * 32 * c.items + lane;
  uint32_t key[kMostItems], token[kMostItems], place[kMostItems];
#pragma unroll
  for (uint32_t i = 0; i < kMostItems; i++) {
    token[i] = rank * cap.d + base + i * 32;
    key[i] = 0xFFFFFFFFu;
    if (i < c.items && token[i] < p.tokens) key[i] = sort_key(p, token[i]);
  }
  for (uint32_t pass = 0; pass < c.passes; pass++) {
    const uint32_t shift = c.bits * pass / c.passes, bits = c.bits * (pass + 1) / c.passes - shift, bins = 1u << bits;
    uint16_t* own = hist + warp * bins;
    for (uint32_t i = threadIdx.x; i < kClusterWarps * bins / 2; i += kClusterThreads)
      reinterpret_cast<uint32_t*>(hist)[i] = 0;
    if (pass) {
      const uint32_t* from = buffers + ((pass + 1) & 1) * 2 * cap.d;
#pragma unroll
      for (uint32_t i = 0; i < kMostItems; i++) {
        if (i >= c.items) break;
        key[i] = from[base + i * 32];
        token[i] = from[cap.d + base + i * 32];
      }
    }
    __syncthreads();
    // a key's place among its digit's in the warp
#pragma unroll
    for (uint32_t i = 0; i < kMostItems; i++) {
      if (i >= c.items) break;
      const bool there = rank * cap.d + base + i * 32 < p.tokens;
      const uint32_t digit = there ? (key[i] >> shift) & (bins - 1) : bins;  // its own class beyond the end
      const uint32_t equal = same_digit(digit, bits + 1), below = equal & lanes_below_mask();
      const uint32_t before = there ? own[digit] : 0;
      place[i] = before + __popc(below);
      __syncwarp();
      if (there && below == 0) own[digit] = static_cast<uint16_t>(before + __popc(equal));
      __syncwarp();
    }
    __syncthreads();
    // the digits' prefix over the warps; every CTA gets to know all CTAs' totals
    for (uint32_t e = threadIdx.x; e < bins; e += kClusterThreads) {
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kClusterWarps; w++) {
        const uint32_t n = hist[w * bins + e];
        hist[w * bins + e] = static_cast<uint16_t>(sum);
        sum += n;
      }
      for (uint32_t k = 0; k < c.ctas; k++) st_shared_of_cta(&totals[rank * kClusterBins + e], k, sum);
    }
    cluster_arrive();
    cluster_wait();
    uint32_t all = 0, before = 0;
    if (threadIdx.x < bins) {
      for (uint32_t k = 0; k < c.ctas; k++) {
        const uint32_t n = totals[k * kClusterBins + threadIdx.x];
        before += k < rank ? n : 0;
        all += n;
      }
    }
    const uint32_t upto = warp_inclusive_scan(all);
    if (lane == 31) warp_totals[warp] = upto;
    __syncthreads();
    uint32_t at = upto - all + before;
    for (uint32_t w = 0; w < warp; w++) at += warp_totals[w];
    if (threadIdx.x < bins) start[threadIdx.x] = at;
    __syncthreads();
    const bool last = pass + 1 == c.passes;
    uint32_t* to = buffers + (pass & 1) * 2 * cap.d;
#pragma unroll
    for (uint32_t i = 0; i < kMostItems; i++) {
      if (i >= c.items || rank * cap.d + base + i * 32 >= p.tokens) break;
      const uint32_t digit = (key[i] >> shift) & (bins - 1), r = start[digit] + own[digit] + place[i];
      if (last) {
        p.keys_out[r] = key[i];
        p.tokens_out[r] = token[i];
      } else {
        const uint32_t cta = cap(r), k = r - cta * cap.d;
        st_shared_of_cta(&to[k], cta, key[i]);
        st_shared_of_cta(&to[cap.d + k], cta, token[i]);
      }
    }
    if (!last) {
      cluster_arrive();
      cluster_wait();
    }
  }
}

// ------------------------------------------------------------------ sums
// A warp adds up a run of up to 32 tokens of the sorted order over 256 columns, a lane eight of them
// (8 / V pieces, 32 apart).  Where a row's tokens all lie in the run, the row is written; where they
// go on in a neighbouring run, the sum is left in the workspace: slot 0 of the run for the tokens of
// a row that began before it, slot 1 for one that begins in it and goes on.  8192 rows of 4096 bf16: 20 us,
// waiting for rows with the 24 warps an SM that 80 registers allow.  Where a run took the tokens that its
// last row has in the next run too, so that fewer rows need a join, the longest warps had twice the work
// (200000 tokens of 32000 x 512 143 us instead of 125).
constexpr uint32_t kSlab = 256;
// Rows on their way at once, as many as 80 registers hold; ADD: with the table's rows that they end in.
template <typename T, bool VEC, bool ADD>
constexpr int kSumRows = (VEC && !ADD ? 8 : 4) / (sizeof(T) / 2);

template <typename T, typename TT, bool VEC>
struct EmbedCols {
  static constexpr int V = kPieceOf<T>, NP = 8 / V;
  AnyValues<T, V, VEC> w[NP];
  __device__ __forceinline__ static uint32_t col(uint32_t slab, int i) {
    return slab * kSlab + (i * 32 + lane_id()) * V;
  }
  __device__ __forceinline__ void load(const T* row, uint32_t slab, uint32_t hidden) {
#pragma unroll
    for (int i = 0; i < NP; i++) {
      const uint32_t c = col(slab, i);
      w[i].clear();
      if (whole_piece<T>(c, hidden)) {
        w[i].load(row + c);
      } else if (c < hidden) {  // the last values of the row, one by one
        uint32_t part[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < V; j++) {
          if (c + j >= hidden) continue;
          if constexpr (sizeof(T) == 4)
            part[j] = reinterpret_cast<const uint32_t*>(row)[c + j];
          else
            part[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[c + j]) << (j & 1) * 16;
        }
        w[i].w[0] = make_uint4(part[0], part[1], part[2], part[3]);
      }
    }
  }
  __device__ __forceinline__ void add(float (&acc)[8]) const {
#pragma unroll
    for (int i = 0; i < NP; i++) {
      float f[V];
      w[i].get(f);
#pragma unroll
      for (int j = 0; j < V; j++) acc[i * V + j] += f[j];
    }
  }
};

// The lane's columns of a table row that the sums are added to, read ahead of them.
template <typename T, typename TT>
struct OldCols {
  static constexpr int V = kPieceOf<T>, W = kPieceOf<TT>;
  uint4 w[8 / W];
  __device__ __forceinline__ void load(const EmbedBwdParams& p, uint64_t row, uint32_t slab) {
    const TT* from = static_cast<const TT*>(p.dtable) + row * p.hidden;
#pragma unroll
    for (int i = 0; i < 8 / V; i++) {
      const uint32_t c = EmbedCols<T, TT, true>::col(slab, i);
      if (c >= p.hidden) continue;
#pragma unroll
      for (int k = 0; k < V / W; k++) w[i * (V / W) + k] = *reinterpret_cast<const uint4*>(from + c + k * W);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8 / W; i++) {
      float v[W];
      Piece<TT, W>{w[i]}.get(v);
#pragma unroll
      for (int j = 0; j < W; j++) f[i * W + j] = v[j];
    }
  }
};

// Writes scale acc + old to the lane's columns of a table row.  Off 16 bytes the warp's columns go
// through shared memory (`tile`, its own), so that the lanes write, and read what they add to,
// neighbouring values.
template <typename T, typename TT, bool VEC>
__device__ __forceinline__ void put_row(const EmbedBwdParams& p, uint64_t row, uint32_t slab, const float (&acc)[8],
                                        const float (&old)[8], float* tile) {
  constexpr int V = kPieceOf<T>, W = kPieceOf<TT>;
  TT* to = static_cast<TT*>(p.dtable) + row * p.hidden;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 8 / V; i++) {
      const uint32_t c = EmbedCols<T, TT, VEC>::col(slab, i);
      if (c >= p.hidden) continue;
#pragma unroll
      for (int k = 0; k < V; k += W) {
        float f[W];
#pragma unroll
        for (int j = 0; j < W; j++) f[j] = fmaf(p.scale, acc[i * V + (k + j) % V], old[i * V + (k + j) % V]);
        Piece<TT, W> o;
        o.set(f);
        o.store(to + c + k);
      }
    }
  } else {
    const uint32_t lane = lane_id(), first = slab * kSlab;
    __syncwarp();  // the last row's values have been read
#pragma unroll
    for (int i = 0; i < 8 / V; i++)
      store_f32<V>(tile + (i * 32 + lane) * V, *reinterpret_cast<const float(*)[V]>(acc + i * V));
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t c = first + j * 32 + lane;
      if (c >= p.hidden) continue;
      const float before = p.accumulate ? to_f32<TT>(to[c]) : 0.f;
      to[c] = from_f32<TT>(fmaf(p.scale, tile[j * 32 + lane], before));
    }
  }
}

__device__ __forceinline__ float* part_of(const EmbedBwdParams& p, uint64_t run, uint32_t slot, uint32_t slab) {
  return p.parts + ((run * 2 + slot) * p.slabs + slab) * kSlab;
}

template <typename T, typename TT, bool VEC, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads, 3) embed_sum_kernel(EmbedBwdParams p) {
  constexpr int kRowLoads = kSumRows<T, VEC, ADD>;
  __shared__ __align__(16) float tiles[VEC ? 1 : kEmbedThreads / 32][VEC ? 4 : kSlab];
  float* tile = tiles[VEC ? 0 : threadIdx.x >> 5];
  pdl_begin();
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * (kEmbedThreads / 32) + (threadIdx.x >> 5), run = i / p.slabs;
  if (run >= p.runs) return;
  const uint32_t lane = lane_id(), slab = static_cast<uint32_t>(i - run * p.slabs);
  const uint64_t first = run * p.run;
  const uint32_t none = static_cast<uint32_t>(p.vocab);
  const bool there = lane < p.run && first + lane < p.tokens;
  const uint32_t key = there ? p.keys_in[first + lane] : none;
  const uint32_t token = there ? p.tokens_in[first + lane] : 0;
  const uint32_t before = first ? p.keys_in[first - 1] : none;
  const uint32_t after = first + p.run < p.tokens ? p.keys_in[first + p.run] : none;
  const uint32_t n = __popc(__ballot_sync(kFull, key != none));  // those with a row come first
  const uint32_t next = __shfl_down_sync(kFull, key, 1);
  const uint32_t ends = __ballot_sync(kFull, lane == 31 || next != key);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; j++) acc[j] = 0.f;
  bool began = __shfl_sync(kFull, key, 0) == before;  // the row at hand began before the run
  const bool leaves = n == p.run && __shfl_sync(kFull, key, p.run - 1) == after;  // its last row goes on behind the run
  for (uint32_t r0 = 0; r0 < n; r0 += kRowLoads) {
    EmbedCols<T, TT, VEC> v[kRowLoads];
    OldCols<T, TT> old[ADD ? kRowLoads : 1];
#pragma unroll
    for (int q = 0; q < kRowLoads; q++) {
      const uint64_t t = __shfl_sync(kFull, token, (r0 + q) & 31);
      const uint32_t row = __shfl_sync(kFull, key, (r0 + q) & 31);
      if (r0 + q >= n) continue;
      v[q].load(static_cast<const T*>(p.dout) + t * p.dout_stride, slab, p.hidden);
      if constexpr (ADD)
        if (ends >> (r0 + q) & 1) old[q].load(p, row, slab);
    }
#pragma unroll
    for (int q = 0; q < kRowLoads; q++) {
      const uint32_t r = r0 + q;
      if (r >= n) break;
      v[q].add(acc);
      if (!(ends >> r & 1)) continue;
      const uint32_t row = __shfl_sync(kFull, key, r);
      if (began || (leaves && r + 1 == p.run)) {
        float* to = part_of(p, run, began ? 0 : 1, slab) + lane * 8;
        *reinterpret_cast<float4*>(to) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      } else {
        float before[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if constexpr (ADD) old[q].get(before);
        put_row<T, TT, VEC>(p, row, slab, acc, before, tile);
      }
      began = false;
#pragma unroll
      for (int j = 0; j < 8; j++) acc[j] = 0.f;
    }
  }
}

// How many sorted keys are below `row`; the warp looks at 32 places at a time.
__device__ __forceinline__ uint64_t keys_below(const EmbedBwdParams& p, uint64_t row) {
  uint64_t from = 0, size = p.tokens;  // the answer is from .. from + size
  while (size) {
    const uint64_t step = (size + 31) / 32, at = from + step * (lane_id() + 1) - 1;
    const bool below = at < from + size && p.keys_in[at] < row;
    const uint32_t n = __popc(__ballot_sync(kFull, below));
    const uint64_t end = from + size;
    from += n * step;
    size = min(step - 1, end - min(end, from));
  }
  return from;
}

// Zeroes the rows that no token asks for: a warp gap_rows of them, up to 32; a lane looks for one of them
// among the keys from the first one's to the last one's.
__device__ __forceinline__ void fill_gaps(const EmbedBwdParams& p, uint64_t warp) {
  const uint64_t first = warp * p.gap_rows, last = min(p.vocab, first + p.gap_rows);
  if (first >= last) return;
  const uint64_t row = first + lane_id(), stop = keys_below(p, last);
  uint64_t from = keys_below(p, first), size = stop - from;
  while (size) {
    const uint64_t half = size / 2;
    const bool below = p.keys_in[from + half] < row;
    from += below ? half + 1 : 0;
    size = below ? size - half - 1 : half;
  }
  const bool there = from < stop && p.keys_in[from] == row;
  const uint64_t bytes = static_cast<uint64_t>(p.hidden) * p.size;
  for (uint32_t gaps = __ballot_sync(kFull, row < last && !there); gaps; gaps &= gaps - 1)
    zero_row(static_cast<uint8_t*>(p.dtable) + (first + __ffs(gaps) - 1) * bytes, bytes);
}

// Rows whose tokens lie in several runs, of one slab.  Each warp looks at one run, and adds the parts of
// the row that begins there and goes on; where those are many the warps of the CTA share them.  About 10 us,
// a chain of keys, parts and barriers; 4 to 16 parts alone, 4 or 8 of them in flight made no difference.
// With more than kEmbedClusterTokens tokens its idle SMs also zero the unused rows (65536 tokens of 32000 x
// 1024 71 us, with a bitmap and a launch for those 80).
constexpr uint32_t kJoinAlone = 16;  // parts that a warp adds by itself
template <typename T, typename TT, bool VEC>
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(EmbedBwdParams p) {
  constexpr uint32_t kWarps = kEmbedThreads / 32;
  __shared__ __align__(16) float sums[kWarps][kSlab];
  __shared__ uint32_t many[kWarps];  // parts of a warp's row that are for all, or 0
  __shared__ uint32_t rows[kWarps];
  pdl_begin();
  if (blockIdx.x >= p.join_ctas) {
    fill_gaps(p, static_cast<uint64_t>(blockIdx.x - p.join_ctas) * kWarps + (threadIdx.x >> 5));
    return;
  }
  const uint64_t group = blockIdx.x / p.slabs;
  const uint32_t slab = static_cast<uint32_t>(blockIdx.x - group * p.slabs), lane = lane_id(), warp = threadIdx.x >> 5;
  const uint64_t run = group * kWarps + warp, first = run * p.run, next = first + p.run;
  uint32_t count = 0, row = 0;
  if (next < p.tokens) {
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    // lane i: the first key of run + 1 + i; with it the last one here, the first one, and the one before
    const uint64_t at = next + static_cast<uint64_t>(lane) * p.run;
    const uint32_t key = at < p.tokens ? p.keys_in[at] : none;
    const uint32_t last = p.keys_in[next - 1], begin = p.keys_in[first], before = first ? p.keys_in[first - 1] : none;
    row = last;
    if (last != none && (begin != last || before != last)) {
      uint32_t more = __ballot_sync(kFull, key == last);
      count = more ? 1 : 0;
      while (more == kFull) {  // 32 runs more
        count += 32;
        const uint64_t far = next + (static_cast<uint64_t>(lane) + count - 1) * p.run;
        more = __ballot_sync(kFull, far < p.tokens && p.keys_in[far] == last);
      }
      count += __popc(more);  // the row's runs come one after another
    }
  }
  // adds parts from .. to of the row that begins in run `of`
  auto add = [&](uint64_t of, uint32_t from, uint32_t to, float (&acc)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) acc[j] = 0.f;
#pragma unroll 4
    for (uint32_t i = from; i < to; i++) {
      const float* part = part_of(p, of + i, i ? 0 : 1, slab) + lane * 8;
      const float4 a = *reinterpret_cast<const float4*>(part), b = *reinterpret_cast<const float4*>(part + 4);
      acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
      acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
    }
  };
  auto put = [&](uint32_t of, const float (&acc)[8]) {
    float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (VEC && p.accumulate) {
      OldCols<T, TT> cols;
      cols.load(p, of, slab);
      cols.get(old);
    }
    put_row<T, TT, VEC>(p, of, slab, acc, old, sums[warp]);
  };
  float acc[8];
  if (count && count <= kJoinAlone) {
    add(run, 0, count, acc);
    put(row, acc);
  }
  if (lane == 0) {
    many[warp] = count > kJoinAlone ? count : 0;
    rows[warp] = row;
  }
  __syncthreads();
  for (uint32_t w = 0; w < kWarps; w++) {
    const uint32_t n = many[w];
    if (n == 0) continue;
    add(group * kWarps + w, static_cast<uint32_t>(static_cast<uint64_t>(n) * warp / kWarps),
        static_cast<uint32_t>(static_cast<uint64_t>(n) * (warp + 1) / kWarps), acc);
#pragma unroll
    for (int j = 0; j < 8; j++) sums[warp][j * 32 + lane] = acc[j];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        acc[j] = 0.f;
#pragma unroll
        for (uint32_t q = 0; q < kWarps; q++) acc[j] += sums[q][j * 32 + lane];
      }
      put(rows[w], acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ launches
uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

cudaError_t run(const void* fn, uint64_t grid, int threads, int smem, cudaStream_t stream, void** args) {
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, stream, args, false);
}

template <typename T, typename TT>
cudaError_t lookup(EmbedParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  if (!vec) {
    uint32_t shares = static_cast<uint32_t>(ceil_div(any_units<T>(p.hidden), 32));
    void* args[] = {&p, &shares};
    return run(reinterpret_cast<const void*>(embed_any_kernel<T, TT>), ceil_div(p.tokens * shares, kEmbedThreads / 32),
               kEmbedThreads, 0, stream, args);
  }
  Divisor pieces(p.hidden / kPieceOf<T>);
  const uint64_t all = p.tokens * pieces.d;
  void* args[] = {&p, &pieces};
  if (all <= 2ull * kEmbedThreads * static_cast<uint64_t>(dev.sm_count))
    return run(reinterpret_cast<const void*>(embed_kernel<T, TT, 1>), ceil_div(all, kEmbedThreads), kEmbedThreads, 0,
               stream, args);
  constexpr uint32_t kUnits = sizeof(TT) > sizeof(T) ? 2 : 4;
  if (pieces.d >= 64) {
    Divisor shares(static_cast<uint32_t>(ceil_div(pieces.d, 32 * kUnits)));
    void* wide[] = {&p, &shares};
    return run(reinterpret_cast<const void*>(embed_wide_kernel<T, TT, kUnits>),
               ceil_div(p.tokens * shares.d, kEmbedThreads / 32), kEmbedThreads, 0, stream, wide);
  }
  return run(reinterpret_cast<const void*>(embed_kernel<T, TT, 2>), ceil_div(all, 2 * kEmbedThreads), kEmbedThreads, 0,
             stream, args);
}

constexpr uint64_t kGapWarps = 16;  // an SM's warps that zero rows beside the joins, or as many as 32 rows each make
template <typename T, typename TT, bool VEC>
cudaError_t sums(EmbedBwdParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  void* args[] = {&p};
  const void* fn = VEC && p.accumulate ? reinterpret_cast<const void*>(embed_sum_kernel<T, TT, VEC, VEC>)
                                       : reinterpret_cast<const void*>(embed_sum_kernel<T, TT, VEC, false>);
  cudaError_t e = run(fn, ceil_div(p.runs * p.slabs, kEmbedThreads / 32), kEmbedThreads, 0, stream, args);
  if (e != cudaSuccess || p.runs < 2) return e;
  const uint64_t join = ceil_div(p.runs, kEmbedThreads / 32) * p.slabs,
                 fill = p.tokens > kEmbedClusterTokens && !p.accumulate ? p.vocab : 0;
  if (join > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  p.join_ctas = static_cast<uint32_t>(join);
  p.gap_rows = static_cast<uint32_t>(ceil_div(fill, kGapWarps * static_cast<uint64_t>(dev.sm_count)));
  if (p.gap_rows > 32) p.gap_rows = 32;
  const uint64_t gaps = fill ? ceil_div(fill, p.gap_rows * (kEmbedThreads / 32)) : 0;
  return run(reinterpret_cast<const void*>(embed_join_kernel<T, TT, VEC>), join + gaps, kEmbedThreads, 0, stream, args);
}
template <typename T, typename TT>
cudaError_t sums(EmbedBwdParams& p, bool vec, cudaStream_t stream, const DeviceInfo& dev) {
  return vec ? sums<T, TT, true>(p, stream, dev) : sums<T, TT, false>(p, stream, dev);
}

// Tokens of a run: those that make the waves of warps, three CTAs an SM, take the least time, a warp
// as long as its run and six rows more (16384 tokens of 4096 columns: 24 of them fill three waves,
// with 32 the third is a quarter full); but no more than kMostShort warps of short runs, whose sums
// take workspace.
constexpr uint64_t kMostShort = 16384;
uint32_t embed_run(uint64_t tokens, uint32_t hidden, const DeviceInfo& dev) {
  const uint64_t slabs = ceil_div(hidden, kSlab), wave = 24ull * static_cast<uint64_t>(dev.sm_count);
  // One run, and no launch for joins: 8 tokens of 1000 x 4096 bf16 7.4 us, in runs of 4 8.5 (host 5.3, 8.0); 16
  // 9.0 and 8.9, 32 11.5 and 9.3.
  if (tokens <= 8) return 8;
  uint64_t least = ~0ull;
  uint32_t best = 32;
  for (uint32_t run = 32; run >= 4; run--) {
    const uint64_t warps = ceil_div(tokens, run) * slabs, time = ceil_div(warps, wave) * (run + 6);
    if ((run < 32 && warps > kMostShort) || time >= least) continue;
    least = time;
    best = run;
  }
  return best;
}
// At most so many runs of `tokens` tokens or fewer, on any device.
uint64_t embed_runs(uint64_t tokens, uint32_t hidden) {
  const uint64_t few = kMostShort / ceil_div(hidden, kSlab) + 1, runs = ceil_div(tokens, 32);
  const uint64_t most = runs > few ? runs : few, all = ceil_div(tokens, 4);
  return most < all ? most : all;
}

// Where a gradient's workspace holds what.
struct EmbedWork {
  uint64_t keys, tokens, counts, totals, parts, bytes;  // byte offsets; keys and tokens have two halves
  EmbedWork(uint64_t n, uint32_t hidden) {
    const uint64_t chunks = ceil_div(n, kEmbedSortChunk), runs = embed_runs(n, hidden);
    uint64_t at = 0;
    auto take = [&](uint64_t words) {
      const uint64_t here = at;
      at += ceil_div(words * 4, 16) * 16;
      return here;
    };
    parts = take(runs * 2 * ceil_div(hidden, kSlab) * kSlab);
    keys = take(2 * n);
    tokens = take(2 * n);
    counts = take(kSortBins * chunks);
    totals = take(kSortBins);
    bytes = at;
  }
};

cudaError_t sort_in_cluster(EmbedBwdParams& p, uint32_t bits, cudaStream_t stream, const DeviceInfo& dev) {
  static KernelPrep prep;
  ClusterSort c = {};
  c.bits = bits;
  c.passes = static_cast<uint32_t>(ceil_div(bits, 9));
  // one CTA holds a few tokens, and more of them a cluster, with as few a thread as that allows
  c.ctas = p.tokens <= 2 * kClusterThreads ? 1 : kEmbedClusterCtas;
  c.items = static_cast<uint32_t>(ceil_div(p.tokens, static_cast<uint64_t>(c.ctas) * kClusterThreads));
  if (c.items < 1) c.items = 1;
  Divisor cap(c.items * kClusterThreads);
  const uint32_t buffers = c.passes > 2 ? 2 : c.passes - 1;
  const int smem = static_cast<int>(kClusterWarps * kClusterBins * 2 + (kEmbedClusterCtas + 1) * kClusterBins * 4 +
                                    buffers * 2 * cap.d * 4);
  constexpr int kMostSmem = static_cast<int>(kClusterWarps * kClusterBins * 2 + (kEmbedClusterCtas + 1) * kClusterBins * 4 +
                                             4 * kMostItems * kClusterThreads * 4);
  int per_sm = 0;
  const void* fn = reinterpret_cast<const void*>(embed_cluster_kernel);
  cudaError_t e = prepare_kernel(prep, fn, kClusterThreads, kMostSmem, dev, &per_sm);
  if (e != cudaSuccess) return e;
  if (!p.accumulate && p.vocab) {
    // One wave of CTAs, two an SM where clusters fit.  The table is cut so that those that take the
    // sort's place after it end with the others: the sort's time, about 10 us and 4 more with every
    // 16384 tokens, at 20 KB a microsecond.
    int fit = 0;
    static RingPrep fits[2];
    e = prepare_ring(fits[c.ctas > 1], fn, kClusterThreads, kMostSmem, dev, static_cast<int>(c.ctas), &fit);
    if (e != cudaSuccess) return e;
    const uint64_t beside = fit > 1 ? (static_cast<uint64_t>(fit) - 1) * c.ctas : 1;
    const uint64_t row = static_cast<uint64_t>(p.hidden) * p.size;
    const uint64_t lost = (10 + p.tokens / 4096) * 20480 / row;
    c.fill = static_cast<uint32_t>(beside);
    c.late = c.ctas;
    const uint64_t all = p.vocab + c.late * lost;
    c.fill_rows = ceil_div(all, beside + c.late);
    if (c.fill_rows <= lost || c.fill_rows * beside >= p.vocab) c.late = 0, c.fill_rows = ceil_div(p.vocab, beside);
    if (c.late) c.late_rows = ceil_div(p.vocab - c.fill_rows * beside, c.late);
  }
  const uint32_t grid = c.ctas + static_cast<uint32_t>(ceil_div(c.fill + c.late, c.ctas)) * c.ctas;
  void* args[] = {&p, &c, &cap};
  return launch_kernel(fn, dim3(grid), dim3(kClusterThreads), smem, stream, args, false, c.ctas);
}

cudaError_t sort_in_launches(EmbedBwdParams& p, uint32_t bits, uint32_t* const (&keys)[2], uint32_t* const (&tokens)[2],
                             cudaStream_t stream, const DeviceInfo& dev) {
  cudaError_t e = cudaSuccess;
  const uint32_t passes = static_cast<uint32_t>(ceil_div(bits, kEmbedDigitBits));
  static KernelPrep prep;
  int per_sm = 0;
  constexpr int kMostSmem = (kSortWarps + 1) * static_cast<int>(kSortBins) * 4;
  e = prepare_kernel(prep, reinterpret_cast<const void*>(embed_place_kernel), kSortThreads, kMostSmem, dev, &per_sm);
  void* args[] = {&p};
  for (uint32_t pass = 0; pass < passes && e == cudaSuccess; pass++) {
    p.shift = bits * pass / passes;
    p.digit_bits = bits * (pass + 1) / passes - p.shift;
    p.keys_in = pass ? keys[(pass + 1) & 1] : nullptr;
    p.tokens_in = pass ? tokens[(pass + 1) & 1] : nullptr;
    p.keys_out = keys[pass & 1];
    p.tokens_out = tokens[pass & 1];
    e = run(reinterpret_cast<const void*>(embed_count_kernel), p.sort_chunks, kSortThreads, 0, stream, args);
    if (e == cudaSuccess)
      e = run(reinterpret_cast<const void*>(embed_prefix_kernel), ceil_div(1u << p.digit_bits, kSortWarps),
              kSortThreads, 0, stream, args);
    if (e == cudaSuccess)
      e = run(reinterpret_cast<const void*>(embed_place_kernel), p.sort_chunks, kSortThreads,
              (kSortWarps + 1) * (4 << p.digit_bits), stream, args);
  }
  if (e != cudaSuccess) return e;
  p.keys_in = keys[(passes + 1) & 1];
  p.tokens_in = tokens[(passes + 1) & 1];
  return e;
}

}  // namespace

cudaError_t launch_embed(const EmbedParams& params, int dtype, int table_f32, bool vec, cudaStream_t stream,
                         const DeviceInfo& dev) {
  if (params.tokens == 0) return cudaSuccess;
  EmbedParams p = params;
  switch (dtype) {
    case ZC_BF16:
      return table_f32 ? lookup<__nv_bfloat16, float>(p, vec, stream, dev)
                       : lookup<__nv_bfloat16, __nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16:
      return table_f32 ? lookup<__half, float>(p, vec, stream, dev) : lookup<__half, __half>(p, vec, stream, dev);
    default: return lookup<float, float>(p, vec, stream, dev);
  }
}

uint64_t embed_workspace_bytes(uint64_t tokens, uint32_t hidden) {
  return EmbedWork(tokens, hidden).bytes;
}

cudaError_t launch_embed_bwd(const EmbedBwdParams& params, int dtype, int table_f32, bool vec, void* ws,
                             cudaStream_t stream, const DeviceInfo& dev) {
  EmbedBwdParams p = params;
  const EmbedWork at(p.tokens, p.hidden);
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(base + at.keys), reinterpret_cast<uint32_t*>(base + at.keys) + p.tokens};
  uint32_t* tokens[2] = {reinterpret_cast<uint32_t*>(base + at.tokens),
                         reinterpret_cast<uint32_t*>(base + at.tokens) + p.tokens};
  p.counts = reinterpret_cast<uint32_t*>(base + at.counts);
  p.totals = reinterpret_cast<uint32_t*>(base + at.totals);
  p.parts = reinterpret_cast<float*>(base + at.parts);
  p.sort_chunks = static_cast<uint32_t>(ceil_div(p.tokens, kEmbedSortChunk));
  p.run = embed_run(p.tokens, p.hidden, dev);
  p.runs = ceil_div(p.tokens, p.run);
  p.slabs = static_cast<uint32_t>(ceil_div(p.hidden, kSlab));
  p.size = dtype == ZC_F32 || table_f32 ? 4 : 2;
  uint32_t bits = 1;  // of the keys 0 .. vocab
  while (p.vocab >> bits) bits++;
  cudaError_t e;
  if (p.tokens <= kEmbedClusterTokens) {
    p.keys_out = keys[0];
    p.tokens_out = tokens[0];
    e = sort_in_cluster(p, bits, stream, dev);
    p.keys_in = keys[0];
    p.tokens_in = tokens[0];
  } else {
    e = sort_in_launches(p, bits, keys, tokens, stream, dev);
  }
  if (e != cudaSuccess) return e;
  if (p.tokens == 0) return e;
  switch (dtype) {
    case ZC_BF16:
      return table_f32 ? sums<__nv_bfloat16, float>(p, vec, stream, dev) : sums<__nv_bfloat16, __nv_bfloat16>(p, vec, stream, dev);
    case ZC_F16: return table_f32 ? sums<__half, float>(p, vec, stream, dev) : sums<__half, __half>(p, vec, stream, dev);
    default: return sums<float, float>(p, vec, stream, dev);
  }
}

}  // namespace zc
