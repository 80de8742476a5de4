// zc_dropout.cu -- dropout with a mask that is never stored (zc_dropout.cuh), and the residual
// addition behind it in the same pass:  out = a residual + D(x),  D(x) = x / (1 - p) where kept.
//
// The gradient of x is the dropout of out's gradient with the same seed, offset and call.  Drawing twice
// costs instructions where a stored mask would cost memory: 16384 x 4096 with a residual bf16 59.4 us and
// fp32 116 (the copy's rate, 6.8 and 6.9 TB/s; 58% of the issue slots), bf16 without one 43 (92%; 67% of the
// issue slots).
#include "zc_dropout.cuh"
#include "zc_internal.h"

namespace zc {

namespace {

constexpr int kDropThreads = 256;

// Rows whose addresses, strides and widths are multiples of 16 bytes: a thread takes UNITS groups of
// eight columns, kDropThreads apart, all loads before the first use, and draws for all of them
// together.  FLAT: all matrices are contiguous, and their rows whole groups.
template <typename T, int UNITS, bool RESIDUAL, bool FLAT>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(DropoutParams p, Divisor groups) {
  constexpr int V = kPieceOf<T>, NP = 8 / V;
  pdl_begin();
  const KeepRng rng(p.drop);
  const bool drops = p.drop.limit != 0;
  const uint64_t i0 = static_cast<uint64_t>(blockIdx.x) * (kDropThreads * UNITS);
  const uint64_t t0 = i0 >> 31 ? i0 / groups.d : groups(static_cast<uint32_t>(i0));
  const uint32_t c0 = static_cast<uint32_t>(i0 - t0 * groups.d) + threadIdx.x;
  Piece<T, V> x[UNITS][NP], r[UNITS][NP];
  uint32_t row[UNITS], group[UNITS];
  bool there[UNITS];
  // where the values of unit q, a row's group, lie in a matrix
  auto at = [&](int q, int k, uint32_t of_row, uint32_t of_group, uint64_t stride) {
    if (FLAT) return (i0 + threadIdx.x + q * kDropThreads) * 8 + k * V;
    return of_row * stride + of_group * 8 + k * V;
  };
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    const uint32_t i = c0 + q * kDropThreads, dt = groups(i);
    group[q] = i - dt * groups.d;
    there[q] = t0 + dt < p.tokens;
    row[q] = static_cast<uint32_t>(t0 + dt);
#pragma unroll
    for (int k = 0; k < NP; k++) {
      const bool here = there[q] && (FLAT || group[q] * 8 + k * V < p.width);
      x[q][k] = r[q][k] = Piece<T, V>::zero();
      if (here) x[q][k] = Piece<T, V>::load(static_cast<const T*>(p.x) + at(q, k, row[q], group[q], p.x_stride));
      if (here && RESIDUAL)
        r[q][k] =
            Piece<T, V>::load(static_cast<const T*>(p.residual) + at(q, k, row[q], group[q], p.residual_stride));
    }
  }
  uint4 g[UNITS];
#pragma unroll
  for (int q = 0; q < UNITS; q++) g[q] = make_uint4(0u, 0u, 0u, 0u);
  if (drops) rng.template groups<UNITS>(row, group, g);
#pragma unroll
  for (int q = 0; q < UNITS; q++) {
    const uint32_t w[4] = {g[q].x, g[q].y, g[q].z, g[q].w};
#pragma unroll
    for (int k = 0; k < NP; k++) {
      float f[V], o[V];
      uint32_t bits[V / 2];
#pragma unroll
      for (int j = 0; j < V / 2; j++) bits[j] = w[k * V / 2 + j];
      x[q][k].get(f);
      if (drops) rng.template apply<V>(f, bits);
      if (RESIDUAL) {
        r[q][k].get(o);
#pragma unroll
        for (int j = 0; j < V; j++) f[j] = fmaf(p.residual_scale, o[j], f[j]);
      }
      Piece<T, V> out;
      out.set(f);
      if (there[q] && (FLAT || group[q] * 8 + k * V < p.width))
        out.store(static_cast<T*>(p.out) + at(q, k, row[q], group[q], p.width));
    }
  }
}

// 8 values at p, which lies anywhere (or, with ALIKE, on a piece), as the pieces that hold them.
template <typename T, bool ALIKE>
struct AnyEight {
  static constexpr int NP = 8 / kPieceOf<T>;
  uint4 w[ALIKE ? NP : NP + 1];
  uint32_t off;
  __device__ __forceinline__ void load(const T* p) {
    off = ALIKE ? 0 : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
#pragma unroll
    for (int k = 0; k < NP; k++) w[k] = from[k];
    if constexpr (!ALIKE) w[NP] = off ? from[NP] : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    constexpr int V = kPieceOf<T>;
#pragma unroll
    for (int k = 0; k < NP; k++) {
      float v[V];
      if constexpr (ALIKE)
        Piece<T, V>{w[k]}.get(v);
      else
        Piece<T, V>{shift_pieces<T>(w[k], w[k + 1], off)}.get(v);
#pragma unroll
      for (int j = 0; j < V; j++) f[k * V + j] = v[j];
    }
  }
};

// 2 W 16-bit values from value `first` on of a run of them in shared memory (4-byte aligned, and the word
// behind them may be read).
template <int W>
__device__ __forceinline__ void load_bits(const uint32_t* run, uint32_t first, uint32_t (&bits)[W]) {
  uint32_t w[W + 1];
#pragma unroll
  for (int j = 0; j <= W; j++) w[j] = run[first / 2 + j];
#pragma unroll
  for (int j = 0; j < W; j++) bits[j] = __funnelshift_r(w[j], w[j + 1], (first & 1) * 16);
}

// Rows off 16 bytes.  A warp takes TURNS times 31 units of a row of the output: eight columns from an
// aligned piece on, or a column outside those (the ones behind the last piece, then the ones before
// the first).  Eight such columns lie in two of the generator's groups: every lane draws one and
// takes the second from the lane above, through shared memory, the last lane drawing for its
// neighbour alone.  (Selecting among the words of both groups took 79 us where this takes 76.)  ALIKE: the rows of all matrices start equally far into a piece.  16384 x 4095 bf16
// with a residual 76 us (78% of the copy's rate, 62% of the issue slots at 42% of the warps), fp32 116.
constexpr uint32_t kDropAnyUnits = 31;
template <typename T, bool RESIDUAL, bool ALIKE, int TURNS>
__global__ void __launch_bounds__(kDropThreads) dropout_any_kernel(DropoutParams p, Divisor shares) {
  constexpr int V = kPieceOf<T>, NP = 8 / V;
  __shared__ uint4 groups_of[kDropThreads / 32][TURNS][33];  // the last is only read past the others
  pdl_begin();
  const KeepRng rng(p.drop);
  const bool drops = p.drop.limit != 0;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5);
  const uint64_t t = i >> 31 ? i / shares.d : shares(static_cast<uint32_t>(i));
  if (t >= p.tokens) return;
  const uint32_t lane = lane_id();
  const uint32_t u0 = static_cast<uint32_t>(i - t * shares.d) * (TURNS * kDropAnyUnits) + lane;
  T* out = static_cast<T*>(p.out) + t * p.width;
  const T* x = static_cast<const T*>(p.x) + t * p.x_stride;
  const T* r = RESIDUAL ? static_cast<const T*>(p.residual) + t * p.residual_stride : nullptr;
  uint32_t head = static_cast<uint32_t>((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / sizeof(T);
  head = head < p.width ? head : p.width;
  // behind the last piece one unit at the least, which draws the group of that piece's last columns
  const uint32_t body = (p.width - head) / 8, tail = p.width - head - body * 8, behind = tail ? tail : 1;
  uint32_t col[TURNS], row[TURNS], group[TURNS];
  bool whole[TURNS], single[TURNS];
  AnyEight<T, ALIKE> xs[TURNS], rs[TURNS];
#pragma unroll
  for (int q = 0; q < TURNS; q++) {
    const uint32_t u = u0 + q * kDropAnyUnits, e = u - body;
    const bool in_front = u >= body && e >= behind;
    col[q] = in_front ? e - behind : head + body * 8 + (u < body ? (u - body) * 8 : e);
    whole[q] = u < body && lane < kDropAnyUnits;
    single[q] = u >= body && lane < kDropAnyUnits && (in_front ? col[q] < head : e < tail);
    row[q] = static_cast<uint32_t>(t);
    group[q] = col[q] / 8;
    if (whole[q]) {
      xs[q].load(x + col[q]);
      if (RESIDUAL) rs[q].load(r + col[q]);
    }
  }
  uint4 g[TURNS];
#pragma unroll
  for (int q = 0; q < TURNS; q++) g[q] = make_uint4(0u, 0u, 0u, 0u);
  if (drops) rng.template groups<TURNS>(row, group, g);
  uint4(*runs)[33] = groups_of[threadIdx.x >> 5];
#pragma unroll
  for (int q = 0; q < TURNS; q++) runs[q][lane] = g[q];
  __syncwarp();
#pragma unroll
  for (int q = 0; q < TURNS; q++) {
    uint32_t bits[4];  // of eight columns, which start head columns into the lane's group
    load_bits<4>(reinterpret_cast<const uint32_t*>(runs[q]), lane * 8 + (head & 7), bits);
    if (single[q]) {
      float f = to_f32<T>(x[col[q]]);
      if (drops) f = rng.keeps(g[q], col[q] & 7) ? f * rng.factor : 0.f;
      if (RESIDUAL) f = fmaf(p.residual_scale, to_f32<T>(r[col[q]]), f);
      out[col[q]] = from_f32<T>(f);
    }
    if (whole[q]) {
      float f[8], o[8];
      xs[q].get(f);
      if (drops) rng.template apply<8>(f, bits);
      if (RESIDUAL) {
        rs[q].get(o);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = fmaf(p.residual_scale, o[j], f[j]);
      }
#pragma unroll
      for (int k = 0; k < NP; k++) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; j++) v[j] = f[k * V + j];
        Piece<T, V> piece;
        piece.set(v);
        piece.store(out + col[q] + k * V);
      }
    }
  }
}

cudaError_t launch(const void* fn, uint64_t grid, cudaStream_t stream, void** args) {
  if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  return launch_kernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kDropThreads), 0, stream, args, false);
}

template <typename T, bool RESIDUAL>
cudaError_t run(DropoutParams& p, bool vec, cudaStream_t stream) {
  if (vec) {
    Divisor groups((p.width + 7) / 8);
    void* args[] = {&p, &groups};
    const bool flat = p.width % 8 == 0 && p.x_stride == p.width && (!RESIDUAL || p.residual_stride == p.width);
    const uint64_t all = p.tokens * groups.d;
    // Two groups a thread, and four of 16-bit values with a residual where they are many (16384 x 4096 bf16
    // 59 us, with two 62, with eight 72; without a residual 43, with four 47; 256 x 1024 1.7, with four 2.2).
    if constexpr (sizeof(T) == 2 && RESIDUAL) {
      if (all >= 4096ull * kDropThreads) {
        return launch(flat ? reinterpret_cast<const void*>(dropout_kernel<T, 4, RESIDUAL, true>)
                           : reinterpret_cast<const void*>(dropout_kernel<T, 4, RESIDUAL, false>),
                      (all + kDropThreads * 4 - 1) / (kDropThreads * 4), stream, args);
      }
    }
    return launch(flat ? reinterpret_cast<const void*>(dropout_kernel<T, 2, RESIDUAL, true>)
                       : reinterpret_cast<const void*>(dropout_kernel<T, 2, RESIDUAL, false>),
                  (all + kDropThreads * 2 - 1) / (kDropThreads * 2), stream, args);
  }
  const auto base = [](const void* q) { return reinterpret_cast<uintptr_t>(q) & 15; };
  const auto apart = [](uint64_t stride) { return stride * sizeof(T) & 15; };
  const bool alike = base(p.x) == base(p.out) && apart(p.x_stride) == apart(p.width) &&
                     (!RESIDUAL || (base(p.residual) == base(p.out) && apart(p.residual_stride) == apart(p.width)));
  // at most 7 columns on either side of the pieces; two turns a warp where the rows have them
  const uint32_t units = p.width / 8 + 14, turns = units > kDropAnyUnits ? 2 : 1;
  Divisor shares((units + turns * kDropAnyUnits - 1) / (turns * kDropAnyUnits));
  const void* fn;
  if (turns == 2)
    fn = alike ? reinterpret_cast<const void*>(dropout_any_kernel<T, RESIDUAL, true, 2>)
               : reinterpret_cast<const void*>(dropout_any_kernel<T, RESIDUAL, false, 2>);
  else
    fn = alike ? reinterpret_cast<const void*>(dropout_any_kernel<T, RESIDUAL, true, 1>)
               : reinterpret_cast<const void*>(dropout_any_kernel<T, RESIDUAL, false, 1>);
  void* args[] = {&p, &shares};
  return launch(fn, (p.tokens * shares.d + kDropThreads / 32 - 1) / (kDropThreads / 32), stream, args);
}

template <typename T>
cudaError_t run_typed(DropoutParams& p, bool vec, cudaStream_t stream) {
  return p.residual ? run<T, true>(p, vec, stream) : run<T, false>(p, vec, stream);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& params, int dtype, bool vec, cudaStream_t stream) {
  if (params.tokens == 0) return cudaSuccess;
  DropoutParams p = params;
  switch (dtype) {
    case ZC_BF16: return run_typed<__nv_bfloat16>(p, vec, stream);
    case ZC_F16: return run_typed<__half>(p, vec, stream);
    default: return run_typed<float>(p, vec, stream);
  }
}

}  // namespace zc
