// The forward products of few tokens (serving): bound by the bytes of the
// weights, which are read once, straight into registers.
//
// A workgroup makes 16 columns of the results (of both projections, if
// gated) for all tokens.  Its waves take the 128-byte pieces of the weights'
// rows in turn: a lane reads 32 consecutive bytes of one of 16 rows, by two
// loads, and is handed the same k of a token, so that a 16 x 16 product of the
// matrix cores takes 16 rows and 16 tokens whatever the order of the k.  The
// waves' sums meet in LDS, in a fixed order.  Nothing has to be aligned.
//
// Bound: HBM.  One token: gated 4096 x 11008 32.9 us (5.5 TB/s; a kernel that
// only reads as many bytes in this order took 31), linear 11008 x 4096 17.8 (5.1
// TB/s; those with three sets of weights in turn, some of whose bytes are still
// in the Infinity Cache; with nine sets 34.1 and 22.1).  With more tokens x,
// which comes out of the L2 for every 16 columns, and outputs too narrow for
// all CUs: takes_few leaves those to the tiles.
#include "k_layer_tile.hpp"

namespace sm {
namespace layer {

namespace {

// 16 bytes of a row from entry k on; TAIL: zeros from entry K on.
template <typename T, bool TAIL>
__device__ __forceinline__ u32x4 load16(const T* row, int k, int K) {
  typedef u32x4 V __attribute__((aligned(2)));
  constexpr int E = 16 / sizeof(T);
  if (!TAIL) return *reinterpret_cast<const V*>(row + k);
  u32x4 v = {};
  if (k + E <= K) {
    v = *reinterpret_cast<const V*>(row + k);
  } else if (k < K) {
#pragma unroll
    for (int e = 0; e < E - 1; ++e) {
      if (k + e >= K) continue;
      if constexpr (sizeof(T) == 2) v[e >> 1] |= (uint32_t)row[k + e] << (16 * (e & 1));
      else v[e] = __float_as_uint(row[k + e]);
    }
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void mma16(f32x4& acc, u32x4 a, u32x4 b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]),
                                                 acc, 0, 0, 0);
  }
}

// W: blocks of 16 weight rows, TB: of 16 tokens (lanes without one load
// nothing: for one token that is a sixteenth of what 16 lanes with its bytes
// would draw through the L1).  U: pieces whose loads are in flight together.
template <typename T, int W, int TB, int U, bool TAIL>
__device__ __forceinline__ void pieces(f32x4 (&acc)[W][TB], const T* const (&w)[W],
                                       const T* const (&x)[TB], int k, int step, int K,
                                       int tokens) {
  constexpr int E = 16 / sizeof(T);
  u32x4 a[U][W][2], b[U][TB][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < W; ++i) a[u][i][h] = load16<T, TAIL>(w[i], k + u * step + h * E, K);
#pragma unroll
  for (int t = 0; t < TB; ++t) {
#pragma unroll
    for (int u = 0; u < U; ++u) b[u][t][0] = b[u][t][1] = u32x4{};
    if (16 * t + (int)(threadIdx.x & 15) < tokens) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) b[u][t][h] = load16<T, TAIL>(x[t], k + u * step + h * E, K);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t) mma16<T>(acc[i][t], a[u][i][h], b[u][t][h]);
}

template <typename T, int KIND, int TB, int U>
__global__ __launch_bounds__(1024) void k_few(Product p) {
  constexpr int W = kind_dual(KIND) ? 2 : 1;
  constexpr int PIECE = 128 / sizeof(T), LANE = PIECE / 4;
  __shared__ f32x4 sums[16][W * TB][64];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16;
  const int r = lane & 15, k0 = (lane >> 4) * LANE;
  const T* w[W];
  const T* x[TB];
#pragma unroll
  for (int i = 0; i < W; ++i)
    w[i] = static_cast<const T*>(p.b[i].p) + min(n0 + r, p.N - 1) * p.b[i].ld + k0;
#pragma unroll
  for (int t = 0; t < TB; ++t)
    x[t] = static_cast<const T*>(p.a[0].p) + min(16 * t + r, p.M - 1) * p.a[0].ld + k0;
  f32x4 acc[W][TB] = {};
  const int step = waves * PIECE;
  int k = wave * PIECE;
  for (; k + (U - 1) * step + PIECE <= p.K; k += U * step)
    pieces<T, W, TB, U, false>(acc, w, x, k, step, p.K - k0, p.M);
  if (k < p.K) pieces<T, W, TB, U, true>(acc, w, x, k, step, p.K - k0, p.M);
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t) sums[wave][i * TB + t][lane] = acc[i][t];
  __syncthreads();
  // wave t finishes the t-th block of tokens: a lane has four columns of one
  if (wave >= TB) return;
  f32x4 s[W] = {};
  for (int q = 0; q < waves; ++q)
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] += sums[q][i * TB + wave][lane];
  const int row = 16 * wave + r, col = n0 + 4 * (lane >> 4);
  if (col >= p.N) return;
  const f32x4 bias = load_bias<T, KIND>(p, col);
  const f32x4 in = load_in<T, KIND>(p, 0, row, col);
  switch (p.act) {
#define SM_ACT(A) \
  case A: finish4<T, KIND, A>(p, 0, row, col, s[0], s[W - 1], bias, in); break;
    SM_ACT(SM_ACT_NONE)
    SM_ACT(SM_ACT_RELU)
    SM_ACT(SM_ACT_SILU)
    SM_ACT(SM_ACT_GELU)
    SM_ACT(SM_ACT_GELU_TANH)
#undef SM_ACT
  }
}

// 16 waves, where the rows have a piece for each, two pieces in flight up to 16
// tokens and one beyond.  No choice is the best everywhere; us, bf16 (nine sets
// of weights):
//                    waves x pieces   8 x 1  8 x 2  16 x 1  16 x 2
//   gated 4096 -> 11008, 1 token       35.5   35.3    34.3    34.1
//   linear 11008 -> 4096, 1 token      22.3   21.3    20.8    22.0
//   gated 4096 -> 11008, 16 tokens     38.3   42.2    38.1    41.1
//   gated 1280 -> 5120, 1 token         8.8    9.3     8.8    11.1
//   gated 11008 -> 4096, 19 tokens     42.4   48.7    44.2    48.0
// and float32, linear 4096 -> 11008, 1 token: 43.4, 38.8, 38.7, 36.6; 19 tokens:
// 59.6, 62.0, 57.4, 63.6.
template <typename T, int KIND>
void launch_kind(const Product& p, hipStream_t s) {
  constexpr int PIECE = 128 / sizeof(T);
  int waves = 16;
  while (waves > 2 && (waves - 1) * PIECE >= p.K) waves /= 2;
  const dim3 grid((p.N + 15) / 16), block(64 * waves);
  if (p.M <= 16) hipLaunchKernelGGL((k_few<T, KIND, 1, 2>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_few<T, KIND, 2, 1>), grid, block, 0, s, p);
}

}  // namespace

void launch_few(const Product& p, hipStream_t s) {
  SM_DISPATCH_DT(p.dt, E, if (p.kind == kLinear) launch_kind<E, kLinear>(p, s);
                 else launch_kind<E, kGated>(p, s));
}

}  // namespace layer
}  // namespace sm
