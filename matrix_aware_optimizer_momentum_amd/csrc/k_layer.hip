// The feed-forward layers' matrix products, for every type, size, stride and
// alignment: 64 x 64 tiles of the result, k steps of 32 staged through LDS
// element by element, one 32 x 32 block of MFMA sums (two for the gated
// kinds) per wave, and the epilogue from the registers.
#include "layer_math.hpp"

namespace sm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 64, kStep = 32;

// LDS pitch of a tile row: 16-byte multiples, rows 4 banks apart or more.
template <typename T>
constexpr int kPitch = kStep + 16 / (int)sizeof(T);

template <typename T, bool KR>
__device__ __forceinline__ void stage(T* lds, const T* p, int64_t ld, int row0, int rows, int k0,
                                      int K) {
#pragma unroll
  for (int i = 0; i < kTile * kStep / 256; ++i) {
    const int e = i * 256 + (int)threadIdx.x;
    const int r = KR ? e % kTile : e / kStep, k = KR ? e / kTile : e % kStep;
    const bool in = row0 + r < rows && k0 + k < K;
    const int64_t at = KR ? (int64_t)(k0 + k) * ld + row0 + r : (int64_t)(row0 + r) * ld + k0 + k;
    lds[r * kPitch<T> + k] = in ? p[at] : T(0);
  }
}

// acc += the products of k step 32 of wave block (wm, wn).
__device__ __forceinline__ void multiply(f32x16& acc, const bf16_t* a, const bf16_t* b) {
  const int lane = threadIdx.x & 63;
  const int at = (lane & 31) * kPitch<bf16_t> + 8 * (lane >> 5);
#pragma unroll
  for (int k = 0; k < kStep; k += 16)
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(a + at + k),
                                                  *reinterpret_cast<const bf16x8*>(b + at + k), acc,
                                                  0, 0, 0);
}
__device__ __forceinline__ void multiply(f32x16& acc, const float* a, const float* b) {
  const int lane = threadIdx.x & 63;
  const int at = (lane & 31) * kPitch<float> + (lane >> 5);
#pragma unroll
  for (int k = 0; k < kStep; k += 2)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[at + k], b[at + k], acc, 0, 0, 0);
}

template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_product(Product p) {
  constexpr bool DUAL = kind_dual(KIND), AKR = kind_a_kr(KIND), BKR = kind_b_kr(KIND);
  constexpr bool FINE = sizeof(T) == 4;
  __shared__ __attribute__((aligned(16))) T la[kTile * kPitch<T>];
  __shared__ __attribute__((aligned(16))) T lb[DUAL ? 2 : 1][kTile * kPitch<T>];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  const int z = blockIdx.z;
  f32x16 acc[DUAL ? 2 : 1] = {};
  const int sums = KIND == kDx ? p.parts : 1;
  for (int q = 0; q < sums; ++q) {
    const Operand A = p.a[KIND == kDw ? z : q], B = p.b[q];
    for (int k0 = 0; k0 < p.K; k0 += kStep) {
      __syncthreads();
      stage<T, AKR>(la, static_cast<const T*>(A.p), A.ld, m0, p.M, k0, p.K);
      stage<T, BKR>(lb[0], static_cast<const T*>(B.p), B.ld, n0, p.N, k0, p.K);
      if constexpr (DUAL)
        stage<T, BKR>(lb[1], static_cast<const T*>(p.b[1].p), p.b[1].ld, n0, p.N, k0, p.K);
      __syncthreads();
      multiply(acc[0], la + wm * kPitch<T>, lb[0] + wn * kPitch<T>);
      if constexpr (DUAL) multiply(acc[1], la + wm * kPitch<T>, lb[1] + wn * kPitch<T>);
    }
  }
  const int col = n0 + wn + (lane & 31);
  if (col >= (p.pad > p.N ? p.pad : p.N)) return;
  T* c0 = static_cast<T*>(p.c[KIND == kDw ? z : 0]);
  const int64_t ldc = p.ldc[KIND == kDw ? z : 0];
  const T* in = static_cast<const T*>(p.in.p);
  const float bias = p.bias && col < p.N ? Elem<T>::load(static_cast<const T*>(p.bias) + col) : 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = m0 + wm + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    if (row >= p.M) continue;
    T* c = c0 + row * ldc + col;
    if (col >= p.N) {   // the padding of dz
      Elem<T>::store(c, 0.f);
      if constexpr (KIND == kGatedSlope)
        Elem<T>::store(static_cast<T*>(p.c[1]) + row * p.ldc[1] + col, 0.f);
      continue;
    }
    float v = acc[0][r];
    if constexpr (KIND == kLinear) {
      v = act_value<FINE>(p.act, v + bias);
      if (in) v += Elem<T>::load(in + row * p.in.ld + col);
    } else if constexpr (KIND == kSlope) {
      v = Elem<T>::load(in + row * p.in.ld + col) * act_both<FINE>(p.act, v + bias).slope;
    } else if constexpr (KIND == kGated) {
      v = act_value<FINE>(p.act, v) * acc[1][r];
    } else if constexpr (KIND == kGatedSlope) {
      const float g = Elem<T>::load(in + row * p.in.ld + col);
      const ActBoth h = act_both<FINE>(p.act, v);
      v = g * acc[1][r] * h.slope;
      Elem<T>::store(static_cast<T*>(p.c[1]) + row * p.ldc[1] + col, g * h.value);
    } else if constexpr (KIND == kDw) {
      if (p.accumulate) v += Elem<T>::load(c);
    }
    Elem<T>::store(c, v);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_column_sums(const T* dz, int64_t ld, int64_t rows, int n,
                                                     T* out, int accumulate) {
  __shared__ float red[256];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  float sum = 0.f;
  if (col < n)
    for (int64_t r = threadIdx.x >> 5; r < rows; r += 8) sum += Elem<T>::load(dz + r * ld + col);
  red[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 32 || col >= n) return;
#pragma unroll
  for (int q = 1; q < 8; ++q) sum += red[threadIdx.x + 32 * q];
  if (accumulate) sum += Elem<T>::load(out + col);
  Elem<T>::store(out + col, sum);
}

template <typename T>
__global__ __launch_bounds__(256) void k_zero(T* p, int64_t ld, int64_t rows, int cols) {
  const int64_t n = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cols;
    p[r * ld + (i - r * cols)] = T(0);
  }
}

template <typename T>
void launch_kind(const Product& p, dim3 grid, hipStream_t s) {
  switch (p.kind) {
#define SM_KIND(K) \
  case K: hipLaunchKernelGGL((k_product<T, K>), grid, dim3(256), 0, s, p); break;
    SM_KIND(kLinear)
    SM_KIND(kSlope)
    SM_KIND(kGated)
    SM_KIND(kGatedSlope)
    SM_KIND(kDx)
    SM_KIND(kDw)
#undef SM_KIND
  }
}

}  // namespace

sm_status launch_product(const Product& p, hipStream_t s) {
  const int cols = std::max(p.N, p.pad);
  const dim3 grid((cols + kTile - 1) / kTile, (p.M + kTile - 1) / kTile,
                  p.kind == kDw ? p.parts : 1);
  if (grid.y > 65535) return SM_ERR_SHAPE;
  prof_begin(SM_K_LAYER, 2.0 * p.M * p.N * p.K * (kind_dual(p.kind) ? 2 : p.parts), s, 0.0);
  SM_DISPATCH_DT(p.dt, E, launch_kind<E>(p, grid, s));
  prof_end(s);
  return check_launch();
}

sm_status launch_column_sums(const void* dz, int64_t ld, int64_t T, int n, int dt, void* out,
                             int accumulate, hipStream_t s) {
  prof_begin(SM_K_ACT8, (double)T * n * dt_size(dt), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_column_sums<E>, dim3((n + 31) / 32), dim3(256), 0, s,
                                           static_cast<const E*>(dz), ld, T, n,
                                           static_cast<E*>(out), accumulate));
  prof_end(s);
  return check_launch();
}

sm_status launch_zero(void* p, int64_t ld, int64_t rows, int cols, int dt, hipStream_t s) {
  const int64_t n = rows * cols;
  const int grid = (int)std::min<int64_t>(4096, (n + 255) / 256);
  prof_begin(SM_K_ACT8, (double)n * dt_size(dt), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_zero<E>, dim3(grid), dim3(256), 0, s,
                                           static_cast<E*>(p), ld, rows, cols));
  prof_end(s);
  return check_launch();
}

}  // namespace sm
