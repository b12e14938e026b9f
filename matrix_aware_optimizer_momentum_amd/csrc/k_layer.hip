// The feed-forward layers' launches: which tiles a product takes, the column
// sums behind dbias, and matrices laid out for the products.
#include "k_layer_tile.hpp"

namespace sm {

namespace {

int cu_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cache[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n <= 0)
      n = 256;
    cache[dev] = n;
  }
  return cache[dev];
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

// rows x cols entries to rows x ld ones, zeros behind them.
template <typename T>
__global__ __launch_bounds__(256) void k_lay_out(const T* p, int64_t ldp, int64_t rows, int cols,
                                                 T* out, int64_t ld) {
  const int64_t n = rows * ld;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / ld, c = i - r * ld;
    out[i] = c < cols ? p[r * ldp + c] : T(0);
  }
}

}  // namespace

sm_status launch_product(const Product& p, hipStream_t s) {
  using namespace layer;
  if (few_tokens(p.kind, p.M)) {
    prof_begin(SM_K_LAYER, 2.0 * p.M * p.N * p.K * (kind_dual(p.kind) ? 2 : 1), s, 0.0);
    launch_few(p, s);
    prof_end(s);
    return check_launch();
  }
  TileArgs a;
  a.p = p;
  const int cols = std::max(p.N, p.pad);
  const int nprob = p.kind == kDw ? p.parts : 1, cus = cu_count();
  auto tiles = [&](int mi) {
    const int rows = 64 * mi, width = kind_dual(p.kind) ? 32 * mi : 64 * mi;
    a.tiles_m = (p.M + rows - 1) / rows;
    a.tiles_n = (cols + width - 1) / width;
    a.per_prob = a.tiles_m * a.tiles_n;
    a.total = a.per_prob * nprob;
    return a.total;
  };
  const bool large = tiles(4) >= cus / 2;
  const int grid = std::min(tiles(large ? 4 : 2), large ? cus : 2 * cus);
  a.xcd_chunk = grid % 8 == 0 ? grid / 8 : 0;
  prof_begin(SM_K_LAYER, 2.0 * p.M * p.N * p.K * (kind_dual(p.kind) ? 2 : p.parts), s, 0.0);
  if (p.dt == BF16) (large ? launch_tile_bf16_4 : launch_tile_bf16_2)(a, grid, s);
  else (large ? launch_tile_f32_4 : launch_tile_f32_2)(a, grid, s);
  prof_end(s);
  return check_launch();
}

sm_status launch_lay_out(const void* p, int64_t ldp, int64_t rows, int cols, int dt, void* out,
                         int64_t ld, hipStream_t s) {
  const int64_t n = rows * ld;
  const int grid = (int)std::min<int64_t>(4096, (n + 255) / 256);
  prof_begin(SM_K_ACT8, 2.0 * n * dt_size(dt), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_lay_out<E>, dim3(grid), dim3(256), 0, s,
                                           static_cast<const E*>(p), ldp, rows, cols,
                                           static_cast<E*>(out), ld));
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
