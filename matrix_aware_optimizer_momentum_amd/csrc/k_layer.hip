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

// Column sums over kSumRows rows, of dz as it was rounded for the products (in
// bf16 an error as large as the rounding of the sums themselves, where terms of
// both signs cancel to a root of their number): a wave takes every eighth row, a lane two
// columns, eight rows in flight.  FINAL: those are all rows, and the sums go to
// out (or onto it); else to sums[blockIdx.y][n] in float32.
constexpr int kSumRows = 256, kSumCols = 128, kSumWaves = 8;
template <typename T, bool FINAL>
__global__ __launch_bounds__(64 * kSumWaves) void k_column_sums(const T* dz, int64_t ld,
                                                                int64_t rows, int n, T* out,
                                                                float* sums, int accumulate) {
  __shared__ float red[kSumWaves][kSumCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * kSumCols + 2 * lane;
  const int64_t r0 = (int64_t)blockIdx.y * kSumRows + wave;
  const int64_t end = r0 - wave + kSumRows < rows ? r0 - wave + kSumRows : rows;
  const bool one = col < n, two = col + 1 < n;
  float a = 0.f, b = 0.f;
  for (int64_t r = r0; r < end; r += 8 * kSumWaves) {
    T v[8][2];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t at = (r + q * kSumWaves) * ld + col;
      const bool in = r + q * kSumWaves < end;
      v[q][0] = in && one ? dz[at] : T(0);
      v[q][1] = in && two ? dz[at + 1] : T(0);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      a += Elem<T>::load(&v[q][0]);
      b += Elem<T>::load(&v[q][1]);
    }
  }
  red[wave][2 * lane] = a;
  red[wave][2 * lane + 1] = b;
  __syncthreads();
  const int c = blockIdx.x * kSumCols + (int)threadIdx.x;
  if (threadIdx.x >= kSumCols || c >= n) return;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < kSumWaves; ++q) s += red[q][threadIdx.x];
  if constexpr (FINAL) {
    if (accumulate) s += Elem<T>::load(out + c);
    Elem<T>::store(out + c, s);
  } else {
    sums[(int64_t)blockIdx.y * n + c] = s;
  }
}
template <typename T>
__global__ __launch_bounds__(64) void k_column_join(const float* sums, int shares, int n, T* out,
                                                    int accumulate) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
  for (int q = 0; q < shares; ++q) s += sums[(int64_t)q * n + c];
  if (accumulate) s += Elem<T>::load(out + c);
  Elem<T>::store(out + c, s);
}

template <typename T>
__global__ __launch_bounds__(256) void k_zero(T* p, int64_t ld, int64_t rows, int cols) {
  const int64_t n = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cols;
    p[r * ld + (i - r * cols)] = T(0);
  }
}

// A matrix a launch row (blockIdx.y): a thread takes 8 entries of the copy, read at
// once where they exist at whatever alignment, its row by one scalar division a workgroup and one in 32 bits.
template <typename T>
__global__ __launch_bounds__(256) void k_lay_out(LayOuts all) {
  constexpr int N = sizeof(T) / 2;   // 16-byte pieces
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef u32x4 V __attribute__((aligned(2)));
  const LayOut& m = all.m[blockIdx.y];
  const int cols = m.cols;
  const int per_row = (int)(m.ld / 8);
  const int64_t n = m.rows * per_row;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < n; first += (int64_t)gridDim.x * 256) {
    const int64_t row0 = first / per_row;
    const uint32_t at = (uint32_t)(first - row0 * per_row) + threadIdx.x;
    const int64_t row = row0 + at / (uint32_t)per_row;
    if (row >= m.rows) break;
    const int col = 8 * (int)(at % (uint32_t)per_row);
    const T* q = static_cast<const T*>(m.p) + row * m.ldp + col;
    u32x4 v[N] = {};
    if (col + 8 <= cols) {
#pragma unroll
      for (int h = 0; h < N; ++h) v[h] = reinterpret_cast<const V*>(q)[h];
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e) {
        if (col + e >= cols) continue;
        if constexpr (sizeof(T) == 2) v[0][e >> 1] |= (uint32_t)q[e] << (16 * (e & 1));
        else v[e >> 2][e & 3] = __float_as_uint(q[e]);
      }
    }
#pragma unroll
    for (int h = 0; h < N; ++h)
      reinterpret_cast<u32x4*>(static_cast<T*>(m.out) + row * m.ld + col)[h] = v[h];
  }
}

}  // namespace

namespace {

Plan plan_of(int kind, int dt, int M, int N, int K, int parts) {
  return plan_product(kind, dt == BF16, M, N, K, parts, cu_count());
}

layer::TileArgs tile_args(const Product& p, int mi, int splits) {
  layer::TileArgs a;
  std::memset(&a, 0, sizeof(a));
  a.p = p;
  a.tiles_m = ceil_div(p.M, tile_rows(mi));
  a.tiles_n = ceil_div(std::max(p.N, p.pad), tile_cols(p.kind, mi));
  a.per_prob = a.tiles_m * a.tiles_n;
  a.splits = splits;
  a.total = a.per_prob * (p.kind == kDw ? p.parts : 1) * splits;
  a.rows = a.tiles_m * tile_rows(mi);
  a.width = a.tiles_n * 64 * mi;
  return a;
}

void launch_tiles(const Product& p, int mi, int splits, void* sums, hipStream_t s) {
  using namespace layer;
  TileArgs a = tile_args(p, mi, splits);
  a.sums = static_cast<float*>(sums);
  const int grid = std::min(a.total, mi == 4 ? cu_count() : 2 * cu_count());
  a.xcd_chunk = grid % 8 == 0 ? grid / 8 : 0;
  if (p.dt == BF16)
    (mi == 4 ? launch_tile_bf16_4 : mi == 2 ? launch_tile_bf16_2 : launch_tile_bf16_1)(a, grid, s);
  else
    (mi == 4 ? launch_tile_f32_4 : mi == 2 ? launch_tile_f32_2 : launch_tile_f32_1)(a, grid, s);
}

}  // namespace

bool few_tokens(int kind, int dt, int64_t T, int n, int d, bool w_in_place, bool x_in_place) {
  return takes_few(kind, dt == BF16, T, n, d, w_in_place, x_in_place, cu_count());
}

size_t product_ws(int kind, int dt, int M, int N, int K, int parts) {
  const Plan plan = plan_of(kind, dt, M, N, K, parts);
  if (plan.splits == 1) return 0;
  Product p;
  std::memset(&p, 0, sizeof(p));
  p.kind = kind;
  p.M = M;
  p.N = N;
  p.pad = (N + 7) / 8 * 8;
  p.parts = parts;
  const layer::TileArgs a = tile_args(p, plan.mi, plan.splits);
  return (size_t)a.rows * a.width * 4 * (kind == kDw ? parts : 1) * plan.splits;
}

// Operands read once, results written once (read first if they are added to).
static double product_bytes(const Product& p) {
  const double a = (double)p.M * p.K, b = (double)p.N * p.K, c = (double)p.M * p.N;
  double n = a * p.parts + b + c;
  if (kind_dual(p.kind)) n += b;
  if (p.kind == kGatedSlope) n += c;
  if (p.kind == kDx && p.parts == 2) n += b;
  if (p.kind == kDw) n += c * (p.parts * (p.accumulate ? 2 : 1) - 1);
  if (p.in.p) n += c;
  return n * dt_size(p.dt);
}

sm_status launch_product(const Product& p, void* sums, hipStream_t s) {
  prof_begin(SM_K_LAYER, 2.0 * p.M * p.N * p.K * (kind_dual(p.kind) ? 2 : p.parts), s,
             product_bytes(p));
  if (p.few) {
    layer::launch_few(p, s);
  } else {
    const Plan plan = plan_of(p.kind, p.dt, p.M, p.N, p.K, p.parts);
    Product q = p;
    q.N = std::min(p.N, plan.cut);
    if (plan.cut < p.N && p.pad) q.pad = q.N;
    launch_tiles(q, plan.mi, plan.splits, sums, s);
    if (plan.cut < p.N) {
      const int64_t size = (int64_t)dt_size(p.dt), at = plan.cut * size;
      auto on = [](const void* m, int64_t bytes) {
        return m ? static_cast<const char*>(m) + bytes : nullptr;
      };
      q = p;
      q.N = p.N - plan.cut;
      q.pad = p.pad ? p.pad - plan.cut : 0;
      for (int i = 0; i < 2; ++i) {
        q.b[i].p = on(p.b[i].p, kind_b_kr(p.kind) ? at : at * p.b[i].ld);
        q.c[i] = const_cast<char*>(on(p.c[i], at));
      }
      q.bias = on(p.bias, at);
      q.in.p = on(p.in.p, at);
      launch_tiles(q, 2, 1, nullptr, s);
    }
  }
  prof_end(s);
  return check_launch();
}

sm_status launch_lay_out(const LayOuts& all, int dt, hipStream_t s) {
  if (all.n == 0) return SM_OK;
  int64_t most = 0;
  double bytes = 0.0;
  for (int i = 0; i < all.n; ++i) {
    const int64_t n = all.m[i].rows * (all.m[i].ld / 8);
    most = std::max(most, n);
    bytes += 16.0 * n * dt_size(dt);
  }
  const dim3 grid((unsigned)std::min<int64_t>((most + 255) / 256, 1 << 20), all.n);
  prof_begin(SM_K_MISC, bytes, s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_lay_out<E>, grid, dim3(256), 0, s, all));
  prof_end(s);
  return check_launch();
}

size_t column_sums_ws(int64_t T, int n) {
  return T > kSumRows ? (size_t)ceil_div(T, kSumRows) * n * 4 : 0;
}

sm_status launch_column_sums(const void* dz, int64_t ld, int64_t T, int n, int dt, void* out,
                             int accumulate, void* sums, hipStream_t s) {
  const int shares = ceil_div(T, kSumRows);
  const dim3 block(64 * kSumWaves);
  float* f = static_cast<float*>(sums);
  prof_begin(SM_K_MISC, (double)T * n * dt_size(dt), s);
  // shares beyond a grid's height: launches of their own
  for (int q = 0; q < shares; q += 65535) {
    const dim3 grid((n + kSumCols - 1) / kSumCols, std::min(shares - q, 65535));
    const int64_t r0 = (int64_t)q * kSumRows;
    SM_DISPATCH_DT(dt, E, const E* z = static_cast<const E*>(dz) + r0 * ld;
                   if (shares == 1)
                     hipLaunchKernelGGL((k_column_sums<E, true>), grid, block, 0, s, z, ld, T, n,
                                        static_cast<E*>(out), f, accumulate);
                   else hipLaunchKernelGGL((k_column_sums<E, false>), grid, block, 0, s, z, ld,
                                           T - r0, n, static_cast<E*>(out), f + (int64_t)q * n,
                                           accumulate));
  }
  if (shares > 1)
    SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_column_join<E>, dim3((n + 63) / 64), dim3(64), 0, s,
                                             f, shares, n, static_cast<E*>(out), accumulate));
  prof_end(s);
  return check_launch();
}

sm_status launch_zero(void* p, int64_t ld, int64_t rows, int cols, int dt, hipStream_t s) {
  const int64_t n = rows * cols;
  const int grid = (int)std::min<int64_t>(4096, (n + 255) / 256);
  prof_begin(SM_K_MISC, (double)n * dt_size(dt), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_zero<E>, dim3(grid), dim3(256), 0, s,
                                           static_cast<E*>(p), ld, rows, cols));
  prof_end(s);
  return check_launch();
}

}  // namespace sm
