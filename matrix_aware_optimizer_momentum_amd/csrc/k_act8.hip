// 8-bit checkpoints of activations: codes and scales of 32-entry blocks, and
// back.  Bound by HBM: every entry is read once and written once.
//
// Four lanes take a block, 8 entries each, and find its largest magnitude by
// two permutations; a lane reads and writes its 8 entries at once where the
// rows allow it.
#include "layer_internal.hpp"

namespace sm {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInf = 0x7F800000u;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Over groups of four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = umax(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));
  return umax(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));
}

// Entries 8 i .. 8 i + 7 of a row, of which `left` exist (the others read as
// 0 and are not written).
template <typename T>
__device__ __forceinline__ void get8(const T* p, int left, float* v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < left ? Elem<T>::load(p + e) : 0.f;
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int left, const float* v) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) Elem<T>::store(p + e, v[e]);
}

// Work item i: lane i % 4 of block i / 4, blocks row by row.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_act8_pack(const T* x, int64_t ldx, int64_t items,
                                                        int blocks, int d, uint8_t* x8,
                                                        uint8_t* scale) {
  // whole groups of four lanes run or do not (items is a multiple of 4)
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t blk = i >> 2;
    const int64_t row = blk / blocks;
    const int col = (int)(blk - row * blocks) * SM_ACT8_BLOCK + 8 * (int)(i & 3);
    const int left = d - col;
    float v[8];
    get8(x + row * ldx + col, left, v);
    uint32_t amax = 0, bad = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      if (b >= kInf) {
        bad |= 1u << e;
        v[e] = 0.f;
      } else {
        amax = umax(amax, b);
      }
    }
    amax = quad_max(amax);
    // biased exponent of the scale: 448 is 1.75 * 2^8
    int e8 = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e8 = e8 < 10 ? 10 : e8;   // 2^-117
    const float q = __uint_as_float((uint32_t)(254 - e8) << 23);
    if (e8 == 247) {   // 256 * 2^120 is infinite: 240 is the largest code here
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e], -0x1.Ep127f), 0x1.Ep127f);
    }
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * q, v[4 * h + 1] * q, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * q, v[4 * h + 3] * q, w, true);
      c[h] = (uint32_t)w;
    }
    uint8_t* out = x8 + row * d + col;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) out[e] = (bad >> e) & 1u ? 0x7Fu : (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
    if ((i & 3) == 0) scale[blk] = (uint8_t)e8;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_act8_unpack(const uint8_t* x8, const uint8_t* scale,
                                                          int64_t items, int blocks, int d, T* x,
                                                          int64_t ldx, bool pad) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t blk = i >> 2;
    const int64_t row = blk / blocks;
    const int col = (int)(blk - row * blocks) * SM_ACT8_BLOCK + 8 * (int)(i & 3);
    const int left = d - col;
    const uint32_t e8 = scale[blk];
    // 2^(e8 - 127); 0 is 2^-127, a subnormal; 255 stands for NaN
    const float q = e8 == 255u ? __uint_as_float(0x7FC00000u)
                               : __uint_as_float(e8 ? e8 << 23 : 0x400000u);
    const uint8_t* in = x8 + row * d + col;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t c = e < left ? in[e] : 0u;
      v[e] = __builtin_amdgcn_cvt_f32_fp8(c, 0) * q;
    }
    put8(x + row * ldx + col, pad && left > 0 ? 8 : left, v);
  }
}

int grid_for(int64_t items) {
  const int64_t g = (items + kThreads - 1) / kThreads;
  return (int)(g < 1 ? 1 : g > 8192 ? 8192 : g);
}

}  // namespace

sm_status launch_act8_pack(const void* x, int64_t ldx, int dt, int64_t T, int d, uint8_t* x8,
                           uint8_t* scale, hipStream_t s) {
  const int blocks = (d + SM_ACT8_BLOCK - 1) / SM_ACT8_BLOCK;
  const int64_t items = T * blocks * 4;
  prof_begin(SM_K_ACT8, (double)T * (d * (1.0 + dt_size(dt)) + blocks), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_act8_pack<E>, dim3(grid_for(items)), dim3(kThreads),
                                           0, s, static_cast<const E*>(x), ldx, items, blocks, d,
                                           x8, scale));
  prof_end(s);
  return check_launch();
}

sm_status launch_act8_unpack(const uint8_t* x8, const uint8_t* scale, int dt, int64_t T, int d,
                             void* x, int64_t ldx, bool pad, hipStream_t s) {
  const int blocks = (d + SM_ACT8_BLOCK - 1) / SM_ACT8_BLOCK;
  const int64_t items = T * blocks * 4;
  prof_begin(SM_K_ACT8, (double)T * (d * (1.0 + dt_size(dt)) + blocks), s);
  SM_DISPATCH_DT(dt, E, hipLaunchKernelGGL(k_act8_unpack<E>, dim3(grid_for(items)), dim3(kThreads),
                                           0, s, x8, scale, items, blocks, d, static_cast<E*>(x),
                                           ldx, pad));
  prof_end(s);
  return check_launch();
}

}  // namespace sm
