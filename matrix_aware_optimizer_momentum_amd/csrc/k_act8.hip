// 8-bit checkpoints of activations: codes and scales of 32-entry blocks, and
// back.  Bound by HBM: every entry is read once and written once.
//
// Four lanes take a block, 8 entries each, and find its largest magnitude by
// two permutations; a wave's accesses are 16 bytes a lane (bf16; twice that in
// float32) and 8 bytes of codes.  A workgroup takes one or four units of 64
// blocks, all of whose loads are in flight before the first is used.  Rows and columns
// come from one scalar division a workgroup: a division per lane in 64 bits
// cost more than the memory (pack of 8192 x 4096 bf16: 44 us with it).
// Measured with one or two sets of buffers in turn, three, and six (less and less
// of what is read is still in the Infinity Cache): that pack 16.5, 16.5 and 20.0
// us (6.2, 6.2, 5.1 TB/s), unpack of 8192 x 11008 to bf16 39.5, 43.9 and 48.5
// (6.9, 6.2, 5.6).
#include "layer_internal.hpp"

namespace sm {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = kThreads / 4;   // of a unit
constexpr uint32_t kInf = 0x7F800000u;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Over groups of four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = umax(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));
  return umax(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));
}

// Eight entries, of which `left` exist (the others read as 0 and are not
// written), at any alignment: global memory takes wide accesses at the
// entries' own.
template <typename T>
struct Raw8 {
  u32x4 a[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> get8(const T* p, int left) {
  typedef u32x4 V __attribute__((aligned(2)));
  Raw8<T> r = {};
  if (left >= 8) {
#pragma unroll
    for (unsigned h = 0; h < sizeof(T) / 2; ++h)
      r.a[h] = *reinterpret_cast<const V*>(p + h * (16 / sizeof(T)));
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (e >= left) continue;
      if constexpr (sizeof(T) == 2) r.a[0][e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
      else r.a[e >> 2][e & 3] = __float_as_uint(p[e]);
    }
  }
  return r;
}
__device__ __forceinline__ void expand8(const Raw8<bf16_t>& r, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(r.a[0][e] << 16);
    v[2 * e + 1] = __uint_as_float(r.a[0][e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void expand8(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.a[e >> 2][e & 3]);
}
template <bool NT, typename V, typename P>
__device__ __forceinline__ void store_v(P* p, V v) {
  typedef V VP __attribute__((aligned(alignof(P))));   // P: an entry
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<VP*>(p));
  else *reinterpret_cast<VP*>(p) = v;
}
template <bool NT>
__device__ __forceinline__ void put8(float* p, int left, const float* v) {
  if (left >= 8) {
    store_v<NT>(p, f32x4{v[0], v[1], v[2], v[3]});
    store_v<NT>(p + 4, f32x4{v[4], v[5], v[6], v[7]});
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) p[e] = v[e];
}
template <bool NT>
__device__ __forceinline__ void put8(bf16_t* p, int left, const float* v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bf16x2 b;
    b[0] = (__bf16)v[2 * e];
    b[1] = (__bf16)v[2 * e + 1];
    w[e] = __builtin_bit_cast(uint32_t, b);
  }
  if (left >= 8) {
    store_v<NT>(p, w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) p[e] = (bf16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// Where a lane's 8 entries are: block `at` of the workgroup's first one (row0,
// block0; `blocks` to a row).
struct Place {
  int64_t row;
  int blk, col, left;
};
__device__ __forceinline__ Place place(int64_t row0, int block0, int at, int blocks, int d) {
  int r = 0, b = block0 + at;
  if (blocks >= 4 * kBlocks) {   // at most one row on
    if (b >= blocks) b -= blocks, r = 1;
  } else {
    r = (int)((uint32_t)b / (uint32_t)blocks);
    b -= r * blocks;
  }
  const int col = b * SM_ACT8_BLOCK + 8 * (int)(threadIdx.x & 3);
  return {row0 + r, b, col, d - col};
}

// Largest magnitude of eight entries, as float32 bits (magnitudes order like
// their bits; kInf or more if some entry is not finite).
__device__ __forceinline__ uint32_t amax8(const Raw8<bf16_t>& r) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.a[0][e] & 0x7FFF7FFFu));
  return umax(m[0], m[1]) << 16;
}
__device__ __forceinline__ uint32_t amax8(const Raw8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = umax(m, r.a[e >> 2][e & 3] & 0x7FFFFFFFu);
  return m;
}
// Eight codes; the hardware's scaled conversions divide by the scale, a power
// of two, and round to nearest even.
__device__ __forceinline__ u32x2 encode8(const Raw8<bf16_t>& r, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    i16x2 w = {};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(
        w, __builtin_bit_cast(bf16x2, (uint32_t)r.a[0][2 * h]), scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(
        w, __builtin_bit_cast(bf16x2, (uint32_t)r.a[0][2 * h + 1]), scale, true);
    c[h] = __builtin_bit_cast(uint32_t, w);
  }
  return c;
}
__device__ __forceinline__ u32x2 encode8(const Raw8<float>& r, float scale) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  float v[8];
  expand8(r, v);
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    i16x2 w = {};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[4 * h], v[4 * h + 1], scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[4 * h + 2], v[4 * h + 3], scale, true);
    c[h] = __builtin_bit_cast(uint32_t, w);
  }
  return c;
}
// Biased exponent of the scale of a block of the largest finite magnitude
// amax: 448 is 1.75 * 2^8, and the least scale 2^-117.
__device__ __forceinline__ uint32_t exponent_for(uint32_t amax) {
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 10 ? 10 : e);
}
// A block with entries that are not finite, or so large that a code's value
// might be infinite: those become NaN, and 240 the largest code under 2^120.
template <typename T>
__device__ __forceinline__ u32x2 encode8_rare(const Raw8<T>& r, uint32_t* e8) {
  float v[8];
  expand8(r, v);
  uint32_t amax = 0, bad = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    if (b >= kInf) bad |= 1u << e, v[e] = 0.f;
    else amax = umax(amax, b);
  }
  *e8 = exponent_for(quad_max(amax));
  if (*e8 == 247u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e], -0x1.Ep127f), 0x1.Ep127f);
  }
  const float q = __uint_as_float((254u - *e8) << 23);
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * q, v[4 * h + 1] * q, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * q, v[4 * h + 3] * q, w, true);
    c[h] = (uint32_t)w;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if ((bad >> e) & 1u) c[e >> 2] |= 0x7Fu << (8 * (e & 3));   // 0 before
  return c;
}

template <typename T, int UNITS, bool NT>
__global__ __launch_bounds__(kThreads) void k_act8_pack(const T* x, int64_t ldx, int64_t rows,
                                                        int blocks, int d, uint8_t* x8,
                                                        uint8_t* scale) {
  const int64_t first = (int64_t)blockIdx.x * (kBlocks * UNITS);
  const int64_t row0 = first / blocks;
  const int block0 = (int)(first - row0 * blocks);
  Place at[UNITS];
  Raw8<T> raw[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    at[u] = place(row0, block0, u * kBlocks + (int)(threadIdx.x >> 2), blocks, d);
    if (at[u].row >= rows) at[u].left = 0;
    raw[u] = get8(x + at[u].row * ldx + at[u].col, at[u].left);
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if (at[u].row >= rows) continue;   // whole groups of four lanes
    uint32_t e8 = exponent_for(quad_max(amax8(raw[u])));
    u32x2 c = encode8(raw[u], __uint_as_float(e8 << 23));
    if (__builtin_expect(e8 >= 247u, 0)) c = encode8_rare(raw[u], &e8);
    uint8_t* out = x8 + at[u].row * d + at[u].col;
    if (at[u].left >= 8) {
      store_v<NT>(out, c);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < at[u].left) out[e] = (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
    }
    if ((threadIdx.x & 3) == 0) scale[at[u].row * blocks + at[u].blk] = (uint8_t)e8;
  }
}

template <typename T, int UNITS, bool NT>
__global__ __launch_bounds__(kThreads) void k_act8_unpack(const uint8_t* x8, const uint8_t* scale,
                                                          int64_t rows, int blocks, int d, T* x,
                                                          int64_t ldx, bool pad) {
  const int64_t first = (int64_t)blockIdx.x * (kBlocks * UNITS);
  const int64_t row0 = first / blocks;
  const int block0 = (int)(first - row0 * blocks);
  Place at[UNITS];
  u32x2 raw[UNITS];
  uint32_t e8[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    at[u] = place(row0, block0, u * kBlocks + (int)(threadIdx.x >> 2), blocks, d);
    if (at[u].row >= rows) at[u].left = 0;
    const uint8_t* p = x8 + at[u].row * d + at[u].col;
    raw[u] = u32x2{};
    e8[u] = 0;
    if (at[u].left > 0) e8[u] = scale[at[u].row * blocks + at[u].blk];
    if (at[u].left >= 8) {
      typedef u32x2 V __attribute__((aligned(1)));
      raw[u] = *reinterpret_cast<const V*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < at[u].left) raw[u][e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if (at[u].left <= 0) continue;
    // 2^(e8 - 127); 0 is 2^-127, a subnormal; 255 stands for NaN
    const float q = e8[u] == 255u ? __uint_as_float(0x7FC00000u)
                                  : __uint_as_float(e8[u] ? e8[u] << 23 : 0x400000u);
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[u][h], false);
      const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[u][h], true);
      v[4 * h] = a[0] * q;
      v[4 * h + 1] = a[1] * q;
      v[4 * h + 2] = b[0] * q;
      v[4 * h + 3] = b[1] * q;
    }
    put8<NT>(x + at[u].row * ldx + at[u].col, pad ? 8 : at[u].left, v);
  }
}

// Blocks from which a workgroup takes four units: 256 workgroups of them.
constexpr int64_t kManyBlocks = 256 * 4 * kBlocks;
// A checkpoint is read in the backward pass: its stores are non-temporal (8192
// x 4096 bf16: 16.5 us, 20.7 cacheable).  Values are used sooner, and theirs
// are cacheable as long as all that a call moves (codes, scales and values)
// may stay in the Infinity Cache.  Just beyond, the call itself is faster with
// non-temporal ones, a reader right behind it with the others: 8192 x 11008 to
// bf16 (273 MB, 180 of them values) 39.6 us and 45.5, with a reading of the
// values 113 and 104; a backward pass with weight gradients alone 660 and 655,
// with dx ahead of them 1246 both.
constexpr double kStreamBytes = 256.0 * 1024 * 1024;

}  // namespace

// Launches KERNEL<E, units, non-temporal> over T x blocks blocks.
#define SM_ACT8_LAUNCH(KERNEL, STREAM, ...)                                              \
  do {                                                                                   \
    const int64_t n = T * blocks;                                                        \
    const bool many = n >= kManyBlocks;                                                  \
    const int group = (many ? 4 : 1) * kBlocks;                                          \
    const dim3 grid((unsigned)((n + group - 1) / group)), block(kThreads);               \
    if (!many)                                                                           \
      hipLaunchKernelGGL((KERNEL<E, 1, false>), grid, block, 0, s, __VA_ARGS__);         \
    else if (!(STREAM))                                                                  \
      hipLaunchKernelGGL((KERNEL<E, 4, false>), grid, block, 0, s, __VA_ARGS__);         \
    else                                                                                 \
      hipLaunchKernelGGL((KERNEL<E, 4, true>), grid, block, 0, s, __VA_ARGS__);          \
  } while (0)

sm_status launch_act8_pack(const void* x, int64_t ldx, int dt, int64_t T, int d, uint8_t* x8,
                           uint8_t* scale, hipStream_t s) {
  const int blocks = (d + SM_ACT8_BLOCK - 1) / SM_ACT8_BLOCK;
  const double bytes = (double)T * (d * (1.0 + dt_size(dt)) + blocks);
  prof_begin(SM_K_ACT8, bytes, s);
  SM_DISPATCH_DT(dt, E, SM_ACT8_LAUNCH(k_act8_pack, true, static_cast<const E*>(x), ldx, T, blocks, d,
                                       x8, scale));
  prof_end(s);
  return check_launch();
}

sm_status launch_act8_unpack(const uint8_t* x8, const uint8_t* scale, int dt, int64_t T, int d,
                             void* x, int64_t ldx, bool pad, hipStream_t s) {
  const int blocks = (d + SM_ACT8_BLOCK - 1) / SM_ACT8_BLOCK;
  const double bytes = (double)T * (d * (1.0 + dt_size(dt)) + blocks);
  prof_begin(SM_K_ACT8, bytes, s);
  SM_DISPATCH_DT(dt, E, SM_ACT8_LAUNCH(k_act8_unpack, bytes > kStreamBytes, x8, scale, T, blocks, d,
                                       static_cast<E*>(x), ldx, pad));
  prof_end(s);
  return check_launch();
}

}  // namespace sm
