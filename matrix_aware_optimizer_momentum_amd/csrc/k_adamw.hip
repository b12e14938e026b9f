// AdamW over sets of parameters (float32 or 8-bit states), the global
// gradient norm, and the conversion of 8-bit states.  All of it is bound by
// HBM: every entry's weights, gradients and states are read once and written
// once, with accesses of up to 16 bytes per lane, contiguous across the wave.
//
// One launch works on a whole set, whatever its lengths and types: each
// workgroup reads its work item (parameter, place) and the parameter's table
// entry, both uniform (scalar loads), and takes one unit of entries, 4 per
// lane.
#include "adamw_internal.hpp"

#include <type_traits>

namespace sm {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = kThreads * 4;   // 4 entries per thread
// The step's accesses are non-temporal: between two steps a forward and a
// backward pass go through the caches, so that nothing of a set is left in
// them.  On data that other sets have pushed out, cacheable / non-temporal,
// by the bytes that a step moves:
//   float32 states, bf16 weights   16 MB 7.0 / 6.9 us, 64 MB 16.5 / 13.8,
//                                  256 MB 52 / 45, 512 MB 100 / 84
//   8-bit states, masters          16 MB 7.3 / 6.9 us, 64 MB 18.2 / 14.7,
//                                  256 MB 53 / 46, 512 MB 100 / 89
// (On a set of 256 MB that is still cached, 41 / 43.)  The norm, whose
// gradients the step reads next, and the states' conversion stay cacheable
// up to the 256 MB of the Infinity Cache:
//   norm   256 MB 48 / 46 us, 400 MB 72 / 67, 512 MB 90 / 84
//   pack   192 MB 35 / 36 us, 256 MB 46 / 46, 400 MB 76 / 70
constexpr double kStreamBytes = 256.0 * 1024 * 1024;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// Pointers that a kernel reads from a table carry no address space; these
// say that they are global memory (else every access is a flat one), and,
// for a kernel's tables and scalars, that nothing writes them while it runs
// (so that uniform ones take scalar loads).
#define SM_GLOBAL __attribute__((address_space(1)))
#define SM_CONST __attribute__((address_space(4)))
template <typename T>
__device__ __forceinline__ T load_const(const T* p) {
  static_assert(sizeof(T) % 4 == 0, "whole words");
  const SM_CONST uint32_t* q = (const SM_CONST uint32_t*)reinterpret_cast<uintptr_t>(p);
  uint32_t w[sizeof(T) / 4];
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 4; ++i) w[i] = q[i];
  T v;
  __builtin_memcpy(&v, w, sizeof(T));
  return v;
}

// A vector V of elements P at an address aligned to P: one access, since
// global memory takes wide accesses at any alignment.  (64 M bf16 entries in
// buffers one element off, by single elements and so: step with float32
// states 440 and 239 us, with 8-bit ones 360 and 133, norm 129 and 26.)
template <bool NT, typename V, typename P>
__device__ __forceinline__ V load_v(const SM_GLOBAL P* p) {
  typedef V VP __attribute__((aligned(alignof(P))));
  if constexpr (NT) return __builtin_nontemporal_load((const SM_GLOBAL VP*)p);
  else return *(const SM_GLOBAL VP*)p;
}
template <bool NT, typename V, typename P>
__device__ __forceinline__ void store_v(SM_GLOBAL P* p, V v) {
  typedef V VP __attribute__((aligned(alignof(P))));
  if constexpr (NT) __builtin_nontemporal_store(v, (SM_GLOBAL VP*)p);
  else *(SM_GLOBAL VP*)p = v;
}
// A table's pointer, moved by a uniform number of entries.
template <typename T>
__device__ __forceinline__ SM_GLOBAL T* at(void* p, int64_t e) {
  return (SM_GLOBAL T*)reinterpret_cast<uintptr_t>(p) + e;
}
template <typename T>
__device__ __forceinline__ const SM_GLOBAL T* at(const void* p, int64_t e) {
  return (const SM_GLOBAL T*)reinterpret_cast<uintptr_t>(p) + e;
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf2f(v); }
__device__ __forceinline__ void from_f32(SM_GLOBAL float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(SM_GLOBAL bf16_t* p, float v) { *p = f2bf(v); }

// Two float32 values as a pair of bf16 ones, to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Four entries as they are stored: two words of bf16 ones, four of float32.
template <typename T>
struct Raw4 {
  typedef u32x4 type;
};
template <>
struct Raw4<bf16_t> {
  typedef u32x2 type;
};
__device__ __forceinline__ void expand4(u32x4 a, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(a[e]);
}
__device__ __forceinline__ void expand4(u32x2 a, float* v) {
  v[0] = __uint_as_float(a.x << 16);
  v[1] = __uint_as_float(a.x & 0xFFFF0000u);
  v[2] = __uint_as_float(a.y << 16);
  v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}

// Sixteen bytes of gradients.
__device__ __forceinline__ void expand_all(u32x4 a, float* v, float) { expand4(a, v); }
__device__ __forceinline__ void expand_all(u32x4 a, float* v, bf16_t) {
  expand4(u32x2{a.x, a.y}, v);
  expand4(u32x2{a.z, a.w}, v + 4);
}

// Four entries from p + l on, of which `left` from p on exist.  full: all of
// them do; otherwise missing ones read as 0 and are not written.  p is
// uniform and l the lane's offset, so that the addresses are a scalar base
// and a 32-bit offset.
template <typename T, bool NT>
__device__ __forceinline__ typename Raw4<T>::type get4(const SM_GLOBAL T* p, uint32_t l,
                                                       uint32_t left, bool full) {
  typedef typename Raw4<T>::type V;
  if (full) return load_v<NT, V>(p + l);
  V a = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (l + e >= left) continue;
    if constexpr (sizeof(T) == 2) a[e >> 1] |= (uint32_t)p[l + e] << (16 * (e & 1));
    else a[e] = __float_as_uint(p[l + e]);
  }
  return a;
}
template <typename T, bool NT>
__device__ __forceinline__ void put4(SM_GLOBAL T* p, uint32_t l, uint32_t left, bool full,
                                     const float* v) {
  if (full) {
    if constexpr (sizeof(T) == 2) {
      store_v<NT>(p + l, u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])});
    } else {
      store_v<NT>(p + l, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                               __float_as_uint(v[2]), __float_as_uint(v[3])});
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (l + e < left) from_f32(p + l + e, v[e]);
  }
}
// Four codes as a word, or four bf16 values as two.
template <bool NT>
__device__ __forceinline__ uint32_t get4_codes(const SM_GLOBAL uint8_t* p, uint32_t l,
                                               uint32_t left, bool full) {
  if (full) return load_v<NT, uint32_t>(p + l);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (l + e < left) w |= (uint32_t)p[l + e] << (8 * e);
  return w;
}
template <bool NT>
__device__ __forceinline__ void put4_codes(SM_GLOBAL uint8_t* p, uint32_t l, uint32_t left,
                                           bool full, uint32_t c) {
  if (full) {
    store_v<NT>(p + l, c);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (l + e < left) p[l + e] = (uint8_t)(c >> (8 * e));
}
template <bool NT>
__device__ __forceinline__ void put4_bf16(SM_GLOBAL bf16_t* p, uint32_t l, uint32_t left,
                                          bool full, uint32_t lo, uint32_t hi) {
  if (full) {
    store_v<NT>(p + l, u32x2{lo, hi});
    return;
  }
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (l + e < left) p[l + e] = (bf16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// ------------------------------------------------------------------ random bits
//
// r = mix32(entry ^ key) gives m 16 bits (its low half) and v 16 (its high
// half); mix32(r ^ 0x9E3779B1) gives the weight 16.  Written with y, the
// value before mix32's last step, r = y ^ (y >> 16): r's high half is y's,
// and since that step undoes itself the second mixing's first step leaves
// y ^ (C ^ (C >> 16)), C = 0x9E3779B1.

__device__ __forceinline__ void opaque(uint32_t& x) { asm("" : "+v"(x)); }

// y of entries e0 .. e0 + 3, e0 a multiple of 4: (e0 + i) ^ key is e0 ^ key
// with i in its two low bits, which the first shift does not reach.
__device__ __forceinline__ void random4(uint32_t e0, uint32_t key, uint32_t* y) {
  uint32_t x = e0 ^ key;
  x ^= x >> 16;
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) {
    y[e] = (x ^ e) * 0x9E3779B1u;
    y[e] = (y[e] ^ (y[e] >> 15)) * 0x85A308D3u;
    opaque(y[e]);   // else shifts of y become multiplications of their own
  }
}
// Seeds of the hardware's stochastic conversions, which add a seed's top
// bits below the result's last one and truncate: 16 random bits and a half
// below them for the codes (codes' own values stay), 16 for bf16.
__device__ __forceinline__ uint32_t seed_v(uint32_t y) {
  uint32_t x = (y & 0xFFFF0000u) | 0x8000u;
  opaque(x);   // one instruction, used for m as well
  return x;
}
__device__ __forceinline__ uint32_t seed_m(uint32_t y, uint32_t sv) { return sv ^ (y << 16); }
__device__ __forceinline__ uint32_t seed_w(uint32_t y) {
  uint32_t x = (y ^ (0x9E3779B1u ^ (0x9E3779B1u >> 16))) * 0x9E3779B1u;
  x = (x ^ (x >> 15)) * 0x85A308D3u;
  opaque(x);
  return x ^ (x << 16);   // its top half: the low one of x ^ (x >> 16)
}
__device__ __forceinline__ uint32_t bf16_pair_stochastic(float a, float b, uint32_t ya,
                                                         uint32_t yb) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r = {};
  r = __builtin_amdgcn_cvt_sr_bf16_f32(r, a, seed_w(ya), false);
  r = __builtin_amdgcn_cvt_sr_bf16_f32(r, b, seed_w(yb), true);
  return __builtin_bit_cast(uint32_t, r);
}

// ------------------------------------------------------------------ 8-bit codes
//
// The conversions are gfx950's scaled ones: they multiply (decode) or divide
// (encode) by the scale, a power of two, so nothing but the code's own
// rounding is lost.

constexpr uint32_t kInf = 0x7F800000u;

__device__ __forceinline__ void decode4_m(uint32_t c, float scale, float* v) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, true);
  v[0] = a[0];
  v[1] = a[1];
  v[2] = b[0];
  v[3] = b[1];
}
__device__ __forceinline__ void decode4_v(uint32_t c, float scale, float* v) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(c, scale, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(c, scale, true);
  v[0] = a[0];
  v[1] = a[1];
  v[2] = b[0];
  v[3] = b[1];
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The wave's largest value, uniform.  Within rows of 16 lanes by
// permutations, then rows 0 -> 1 and 2 -> 3, then both into row 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  // lanes that the control leaves out get 0, the identity
  return umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = dpp_max<0xB1, 0xF>(x);    // quad_perm [1, 0, 3, 2]
  x = dpp_max<0x4E, 0xF>(x);    // quad_perm [2, 3, 0, 1]
  x = dpp_max<0x141, 0xF>(x);   // row_half_mirror
  x = dpp_max<0x140, 0xF>(x);   // row_mirror
  x = dpp_max<0x142, 0xA>(x);   // row_bcast:15
  x = dpp_max<0x143, 0xC>(x);   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// Largest magnitude of a block's first moments, and largest second moment,
// as bits (magnitudes order like their bits).  kInf or more if some value is
// not finite (a negative second moment counts as such).
__device__ __forceinline__ uint32_t amax_m(const float* m) {
  int pos = 0;         // the largest positive value; any negative one is
  uint32_t any = 0;    // above it as unsigned, the largest magnitude on top
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t b = __float_as_uint(m[e]);
    pos = (int)b > pos ? (int)b : pos;
    any = umax(any, b);
  }
  return wave_max(umax((uint32_t)pos, any & 0x7FFFFFFFu));
}
__device__ __forceinline__ uint32_t amax_v(const float* v) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) a = umax(a, __float_as_uint(v[e]));
  return wave_max(a);
}

// The block's scale, 2^e with e >= -126 the smallest with amax <= 1.75 *
// 2^top * 2^e.
__device__ __forceinline__ float scale_for(uint32_t amax, int top) {
  const int e = (int)(amax >> 23) - top + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// Four first / second moments (finite) as codes, rounded stochastically: up
// with the probability that the dropped part is of a code's step, to 2^-17.
// y: the entries' random bits.
__device__ __forceinline__ uint32_t encode4_m(const float* m, float scale, const uint32_t* y,
                                              const uint32_t* sv) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(0u, m[0], seed_m(y[0], sv[0]), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, m[1], seed_m(y[1], sv[1]), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, m[2], seed_m(y[2], sv[2]), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, m[3], seed_m(y[3], sv[3]), scale, 3);
}
// A positive v takes at least the smallest code, 1: only its own code may be
// 0 (codes are below 0x7F, so that adding 0x7F sets a byte's top bit iff it
// is not 0).
__device__ __forceinline__ uint32_t floor_codes(const float* v, uint32_t c) {
  const uint32_t zeros = ~(c + 0x7F7F7F7Fu) & 0x80808080u;
  if (__builtin_expect(__any(zeros != 0u), 0)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v[e] > 0.f) c |= (zeros >> 7) & (1u << (8 * e));
  }
  return c;
}
__device__ __forceinline__ uint32_t encode4_v(const float* v, float scale, const uint32_t* sv) {
  uint32_t c = __builtin_amdgcn_cvt_scalef32_sr_bf8_f32(0u, v[0], sv[0], scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_sr_bf8_f32(c, v[1], sv[1], scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_sr_bf8_f32(c, v[2], sv[2], scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_sr_bf8_f32(c, v[3], sv[3], scale, 3);
  return floor_codes(v, c);
}
__device__ __forceinline__ float reciprocal(float scale) {   // of 2^e, e >= -126: exact
  return __uint_as_float(0x7F000000u - __float_as_uint(scale));
}
// The same to nearest even.
__device__ __forceinline__ uint32_t encode4_m_nearest(const float* m, float scale) {
  const float q = reciprocal(scale);
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(m[0] * q, m[1] * q, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m[2] * q, m[3] * q, c, true);
}
__device__ __forceinline__ uint32_t encode4_v_nearest(const float* v, float scale) {
  const float q = reciprocal(scale);
  int c = __builtin_amdgcn_cvt_pk_bf8_f32(v[0] * q, v[1] * q, 0, false);
  c = __builtin_amdgcn_cvt_pk_bf8_f32(v[2] * q, v[3] * q, c, true);
  return floor_codes(v, (uint32_t)c);
}

// A block with values that are not finite: those (and negative second
// moments) are taken out before the codes are made, and put in afterwards:
// NaN for m; NaN, infinity or 0 for v.
__device__ __forceinline__ void split_m(float* m, uint32_t* keep, uint32_t* put) {
  *keep = 0xFFFFFFFFu;
  *put = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((__float_as_uint(m[e]) & 0x7FFFFFFFu) < kInf) continue;
    m[e] = 0.f;
    *keep &= ~(0xFFu << (8 * e));
    *put |= 0x7Fu << (8 * e);
  }
}
__device__ __forceinline__ void split_v(float* v, uint32_t* keep, uint32_t* put) {
  *keep = 0xFFFFFFFFu;
  *put = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t b = __float_as_uint(v[e]);
    if (b < kInf) continue;
    v[e] = 0.f;
    *keep &= ~(0xFFu << (8 * e));
    *put |= (b == kInf ? 0x7Cu : (b & 0x7FFFFFFFu) > kInf ? 0x7Fu : 0u) << (8 * e);
  }
}

struct Codes {
  uint32_t m, v;
  float ms, vs;
};
template <bool STOCHASTIC>
__device__ __forceinline__ void encode_finite(const float* m, const float* v, uint32_t am,
                                              uint32_t av, const uint32_t* y, Codes& c) {
  c.ms = scale_for(am, 8);
  c.vs = scale_for(av, 15);
  if constexpr (STOCHASTIC) {
    uint32_t sv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sv[e] = seed_v(y[e]);
    c.m = encode4_m(m, c.ms, y, sv);
    c.v = encode4_v(v, c.vs, sv);
  } else {
    c.m = encode4_m_nearest(m, c.ms);
    c.v = encode4_v_nearest(v, c.vs);
  }
}
// Codes and scales of the wave's block; y: random bits (null: to nearest).
// All lanes of the wave must call it.
template <bool STOCHASTIC>
__device__ __forceinline__ Codes encode_block(float* m, float* v, const uint32_t* y) {
  const uint32_t am = amax_m(m), av = amax_v(v);
  Codes c;
  if (__builtin_expect(am >= kInf || av >= kInf, 0)) {   // uniform
    uint32_t km, kv, pm, pv;
    split_m(m, &km, &pm);
    split_v(v, &kv, &pv);
    encode_finite<STOCHASTIC>(m, v, amax_m(m), amax_v(v), y, c);
    c.m = (c.m & km) | pm;
    c.v = (c.v & kv) | pv;
  } else {
    encode_finite<STOCHASTIC>(m, v, am, av, y, c);
  }
  return c;
}

// ------------------------------------------------------------------ set tables

__global__ __launch_bounds__(kThreads) void k_set_fill(FillTbl t, int index0, ParamEnt* ents,
                                                       WorkItem* items, WorkItem* norm_out,
                                                       uint32_t* counter) {
  const int q = blockIdx.y;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    ents[index0 + q] = t.e[q];
    *counter = 0;
  }
  const int64_t n = step_items(t.e[q]);
  const int64_t nn = norm_items(t.e[q].count);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    WorkItem it;
    it.tensor = (uint32_t)(index0 + q);
    it.chunk = (uint32_t)i;
    items[t.first[q] + i] = it;
    if (i < nn) norm_out[t.norm_first[q] + i] = it;   // n >= nn
  }
}

// ------------------------------------------------------------------ AdamW

__device__ __forceinline__ bool is_finite(float v) {
  return (__float_as_uint(v) & kInf) != kInf;
}

__global__ void k_adamw_prep(sm_adamw_config c, int64_t* step, const float* gscale,
                             const float* lr_scale, AdamwScalars* out) {
  if (threadIdx.x != 0) return;
  const int64_t done = *step, t = done < 0 ? 1 : done + 1;
  AdamwScalars a = adamw_scalars(c, t);
  a.skip = done < 0 || (gscale && !is_finite(*gscale)) || (lr_scale && !is_finite(*lr_scale));
  *out = a;
  if (!a.skip) *step = t;
}

// Sum of the workers' gradients of four entries over P (ParamSetDev), in
// float64 and rounded once.  (Gradients of one entry less than 2^23 apart are
// summed exactly, whatever M.)
template <typename TG>
__device__ __forceinline__ u32x4 sum_grad4(const ParamEnt& p, int M, double inv_P, int64_t u0,
                                           uint32_t l, uint32_t left, bool full) {
  const SM_GLOBAL TG* gp = at<TG>(p.g, u0);
  double s[4] = {};
#pragma unroll 4
  for (int k = 0; k < M; ++k) {
    float x[4];
    expand4(get4<TG, true>(gp + k * p.gstride, l, left, full), x);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += (double)x[e];
  }
  u32x4 g;
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = __float_as_uint((float)(s[e] * inv_P));
  return g;
}

// An infinite value as the largest finite one: under a decay it would be taken
// from itself.  (Two instructions with their constants inside them: a med3
// would hold its own in registers, of which the step has none left.)
__device__ __forceinline__ float clamp_finite(float w) {
  float r;
  asm("v_min_f32 %0, 0x7f7fffff, %1" : "=v"(r) : "v"(w));
  asm("v_max_f32 %0, 0xff7fffff, %0" : "+v"(r));
  return r;
}

// The moments' averages and the weights' change, the same for both kinds of
// states.  sqrt and the reciprocal are the hardware's (each within an ulp):
// their error is relative to one step's change, not to the weight.  SCALED:
// powers of two keep their arguments and results normal (scaled_roots).  The
// decay and the change are one term, so that a weight is rounded once: a
// factor 1 - lr wd in float32 would be off by 3 % of a decay of 1e-6 and leave
// out one below 3e-8, the same way at every step.
template <bool SCALED>
__device__ __forceinline__ void adamw4(const AdamwScalars& a, float decay, float step,
                                       const float* g, float* m, float* v, float* w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    m[e] = a.b1 * m[e] + a.a1 * g[e];
    v[e] = a.b2 * v[e] + a.a2 * (g[e] * g[e]);
    float d;
    if constexpr (SCALED) {
      const bool low = v[e] < 0x1p-126f;
      const float root = __builtin_amdgcn_sqrtf(low ? v[e] * 0x1p64f : v[e]);
      const float den = __fmaf_rn(low ? root * 0x1p-32f : root, a.root, a.eps);
      d = m[e] * __builtin_amdgcn_rcpf(den * 0x1p-32f) * 0x1p-32f;
    } else {
      d = m[e] * __builtin_amdgcn_rcpf(__fmaf_rn(__builtin_amdgcn_sqrtf(v[e]), a.root, a.eps));
    }
    w[e] = w[e] - __fmaf_rn(step, d, decay * clamp_finite(w[e]));
  }
}

// What a thread holds of one unit (4 entries, the wave's 256 one block of an
// 8-bit state), as loaded: nothing waits for these loads until finish_unit.
// TS: the weights that are read; TG: the gradients, or float for the sum of
// several workers'.
template <typename TS, typename TG, bool FP8>
struct Held {
  typename Raw4<TG>::type g;
  typename Raw4<TS>::type w;
  u32x4 m, v;
  uint32_t mc, vc;
  float ms, vs;
};

// Entries of a unit from u0 on, at most a unit.
template <int UNIT>
__device__ __forceinline__ uint32_t unit_left(int64_t count, int64_t u0) {
  const int64_t n = count - u0;
  return (uint32_t)(n < UNIT ? n : UNIT);
}

// full: the thread has all four entries.  ONE: a single worker.
template <typename TS, typename TG, bool FP8, bool ONE, typename H>
__device__ __forceinline__ void load_unit(const ParamEnt& p, int M, double inv_P, int64_t u0,
                                          uint32_t left, bool full, H& h) {
  const uint32_t l = threadIdx.x * 4;
  if constexpr (FP8) {
    // the wave's block, uniform
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t blk = u0 / kStateBlock + wave;
    const bool inside = wave * kStateBlock < left;
    h.mc = get4_codes<true>(at<uint8_t>(p.m, u0), l, left, full);
    h.vc = get4_codes<true>(at<uint8_t>(p.v, u0), l, left, full);
    h.ms = inside ? *at<float>(p.ms, blk) : 1.0f;
    h.vs = inside ? *at<float>(p.vs, blk) : 1.0f;
  } else {
    h.m = get4<float, true>(at<float>(p.m, u0), l, left, full);
    h.v = get4<float, true>(at<float>(p.v, u0), l, left, full);
  }
  h.w = get4<TS, true>(at<TS>(sizeof(TS) == 4 && p.master ? p.master : p.w, u0), l, left, full);
  if constexpr (ONE) h.g = get4<TG, true>(at<TG>(p.g, u0), l, left, full);
  else h.g = sum_grad4<TG>(p, M, inv_P, u0, l, left, full);
}

// TW: the weights' type.  TS float32 with bf16 weights: they have a master.
template <typename TW, typename TS, bool FP8, bool SCALED, typename H>
__device__ __forceinline__ void finish_unit(const ParamEnt& p, const AdamwScalars& a, float f,
                                            float decay, float step, uint32_t key0, int64_t u0,
                                            uint32_t left, bool full, const H& h) {
  const uint32_t l = threadIdx.x * 4;
  float g[4], w[4], m[4], v[4];
  expand4(h.g, g);
  expand4(h.w, w);
  if constexpr (FP8) {
    decode4_m(h.mc, h.ms, m);
    decode4_v(h.vc, h.vs, v);
  } else {
    expand4(h.m, m);
    expand4(h.v, v);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = g[e] * f;
  adamw4<SCALED>(a, decay, step, g, m, v, w);
  constexpr bool SR_W = sizeof(TS) == 2, MASTER = sizeof(TW) == 2 && sizeof(TS) == 4;
  uint32_t y[4];
  if (FP8 || (SR_W && a.stochastic))
    random4((uint32_t)u0 + l, mix_key(key0, (uint32_t)((uint64_t)u0 >> 32)), y);
  SM_GLOBAL TW* wp = at<TW>(p.w, u0);
  if constexpr (SR_W) {
    if (a.stochastic)
      put4_bf16<true>(wp, l, left, full, bf16_pair_stochastic(w[0], w[1], y[0], y[1]),
                      bf16_pair_stochastic(w[2], w[3], y[2], y[3]));
    else
      put4<TW, true>(wp, l, left, full, w);
  } else {
    put4<TW, true>(wp, l, left, full, w);
  }
  if constexpr (MASTER) put4<float, true>(at<float>(p.master, u0), l, left, full, w);
  if constexpr (FP8) {
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t blk = u0 / kStateBlock + wave;
    const Codes c = encode_block<true>(m, v, y);
    put4_codes<true>(at<uint8_t>(p.m, u0), l, left, full, c.m);
    put4_codes<true>(at<uint8_t>(p.v, u0), l, left, full, c.v);
    if (wave * kStateBlock < left && (threadIdx.x & 63) == 0) {
      *at<float>(p.ms, blk) = c.ms;
      *at<float>(p.vs, blk) = c.vs;
    }
  } else {
    put4<float, true>(at<float>(p.m, u0), l, left, full, m);
    put4<float, true>(at<float>(p.v, u0), l, left, full, v);
  }
}

// The item of workgroup b: workgroups go to the 8 XCDs in turn, and of every
// 8 * RUN items each XCD takes RUN that follow one another (the last ones,
// fewer than that, stay in turn).  495 M entries with float32 states: 1.87
// ms in turn, 1.84 in runs of 64, 1.81 of 256, 1.81 of 512; a 64 M-entry
// embedding with 8-bit states and masters: 169, 164, 166 and 167 us.
template <int RUN>
__device__ __forceinline__ int xcd_run(int b, int items) {
  const int in = b % (8 * RUN), first = b - in;
  return first + 8 * RUN <= items ? first + (in % 8) * RUN + in / 8 : b;
}

// One work item: one unit, or kUnitsFp8 of them.  HBM bounds it: 1.83-1.85
// ms for 495 M bf16 entries with float32 states (22 bytes each, 5.9-6.0
// TB/s), 163 us for a 64 M-entry embedding with 8-bit states and masters (16
// bytes, 6.3 TB/s).  With 8-bit states and stochastic weights (10 bytes,
// 0.81-0.84 ms, 5.9-6.2 TB/s) the vector units are busy throughout as well, at
// 53 instructions an entry, half of them for the random bits.
template <bool FP8, bool SCALED>
__device__ __forceinline__ void adamw_item(const ParamSetDev& set, const AdamwScalars& arg,
                                           bool device, const float* gscale,
                                           const float* lr_scale) {
  constexpr int UNIT = step_unit(FP8);
  const WorkItem it = load_const(set.items + xcd_run<FP8 ? 64 : 256>(blockIdx.x, set.nitems));
  const ParamEnt p = load_const(set.ents + it.tensor);
  AdamwScalars a = arg;
  if (device) a = load_const(set.scalars);
  const float gs = gscale ? load_const(gscale) : 1.0f;
  const float ls = lr_scale ? load_const(lr_scale) : 1.0f;
  if (a.skip || !is_finite(gs) || !is_finite(ls)) return;
  const float mult = ls * p.lr_mult;
  const float decay = a.lr * mult * p.wd;
  const float step = a.step * mult;
  const float f = gs * set.P_over_M;
  const int64_t span = p.span, first = (int64_t)it.chunk * span;
  const uint32_t key0 = mix_key(a.key, it.tensor);
  auto item = [&](auto tw, auto ts, auto tg, auto fp8) {
    typedef decltype(tw) TW;
    typedef decltype(ts) TS;
    typedef decltype(tg) TG;
    constexpr bool F8 = decltype(fp8)::value;
    const bool whole = first + span <= p.count;
    if (whole && set.M == 1) {
      constexpr int units = sizeof(TS) == 2 && F8 ? kUnitsFp8 : 1;
      Held<TS, TG, F8> h[units];
#pragma unroll
      for (int u = 0; u < units; ++u)
        load_unit<TS, TG, F8, true>(p, 1, 1.0, first + u * UNIT, UNIT, true, h[u]);
#pragma unroll
      for (int u = 0; u < units; ++u)
        finish_unit<TW, TS, F8, SCALED>(p, a, f, decay, step, key0, first + u * UNIT, UNIT, true,
                                        h[u]);
    } else if (whole) {
      Held<TS, float, F8> h;
      load_unit<TS, TG, F8, false>(p, set.M, set.inv_P, first, UNIT, true, h);
      finish_unit<TW, TS, F8, SCALED>(p, a, f, decay, step, key0, first, UNIT, true, h);
    } else {
      for (int64_t u0 = first; u0 < first + span && u0 < p.count; u0 += UNIT) {
        const uint32_t left = unit_left<UNIT>(p.count, u0);
        const bool full = threadIdx.x * 4 + 4 <= left;
        Held<TS, float, F8> h;
        load_unit<TS, TG, F8, false>(p, set.M, set.inv_P, u0, left, full, h);
        finish_unit<TW, TS, F8, SCALED>(p, a, f, decay, step, key0, u0, left, full, h);
      }
    }
  };
  auto grads = [&](auto tw, auto ts, auto fp8) {
    if (p.flags & kPF_G16) item(tw, ts, bf16_t(), fp8);
    else item(tw, ts, float(), fp8);
  };
  auto weights = [&](auto fp8) {
    if (!(p.flags & kPF_W16)) grads(float(), float(), fp8);
    else if (p.master) grads(bf16_t(), float(), fp8);
    else grads(bf16_t(), bf16_t(), fp8);
  };
  if constexpr (FP8) {
    if (p.flags & kPF_FP8) {
      weights(std::true_type());
      return;
    }
  }
  weights(std::false_type());
}
// 72 registers: seven waves per SIMD.
template <bool FP8>
__global__ __launch_bounds__(step_threads(FP8)) __attribute__((amdgpu_num_vgpr(72))) void k_adamw(
    ParamSetDev set, AdamwScalars arg, bool device, const float* gscale, const float* lr_scale) {
  adamw_item<FP8, false>(set, arg, device, gscale, lr_scale);
}
// A kernel of its own: behind a uniform branch of the one above the scaling
// costs every step 73 registers, where seven waves per SIMD leave 72, and 30
// spilled scalars.
template <bool FP8>
__global__ __launch_bounds__(step_threads(FP8)) void k_adamw_scaled(
    ParamSetDev set, AdamwScalars arg, bool device, const float* gscale, const float* lr_scale) {
  adamw_item<FP8, true>(set, arg, device, gscale, lr_scale);
}

// ------------------------------------------------------------------ gradient norm

// Fixed-order block sum of doubles: wave butterfly, then the four waves.
__device__ double block_sum64(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename TG>
__device__ __forceinline__ float sumsq16(u32x4 a) {
  constexpr int E = 16 / sizeof(TG);
  float x[E], s = 0.f;
  expand_all(a, x, TG());
#pragma unroll
  for (int e = 0; e < E; ++e) s = __fmaf_rn(x[e], x[e], s);
  return s;
}

// The thread's share of a work item (`left` entries).  One worker: kNormFlight
// 16-byte loads in flight.
constexpr int kNormFlight = 8;
template <typename TG, bool NT>
__device__ __forceinline__ double sumsq_item(const SM_GLOBAL TG* g, int M, double inv_P,
                                             int64_t gstride, uint32_t left) {
  constexpr uint32_t E = 16 / sizeof(TG), STEP = kThreads * E;
  static_assert(kNormSpan % (STEP * kNormFlight) == 0, "whole rounds");
  const uint32_t l = threadIdx.x * E;
  double acc = 0.0;
  auto round = [&](uint32_t i, auto whole) {
    u32x4 a[kNormFlight];
#pragma unroll
    for (uint32_t q = 0; q < kNormFlight; ++q) {
      const bool in = decltype(whole)::value || i + q * STEP + E <= left;
      a[q] = u32x4{0u, 0u, 0u, 0u};
      if (in) a[q] = load_v<NT, u32x4>(g + (i + q * STEP));
    }
#pragma unroll
    for (uint32_t q = 0; q < kNormFlight; ++q) acc += (double)sumsq16<TG>(a[q]);
  };
  if (M == 1 && left == kNormSpan) {
    for (uint32_t i = 0; i < kNormSpan; i += STEP * kNormFlight) round(i + l, std::true_type());
  } else if (M == 1) {
    for (uint32_t i = l; i < left; i += STEP * kNormFlight) round(i, std::false_type());
  } else {
    for (uint32_t i = l; i + E <= left; i += STEP) {
      double s[E] = {};
#pragma unroll 8
      for (int k = 0; k < M; ++k) {
        float x[E];
        expand_all(load_v<NT, u32x4>(g + k * gstride + i), x, TG());
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) s[e] += (double)x[e];
      }
      float q = 0.f;
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        const float x = (float)(s[e] * inv_P);
        q = __fmaf_rn(x, x, q);
      }
      acc += (double)q;
    }
  }
  // the last entries, fewer than a load
  const uint32_t tail = left - left % E;
  if (threadIdx.x < left - tail) {
    double s = 0.0;
    for (int k = 0; k < M; ++k) s += (double)to_f32(g[k * gstride + tail + threadIdx.x]);
    const float x = (float)(s * inv_P);
    acc += (double)(x * x);
  }
  return acc;
}

// The sums of squares of a set, one per workgroup (495 M bf16 entries in
// 143-148 us, 6.7-6.9 TB/s).  A call's last launch also joins the sums of all
// its sets: its last workgroup to come adds them, in their order.  The
// counter wraps to 0 with that one, ready for the next call.  The sums are
// written and read by atomics at device scope, past the XCDs' own L2s: a
// release fence in each workgroup, which writes back its XCD's L2, took 90
// us over 2048 workgroups.  A second launch for the joining took a small set
// (290 vectors) from 8.7 to 11 us.
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_grad_norm(ParamSetDev set, NormJoin f) {
  __shared__ double red[4];
  __shared__ bool last;
  double acc = 0.0;
  for (int i = blockIdx.x; i < set.norm_items; i += gridDim.x) {
    const WorkItem it = load_const(set.norm_at + i);
    const ParamEnt p = load_const(set.ents + it.tensor);
    const int64_t first = (int64_t)it.chunk * kNormSpan;
    const uint32_t left = unit_left<kNormSpan>(p.count, first);
    acc += (p.flags & kPF_G16)
               ? sumsq_item<bf16_t, NT>(at<bf16_t>(p.g, first), set.M, set.inv_P, p.gstride, left)
               : sumsq_item<float, NT>(at<float>(p.g, first), set.M, set.inv_P, p.gstride, left);
  }
  const double P_over_M = 1.0 / (set.inv_P * (double)set.M);
  const double s = block_sum64(acc, red) * (P_over_M * P_over_M);
  if (threadIdx.x == 0) {
    // returns once the sum is where every XCD sees it
    const unsigned long long was =
        __hip_atomic_exchange(reinterpret_cast<unsigned long long*>(set.parts) + blockIdx.x,
                              __builtin_bit_cast(unsigned long long, s), __ATOMIC_RELAXED,
                              __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::"v"(was) : "memory");   // waits for it
    last = f.nsets > 0 && atomicInc(set.counter, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  acc = 0.0;
  for (int q = 0; q < f.nsets; ++q)
    for (int i = threadIdx.x; i < f.n[q]; i += kThreads)
      acc += __builtin_bit_cast(
          double, __hip_atomic_load(reinterpret_cast<unsigned long long*>(f.parts[q]) + i,
                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  const double total = block_sum64(acc, red);
  if (threadIdx.x == 0) {
    const float norm = (float)(sqrt(total) * fabs((double)f.scale));
    const double c = (double)f.max_norm / ((double)norm + 1e-6);
    f.out[0] = norm;
    f.out[1] = is_finite(norm) ? (float)((double)f.scale * (c < 1.0 ? c : 1.0))
                               : __uint_as_float(0x7FC00000u);
  }
}

// ------------------------------------------------------------------ 8-bit states

// A wave per block, 4 entries per lane (64 M entries: 102-106 us each way,
// 6.1-6.3 TB/s).
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_state8_pack(const float* m, const float* v,
                                                          int64_t count, uint8_t* m8, uint8_t* v8,
                                                          float* ms, float* vs) {
  const uint32_t l = threadIdx.x * 4;
  for (int64_t u0 = (int64_t)blockIdx.x * kUnit; u0 < count; u0 += (int64_t)gridDim.x * kUnit) {
    const uint32_t left = unit_left<kUnit>(count, u0);
    const bool full = l + 4 <= left;
    float x[4], y[4];
    expand4(get4<float, NT>(at<float>(m, u0), l, left, full), x);
    expand4(get4<float, NT>(at<float>(v, u0), l, left, full), y);
    const Codes c = encode_block<false>(x, y, nullptr);
    put4_codes<NT>(at<uint8_t>(m8, u0), l, left, full, c.m);
    put4_codes<NT>(at<uint8_t>(v8, u0), l, left, full, c.v);
    if (l < left && (threadIdx.x & 63) == 0) {
      ms[u0 / kStateBlock + (threadIdx.x >> 6)] = c.ms;
      vs[u0 / kStateBlock + (threadIdx.x >> 6)] = c.vs;
    }
  }
}

template <bool NT>
__global__ __launch_bounds__(kThreads) void k_state8_unpack(const uint8_t* m8, const uint8_t* v8,
                                                            const float* ms, const float* vs,
                                                            int64_t count, float* m, float* v) {
  const uint32_t l = threadIdx.x * 4;
  for (int64_t u0 = (int64_t)blockIdx.x * kUnit; u0 < count; u0 += (int64_t)gridDim.x * kUnit) {
    const uint32_t left = unit_left<kUnit>(count, u0);
    if (l >= left) continue;
    const bool full = l + 4 <= left;
    const int64_t blk = u0 / kStateBlock + (threadIdx.x >> 6);
    float x[4], y[4];
    decode4_m(get4_codes<NT>(at<uint8_t>(m8, u0), l, left, full), ms[blk], x);
    decode4_v(get4_codes<NT>(at<uint8_t>(v8, u0), l, left, full), vs[blk], y);
    put4<float, NT>(at<float>(m, u0), l, left, full, x);
    put4<float, NT>(at<float>(v, u0), l, left, full, y);
  }
}

// One workgroup per unit, up to a launch's limit of 2^32 threads.
int unit_blocks(int64_t count) {
  const int64_t n = (count + kUnit - 1) / kUnit;
  return (int)(n < (1 << 23) ? n : (1 << 23));
}

}  // namespace

// ------------------------------------------------------------------ launchers

sm_status launch_set_fill(const FillTbl& t, int n, int index0, ParamEnt* ents, WorkItem* items,
                          WorkItem* norm_items, uint32_t* counter, hipStream_t s) {
  int64_t most = 1;
  for (int q = 0; q < n; ++q)
    most = std::max<int64_t>(most, step_items(t.e[q]));
  const dim3 grid((unsigned)std::min<int64_t>((most + kThreads - 1) / kThreads, 1024), n);
  double bytes = 0.0;   // written
  for (int q = 0; q < n; ++q)
    bytes += sizeof(ParamEnt) + sizeof(WorkItem) * (double)(step_items(t.e[q]) +
                                                            sm::norm_items(t.e[q].count));
  prof_begin(SM_K_MISC, bytes, s);
  hipLaunchKernelGGL(k_set_fill, grid, dim3(kThreads), 0, s, t, index0, ents, items, norm_items,
                     counter);
  prof_end(s);
  return check_launch();
}

sm_status launch_adamw_prep(const sm_adamw_config& c, int64_t* step, const float* gscale,
                            const float* lr_scale, AdamwScalars* out, hipStream_t s) {
  // the step's index read and written, the factors, the scalars
  prof_begin(SM_K_MISC, 16.0 + (gscale ? 4 : 0) + (lr_scale ? 4 : 0) + sizeof(AdamwScalars), s);
  hipLaunchKernelGGL(k_adamw_prep, dim3(1), dim3(64), 0, s, c, step, gscale, lr_scale, out);
  prof_end(s);
  return check_launch();
}

sm_status launch_adamw(const ParamSetDev& set, const AdamwScalars& a, bool device,
                       const float* gscale, const float* lr_scale, bool fp8, bool scaled,
                       double bytes, hipStream_t s) {
  if (set.nitems == 0) return SM_OK;
  const auto kernel = scaled ? (fp8 ? k_adamw_scaled<true> : k_adamw_scaled<false>)
                             : (fp8 ? k_adamw<true> : k_adamw<false>);
  prof_begin(SM_K_ADAMW, bytes, s);
  hipLaunchKernelGGL(kernel, dim3(set.nitems), dim3(step_threads(fp8)), 0, s, set, a, device,
                     gscale, lr_scale);
  prof_end(s);
  return check_launch();
}

sm_status launch_grad_norm(const ParamSetDev& set, const NormJoin& f, double bytes,
                           hipStream_t s) {
  prof_begin(SM_K_GRAD_NORM, bytes, s);
  const auto kernel = bytes > kStreamBytes ? k_grad_norm<true> : k_grad_norm<false>;
  hipLaunchKernelGGL(kernel, dim3(norm_set_parts(set.norm_items, set.M)), dim3(kThreads), 0, s,
                     set, f);
  prof_end(s);
  return check_launch();
}

sm_status launch_state8_pack(const float* m, const float* v, int64_t count, uint8_t* m8,
                             uint8_t* v8, float* ms, float* vs, hipStream_t s) {
  const double bytes = 10.03125 * (double)count;
  prof_begin(SM_K_STATE8, bytes, s);
  const auto kernel = bytes > kStreamBytes ? k_state8_pack<true> : k_state8_pack<false>;
  hipLaunchKernelGGL(kernel, dim3(unit_blocks(count)), dim3(kThreads), 0, s, m, v, count, m8, v8,
                     ms, vs);
  prof_end(s);
  return check_launch();
}

sm_status launch_state8_unpack(const uint8_t* m8, const uint8_t* v8, const float* ms,
                               const float* vs, int64_t count, float* m, float* v,
                               hipStream_t s) {
  const double bytes = 10.03125 * (double)count;
  prof_begin(SM_K_STATE8, bytes, s);
  const auto kernel = bytes > kStreamBytes ? k_state8_unpack<true> : k_state8_unpack<false>;
  hipLaunchKernelGGL(kernel, dim3(unit_blocks(count)), dim3(kThreads), 0, s, m8, v8, ms, vs,
                     count, m, v);
  prof_end(s);
  return check_launch();
}

}  // namespace sm
