// AdamW over sets of parameters (float32 or 8-bit states), the global
// gradient norm, and the conversion of 8-bit states.  All of it is bound by
// HBM: every entry's weights, gradients and states are read once and written
// once, with 16-byte accesses where the addresses allow.
//
// One launch works on a whole set, whatever its lengths and types: each
// workgroup reads its work item (parameter, place) and the parameter's table
// entry, both uniform (scalar loads), and takes units of 2048 entries, 8 per
// thread.
#include "adamw_internal.hpp"

namespace sm {

namespace {

constexpr int kThreads = 256;
static_assert(kUnit == kThreads * 8, "8 entries per thread");

// Eight entries from e0 on (missing ones read as 0).
template <typename T>
__device__ __forceinline__ void get8(const T* p, int64_t e0, int64_t count, bool vec, float* v) {
  if (vec && e0 + 8 <= count) {
    load8<T>(p + e0, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e0 + e < count ? Elem<T>::load(p + e0 + e) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t e0, int64_t count, bool vec, const float* v) {
  if (vec && e0 + 8 <= count) {
    store8<T>(p + e0, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e0 + e < count) Elem<T>::store(p + e0 + e, v[e]);
  }
}
// Eight codes, as two words (missing ones read as 0).
__device__ __forceinline__ uint2 get8_codes(const uint8_t* p, int64_t e0, int64_t count,
                                            bool vec) {
  if (vec && e0 + 8 <= count) return *reinterpret_cast<const uint2*>(p + e0);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e0 + e < count) w[e >> 2] |= (uint32_t)p[e0 + e] << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put8_codes(uint8_t* p, int64_t e0, int64_t count, bool vec,
                                           uint2 c) {
  if (vec && e0 + 8 <= count) {
    *reinterpret_cast<uint2*>(p + e0) = c;
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e0 + e < count) p[e0 + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
}

// ------------------------------------------------------------------ 8-bit codes

// Values of eight codes times the block's scale (a power of two: exact).
__device__ __forceinline__ void decode8_m(uint2 c, float scale, float* v) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w[q], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(w[q], true);
    v[4 * q] = a[0] * scale;
    v[4 * q + 1] = a[1] * scale;
    v[4 * q + 2] = b[0] * scale;
    v[4 * q + 3] = b[1] * scale;
  }
}
__device__ __forceinline__ void decode8_v(uint2 c, float scale, float* v) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(w[q], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_bf8(w[q], true);
    v[4 * q] = a[0] * scale;
    v[4 * q + 1] = a[1] * scale;
    v[4 * q + 2] = b[0] * scale;
    v[4 * q + 3] = b[1] * scale;
  }
}

constexpr uint32_t kInf = 0x7F800000u;

// The largest finite magnitude of the thread's eight values, as bits
// (magnitudes order like their bits).
__device__ __forceinline__ uint32_t amax8(const float* v) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    a = b < kInf && b > a ? b : a;
  }
  return a;
}
// ... of the 32 threads that share a block.  All lanes must call it.
__device__ __forceinline__ uint32_t block_amax(uint32_t a) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t b = (uint32_t)__shfl_xor((int)a, o, 64);
    a = b > a ? b : a;
  }
  return a;
}
// Biased exponent (>= 1) of the block's scale: the smallest with amax <=
// 1.75 * 2^top * scale.
__device__ __forceinline__ uint32_t scale_exp(uint32_t amax, int top) {
  const int e = (int)(amax >> 23) - top + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}
__device__ __forceinline__ float exp_value(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float exp_recip(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Code of a magnitude x (scaled by its block) with KEEP mantissa bits and
// normals from 2^LOWEST on, rounded stochastically by 16 random bits r.
// Dropping the low mantissa bits after adding random ones rounds up with the
// probability that the dropped part is of a code's step (to 2^-17; codes'
// own values stay).  Below 2^LOWEST the codes are equally spaced: x +
// 2^LOWEST lies in a binade with just that spacing.
template <int KEEP, int LOWEST>
__device__ __forceinline__ uint32_t code_stochastic(float x, uint32_t r) {
  constexpr int DROP = 23 - KEEP;
  constexpr uint32_t BASE = (uint32_t)(127 + LOWEST) << KEEP;
  const float lim = __uint_as_float((uint32_t)(127 + LOWEST) << 23);
  const bool low = x < lim;
  const uint32_t bits = __float_as_uint(low ? x + lim : x);
  const uint32_t up = (r << (DROP - 16)) | (1u << (DROP - 17));
  return ((bits + up) >> DROP) - (low ? BASE : BASE - (1u << KEEP));
}

__device__ __forceinline__ uint32_t code_m(float m, float recip, uint32_t r) {
  const uint32_t b = __float_as_uint(m);
  if ((b & 0x7FFFFFFFu) >= kInf) return 0x7Fu;
  const float x = __uint_as_float(b & 0x7FFFFFFFu) * recip;
  return code_stochastic<3, -6>(x, r) | ((b >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t code_v(float v, float recip, uint32_t r) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) >= kInf) return b == kInf ? 0x7Cu : 0x7Fu;
  if (!(v > 0.f)) return 0u;
  const uint32_t c = code_stochastic<2, -14>(v * recip, r);
  return c == 0u ? 1u : c;
}

// bf16 of v rounded stochastically by 16 random bits.
__device__ __forceinline__ bf16_t f2bf_stochastic(float v, uint32_t r16) {
  const uint32_t b = __float_as_uint(v);
  if ((b & kInf) == kInf) return f2bf(v);
  return (bf16_t)((b + r16) >> 16);
}

// ------------------------------------------------------------------ set tables

__global__ __launch_bounds__(kThreads) void k_set_fill(FillTbl t, int index0, ParamEnt* ents,
                                                       WorkItem* items, int units) {
  const int q = blockIdx.y;
  const ParamEnt& e = t.e[q];
  if (blockIdx.x == 0 && threadIdx.x == 0) ents[index0 + q] = e;
  const int64_t span = (int64_t)units * kUnit;
  const int64_t n = (e.count + span - 1) / span;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    WorkItem it;
    it.tensor = (uint32_t)(index0 + q);
    it.chunk = (uint32_t)i;
    items[t.first[q] + i] = it;
  }
}

// ------------------------------------------------------------------ AdamW

__device__ __forceinline__ bool is_finite(float v) {
  return (__float_as_uint(v) & kInf) != kInf;
}

__global__ void k_adamw_prep(sm_adamw_config c, int64_t* step, const float* gscale,
                             const float* lr_scale, AdamwScalars* out) {
  if (threadIdx.x != 0) return;
  const int64_t t = *step + 1;
  AdamwScalars a = adamw_scalars(c, t);
  a.skip = (gscale && !is_finite(*gscale)) || (lr_scale && !is_finite(*lr_scale));
  *out = a;
  if (!a.skip) *step = t;
}

// The mean gradient of eight entries, times the step's factor f =
// gscale / M.  Several workers' gradients are summed in float64: the sum
// does not depend on their order, and is rounded once.
template <typename TG>
__device__ __forceinline__ void mean_grad8(const ParamEnt& p, int M, int64_t e0, bool vec,
                                           float f, float* g) {
  const TG* gp = static_cast<const TG*>(p.g);
  if (M == 1) {
    get8<TG>(gp, e0, p.count, vec, g);
  } else {
    double s[8] = {};
    for (int k = 0; k < M; ++k) {
      float x[8];
      get8<TG>(gp + k * p.gstride, e0, p.count, vec, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += (double)x[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = (float)s[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] = g[e] * f;
}

// The moments' averages and the weights' change, the same for both kinds of
// states.  sqrt and the reciprocal are the hardware's (each within an ulp):
// their error is relative to one step's change, not to the weight.
__device__ __forceinline__ void adamw8(const AdamwScalars& a, float keep, float step,
                                       const float* g, float* m, float* v, float* w) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = a.b1 * m[e] + a.a1 * g[e];
    v[e] = a.b2 * v[e] + a.a2 * (g[e] * g[e]);
    const float den = __builtin_amdgcn_sqrtf(v[e]) * a.root + a.eps;
    w[e] = w[e] * keep - step * (m[e] * __builtin_amdgcn_rcpf(den));
  }
}

template <typename TW, typename TG, bool FP8>
__device__ __forceinline__ void adamw_unit(const ParamEnt& p, const AdamwScalars& a, int M,
                                           float f, float keep, float step, uint32_t key0,
                                           int64_t e0, bool vec) {
  float g[8], m[8], v[8], w[8];
  mean_grad8<TG>(p, M, e0, vec, f, g);
  const int64_t blk = e0 / kStateBlock;
  const bool inside = e0 < p.count;
  if constexpr (FP8) {
    const uint2 mc = get8_codes(static_cast<const uint8_t*>(p.m), e0, p.count, vec);
    const uint2 vc = get8_codes(static_cast<const uint8_t*>(p.v), e0, p.count, vec);
    decode8_m(mc, inside ? p.ms[blk] : 0.f, m);
    decode8_v(vc, inside ? p.vs[blk] : 0.f, v);
  } else {
    get8<float>(static_cast<const float*>(p.m), e0, p.count, vec, m);
    get8<float>(static_cast<const float*>(p.v), e0, p.count, vec, v);
  }
  const bool master = sizeof(TW) == 2 && p.master;
  if (master) get8<float>(p.master, e0, p.count, vec, w);
  else get8<TW>(static_cast<const TW*>(p.w), e0, p.count, vec, w);

  adamw8(a, keep, step, g, m, v, w);

  uint32_t r[8];
  if (FP8 || (sizeof(TW) == 2 && a.stochastic)) {
    const uint32_t key = mix_key(key0, (uint32_t)((uint64_t)e0 >> 32));
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = mix32(((uint32_t)e0 + e) ^ key);
  }
  if constexpr (FP8) {
    const uint32_t em = scale_exp(block_amax(amax8(m)), 8);
    const uint32_t ev = scale_exp(block_amax(amax8(v)), 15);
    const float rm = exp_recip(em), rv = exp_recip(ev);
    uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cm[e >> 2] |= code_m(m[e], rm, r[e] & 0xFFFFu) << (8 * (e & 3));
      cv[e >> 2] |= code_v(v[e], rv, r[e] >> 16) << (8 * (e & 3));
    }
    put8_codes(static_cast<uint8_t*>(p.m), e0, p.count, vec, make_uint2(cm[0], cm[1]));
    put8_codes(static_cast<uint8_t*>(p.v), e0, p.count, vec, make_uint2(cv[0], cv[1]));
    if (inside && (threadIdx.x & 31) == 0) {
      p.ms[blk] = exp_value(em);
      p.vs[blk] = exp_value(ev);
    }
  } else {
    put8<float>(static_cast<float*>(p.m), e0, p.count, vec, m);
    put8<float>(static_cast<float*>(p.v), e0, p.count, vec, v);
  }
  if (master) {
    put8<float>(p.master, e0, p.count, vec, w);
  } else if (sizeof(TW) == 2 && a.stochastic) {
    // the rounded values are bf16 values, which the store below keeps
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = bf2f(f2bf_stochastic(w[e], mix32(r[e] ^ 0x9E3779B1u) & 0xFFFFu));
  }
  put8<TW>(static_cast<TW*>(p.w), e0, p.count, vec, w);
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void k_adamw(ParamSetDev set, AdamwScalars arg, bool device,
                                                    const float* gscale, const float* lr_scale) {
  const WorkItem it = set.items[blockIdx.x];
  const ParamEnt p = set.ents[it.tensor];
  const AdamwScalars a = device ? *set.scalars : arg;
  const float gs = gscale ? *gscale : 1.0f;
  const float ls = lr_scale ? *lr_scale : 1.0f;
  if (a.skip || !is_finite(gs) || !is_finite(ls)) return;
  const float mult = ls * p.lr_mult;
  const float keep = (float)(1.0 - (double)(a.lr * mult) * (double)p.wd);
  const float step = a.step * mult;
  const float f = gs * (1.0f / (float)set.M);
  const uint32_t key0 = mix_key(a.key, it.tensor);
  const bool vec = p.flags & kPF_VEC;
  const int64_t first = (int64_t)it.chunk * set.units * kUnit;
  for (int u = 0; u < set.units; ++u) {
    const int64_t u0 = first + (int64_t)u * kUnit;
    if (u0 >= p.count) break;
    const int64_t e0 = u0 + threadIdx.x * 8;
    auto run = [&](auto tw, auto tg) {
      typedef decltype(tw) TW;
      typedef decltype(tg) TG;
      if (FP8 && (p.flags & kPF_FP8))
        adamw_unit<TW, TG, FP8>(p, a, set.M, f, keep, step, key0, e0, vec);
      else
        adamw_unit<TW, TG, false>(p, a, set.M, f, keep, step, key0, e0, vec);
    };
    if (p.flags & kPF_W16) {
      if (p.flags & kPF_G16) run(bf16_t(), bf16_t());
      else run(bf16_t(), float());
    } else {
      if (p.flags & kPF_G16) run(float(), bf16_t());
      else run(float(), float());
    }
  }
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

__global__ __launch_bounds__(kThreads) void k_grad_sumsq(ParamSetDev set, double* parts) {
  __shared__ double red[4];
  double acc = 0.0;
  for (int i = blockIdx.x; i < set.nitems; i += gridDim.x) {
    const WorkItem it = set.items[i];
    const ParamEnt p = set.ents[it.tensor];
    const bool vec = p.flags & kPF_VEC;
    const int64_t first = (int64_t)it.chunk * set.units * kUnit;
    for (int u = 0; u < set.units; ++u) {
      const int64_t e0 = first + (int64_t)u * kUnit + threadIdx.x * 8;
      if (e0 >= p.count) break;
      float g[8];
      if (p.flags & kPF_G16) mean_grad8<bf16_t>(p, set.M, e0, vec, 1.0f, g);
      else mean_grad8<float>(p, set.M, e0, vec, 1.0f, g);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __fmaf_rn(g[e], g[e], s);
      acc += (double)s;
    }
  }
  const double s = block_sum64(acc, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = s / ((double)set.M * (double)set.M);
}

__global__ __launch_bounds__(kThreads) void k_norm_finalize(const double* parts, int n,
                                                            float scale, float max_norm,
                                                            float* out) {
  __shared__ double red[4];
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += parts[i];
  const double s = block_sum64(acc, red);
  if (threadIdx.x == 0) {
    const float norm = (float)(sqrt(s) * fabs((double)scale));
    const double c = (double)max_norm / ((double)norm + 1e-6);
    out[0] = norm;
    out[1] = is_finite(norm) ? (float)((double)scale * (c < 1.0 ? c : 1.0))
                             : __uint_as_float(0x7FC00000u);
  }
}

// ------------------------------------------------------------------ 8-bit states

__global__ __launch_bounds__(kThreads) void k_state8_pack(const float* m, const float* v,
                                                          int64_t count, uint8_t* m8, uint8_t* v8,
                                                          float* ms, float* vs, bool vec) {
  for (int64_t u0 = (int64_t)blockIdx.x * kUnit; u0 < count; u0 += (int64_t)gridDim.x * kUnit) {
    const int64_t e0 = u0 + threadIdx.x * 8;
    float x[8], y[8];
    get8<float>(m, e0, count, vec, x);
    get8<float>(v, e0, count, vec, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = y[e] < 0.f ? 0.f : y[e];
    const uint32_t em = scale_exp(block_amax(amax8(x)), 8);
    const uint32_t ev = scale_exp(block_amax(amax8(y)), 15);
    const float rm = exp_recip(em), rv = exp_recip(ev);
    uint32_t cm[2], cv[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float* xs = x + 4 * q;
      float* ys = y + 4 * q;
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(xs[0] * rm, xs[1] * rm, 0, false);
      cm[q] = __builtin_amdgcn_cvt_pk_fp8_f32(xs[2] * rm, xs[3] * rm, c, true);
      c = __builtin_amdgcn_cvt_pk_bf8_f32(ys[0] * rv, ys[1] * rv, 0, false);
      cv[q] = __builtin_amdgcn_cvt_pk_bf8_f32(ys[2] * rv, ys[3] * rv, c, true);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t sh = 8 * e, bx = __float_as_uint(xs[e]) & 0x7FFFFFFFu;
        const uint32_t by = __float_as_uint(ys[e]) & 0x7FFFFFFFu;
        if (bx >= kInf) cm[q] = (cm[q] & ~(0xFFu << sh)) | (0x7Fu << sh);
        if (by >= kInf) cv[q] = (cv[q] & ~(0xFFu << sh)) | ((by == kInf ? 0x7Cu : 0x7Fu) << sh);
        else if (by != 0u && ((cv[q] >> sh) & 0xFFu) == 0u) cv[q] |= 1u << sh;
      }
    }
    put8_codes(m8, e0, count, vec, make_uint2(cm[0], cm[1]));
    put8_codes(v8, e0, count, vec, make_uint2(cv[0], cv[1]));
    if (e0 < count && (threadIdx.x & 31) == 0) {
      ms[e0 / kStateBlock] = exp_value(em);
      vs[e0 / kStateBlock] = exp_value(ev);
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_state8_unpack(const uint8_t* m8, const uint8_t* v8,
                                                            const float* ms, const float* vs,
                                                            int64_t count, float* m, float* v,
                                                            bool vec) {
  for (int64_t u0 = (int64_t)blockIdx.x * kUnit; u0 < count; u0 += (int64_t)gridDim.x * kUnit) {
    const int64_t e0 = u0 + threadIdx.x * 8;
    if (e0 >= count) continue;
    float x[8], y[8];
    decode8_m(get8_codes(m8, e0, count, vec), ms[e0 / kStateBlock], x);
    decode8_v(get8_codes(v8, e0, count, vec), vs[e0 / kStateBlock], y);
    put8<float>(m, e0, count, vec, x);
    put8<float>(v, e0, count, vec, y);
  }
}

int unit_blocks(int64_t count) {
  const int64_t n = (count + kUnit - 1) / kUnit;
  return (int)(n < 65536 ? n : 65536);
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool state8_vec(const void* m, const void* v, const void* m8, const void* v8) {
  return aligned(m, 16) && aligned(v, 16) && aligned(m8, 8) && aligned(v8, 8);
}

}  // namespace

// ------------------------------------------------------------------ launchers

sm_status launch_set_fill(const FillTbl& t, int n, int index0, ParamEnt* ents, WorkItem* items,
                          int units, hipStream_t s) {
  int64_t most = 1;
  for (int q = 0; q < n; ++q) {
    const int64_t span = (int64_t)units * kUnit;
    most = std::max<int64_t>(most, (t.e[q].count + span - 1) / span);
  }
  const dim3 grid((unsigned)std::min<int64_t>((most + kThreads - 1) / kThreads, 1024), n);
  hipLaunchKernelGGL(k_set_fill, grid, dim3(kThreads), 0, s, t, index0, ents, items, units);
  return check_launch();
}

sm_status launch_adamw_prep(const sm_adamw_config& c, int64_t* step, const float* gscale,
                            const float* lr_scale, AdamwScalars* out, hipStream_t s) {
  hipLaunchKernelGGL(k_adamw_prep, dim3(1), dim3(64), 0, s, c, step, gscale, lr_scale, out);
  return check_launch();
}

sm_status launch_adamw(const ParamSetDev& set, const AdamwScalars& a, bool device,
                       const float* gscale, const float* lr_scale, bool fp8, bool stream,
                       double bytes, hipStream_t s) {
  if (set.nitems == 0) return SM_OK;
  (void)stream;
  prof_begin(SM_K_ADAMW, bytes, s);
  if (fp8)
    hipLaunchKernelGGL((k_adamw<true>), dim3(set.nitems), dim3(kThreads), 0, s, set, a, device,
                       gscale, lr_scale);
  else
    hipLaunchKernelGGL((k_adamw<false>), dim3(set.nitems), dim3(kThreads), 0, s, set, a, device,
                       gscale, lr_scale);
  prof_end(s);
  return check_launch();
}

sm_status launch_grad_sumsq(const ParamSetDev& set, double* parts, double bytes, hipStream_t s) {
  if (set.nitems == 0) return SM_OK;
  prof_begin(SM_K_GRAD_NORM, bytes, s);
  hipLaunchKernelGGL(k_grad_sumsq, dim3(norm_set_parts(set.nitems)), dim3(kThreads), 0, s, set,
                     parts);
  prof_end(s);
  return check_launch();
}

sm_status launch_norm_finalize(const double* parts, int n, float scale, float max_norm,
                               float* out, hipStream_t s) {
  prof_begin(SM_K_GRAD_NORM, 8.0 * n, s);
  hipLaunchKernelGGL(k_norm_finalize, dim3(1), dim3(kThreads), 0, s, parts, n, scale, max_norm,
                     out);
  prof_end(s);
  return check_launch();
}

sm_status launch_state8_pack(const float* m, const float* v, int64_t count, uint8_t* m8,
                             uint8_t* v8, float* ms, float* vs, hipStream_t s) {
  prof_begin(SM_K_STATE8, 10.03125 * (double)count, s);
  hipLaunchKernelGGL(k_state8_pack, dim3(unit_blocks(count)), dim3(kThreads), 0, s, m, v, count,
                     m8, v8, ms, vs, state8_vec(m, v, m8, v8));
  prof_end(s);
  return check_launch();
}

sm_status launch_state8_unpack(const uint8_t* m8, const uint8_t* v8, const float* ms,
                               const float* vs, int64_t count, float* m, float* v,
                               hipStream_t s) {
  prof_begin(SM_K_STATE8, 10.03125 * (double)count, s);
  hipLaunchKernelGGL(k_state8_unpack, dim3(unit_blocks(count)), dim3(kThreads), 0, s, m8, v8, ms,
                     vs, count, m, v, state8_vec(m, v, m8, v8));
  prof_end(s);
  return check_launch();
}

}  // namespace sm
