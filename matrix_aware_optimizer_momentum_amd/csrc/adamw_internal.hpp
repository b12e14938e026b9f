// Declarations shared by the AdamW kernels (k_adamw.hip) and their C ABI
// (sm_adamw.hip): the device tables of a parameter set and the launchers.
#pragma once

#include "sm_internal.hpp"

namespace sm {

// The block of entries that share an 8-bit state's scales: one wave's, 4 per
// lane.
constexpr int kStateBlock = SM_STATE8_BLOCK;
static_assert(kStateBlock == 64 * 4, "a wave holds one block");
// Threads of a workgroup of the step, with and without 8-bit states in the
// set, and the unit of entries that it takes at a time; a work item is one
// unit, or kUnitsFp8 (entry_of in sm_adamw.hip).
__host__ __device__ constexpr int step_threads(bool fp8) { return fp8 ? 256 : 128; }
__host__ __device__ constexpr int step_unit(bool fp8) { return 4 * step_threads(fp8); }
constexpr int kUnitsFp8 = 3;
// Entries of a work item of the norm.
constexpr int kNormSpan = 16384;

// One parameter in a set's device table.
enum : uint32_t {
  kPF_W16 = 1,     // bf16 weights
  kPF_G16 = 2,     // bf16 gradients
  kPF_FP8 = 4,     // 8-bit states
};
struct ParamEnt {
  void* w;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t count, gstride;
  float wd, lr_mult;
  uint32_t flags;
  int32_t span;   // entries of a work item
};

__host__ __device__ inline int64_t step_items(const ParamEnt& p) {
  return (p.count + p.span - 1) / p.span;
}
__host__ __device__ inline int64_t norm_items(int64_t count) {
  return (count + kNormSpan - 1) / kNormSpan;
}

// A share of a set: `span` entries (the parameter's, or kNormSpan) of
// parameter `tensor` from entry chunk * span on.
struct WorkItem {
  uint32_t tensor, chunk;
};

// The 32-bit mixing behind the random bits of stochastic rounding: two
// multiplications (2^32 / golden ratio, digits of pi) between shifts.
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x85A308D3u;
  return x ^ (x >> 16);
}
__host__ __device__ inline uint32_t mix_key(uint32_t key, uint32_t word) {
  return mix32((key ^ word) + 0x9E3779B9u);
}
__host__ __device__ inline uint32_t step_key(uint64_t seed, int64_t t) {
  uint32_t k = mix_key(0u, (uint32_t)seed);
  k = mix_key(k, (uint32_t)(seed >> 32));
  k = mix_key(k, (uint32_t)(uint64_t)t);
  return mix_key(k, (uint32_t)((uint64_t)t >> 32));
}

// Scalars of a step, computed in float64 and rounded once.
struct AdamwScalars {
  float lr, b1, a1, b2, a2;   // a = 1 - b
  float step;                 // lr / (1 - b1^t)
  float root;                 // 1 / sqrt(1 - b2^t)
  float eps;
  uint32_t key;               // of (seed, t)
  int32_t stochastic;
  int32_t skip;
};

__host__ __device__ inline AdamwScalars adamw_scalars(const sm_adamw_config& c, int64_t t) {
  AdamwScalars a;
  a.lr = c.lr;
  a.b1 = c.beta1;
  a.a1 = 1.0f - c.beta1;
  a.b2 = c.beta2;
  a.a2 = 1.0f - c.beta2;
  a.step = (float)((double)c.lr / (1.0 - pow((double)c.beta1, (double)t)));
  a.root = (float)(1.0 / sqrt(1.0 - pow((double)c.beta2, (double)t)));
  a.eps = c.eps;
  a.key = step_key(c.seed, t);
  a.stochastic = c.rounding;
  a.skip = 0;
  return a;
}

// The hardware's square root takes values below 2^-126 as 0, and its
// reciprocal is 0 above 2^126.  The first moves the denominator, at least eps,
// by up to 2^-63 / sqrt(1 - b2^t), most at t = 1: by 2^-22 of it or less
// unless eps is tiny (at b2 = 0.999 below 1.4e-11).  The second needs a huge
// eps.  For such an eps the step scales both.
inline bool scaled_roots(const sm_adamw_config& c) {
  return 0x1p-41f / sqrtf(1.0f - c.beta2) > c.eps || c.eps > 0x1p100f;
}

struct ParamSetDev {
  const ParamEnt* ents;
  const WorkItem* items;      // the step's
  const WorkItem* norm_at;    // the norm's
  AdamwScalars* scalars;      // of a step with a device-side index
  uint32_t* counter;          // of a norm's workgroups, 0 between calls
  double* parts;              // a norm's sums of squares, one per workgroup
  int nitems, norm_items, M;
  // The workers' sum is rounded to float32 after a division by P, the power
  // of two from M on: it is in the mean's range then.  The rest is P / M.
  double inv_P;
  float P_over_M;
};

// Tables of up to kFillMax parameters written per launch (they ride in the
// arguments); first[i], norm_first[i]: parameter i's first work items.
constexpr int kFillMax = 32;
struct FillTbl {
  ParamEnt e[kFillMax];
  int64_t first[kFillMax], norm_first[kFillMax];
};
static_assert(sizeof(FillTbl) <= 3584, "the table rides in the arguments");
sm_status launch_set_fill(const FillTbl& t, int n, int index0, ParamEnt* ents, WorkItem* items,
                          WorkItem* norm_items, uint32_t* counter, hipStream_t s);

// The scalars of a step whose index *step holds, and *step + 1 written back
// unless the step is skipped.
sm_status launch_adamw_prep(const sm_adamw_config& c, int64_t* step, const float* gscale,
                            const float* lr_scale, AdamwScalars* out, hipStream_t s);
// The step itself: scalars from the arguments, or from set.scalars if
// `device`.  fp8: some parameter has 8-bit states.  scaled: scaled_roots.
// bytes: what the step reads and writes.
sm_status launch_adamw(const ParamSetDev& set, const AdamwScalars& a, bool device,
                       const float* gscale, const float* lr_scale, bool fp8, bool scaled,
                       double bytes, hipStream_t s);

// Workgroups of a set's gradient norm, one sum of squares of the mean each.
// Few, since each adds to one counter: 495 M bf16 entries of one worker take
// 143 us with 512 workgroups, 148 with 1024, 158 with 2048.
// Several workers' rows are read with fewer bytes in flight per lane: 67.5 M
// float32 entries of four workers (1.08 GB) take 207 us with 1024, 317 with
// 512, 195 with 2048; 135 M bf16 entries of four 202, 322 and 205; 60 M bf16
// entries of eight (0.96 GB) 150, 145 and 159.
constexpr int kNormParts1 = 512, kNormPartsM = 1024;
inline int norm_set_parts(int items, int M) {
  const int most = M == 1 ? kNormParts1 : kNormPartsM;
  return items < 1 ? 1 : items < most ? items : most;
}
// What a call's last launch needs to join the sums of all its sets.
constexpr int kNormSets = 8;
struct NormJoin {
  double* parts[kNormSets];
  int n[kNormSets];
  int nsets;       // 0: not the last launch
  float scale, max_norm;
  float* out;      // {norm, factor}
};
sm_status launch_grad_norm(const ParamSetDev& set, const NormJoin& f, double bytes,
                           hipStream_t s);

sm_status launch_state8_pack(const float* m, const float* v, int64_t count, uint8_t* m8,
                             uint8_t* v8, float* ms, float* vs, hipStream_t s);
sm_status launch_state8_unpack(const uint8_t* m8, const uint8_t* v8, const float* ms,
                               const float* vs, int64_t count, float* m, float* v, hipStream_t s);

}  // namespace sm
