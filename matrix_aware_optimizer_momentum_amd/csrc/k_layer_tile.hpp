// The feed-forward layers' matrix products on the matrix cores.
//
// Work split.  A launch walks the flat list of output tiles (of both results,
// where a call makes two weight gradients at once) with one workgroup per CU,
// or two of the smaller ones; workgroups of one XCD take consecutive tiles, in
// bands of four tile rows, so that they share operand panels in that XCD's L2.
// A wave owns MI x 2 blocks of 32 x 32 sums; tiles of 256 x 256 have 2 x 4 waves
// with MI 4, tiles of 128 x 128 2 x 2 with MI 2, tiles of 64 x 64, for products
// with few tiles, 2 x 1 with MI 1.  In the larger ones two waves share a SIMD:
// while one waits, or issues a load (which holds it up for as long as two
// products), the other multiplies (four waves of 128 x 128 took 7 % longer).
//
// A gated layer's tile holds both projections of the same columns: of the 64
// rows of B that a wave multiplies 32 are Wg's and 32 the same ones of Wu, so
// that the wave has act's argument and the factor of an output in its own
// registers, and x is read once for both.
//
// Pipeline.  Operands go HBM -> LDS with direct-to-LDS buffer loads, in stages
// of 128 bytes a row (64 bf16 or 32 float32 of k): whole lines, since the L2
// serves a line or half of one in the same time (stages of 64 bytes a row
// asked it for twice as many).  There are two stage buffers (four of the least
// tiles).  A step multiplies
// a stage in four slices of its k, reading the next slice's fragments
// meanwhile; ahead of the last slice each wave waits for its reads of this
// stage and its loads of the next one, and the workgroup meets; during the
// last slice the next stage's first fragments are read and the loads of the
// stage that is as many ahead as there are buffers are issued into this one's.
// So loads have a step (three) less a slice to land.  The stages run on across
// tiles and across the two parts of a sum (da Wg + db Wu): a tile's first ones
// load during the last step and the epilogue of the one before.
//
// Bound.  8192 tokens, 4096 x 11008, bf16: 1.29 PFLOP/s by both projections (a
// long run; the others by a profile), 1.27 with the backward epilogue, 1.30 by
// da Wg + db Wu, 1.12 by the weight gradients; the matrix pipes 75, 69, 75 and
// 59 % busy at 1.3 to 1.7 GHz while counted.  The chip lowers its clock under
// this load, so that what counts is the data moved for a product, not only the
// instructions around it.
//
// Edges.  Rows past an operand's last read the last one (their sums are not
// stored).  Where k ends inside a stage, the lanes past it load from beyond
// the buffer descriptor's range, which puts zeros into LDS: no garbage meets
// the sums, and no NaN of memory behind a matrix.
//
// Epilogue.  The products are taken as B A^T, whose sums a lane holds as four
// consecutive columns of one row at a time.  Results are made from them in the
// registers; residual, dy or old gradients come to them, and they go to
// memory, through 4 KB of LDS of the wave's own.
// dz, da and db are rounded to the layer's type there, as operands of the
// products that follow: in bf16 the gradients' error is then the square root of
// two times what rounding them alone leaves (2.4e-3 of a result, 1.7e-3).  A
// second operand with what the rounding cut off would double the products of
// dx and dW (8192 tokens, 4096 x 11008: 2.45 ms more on 3.6).
#pragma once

#include "layer_math.hpp"

namespace sm {
namespace layer {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int ROW = 128;   // bytes of an operand row in a stage

struct TileArgs {
  Product p;
  int tiles_m, tiles_n, per_prob, total, xcd_chunk;
  // Of a product whose sums are split (splits > 1), each share of the stages
  // is a tile of its own and leaves its float32 sums, of every row and column
  // of the tiles (a gated layer's 32 of Wg and 32 of Wu in turn), to
  // sums[share][product]: `rows` rows of `width`.
  int splits, rows, width;
  float* sums;
};

// ---------------------------------------------------------------- four results

// Four consecutive entries, at any alignment (global memory takes wide
// accesses at the entries' own).
__device__ __forceinline__ f32x4 load4(const float* p) {
  typedef f32x4 V __attribute__((aligned(4)));
  return *reinterpret_cast<const V*>(p);
}
__device__ __forceinline__ f32x4 load4(const bf16_t* p) {
  typedef u32x2 V __attribute__((aligned(2)));
  const u32x2 a = *reinterpret_cast<const V*>(p);
  return f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u),
               __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xFFFF0000u)};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) {
  typedef f32x4 V __attribute__((aligned(4)));
  *reinterpret_cast<V*>(p) = v;
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) {
  typedef u32x2 V __attribute__((aligned(2)));
  const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
  *reinterpret_cast<V*>(p) =
      u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2)),
            __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2))};
}
// Four entries as they are stored (in half the registers, of bf16 ones).
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  f32x4 r;
  __device__ __forceinline__ f32x4 value() const { return r; }
};
template <> struct Raw4<bf16_t> {
  u32x2 r;
  __device__ __forceinline__ f32x4 value() const {
    return f32x4{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                 __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u)};
  }
};
template <typename T>
__device__ __forceinline__ Raw4<T> load_raw4(const T* p) {
  typedef decltype(Raw4<T>::r) V __attribute__((aligned(2)));
  return Raw4<T>{*reinterpret_cast<const V*>(p)};
}
// Of which `left` exist.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p, int left) {
  if (left >= 4) return load4(p);
  f32x4 v = {};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < left) v[e] = Elem<T>::load(p + e);
  return v;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v, int left) {
  if (left >= 4) {
    store4(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < left) Elem<T>::store(p + e, v[e]);
}

template <typename T, int KIND>
__device__ __forceinline__ f32x4 load_bias(const Product& p, int col) {
  if constexpr (KIND == kLinear || KIND == kSlope)
    if (p.bias && col < p.N) return load4(static_cast<const T*>(p.bias) + col, p.N - col);
  return f32x4{};
}
// The entries that the results are combined with, ahead of their use.
template <typename T, int KIND>
__device__ __forceinline__ f32x4 load_in(const Product& p, int prob, int row, int col) {
  if (row < p.M && col < p.N) {
    if constexpr (KIND == kDw) {
      if (p.accumulate)
        return load4(static_cast<const T*>(prob ? p.c[1] : p.c[0]) +
                         row * (prob ? p.ldc[1] : p.ldc[0]) + col,
                     p.N - col);
    } else if constexpr (KIND != kGated && KIND != kDx) {
      if (p.in.p) return load4(static_cast<const T*>(p.in.p) + row * p.in.ld + col, p.N - col);
    }
  }
  return f32x4{};
}
// Four columns of a row's results, from the sums g (and u of a gated layer).
struct Results4 {
  f32x4 v, v2;
};
template <typename T, int KIND, int ACT>
__device__ __forceinline__ Results4 results4(f32x4 g, f32x4 u, f32x4 bias, f32x4 in) {
  constexpr bool FINE = sizeof(T) == 4;
  f32x4 v, v2 = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (KIND == kLinear) {
      v[e] = act_value<FINE>(ACT, g[e] + bias[e]) + in[e];
    } else if constexpr (KIND == kSlope) {
      v[e] = in[e] * act_both<FINE>(ACT, g[e] + bias[e]).slope;
    } else if constexpr (KIND == kGated) {
      v[e] = act_value<FINE>(ACT, g[e]) * u[e];
    } else if constexpr (KIND == kGatedSlope) {
      const ActBoth h = act_both<FINE>(ACT, g[e]);
      v[e] = in[e] * u[e] * h.slope;
      v2[e] = in[e] * h.value;
    } else if constexpr (KIND == kDw) {
      v[e] = g[e] + in[e];
    } else {
      v[e] = g[e];
    }
  }
  return {v, v2};
}
// And stored, where they exist.
template <typename T, int KIND, int ACT>
__device__ __forceinline__ void finish4(const Product& p, int prob, int row, int col, f32x4 g,
                                        f32x4 u, f32x4 bias, f32x4 in) {
  if (row >= p.M) return;
  Results4 r = results4<T, KIND, ACT>(g, u, bias, in);
  int left = p.N - col;
  if constexpr (KIND == kSlope || KIND == kGatedSlope) {
    // dz has zeros up to a multiple of 8 columns
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= left) r.v[e] = 0.f;
      if (e >= left) r.v2[e] = 0.f;
    }
    left = p.pad - col;
  }
  store4(static_cast<T*>(prob ? p.c[1] : p.c[0]) + row * (prob ? p.ldc[1] : p.ldc[0]) + col, r.v,
         left);
  if constexpr (KIND == kGatedSlope)
    store4(static_cast<T*>(p.c[1]) + row * p.ldc[1] + col, r.v2, left);
}

// ---------------------------------------------------------------- small things

// The thread id, opaque to the optimizer: what is derived from it where it is
// used does not stay live across the k loop.
__device__ __forceinline__ int fresh_tid() {
  int t = (int)threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | lo;
}

// s_waitcnt vmcnt(N), other counters untouched.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Workgroup barrier without a memory fence: no wait for the loads in flight.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One direct-to-LDS load: each lane's 16 bytes at base + voff land at LDS
// byte address m0 + 16 lane, zeros where voff is kNowhere.  In inline
// assembly so that the compiler, which cannot tell which LDS bytes a pending
// load writes, adds no wait for all of them before every LDS read.  It has no
// register result.  Of its wait states the one after M0's write is here; the
// five after a VALU write of the descriptor's registers are kept by the
// distance (set's s_nop; 8192 x 11008 x 4096 backward 1311 us with five
// before every load, 1290 without), which a test of the generated code checks.
constexpr uint32_t kNowhere = 0x80000000u;   // the range that the descriptor allows
__device__ __forceinline__ void dma16(uint64_t base, uint32_t voff, uint32_t m0) {
  const i32x4 r = {(int)(uint32_t)base, (int)(uint32_t)(base >> 32), (int)kNowhere, 0x00020000};
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "s"(m0)
               : "memory", "m0");
}

// ---------------------------------------------------------------- stages in LDS
//
// KC: rows of 128 bytes; the 16-byte chunk c of row R sits at position c ^
// ((R >> 1) & 7), so that 16 rows read at one chunk hit 16 different 4-bank
// groups.  KR: k rows of 64 MI entries; of bf16, chunk c of k row r sits at
// position c ^ (4 (r & 3)), so that the four k rows of a transposing read lie
// in four different 64-byte bank ranges.
template <typename T, int MI>
struct Geo {
  static constexpr int SIZE = sizeof(T);
  static constexpr int EPC = 16 / SIZE;              // entries of a chunk
  static constexpr int BK = ROW / SIZE;              // k of a stage
  static constexpr int ROWS = 64 * MI;               // operand rows of a tile
  static constexpr int HALF = ROWS * ROW;            // bytes of an operand's stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int CPR = ROWS * SIZE / 16;       // chunks of a k row (KR)
  static constexpr int WN = MI;                      // waves: 2 rows of WN
  // Stage buffers: of small stages more, since a step of theirs is shorter
  // than memory is far.
  static constexpr int NBUF = MI == 1 ? 4 : 2;
  static constexpr int THREADS = 128 * WN;
  static __device__ __forceinline__ int swz(int krow) {
    return SIZE == 2 ? 4 * (krow & 3) & (CPR - 1) : 0;
  }
};

// A wave loads 32 rows' worth of each operand's stage, by four loads of 1 KB.
constexpr int LQ = 4;

// This lane's byte offsets, from the tile's first entry of a stage, of its
// loads, and the first k of each within the stage.
template <typename T, int MI, bool KR, bool DUAL>
struct LoadOffs {
  typedef Geo<T, MI> G;
  uint32_t off[LQ];
  // KC: the lane's chunk starts at k, of odd loads 4 chunks from there; KR:
  // load q reads k row k + q * STEP
  int k;
  static_assert(G::CPR <= 64, "a load covers whole k rows");
  static constexpr int STEP = KR ? 64 / G::CPR : 0;
  __device__ __forceinline__ int k_of(int q) const {
    if constexpr (KR) return k + q * STEP;
    else return q & 1 ? k ^ (4 * G::EPC) : k;
  }

  // row0: the tile's first row (column, KR) of the operand; rows: how many it has.
  __device__ __forceinline__ void set(int64_t ld, int row0, int rows) {
    const int tid = fresh_tid(), lane = tid & 63, wave = uniform(tid >> 6);
    if constexpr (!KR) {
      // load q covers rows 8 (4 wave + q) + lane / 8
      k = ((lane & 7) ^ (lane >> 4)) * G::EPC;
#pragma unroll
      for (int q = 0; q < LQ; ++q) {
        // of both projections, even waves load 32 rows of Wg and odd ones
        // the same rows of Wu
        int r = 32 * (DUAL ? wave >> 1 : wave) + 8 * q + (lane >> 3);
        r = min(r, rows - 1 - row0);
        off[q] = (uint32_t)r * (uint32_t)(ld * G::SIZE) + (uint32_t)(k_of(q) * G::SIZE);
      }
    } else {
      const int last = (rows + G::EPC - 1) / G::EPC * G::EPC - G::EPC - row0;
#pragma unroll
      for (int q = 0; q < LQ; ++q) {
        const int at = (LQ * wave + q) * 64 + lane;
        const int krow = at / G::CPR, chunk = (at % G::CPR) ^ G::swz(krow);
        if (q == 0) k = krow;
        off[q] = (uint32_t)krow * (uint32_t)(ld * G::SIZE) +
                 (uint32_t)(min(chunk * G::EPC, last) * G::SIZE);
      }
    }
  }
  // left: the k that exist from the stage's first on.
  __device__ __forceinline__ uint32_t at(int q, int left) const {
    return k_of(q) < left ? off[q] : kNowhere;
  }
};

// Fragments: 16 bytes of a row for a lane, whose k are one slice's (a quarter
// of a stage): 8 bf16, or 4 float32 of which the e-th goes into the e-th product
// (lanes 0-31 and 32-63 hold different k; A and B the same ones).
template <int MI>
struct Frags {
  u32x4 a[MI], b[2];
};

// Of NB blocks of an operand.
template <typename T, int MI, int NB, bool KR>
struct FragOffs {
  typedef Geo<T, MI> G;
  uint32_t o[KR ? (G::SIZE == 2 ? 2 * NB : 1) : 4];
  __device__ __forceinline__ explicit FragOffs(int rbase) {
    const int lane = fresh_tid() & 63;
    if constexpr (!KR) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int R = rbase + (lane & 31), c = 2 * s + (lane >> 5);
        o[s] = (uint32_t)(R * ROW + 16 * (c ^ ((R >> 1) & 7)));
      }
    } else if constexpr (G::SIZE == 2) {
      const int g = lane >> 4, j = lane & 15;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int krow = 8 * (g >> 1) + 4 * r + (j >> 2);
          const int col = rbase + 32 * i + 16 * (g & 1) + 4 * (j & 3);
          o[2 * i + r] = (uint32_t)(krow * G::ROWS * 2 + 16 * ((col >> 3) ^ G::swz(krow)) +
                                    2 * (col & 7));
        }
    } else {
      o[0] = (uint32_t)((4 * (lane >> 5) * G::ROWS + rbase + (lane & 31)) * 4);
    }
  }
  // Block i of slice s of the operand half at h.
  __device__ __forceinline__ u32x4 read(const char* h, int i, int s) const {
    if constexpr (!KR) {
      return *reinterpret_cast<const u32x4*>(h + o[s] + i * 32 * ROW);
    } else if constexpr (G::SIZE == 2) {
      typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
      const char* p0 = h + o[2 * i] + s * 16 * G::ROWS * 2;
      const char* p1 = h + o[2 * i + 1] + s * 16 * G::ROWS * 2;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4*)(__attribute__((address_space(3))) void*)(p0));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4*)(__attribute__((address_space(3))) void*)(p1));
      const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
      return u32x4{l2.x, l2.y, h2.x, h2.y};
    } else {
      const char* p = h + o[0] + (s * 8 * G::ROWS + 32 * i) * 4;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = *reinterpret_cast<const uint32_t*>(p + e * G::ROWS * 4);
      return v;
    }
  }
};

template <typename T>
__device__ __forceinline__ void mma(f32x16& acc, u32x4 a, u32x4 b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]),
                                                 acc, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- tiles

struct Tile {
  int share, prob, tm, tn;
};
template <int KIND>
__device__ __forceinline__ Tile decode_tile(const TileArgs& A, int t) {
  Tile r;
  const int q = t / A.per_prob;   // share by share, and in each problem by problem
  const int probs = KIND == kDw ? A.p.parts : 1;
  r.share = q / probs;
  r.prob = q - r.share * probs;
  // bands of four tile rows, column by column, each from the top
  const int u = t - q * A.per_prob, band = u / (4 * A.tiles_n), v = u - band * 4 * A.tiles_n;
  const int height = min(4, A.tiles_m - 4 * band);
  r.tn = v / height;
  r.tm = 4 * band + v - r.tn * height;
  return r;
}
// The stages of a share: from..to - 1 of `all`.
struct Stages {
  int from, to;
};
__device__ __forceinline__ Stages stages_of(const TileArgs& A, int share, int all) {
  return {(int)((int64_t)all * share / A.splits), (int)((int64_t)all * (share + 1) / A.splits)};
}

// Where the loads are: a stage of a tile (or of a part of its sums).
template <typename T, int KIND, int MI>
struct LoadPos {
  typedef Geo<T, MI> G;
  static constexpr bool AKR = kind_a_kr(KIND), BKR = kind_b_kr(KIND), DUAL = kind_dual(KIND);
  LoadOffs<T, MI, AKR, false> a;
  LoadOffs<T, MI, BKR, DUAL> b;
  uint64_t abase, bbase;    // of the stage
  uint64_t astep, bstep;    // bytes from a stage to the next
  int left;                 // k that exist from the stage's first on
  int todo;                 // stages of the tile from this one on
  int part, tile;

  static __device__ __forceinline__ int stages(const TileArgs& A) {   // of a part
    return (A.p.K + G::BK - 1) / G::BK;
  }
  // Stage `from` of part q.
  __device__ __forceinline__ void set(const TileArgs& A, const Tile& tl, int q, int from) {
    const Product& p = A.p;
    q = uniform(q);
    from = uniform(from);
    const Operand oa = (KIND == kDw ? tl.prob : KIND == kDx ? q : 0) ? p.a[1] : p.a[0];
    Operand ob = (KIND == kDx && q) ? p.b[1] : p.b[0];
    if constexpr (DUAL)   // odd waves load Wu's rows
      if (uniform(fresh_tid() >> 6) & 1) ob = p.b[1];
    constexpr int NB = DUAL ? G::ROWS / 2 : G::ROWS;
    const int am = tl.tm * G::ROWS, bn = tl.tn * NB;
    a.set(oa.ld, am, p.M);
    b.set(ob.ld, bn, p.N);
    abase = reinterpret_cast<uint64_t>(oa.p) + (uint64_t)((AKR ? am : am * oa.ld) * G::SIZE);
    bbase = reinterpret_cast<uint64_t>(ob.p) + (uint64_t)((BKR ? bn : bn * ob.ld) * G::SIZE);
    astep = uniform64((uint64_t)(AKR ? G::BK * oa.ld * G::SIZE : ROW));
    bstep = uniform64((uint64_t)(BKR ? G::BK * ob.ld * G::SIZE : ROW));
    abase = uniform64(abase + from * astep);
    bbase = uniform64(bbase + from * bstep);
    left = p.K - from * G::BK;
    part = q;
    // the bases come from readfirstlane: see dma16
    asm volatile("s_nop 4" : "+s"(abase), "+s"(bbase));
  }
  __device__ __forceinline__ void set_tile(const TileArgs& A, int t) {
    t = uniform(t);
    const Tile tl = decode_tile<KIND>(A, t);
    const int each = stages(A);
    const Stages s = stages_of(A, tl.share, each * (KIND == kDx ? A.p.parts : 1));
    const int q = KIND == kDx && s.from >= each ? 1 : 0;
    set(A, tl, q, s.from - q * each);
    todo = s.to - s.from;
    tile = t;
  }
  // The next stage: of this part, of the next part, of the workgroup's next
  // tile; past the last one it stays (that stage is then loaded again, into
  // buffers that nobody multiplies).
  __device__ __forceinline__ void advance(const TileArgs& A, int stride) {
    if (todo > 1) {
      --todo;
      if (KIND != kDx || left > G::BK) {
        left -= G::BK;
        abase += astep;
        bbase += bstep;
      } else {
        set(A, decode_tile<KIND>(A, tile), 1, 0);
      }
    } else if (tile + stride < A.total) {
      set_tile(A, tile + stride);
    }
  }
  // Load q of this wave (A's, then B's) into the stage buffer at LDS address buf.
  __device__ __forceinline__ void load(uint32_t buf, int q) const {
    if (q < LQ) dma16(abase, a.at(q, left), buf + 1024u * q);
    else dma16(bbase, b.at(q - LQ, left), buf + (uint32_t)G::HALF + 1024u * (q - LQ));
  }
};

// One step: see the pipeline above.  cur, nxt: this stage and the next one;
// ldb: LDS address of this wave's slots in cur.  f[0] holds the fragments of
// the stage's first slice, and on return those of the next one's.
// sched_barrier keeps the order of the products and the memory instructions
// between them.
template <typename T, int KIND, int MI>
__device__ __forceinline__ void step(f32x16 (&acc)[MI][2], Frags<MI> (&f)[2], const char* cur,
                                     const char* nxt, uint32_t ldb,
                                     const LoadPos<T, KIND, MI>& L,
                                     const FragOffs<T, MI, MI, kind_a_kr(KIND)>& fa,
                                     const FragOffs<T, MI, 2, kind_b_kr(KIND)>& fb) {
  typedef Geo<T, MI> G;
  constexpr int Q = 2 * MI;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const Frags<MI>& now = f[s & 1];
    Frags<MI>& then = f[(s + 1) & 1];
    const char* from = s < 3 ? cur : nxt;
    if (s == 3) {
      // this wave's reads of cur are done, and its loads of nxt; those of the
      // stages after it may be in flight
      constexpr int FLY = (G::NBUF - 2) * 2 * LQ;
      __builtin_amdgcn_s_waitcnt((FLY & 15) | (7 << 4) | ((FLY >> 4) << 14));   // lgkmcnt(0)
      meet();
    }
    // the wave that is past the meeting first goes on first
    if (s == 3) __builtin_amdgcn_s_setprio(1);
    if (s == 0) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      mma<T>(acc[q / 2][q % 2], now.b[q % 2], now.a[q / 2]);
      if (q < 2) then.b[q] = fb.read(from + G::HALF, q, (s + 1) & 3);
      else if (q - 2 < MI) then.a[q - 2] = fa.read(from, q - 2, (s + 1) & 3);
      if (MI == 1 && q == 1) then.a[0] = fa.read(from, 0, (s + 1) & 3);
      if (s == 3) {
#pragma unroll
        for (int l = 0; l < 2 * LQ / Q; ++l) L.load(ldb, 2 * LQ / Q * q + l);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The results of this wave's blocks, some of which lie past an edge: from the
// registers, entry by entry where a row ends.
template <typename T, int KIND, int ACT, int MI>
__device__ __forceinline__ void epilogue_edge(const f32x16 (&acc)[MI][2], const Product& p,
                                              int prob, int row0, int col0) {
  constexpr bool DUAL = kind_dual(KIND);
  const int lane = fresh_tid() & 63;
  const int row = row0 + (lane & 31), col = col0 + 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < (DUAL ? 1 : 2); ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = col + 32 * j + 8 * q;
      const f32x4 bias = load_bias<T, KIND>(p, c);
      f32x4 in[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i)
        in[i] = load_in<T, KIND>(p, prob, row + 32 * i, c);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        f32x4 g, u = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = acc[i][j][4 * q + e];
          if constexpr (DUAL) u[e] = acc[i][1][4 * q + e];
        }
        finish4<T, KIND, ACT>(p, prob, row + 32 * i, c, g, u, bias, in[i]);
      }
    }
}

// A patch of 32 rows of RB bytes in LDS, by which a wave turns between its
// sums' layout (a row to a lane) and whole lines: the 16-byte pieces of row r
// are permuted so that neither side's accesses meet in few banks.  One wave's
// LDS accesses take effect in order, so no barrier is needed between them, but
// the compiler has to keep that order (a lane's accesses are not its own alone).
__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }
template <int RB>
__device__ __forceinline__ uint32_t patch_at(int row, int byte) {
  const int s = RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
  return (uint32_t)(row * RB + (((byte >> 4) ^ s) << 4) + (byte & 15));
}

// The same where all of them exist: what they are combined with, and they
// themselves, go through a patch, so that memory sees 16 bytes a lane and
// whole lines.  (Straight from the registers, 16 bytes of each of 32 rows at
// a time, a 256 x 256 tile took 15 us longer to store.)
template <typename T, int KIND, int ACT, int MI>
__device__ __forceinline__ void epilogue_inside(const f32x16 (&acc)[MI][2], const Product& p,
                                                int prob, int row0, int col0, char* patch) {
  constexpr bool DUAL = kind_dual(KIND);
  constexpr int SIZE = sizeof(T);
  constexpr int JC = !DUAL && SIZE == 2 ? 2 : 1;      // column blocks of a patch
  constexpr int RB = 32 * JC * SIZE;                  // bytes of its rows
  constexpr int LPR = RB / 16, RPI = 64 / LPR;        // lanes of a row, rows of an access
  constexpr int NR = 32 / RPI;
  constexpr int JP = DUAL ? 1 : 2 / JC;               // patches side by side
  constexpr int NP = MI * JP;
  constexpr bool HAS_IN = KIND == kLinear || KIND == kSlope || KIND == kGatedSlope || KIND == kDw;
  typedef u32x4 V __attribute__((aligned(2)));
  const int lane = fresh_tid() & 63;
  const int prow = lane / LPR, pbyte = 16 * (lane % LPR);
  const int srow = lane & 31, sbyte = 4 * SIZE * (lane >> 5);
  char* c0 = static_cast<char*>(prob ? p.c[1] : p.c[0]);
  const int64_t ldc = (prob ? p.ldc[1] : p.ldc[0]) * SIZE;
  const char* in0 = nullptr;
  int64_t ldin = 0;
  if constexpr (KIND == kDw) {
    if (p.accumulate) in0 = c0, ldin = ldc;
  } else if constexpr (HAS_IN) {
    in0 = static_cast<const char*>(p.in.p);
    ldin = p.in.ld * SIZE;
  }
  // this lane's place in a patch's first rows, and a patch's k-th ones from there
  const int64_t at_in = prow * ldin + pbyte, at_c = prow * ldc + pbyte;
  auto patch_of = [&](int n, int k, int64_t ld) {
    return (row0 + 32 * (n % MI) + RPI * k) * ld + (col0 + 32 * (n / MI)) * SIZE;
  };
  u32x4 ahead[NR] = {};
  auto load_patch = [&](int n) {
    if (in0) {
#pragma unroll
      for (int k = 0; k < NR; ++k)
        ahead[k] = *reinterpret_cast<const V*>(in0 + patch_of(n, k, ldin) + at_in);
    }
  };
  if constexpr (HAS_IN) load_patch(0);
  constexpr int Q = 4 * JC;   // a lane's fours of columns in a patch
  constexpr bool HAS_BIAS = KIND == kLinear || KIND == kSlope;
  Raw4<T> bias[HAS_BIAS ? Q : 1] = {};
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    if constexpr (HAS_BIAS) {
      if (n % MI == 0 && p.bias) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          bias[q] = load_raw4(static_cast<const T*>(p.bias) + col0 + 32 * (n / MI) + 8 * q +
                              4 * (lane >> 5));
      }
    }
    Raw4<T> in[Q] = {}, out2[Q];
    if constexpr (HAS_IN) {
      if (in0) {
#pragma unroll
        for (int k = 0; k < NR; ++k)
          *reinterpret_cast<u32x4*>(patch + patch_at<RB>(prow + RPI * k, pbyte)) = ahead[k];
        in_order();
        if (n + 1 < NP) load_patch(n + 1);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          in[q] = load_raw4(
              reinterpret_cast<const T*>(patch + patch_at<RB>(srow, 8 * SIZE * q + sbyte)));
        in_order();
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = n % MI, j = DUAL ? 0 : n / MI + q / 4;
      f32x4 g, u = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = acc[i][j][4 * (q % 4) + e];
        if constexpr (DUAL) u[e] = acc[i][1][4 * (q % 4) + e];
      }
      const f32x4 b = HAS_BIAS ? bias[HAS_BIAS ? q : 0].value() : f32x4{};
      const Results4 r = results4<T, KIND, ACT>(g, u, b, in[q].value());
      store4(reinterpret_cast<T*>(patch + patch_at<RB>(srow, 8 * SIZE * q + sbyte)), r.v);
      if constexpr (KIND == kGatedSlope) store4(reinterpret_cast<T*>(&out2[q]), r.v2);
    }
    auto write_patch = [&](char* c) {
      in_order();
#pragma unroll
      for (int k = 0; k < NR; ++k)
        *reinterpret_cast<V*>(c + patch_of(n, k, ldc) + at_c) =
            *reinterpret_cast<const u32x4*>(patch + patch_at<RB>(prow + RPI * k, pbyte));
      in_order();
    };
    write_patch(c0);
    if constexpr (KIND == kGatedSlope) {   // da and db have one ld
#pragma unroll
      for (int q = 0; q < Q; ++q)
        *reinterpret_cast<Raw4<T>*>(patch + patch_at<RB>(srow, 8 * SIZE * q + sbyte)) = out2[q];
      write_patch(static_cast<char*>(p.c[1]));
    }
    __builtin_amdgcn_sched_barrier(0);   // one patch at a time keeps few values live
  }
}

template <typename T, int KIND, int ACT, int MI>
__device__ __forceinline__ void epilogue_of(const f32x16 (&acc)[MI][2], const Product& p,
                                            int prob, int row0, int col0, bool inside,
                                            char* patch) {
  if (inside) epilogue_inside<T, KIND, ACT, MI>(acc, p, prob, row0, col0, patch);
  else epilogue_edge<T, KIND, ACT, MI>(acc, p, prob, row0, col0);
}

template <typename T, int KIND, int MI>
__device__ __forceinline__ void epilogue(const f32x16 (&acc)[MI][2], const TileArgs& A, Tile t,
                                         char* patch) {
  typedef Geo<T, MI> G;
  const Product& p = A.p;
  if (A.splits > 1) {
    Product s;
    s.c[0] = A.sums + (int64_t)(t.share * (KIND == kDw ? p.parts : 1) + t.prob) * A.rows * A.width;
    s.ldc[0] = A.width;
    const int wave = uniform(fresh_tid() >> 6);
    epilogue_inside<float, kDx, SM_ACT_NONE, MI>(acc, s, 0,
                                                 t.tm * G::ROWS + (wave / G::WN) * (32 * MI),
                                                 (t.tn * G::WN + wave % G::WN) * 64, patch);
    return;
  }
  constexpr int OUT = kind_dual(KIND) ? 32 : 64;   // a wave's result columns
  const int wave = uniform(fresh_tid() >> 6);
  const int row0 = uniform(t.tm * G::ROWS + (wave / G::WN) * (32 * MI));
  const int col0 = uniform((t.tn * G::WN + wave % G::WN) * OUT);
  const bool inside = row0 + 32 * MI <= p.M && col0 + OUT <= p.N;
  if constexpr (kind_acts(KIND)) {
    switch (p.act) {
#define SM_ACT(A) \
  case A: epilogue_of<T, KIND, A, MI>(acc, p, t.prob, row0, col0, inside, patch); break;
      SM_ACT(SM_ACT_NONE)
      SM_ACT(SM_ACT_RELU)
      SM_ACT(SM_ACT_SILU)
      SM_ACT(SM_ACT_GELU)
      SM_ACT(SM_ACT_GELU_TANH)
#undef SM_ACT
    }
  } else {
    epilogue_of<T, KIND, SM_ACT_NONE, MI>(acc, p, t.prob, row0, col0, inside, patch);
  }
}

// Two waves to a SIMD; of the least tiles, whose workgroups of two waves fill
// the LDS of a CU in pairs, one.
template <typename T, int KIND, int MI>
__global__ __launch_bounds__(128 * MI) __attribute__((amdgpu_waves_per_eu(MI == 1 ? 1 : 2, 2)))
void k_tile(TileArgs A) {
  typedef Geo<T, MI> G;
  __shared__ __attribute__((aligned(16))) char smem[G::NBUF * G::STAGE + 4096 * (2 * G::WN)];
  int t = blockIdx.x;
  if (A.xcd_chunk > 0) t = (t & 7) * A.xcd_chunk + (t >> 3);
  const int stride = gridDim.x;
  if (t >= A.total) return;
  const int wave = uniform(fresh_tid() >> 6);
  const uint32_t la0 =
      (uint32_t)uniform((int)(uint32_t)(size_t)(__attribute__((address_space(3))) void*)smem) +
      1024u * LQ * wave;
  LoadPos<T, KIND, MI> L;
  L.set_tile(A, t);
#pragma unroll
  for (int s = 0; s < G::NBUF; ++s) {
#pragma unroll
    for (int q = 0; q < 2 * LQ; ++q) L.load(la0 + s * G::STAGE, q);
    L.advance(A, stride);
  }
  wait_vm<(G::NBUF - 1) * 2 * LQ>();
  meet();
  const FragOffs<T, MI, MI, kind_a_kr(KIND)> fa((wave / G::WN) * 32 * MI);
  const FragOffs<T, MI, 2, kind_b_kr(KIND)> fb((wave % G::WN) * 64);
  int cb = 0;   // the current stage's buffer
  const int all = L.stages(A) * (KIND == kDx ? A.p.parts : 1);
  for (; t < A.total; t += stride) {
    const Stages mine = stages_of(A, decode_tile<KIND>(A, uniform(t)).share, all);
    const int steps = uniform(mine.to - mine.from);
    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    // the first stage's first fragments, again after an epilogue (whose
    // registers they would take)
    Frags<MI> f[2];
#pragma unroll
    for (int i = 0; i < MI; ++i) f[0].a[i] = fa.read(smem + cb * G::STAGE, i, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) f[0].b[j] = fb.read(smem + cb * G::STAGE + G::HALF, j, 0);
    for (int k = 0; k < steps; ++k) {
      const int nb = cb + 1 == G::NBUF ? 0 : cb + 1;
      step<T, KIND, MI>(acc, f, smem + cb * G::STAGE, smem + nb * G::STAGE, la0 + cb * G::STAGE, L,
                        fa, fb);
      L.advance(A, stride);
      cb = nb;
    }
    epilogue<T, KIND, MI>(acc, A, decode_tile<KIND>(A, uniform(t)),
                          smem + G::NBUF * G::STAGE + 4096 * wave);
  }
  wait_vm<0>();   // loads past the last stage target this workgroup's LDS
}

// A split product's shares joined, and its results made of them: one thread
// takes four columns of a row, the shares in order.
template <typename T, int KIND, int ACT>
__device__ __forceinline__ void join4(const TileArgs& A, int prob, int row, int col) {
  const Product& p = A.p;
  const int probs = KIND == kDw ? p.parts : 1;
  const int64_t size = (int64_t)A.rows * A.width;
  const int at = kind_dual(KIND) ? col / 32 * 64 + col % 32 : col;
  const float* s = A.sums + prob * size + (int64_t)row * A.width + at;
  f32x4 g = {}, u = {};
  for (int q = 0; q < A.splits; ++q, s += probs * size) {
    g += *reinterpret_cast<const f32x4*>(s);
    if constexpr (kind_dual(KIND)) u += *reinterpret_cast<const f32x4*>(s + 32);
  }
  finish4<T, KIND, ACT>(p, prob, row, col, g, u, load_bias<T, KIND>(p, col),
                        load_in<T, KIND>(p, prob, row, col));
}
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_join(TileArgs A, int fours) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(i / fours), col = 4 * (int)(i % fours), prob = blockIdx.y;
  if (row >= A.p.M) return;
  if constexpr (kind_acts(KIND)) {
    switch (A.p.act) {
#define SM_ACT(V) \
  case V: join4<T, KIND, V>(A, prob, row, col); break;
      SM_ACT(SM_ACT_NONE)
      SM_ACT(SM_ACT_RELU)
      SM_ACT(SM_ACT_SILU)
      SM_ACT(SM_ACT_GELU)
      SM_ACT(SM_ACT_GELU_TANH)
#undef SM_ACT
    }
  } else {
    join4<T, KIND, SM_ACT_NONE>(A, prob, row, col);
  }
}

template <typename T, int MI>
void launch_tile(const TileArgs& a, int grid, hipStream_t s) {
  const int fours = (std::max(a.p.N, a.p.pad) + 3) / 4;
  const dim3 join((unsigned)(((int64_t)a.p.M * fours + 255) / 256),
                  a.p.kind == kDw ? a.p.parts : 1);
  constexpr int threads = Geo<T, MI>::THREADS;
  switch (a.p.kind) {
#define SM_KIND(K) \
  case K: \
    hipLaunchKernelGGL((k_tile<T, K, MI>), dim3(grid), dim3(threads), 0, s, a); \
    if constexpr (MI == 2) { \
      if (a.splits > 1) hipLaunchKernelGGL((k_join<T, K>), join, dim3(256), 0, s, a, fours); \
    } \
    break;
    SM_KIND(kLinear)
    SM_KIND(kSlope)
    SM_KIND(kGated)
    SM_KIND(kGatedSlope)
    SM_KIND(kDx)
    SM_KIND(kDw)
#undef SM_KIND
  }
}

// kLinear and kGated of few tokens (k_layer_few.hip).
void launch_few(const Product& p, hipStream_t s);

// One translation unit for each type and tile.
void launch_tile_bf16_4(const TileArgs& a, int grid, hipStream_t s);
void launch_tile_bf16_2(const TileArgs& a, int grid, hipStream_t s);
void launch_tile_bf16_1(const TileArgs& a, int grid, hipStream_t s);
void launch_tile_f32_4(const TileArgs& a, int grid, hipStream_t s);
void launch_tile_f32_2(const TileArgs& a, int grid, hipStream_t s);
void launch_tile_f32_1(const TileArgs& a, int grid, hipStream_t s);

}  // namespace layer
}  // namespace sm
