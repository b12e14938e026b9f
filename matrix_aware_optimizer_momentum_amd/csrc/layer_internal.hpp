// Declarations shared by the feed-forward layers' kernels (k_layer*.hip,
// k_act8.hip) and their C ABI (sm_layer.hip).
#pragma once

#include "layer_plan.hpp"
#include "sm_internal.hpp"

namespace sm {

struct Operand {
  const void* p;
  int64_t ld;   // entries
};
struct Product {
  int kind, dt, act;
  int M, N, K;        // c is M x N, sums over K
  int parts;          // kDx: 2 with a[1], b[1]; kDw: 2 with a[1], c[1]
  Operand a[2], b[2]; // kGated*: b[1] is Wu
  Operand in;         // residual or null; dy
  const void* bias;   // or null
  void* c[2];
  int64_t ldc[2];
  int pad;            // kSlope, kGatedSlope: columns N .. pad - 1 of c get zeros
  int accumulate;     // kDw
  int few;            // by the kernel for few tokens
};

// takes_few of layer_plan.hpp on this GPU.
bool few_tokens(int kind, int dt, int64_t T, int n, int d, bool w_in_place, bool x_in_place);
// Launches p.  Unless p.few, every operand's rows (as they are stored) are
// 16-byte aligned, less than 2^31 / 256 bytes apart, and a multiple of 16 bytes
// long, or have readable memory up to one, zeros if they run along k.
// sums: scratch of product_ws bytes (none if p.few), 256-byte aligned.
size_t product_ws(int kind, int dt, int M, int N, int K, int parts);
sm_status launch_product(const Product& p, void* sums, hipStream_t s);
inline bool laid_out(const void* p, int64_t ld, int64_t len, int dt) {
  const int64_t size = (int64_t)dt_size(dt);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && len * size % 16 == 0 &&
         ld * size < (int64_t(1) << 31) / 256;
}
// Copies of matrices that are so: rows x cols entries (ldp apart) to rows x ld
// ones (ld a multiple of 8), zeros behind them; all in one launch.
struct LayOut {
  const void* p;
  int64_t ldp, rows;
  int cols;
  void* out;
  int64_t ld;
};
struct LayOuts {
  LayOut m[4];
  int n;
};
sm_status launch_lay_out(const LayOuts& all, int dt, hipStream_t s);

// The sums over T rows of dz (ld entries apart) of n columns, in float32, to
// out (added to it with accumulate).  sums: scratch of column_sums_ws bytes.
size_t column_sums_ws(int64_t T, int n);
sm_status launch_column_sums(const void* dz, int64_t ld, int64_t T, int n, int dt, void* out,
                             int accumulate, void* sums, hipStream_t s);

// rows x cols entries (row stride ld) set to 0.
sm_status launch_zero(void* p, int64_t ld, int64_t rows, int cols, int dt, hipStream_t s);

// 8-bit checkpoints (sm_act8_pack, sm_act8_unpack).
sm_status launch_act8_pack(const void* x, int64_t ldx, int dt, int64_t T, int d, uint8_t* x8,
                           uint8_t* scale, hipStream_t s);
// pad: entries d .. round_up(d, 8) - 1 of the rows of x get zeros.
sm_status launch_act8_unpack(const uint8_t* x8, const uint8_t* scale, int dt, int64_t T, int d,
                             void* x, int64_t ldx, bool pad, hipStream_t s);

}  // namespace sm
