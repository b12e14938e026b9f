// Which kernel and which tiles a product of the feed-forward layers takes.
// Plain host code: it is compiled by itself to be tested.
#pragma once

#include <algorithm>
#include <cstdint>

namespace sm {

// What a product of a layer computes, and with it its operands' layouts.
// An operand is k-contiguous (KC: rows x K, row-major) or k-major (KR: K x
// rows).
//   kLinear      c = act(A B^T + bias) + in          A = x KC,  B = W KC
//   kSlope       c = in * act'(A B^T + bias)         A = x KC,  B = W KC
//   kGated       c = act(a) b,  a = A B^T, b = A B2^T      x, Wg and Wu KC
//   kGatedSlope  c = in b act'(a),  c2 = in act(a)         x, Wg and Wu KC
//   kDx          c = A B (+ A2 B2)                   A = dz KC, B = W KR
//   kDw          c (+)= A^T B  (and c2 (+)= A2^T B)  A = dz KR, B = x KR
enum ProductKind : int { kLinear, kSlope, kGated, kGatedSlope, kDx, kDw };
constexpr bool kind_dual(int k) { return k == kGated || k == kGatedSlope; }
constexpr bool kind_acts(int k) { return k == kLinear || k == kSlope || kind_dual(k); }
constexpr bool kind_a_kr(int k) { return k == kDw; }
constexpr bool kind_b_kr(int k) { return k == kDx || k == kDw; }

// The kernel for few tokens takes the product, operands of any alignment.  (us
// by it / by tiles: 17 tokens, gated 4096 x 11008 44.6 / 45.7, linear 11008 x
// 4096 26.7 / 32.4; 32 tokens 49.5 / 45.4, 31.7 / 34.0.)
inline bool few_tokens(int kind, int64_t T) {
  return (kind == kLinear || kind == kGated) && T <= 32;
}

// How a product is launched: tiles of 64 mi rows, columns from `cut` on by a
// second launch of small tiles, sums in `splits` shares.
struct Plan {
  int mi, splits, cut;
};

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline int tile_rows(int mi) { return 64 * mi; }
inline int tile_cols(int kind, int mi) { return kind_dual(kind) ? 32 * mi : 64 * mi; }

// b: bf16, else float32.
inline Plan plan_product(int kind, bool b, int M, int N, int K, int parts, int cus) {
  const int nprob = kind == kDw ? parts : 1;
  const int steps = ceil_div(K, b ? 64 : 32) * (kind == kDx ? parts : 1);
  const int64_t large = (int64_t)ceil_div(M, tile_rows(4)) * ceil_div(N, tile_cols(kind, 4)) * nprob;
  const int64_t small = (int64_t)ceil_div(M, tile_rows(2)) * ceil_div(N, tile_cols(kind, 2)) * nprob;
  // us, as measured: a step of a large tile, of one small tile on a CU and of
  // two, of up to two least ones; around a tile; joining (the sums are written
  // and read).  What the choice gains: GPT-2 large's first product for 4096
  // tokens 81 -> 66 us (the cut), gated backward 1003 x 1280 x 3416 140 -> 91,
  // float32 backward 515 x 771 x 1283 239 -> 99 (the shares), 1000 x 1024 x
  // 1024 bf16 19 -> 14 (the least tiles).
  const double t4 = b ? 1.5 : 8.0, t1 = b ? 0.75 : 2.25, t2 = b ? 1.0 : 4.0, c4 = 9.0, c2 = 6.0;
  const double u1 = b ? 0.4 : 1.4, c1 = 5.0;
  const double join = 3.0, per_sum = 8.0 / 8.0e6;
  auto smalls = [&](int64_t n, double st) {   // n small tiles of st steps
    return ceil_div(n, 2 * cus) > 1 || n > cus ? ceil_div(n, 2 * cus) * (st * t2 + c2)
                                               : st * t1 + c2;
  };
  Plan best = {4, 1, N};
  double least = ceil_div(large, cus) * (steps * t4 + c4);
  auto consider = [&](Plan p, double us) {
    if (us < least) least = us, best = p;
  };
  consider({2, 1, N}, smalls(small, steps));
  const int64_t least_tiles =
      (int64_t)ceil_div(M, tile_rows(1)) * ceil_div(N, tile_cols(kind, 1)) * nprob;
  consider({1, 1, N}, ceil_div(least_tiles, 2 * cus) * (steps * u1 + c1));
  for (int s = 2; s <= 16 && s * 2 <= steps; ++s) {
    const double sums = (double)ceil_div(M, 128) * 128 * ceil_div(N, tile_cols(kind, 2)) * 128 *
                        nprob * s;
    consider({2, s, N}, smalls(small * s, (double)steps / s) + join + sums * per_sum);
  }
  if (nprob == 1 && large > cus) {   // whole rounds of large tiles, the rest by small ones
    const int tm = ceil_div(M, tile_rows(4));
    const int n1 = (int)(large / cus * cus / tm) * tile_cols(kind, 4);
    if (n1 > 0 && n1 < N) {
      const int64_t rest = (int64_t)ceil_div(M, 128) * ceil_div(N - n1, tile_cols(kind, 2));
      consider({4, 1, n1}, large / cus * (steps * t4 + c4) + smalls(rest, steps) + 2.0);
    }
  }
  return best;
}

}  // namespace sm
