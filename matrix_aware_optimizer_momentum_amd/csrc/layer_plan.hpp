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

// How a product is launched: tiles of 64 mi rows, columns from `cut` on by a
// second launch of small tiles, sums in `splits` shares.
struct Plan {
  int mi, splits, cut;
  double us, join;   // what it is taken to cost; and of that, joining the shares
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
  Plan best = {4, 1, N, ceil_div(large, cus) * (steps * t4 + c4), 0.0};
  auto consider = [&](const Plan& p) {
    if (p.us < best.us) best = p;
  };
  consider({2, 1, N, smalls(small, steps), 0.0});
  const int64_t least_tiles =
      (int64_t)ceil_div(M, tile_rows(1)) * ceil_div(N, tile_cols(kind, 1)) * nprob;
  consider({1, 1, N, ceil_div(least_tiles, 2 * cus) * (steps * u1 + c1), 0.0});
  for (int s = 2; s <= 16 && s * 2 <= steps; ++s) {
    const double sums = (double)ceil_div(M, 128) * 128 * ceil_div(N, tile_cols(kind, 2)) * 128 *
                        nprob * s;
    const double joining = join + sums * per_sum;
    consider({2, s, N, smalls(small * s, (double)steps / s) + joining, joining});
  }
  if (nprob == 1 && large > cus) {   // whole rounds of large tiles, the rest by small ones
    const int tm = ceil_div(M, tile_rows(4));
    const int n1 = (int)(large / cus * cus / tm) * tile_cols(kind, 4);
    if (n1 > 0 && n1 < N) {
      const int64_t rest = (int64_t)ceil_div(M, 128) * ceil_div(N - n1, tile_cols(kind, 2));
      consider({4, 1, n1, large / cus * (steps * t4 + c4) + smalls(rest, steps) + 2.0, 0.0});
    }
  }
  return best;
}

// The kernel for few tokens takes a forward product (of any alignment), and not
// the tiles.  Its workgroups, one to 16 columns, read whole rows of weights and
// all of x, so that a CU takes these in at a rate of its own (29 and 48 GB/s up
// to 16 tokens, 25 and 42 beyond, where half as many loads are in flight); the
// tiles split sums, and so use all CUs for narrow outputs.  Both wait for the
// weights (5 TB/s), the tiles ahead of joining.  us by it / by tiles, bf16:
//   tokens                  1          8          17         24         32
//   4096 -> 11008       20.5/30.7  23.2/29.0  27.3/29.2  31.1/29.3  34.8/29.4
//   the same, gated     34.1/41.1  36.8/39.7  43.7/39.8  45.9/40.3  49.2/41.1
//   11008 -> 4096       22.1/33.6  23.6/33.8  28.5/34.1  29.8/34.1  33.2/34.6
//   11008 -> 512        14.7/18.5  18.1/19.0  25.3/19.2  27.3/19.1  30.8/19.3
//   the same, gated     25.0/20.6  28.0/21.1  35.3/21.3  37.3/21.3  40.8/21.2
// and float32:
//   4096 -> 11008       36.5/112   40.5/111   55.7/112   60.6/112   67.2/112
//   11008 -> 512, gated 56.4/58.7  59.8/58.9  86.0/58.8  89.2/58.9  93.6/59.0
// (weights out of HBM, times of captured launches).  The rates are fitted to
// 584 such pairs of 17 shapes; where the slower kernel is taken it costs at
// most 8 %.  Laying weights out for the tiles is taken to cost more than it
// gains, laying out x alone 4 us.
inline bool takes_few(int kind, bool b, int64_t T, int n, int d, bool w_in_place, bool x_in_place,
                      int cus) {
  if ((kind != kLinear && kind != kGated) || T > 32) return false;
  if (!w_in_place) return true;
  const double row = (double)d * (b ? 2 : 4), both = kind_dual(kind) ? 2.0 : 1.0;
  const double groups = std::max(1.0, (double)ceil_div(n, 16) / cus);   // workgroups of a CU
  const double w = both * 16 * row * groups, x = T * row * groups;
  const double memory = 2.0 + both * n * row / 5.0e6;
  const double few = 2.0 + (T <= 16 ? w / 29.0e3 + x / 48.0e3 : w / 25.0e3 + x / 42.0e3);
  const Plan p = plan_product(kind, b, (int)T, n, d, 1, cus);
  const double tiles = std::max(p.us - p.join, memory) + p.join + (x_in_place ? 0.0 : 4.0);
  return std::max(few, memory) <= tiles;
}

}  // namespace sm
