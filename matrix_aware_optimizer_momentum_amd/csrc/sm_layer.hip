// C ABI of the feed-forward layers and of the 8-bit checkpoints of their
// inputs.  Arguments are validated on the host before any HIP call.
#include "layer_internal.hpp"

namespace sm {

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int kMaxWidth = 1 << 20;
constexpr int64_t kMaxCount = int64_t(1) << 40;   // entries of x or y: their tiles stay countable
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr int64_t kMaxSpan = int64_t(1) << 46;   // entries from a matrix's first row to past its last

bool multiple_of(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// A matrix that a call reads or writes, in bytes.
struct Area {
  uintptr_t p;
  int64_t ld, rows, len;
  bool written;
};
// Some byte lies in both.  Matrices of one ld may be columns of one wider
// matrix, and a single row may lie between a matrix's: they share none if their
// rows' places modulo ld do not meet.
bool meet(const Area& x, const Area& y) {
  const Area &a = x.p <= y.p ? x : y, &b = x.p <= y.p ? y : x;
  const uintptr_t off = b.p - a.p;
  if (off >= (uintptr_t)((a.rows - 1) * a.ld + a.len)) return false;
  if (a.ld != b.ld && b.rows > 1) return true;
  const int64_t at = (int64_t)(off % (uintptr_t)a.ld);
  return at < a.len || at + b.len > a.ld;
}
class Areas {
 public:
  void add(const void* p, int64_t ld, int64_t rows, int64_t len, bool written) {
    if (p && rows > 0 && len > 0)
      v_[n_++] = Area{reinterpret_cast<uintptr_t>(p), rows == 1 ? len : ld, rows, len, written};
  }
  bool conflict() const {
    for (int i = 0; i < n_; ++i)
      for (int k = 0; k < i; ++k)
        if ((v_[i].written || v_[k].written) && meet(v_[i], v_[k])) return true;
    return false;
  }

 private:
  Area v_[16];
  int n_ = 0;
};

sm_status check_sizes(int64_t T, int d, int dt) {
  if (dt != SM_F32 && dt != SM_BF16) return SM_ERR_DTYPE;
  if (T < 0 || T > kMaxTokens || d < 1 || d > kMaxWidth) return SM_ERR_SHAPE;
  return SM_OK;
}
sm_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t len, size_t size) {
  if (!p || !multiple_of(p, size) || ld < len || ld > kMaxLd) return SM_ERR_ARG;
  return rows > 1 && ld > kMaxSpan / rows ? SM_ERR_ARG : SM_OK;
}

int act8_blocks(int d) { return (d + SM_ACT8_BLOCK - 1) / SM_ACT8_BLOCK; }

sm_status check_act8(const void* x, int64_t ldx, int dt, int64_t T, int32_t d, const uint8_t* x8,
                     const uint8_t* scale, bool pack) {
  SM_TRY(check_sizes(T, d, dt));
  if (T * d > kMaxCount) return SM_ERR_SHAPE;
  if (T == 0) return SM_OK;
  SM_TRY(check_matrix(x, ldx, T, d, dt_size(dt)));
  if (!x8 || !scale) return SM_ERR_ARG;
  const int64_t size = (int64_t)dt_size(dt);
  Areas a;
  a.add(x, ldx * size, T, d * size, !pack);
  a.add(x8, d, T, d, pack);
  a.add(scale, act8_blocks(d), T, act8_blocks(d), pack);
  return a.conflict() ? SM_ERR_ARG : SM_OK;
}

enum Call { kCallLinear, kCallLinearGrad, kCallGated, kCallGatedGrad };
bool is_grad(Call c) { return c == kCallLinearGrad || c == kCallGatedGrad; }
bool is_gated(Call c) { return c == kCallGated || c == kCallGatedGrad; }

// The call makes z (or a and b) and dz anew: not for act none of a linear
// layer, whose dz is dy, nor if only dx of it were wanted of nothing.
bool makes_dz(const sm_layer& l, Call c) { return is_gated(c) || l.act != SM_ACT_NONE; }
// The call reads x (or its checkpoint).
bool reads_x(const sm_layer& l, Call c) {
  return !is_grad(c) || makes_dz(l, c) || l.dw;
}

// all: empty, gets the call's matrices.
sm_status check_layer(const sm_layer* lp, Call c, Areas* all) {
  if (!lp) return SM_ERR_ARG;
  const sm_layer& l = *lp;
  Areas& areas = *all;
  SM_TRY(check_sizes(l.T, l.d, l.dt));
  if (l.n < 1 || l.n > kMaxWidth) return SM_ERR_SHAPE;
  if (l.T * std::max(l.d, l.n) > kMaxCount) return SM_ERR_SHAPE;
  if (l.act < SM_ACT_NONE || l.act > SM_ACT_GELU_TANH) return SM_ERR_ARG;
  const size_t z = dt_size(l.dt);
  const int64_t size = (int64_t)z;
  SM_TRY(check_matrix(l.w, l.ldw, l.n, l.d, z));
  areas.add(l.w, l.ldw * size, l.n, l.d * size, false);
  if (is_gated(c)) {
    SM_TRY(check_matrix(l.w2, l.ldw2, l.n, l.d, z));
    areas.add(l.w2, l.ldw2 * size, l.n, l.d * size, false);
  } else if (l.bias) {
    if (!multiple_of(l.bias, z)) return SM_ERR_ARG;
    areas.add(l.bias, 0, 1, l.n * size, false);
  }
  if (is_grad(c) && l.x8) {
    if (l.x || !l.x8_scale) return SM_ERR_ARG;
    areas.add(l.x8, l.d, l.T, l.d, false);
    areas.add(l.x8_scale, act8_blocks(l.d), l.T, act8_blocks(l.d), false);
  } else if (l.T > 0) {
    SM_TRY(check_matrix(l.x, l.ldx, l.T, l.d, z));
    areas.add(l.x, l.ldx * size, l.T, l.d * size, false);
  }
  if (!is_grad(c)) {
    if (l.T > 0) {
      SM_TRY(check_matrix(l.y, l.ldy, l.T, l.n, z));
      areas.add(l.y, l.ldy * size, l.T, l.n * size, true);
      if (c == kCallLinear && l.residual) {
        SM_TRY(check_matrix(l.residual, l.ldr, l.T, l.n, z));
        if (l.residual != l.y || l.ldr != l.ldy)
          areas.add(l.residual, l.ldr * size, l.T, l.n * size, false);
      }
    }
    return areas.conflict() ? SM_ERR_ARG : SM_OK;
  }
  const void* dw2 = is_gated(c) ? l.dw2 : nullptr;
  const void* dbias = is_gated(c) ? nullptr : l.dbias;
  if (!l.dx && !l.dw && !dw2 && !dbias) return SM_ERR_ARG;
  if (l.T > 0) {
    SM_TRY(check_matrix(l.dy, l.lddy, l.T, l.n, z));
    areas.add(l.dy, l.lddy * size, l.T, l.n * size, false);
    if (l.dx) {
      SM_TRY(check_matrix(l.dx, l.lddx, l.T, l.d, z));
      areas.add(l.dx, l.lddx * size, l.T, l.d * size, true);
    }
  }
  if (l.dw) {
    SM_TRY(check_matrix(l.dw, l.lddw, l.n, l.d, z));
    areas.add(l.dw, l.lddw * size, l.n, l.d * size, true);
  }
  if (dw2) {
    SM_TRY(check_matrix(l.dw2, l.lddw2, l.n, l.d, z));
    areas.add(l.dw2, l.lddw2 * size, l.n, l.d * size, true);
  }
  if (dbias) {
    if (!multiple_of(dbias, z)) return SM_ERR_ARG;
    areas.add(dbias, 0, 1, l.n * size, true);
  }
  return areas.conflict() ? SM_ERR_ARG : SM_OK;
}

// What a call keeps in its workspace: offsets of the operands that it lays out
// anew, of x from a checkpoint, and of dz.
struct LayerWs {
  bool few;   // a forward product by the kernel for few tokens: nothing of this
  bool lay_x, lay_w, lay_w2, lay_dy;
  size_t x, w, w2, dy, dz, dz2, sums, bytes;   // sums: of a split product
  int64_t ldd, ldn;   // rows of d and of n entries
};
LayerWs layer_ws(const sm_layer& l, Call c) {
  LayerWs w{};
  auto take = [&](bool wanted, int64_t rows, int64_t ld) {
    const size_t at = w.bytes;
    if (wanted) w.bytes += (size_t)round_up(rows * ld * (int64_t)dt_size(l.dt), 256);
    return at;
  };
  w.ldd = round_up(l.d, 8);
  w.ldn = round_up(l.n, 8);
  if (l.T == 0) return w;
  if (!is_grad(c)) {
    const bool in_place = laid_out(l.w, l.ldw, l.d, l.dt) &&
                          (!is_gated(c) || laid_out(l.w2, l.ldw2, l.d, l.dt));
    w.few = few_tokens(is_gated(c) ? kGated : kLinear, l.dt, l.T, l.n, l.d, in_place,
                       laid_out(l.x, l.ldx, l.d, l.dt));
    if (w.few) return w;
  }
  const bool grad = is_grad(c), x8 = grad && l.x8;
  const bool again = !grad || makes_dz(l, c);   // x W^T is computed
  w.lay_x = !x8 && reads_x(l, c) && !laid_out(l.x, l.ldx, l.d, l.dt);
  w.lay_w = (again || l.dx) && !laid_out(l.w, l.ldw, l.d, l.dt);
  w.lay_w2 = is_gated(c) && !laid_out(l.w2, l.ldw2, l.d, l.dt);
  w.lay_dy = grad && !again && (l.dx || l.dw) && !laid_out(l.dy, l.lddy, l.n, l.dt);
  w.x = take(w.lay_x || (x8 && reads_x(l, c)), l.T, w.ldd);
  w.w = take(w.lay_w, l.n, w.ldd);
  w.w2 = take(w.lay_w2, l.n, w.ldd);
  w.dy = take(w.lay_dy, l.T, w.ldn);
  w.dz = take(grad && again, l.T, w.ldn);
  w.dz2 = take(grad && is_gated(c), l.T, w.ldn);
  const int T = (int)l.T, two = is_gated(c) ? 2 : 1;
  w.sums = w.bytes;
  size_t most = 0;
  auto product = [&](int kind, int M, int N, int K, int parts) {
    most = std::max(most, product_ws(kind, l.dt, M, N, K, parts));
  };
  if (!grad) {
    product(is_gated(c) ? kGated : kLinear, T, l.n, l.d, 1);
  } else {
    if (again) product(is_gated(c) ? kGatedSlope : kSlope, T, l.n, l.d, 1);
    if (l.dx) product(kDx, T, l.d, l.n, two);
    const int dws = (l.dw ? 1 : 0) + (is_gated(c) && l.dw2 ? 1 : 0);
    if (dws) product(kDw, l.n, l.d, T, dws);
    if (!is_gated(c) && l.dbias) most = std::max(most, column_sums_ws(l.T, l.n));
  }
  w.bytes += (size_t)round_up((int64_t)most, 256);
  return w;
}

sm_status layer_query(const sm_layer* l, Call c, size_t* bytes) {
  if (!bytes) return SM_ERR_ARG;
  Areas areas;
  SM_TRY(check_layer(l, c, &areas));
  *bytes = layer_ws(*l, c).bytes;
  return SM_OK;
}

// The operands of a call, laid out if they have to be.
struct Operands {
  Operand x, w, w2, dz[2];
};
sm_status lay_out(const sm_layer& l, const LayerWs& w, char* ws, Operands* o, bool checkpoint,
                  hipStream_t s) {
  o->x = {l.x, l.ldx};
  o->w = {l.w, l.ldw};
  o->w2 = {l.w2, l.ldw2};
  o->dz[0] = {l.dy, l.lddy};
  o->dz[1] = {nullptr, 0};
  if (checkpoint) {
    o->x = {ws + w.x, w.ldd};
    SM_TRY(launch_act8_unpack(l.x8, l.x8_scale, l.dt, l.T, l.d, ws + w.x, w.ldd, true, s));
  }
  LayOuts all;
  all.n = 0;
  auto lay = [&](bool wanted, Operand* m, int64_t rows, int cols, size_t at, int64_t ld) {
    if (!wanted) return;
    all.m[all.n++] = LayOut{m->p, m->ld, rows, cols, ws + at, ld};
    *m = {ws + at, ld};
  };
  lay(w.lay_x, &o->x, l.T, l.d, w.x, w.ldd);
  lay(w.lay_w, &o->w, l.n, l.d, w.w, w.ldd);
  lay(w.lay_w2, &o->w2, l.n, l.d, w.w2, w.ldd);
  lay(w.lay_dy, &o->dz[0], l.T, l.n, w.dy, w.ldn);
  return launch_lay_out(all, l.dt, s);
}

// What the call uses of the workspace lies over none of its matrices.
sm_status check_ws(const LayerWs& w, const void* ws, size_t ws_bytes, Areas* areas) {
  if (w.bytes && (!ws || !multiple_of(ws, 256))) return SM_ERR_ARG;
  if (ws_bytes < w.bytes) return SM_ERR_WORKSPACE;
  areas->add(ws, 0, w.bytes ? 1 : 0, (int64_t)w.bytes, true);
  return areas->conflict() ? SM_ERR_ARG : SM_OK;
}

Product product_of(const sm_layer& l, int kind, const Operands& o) {
  Product p;
  std::memset(&p, 0, sizeof(p));
  p.kind = kind;
  p.dt = l.dt;
  p.act = l.act;
  p.M = (int)l.T;
  p.N = l.n;
  p.K = l.d;
  p.parts = 1;
  p.a[0] = o.x;
  p.b[0] = o.w;
  p.b[1] = o.w2;
  if (kind == kLinear || kind == kSlope) p.bias = l.bias;
  return p;
}

sm_status run_forward(const sm_layer* lp, Call c, void* ws, size_t ws_bytes, hipStream_t s) {
  Areas areas;
  SM_TRY(check_layer(lp, c, &areas));
  const sm_layer& l = *lp;
  const LayerWs w = layer_ws(l, c);
  SM_TRY(check_ws(w, ws, ws_bytes, &areas));
  if (l.T == 0) return SM_OK;
  Operands o;
  SM_TRY(lay_out(l, w, static_cast<char*>(ws), &o, false, s));
  Product p = product_of(l, c == kCallGated ? kGated : kLinear, o);
  if (c == kCallLinear) p.in = {l.residual, l.ldr};
  p.c[0] = l.y;
  p.ldc[0] = l.ldy;
  p.few = w.few;
  return launch_product(p, static_cast<char*>(ws) + w.sums, s);
}

sm_status run_grad(const sm_layer* lp, Call c, void* wsp, size_t ws_bytes, hipStream_t s) {
  Areas areas;
  SM_TRY(check_layer(lp, c, &areas));
  const sm_layer& l = *lp;
  const bool gated = is_gated(c);
  void* dw2 = gated ? l.dw2 : nullptr;
  void* dbias = gated ? nullptr : l.dbias;
  const LayerWs w = layer_ws(l, c);
  SM_TRY(check_ws(w, wsp, ws_bytes, &areas));
  if (l.T == 0) {
    if (l.accumulate) return SM_OK;
    if (l.dw) SM_TRY(launch_zero(l.dw, l.lddw, l.n, l.d, l.dt, s));
    if (dw2) SM_TRY(launch_zero(dw2, l.lddw2, l.n, l.d, l.dt, s));
    if (dbias) SM_TRY(launch_zero(dbias, l.n, 1, l.n, l.dt, s));
    return SM_OK;
  }
  char* ws = static_cast<char*>(wsp);
  Operands o;
  SM_TRY(lay_out(l, w, ws, &o, l.x8 && reads_x(l, c), s));
  if (makes_dz(l, c)) {
    Product p = product_of(l, gated ? kGatedSlope : kSlope, o);
    p.in = {l.dy, l.lddy};
    p.c[0] = ws + w.dz;
    p.c[1] = ws + w.dz2;
    p.ldc[0] = p.ldc[1] = w.ldn;
    p.pad = (int)w.ldn;
    o.dz[0] = {ws + w.dz, w.ldn};
    o.dz[1] = {ws + w.dz2, w.ldn};
    SM_TRY(launch_product(p, ws + w.sums, s));
  }
  if (l.dx) {
    Product p = product_of(l, kDx, o);
    p.N = l.d;
    p.K = l.n;
    p.parts = gated ? 2 : 1;
    p.a[0] = o.dz[0];
    p.a[1] = o.dz[1];
    p.c[0] = l.dx;
    p.ldc[0] = l.lddx;
    SM_TRY(launch_product(p, ws + w.sums, s));
  }
  if (l.dw || dw2) {
    Product p = product_of(l, kDw, o);
    p.M = l.n;
    p.N = l.d;
    p.K = (int)l.T;
    p.b[0] = o.x;
    p.accumulate = l.accumulate;
    int q = 0;
    if (l.dw) p.a[q] = o.dz[0], p.c[q] = l.dw, p.ldc[q++] = l.lddw;
    if (dw2) p.a[q] = o.dz[1], p.c[q] = dw2, p.ldc[q++] = l.lddw2;
    p.parts = q;
    SM_TRY(launch_product(p, ws + w.sums, s));
  }
  if (dbias)
    SM_TRY(launch_column_sums(o.dz[0].p, o.dz[0].ld, l.T, l.n, l.dt, dbias, l.accumulate,
                              ws + w.sums, s));
  return SM_OK;
}

}  // namespace
}  // namespace sm

using namespace sm;

extern "C" {

sm_status sm_act8_pack(const void* x, int64_t ldx, int dt, int64_t T, int32_t d, uint8_t* x8,
                       uint8_t* scale, hipStream_t s) {
  SM_TRY(check_act8(x, ldx, dt, T, d, x8, scale, true));
  return T == 0 ? SM_OK : launch_act8_pack(x, ldx, dt, T, d, x8, scale, s);
}

sm_status sm_act8_unpack(const uint8_t* x8, const uint8_t* scale, int dt, int64_t T, int32_t d,
                         void* x, int64_t ldx, hipStream_t s) {
  SM_TRY(check_act8(x, ldx, dt, T, d, x8, scale, false));
  return T == 0 ? SM_OK : launch_act8_unpack(x8, scale, dt, T, d, x, ldx, false, s);
}

sm_status sm_linear_ws(const sm_layer* l, size_t* ws_bytes) {
  return layer_query(l, kCallLinear, ws_bytes);
}
sm_status sm_linear(const sm_layer* l, void* ws, size_t ws_bytes, hipStream_t s) {
  return run_forward(l, kCallLinear, ws, ws_bytes, s);
}
sm_status sm_linear_grad_ws(const sm_layer* l, size_t* ws_bytes) {
  return layer_query(l, kCallLinearGrad, ws_bytes);
}
sm_status sm_linear_grad(const sm_layer* l, void* ws, size_t ws_bytes, hipStream_t s) {
  return run_grad(l, kCallLinearGrad, ws, ws_bytes, s);
}
sm_status sm_gated_ws(const sm_layer* l, size_t* ws_bytes) {
  return layer_query(l, kCallGated, ws_bytes);
}
sm_status sm_gated(const sm_layer* l, void* ws, size_t ws_bytes, hipStream_t s) {
  return run_forward(l, kCallGated, ws, ws_bytes, s);
}
sm_status sm_gated_grad_ws(const sm_layer* l, size_t* ws_bytes) {
  return layer_query(l, kCallGatedGrad, ws_bytes);
}
sm_status sm_gated_grad(const sm_layer* l, void* ws, size_t ws_bytes, hipStream_t s) {
  return run_grad(l, kCallGatedGrad, ws, ws_bytes, s);
}

}  // extern "C"
