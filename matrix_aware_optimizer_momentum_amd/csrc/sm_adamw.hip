// C ABI of the AdamW operators: parameter sets, the step, the global
// gradient norm and the conversion of 8-bit states.  Arguments are validated
// on the host before any HIP call.
#include "adamw_internal.hpp"

#include <cmath>
#include <new>

struct sm_param_set_s {
  sm::ParamSetDev dev;
  bool update;        // every parameter has weights and states
  bool fp8;           // some have 8-bit states
  double step_bytes;  // of one AdamW step
  double grad_bytes;
};

namespace sm {

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 40;
constexpr int kMaxParams = 1 << 20;
// The slowest averages of 8-bit states, whose codes are left with a chance in
// steps of 2^-16: at 0.999999 a decaying v (0.33 to 0.52 of one) would hardly
// ever fall, at 0.99999 it falls with 3 to 5 of them for 3.3 to 5.2.
constexpr float kBetaMost8 = 0.99999f;
// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;

bool multiple_of(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool valid_dt(int dt) { return dt == SM_F32 || dt == SM_BF16; }
bool finite(float v) { return std::isfinite(v); }
int64_t state_blocks(int64_t count) { return (count + kStateBlock - 1) / kStateBlock; }
bool norm_only(const sm_param& p) { return !p.w && !p.m && !p.v; }

// Some parameter of the set has 8-bit states.
bool has_fp8(const sm_param* params, int n) {
  for (int i = 0; i < n; ++i)
    if (params[i].count > 0 && !norm_only(params[i]) && params[i].state == SM_STATE_FP8)
      return true;
  return false;
}

// Where a set's tables lie in its workspace, with room for work items of one
// unit each (wider ones need less).
struct SetWs {
  size_t scalars, counter, parts, ents, items, norm_items, bytes;
};
sm_status set_ws(const sm_param* params, int n, SetWs* w) {
  if (!params || n < 1) return SM_ERR_ARG;
  if (n > kMaxParams) return SM_ERR_SHAPE;
  const bool fp8 = has_fp8(params, n);
  const int64_t unit = step_unit(fp8);
  int64_t nitems = 0, nnorm = 0;
  for (int i = 0; i < n; ++i) {
    if (params[i].count < 0 || params[i].count > kMaxCount) return SM_ERR_SHAPE;
    nitems += (params[i].count + unit - 1) / unit;   // < 2^52
    nnorm += norm_items(params[i].count);
  }
  if (nitems * step_threads(fp8) > kMaxThreads) return SM_ERR_SHAPE;
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  w->scalars = 0;
  w->counter = up(sizeof(AdamwScalars));
  w->parts = w->counter + 256;
  w->ents = w->parts + up(kNormPartsM * sizeof(double));
  w->items = w->ents + up((size_t)n * sizeof(ParamEnt));
  w->norm_items = w->items + up((size_t)nitems * sizeof(WorkItem));
  w->bytes = w->norm_items + up((size_t)nnorm * sizeof(WorkItem));
  return SM_OK;
}

// A range of addresses that a set reads or writes.
struct Range {
  uintptr_t a, b;
  bool written;
};
void add_range(std::vector<Range>& v, const void* p, size_t bytes, bool written) {
  if (p && bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    v.push_back(Range{a, a + bytes, written});
  }
}
// Some written range overlaps another range.
bool conflict(std::vector<Range>& v) {
  std::sort(v.begin(), v.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
  uintptr_t end_any = 0, end_written = 0;
  for (const Range& r : v) {
    if (r.a < (r.written ? end_any : end_written)) return true;
    end_any = std::max(end_any, r.b);
    if (r.written) end_written = std::max(end_written, r.b);
  }
  return false;
}

sm_status check_param(const sm_param& p, int M) {
  if (!valid_dt(p.gdt)) return SM_ERR_DTYPE;
  if (p.count == 0) return SM_OK;
  const size_t gs = dt_size(p.gdt);
  if (!p.grad || !multiple_of(p.grad, gs)) return SM_ERR_ARG;
  if (M > 1) {
    if (p.grad_stride < p.count) return SM_ERR_ARG;
    if (p.grad_stride > kMaxCount) return SM_ERR_SHAPE;
  }
  if (norm_only(p)) return SM_OK;
  if (!valid_dt(p.wdt)) return SM_ERR_DTYPE;
  if (p.state != SM_STATE_F32 && p.state != SM_STATE_FP8) return SM_ERR_DTYPE;
  if (!p.w || !p.m || !p.v || !multiple_of(p.w, dt_size(p.wdt))) return SM_ERR_ARG;
  if (p.master && (p.wdt != SM_BF16 || !multiple_of(p.master, 4))) return SM_ERR_ARG;
  if (p.state == SM_STATE_FP8) {
    if (!p.m_scale || !p.v_scale || !multiple_of(p.m_scale, 4) || !multiple_of(p.v_scale, 4))
      return SM_ERR_ARG;
  } else if (p.m_scale || p.v_scale || !multiple_of(p.m, 4) || !multiple_of(p.v, 4)) {
    return SM_ERR_ARG;
  }
  if (!finite(p.weight_decay) || p.weight_decay < 0.f || !finite(p.lr_mult) || p.lr_mult < 0.f)
    return SM_ERR_ARG;
  return SM_OK;
}

ParamEnt entry_of(const sm_param& p, int M, bool fp8) {
  ParamEnt e;
  std::memset(&e, 0, sizeof(e));
  e.g = p.grad;
  e.count = p.count;
  e.gstride = M > 1 ? p.grad_stride : 0;
  e.lr_mult = 1.0f;
  e.span = step_unit(fp8);
  if (p.gdt == SM_BF16) e.flags |= kPF_G16;
  if (!norm_only(p)) {
    e.w = p.w;
    e.master = p.master;
    e.m = p.m;
    e.v = p.v;
    e.ms = p.m_scale;
    e.vs = p.v_scale;
    e.wd = p.weight_decay;
    e.lr_mult = p.lr_mult;
    if (p.wdt == SM_BF16) e.flags |= kPF_W16;
    // bf16 weights alone with 8-bit states, of one worker, move the fewest
    // bytes per entry (10): their items hold several units, whose loads are
    // all in flight before the first one is used.  495 M entries: 0.91 ms
    // with one unit, 0.87 with two, 0.81 with three, 0.85 with four; float32
    // states lose by it (1.82 ms with one, 1.88 with two).
    if (p.wdt == SM_BF16 && !p.master && M == 1 && p.state == SM_STATE_FP8)
      e.span *= kUnitsFp8;
    if (p.state == SM_STATE_FP8) e.flags |= kPF_FP8;
  }
  return e;
}

}  // namespace
}  // namespace sm

using namespace sm;

extern "C" {

sm_status sm_param_set_ws(const sm_param* params, int n, size_t* ws_bytes) {
  if (!ws_bytes) return SM_ERR_ARG;
  SetWs lay;
  SM_TRY(set_ws(params, n, &lay));
  *ws_bytes = lay.bytes;
  return SM_OK;
}

sm_status sm_param_set_create(const sm_param* params, int n, int M, void* ws, size_t ws_bytes,
                              hipStream_t s, sm_param_set* out) {
  if (!out) return SM_ERR_ARG;
  *out = nullptr;
  SetWs lay;
  SM_TRY(set_ws(params, n, &lay));
  if (M < 1 || M > 64) return SM_ERR_UNSUPPORTED;
  if (!ws || !multiple_of(ws, 256)) return SM_ERR_ARG;
  if (ws_bytes < lay.bytes) return SM_ERR_WORKSPACE;
  for (int i = 0; i < n; ++i) SM_TRY(check_param(params[i], M));

  try {
    std::vector<Range> ranges;
    ranges.reserve((size_t)n * (6 + M) + 1);
    add_range(ranges, ws, lay.bytes, true);
    for (int i = 0; i < n; ++i) {
      const sm_param& p = params[i];
      if (p.count == 0) continue;
      const size_t gs = dt_size(p.gdt), c = (size_t)p.count;
      for (int k = 0; k < M; ++k)
        add_range(ranges, static_cast<const char*>(p.grad) + (size_t)k * p.grad_stride * gs,
                  c * gs, false);
      if (norm_only(p)) continue;
      const size_t ss = p.state == SM_STATE_FP8 ? 1 : 4, sb = 4 * (size_t)state_blocks(p.count);
      add_range(ranges, p.w, c * dt_size(p.wdt), true);
      add_range(ranges, p.master, c * 4, true);
      add_range(ranges, p.m, c * ss, true);
      add_range(ranges, p.v, c * ss, true);
      add_range(ranges, p.m_scale, sb, true);
      add_range(ranges, p.v_scale, sb, true);
    }
    if (conflict(ranges)) return SM_ERR_ARG;
  } catch (const std::bad_alloc&) {
    return hip_fail(hipErrorOutOfMemory);
  }

  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  hipError_t e = hipStreamIsCapturing(s, &cap);
  if (e != hipSuccess) return hip_fail(e);
  if (cap != hipStreamCaptureStatusNone) return SM_ERR_UNSUPPORTED;

  sm_param_set h = new (std::nothrow) sm_param_set_s();
  if (!h) return hip_fail(hipErrorOutOfMemory);
  char* base = static_cast<char*>(ws);
  ParamEnt* ents = reinterpret_cast<ParamEnt*>(base + lay.ents);
  WorkItem* wi = reinterpret_cast<WorkItem*>(base + lay.items);
  h->dev.ents = ents;
  h->dev.items = wi;
  WorkItem* ni = reinterpret_cast<WorkItem*>(base + lay.norm_items);
  h->dev.norm_at = ni;
  h->dev.scalars = reinterpret_cast<AdamwScalars*>(base + lay.scalars);
  h->dev.counter = reinterpret_cast<uint32_t*>(base + lay.counter);
  h->dev.parts = reinterpret_cast<double*>(base + lay.parts);
  h->dev.M = M;
  int P = 1;
  while (P < M) P *= 2;
  h->dev.inv_P = 1.0 / P;
  h->dev.P_over_M = (float)P / (float)M;
  h->update = true;
  h->fp8 = has_fp8(params, n);
  h->step_bytes = h->grad_bytes = 0.0;

  int64_t first = 0, norm_first = 0;
  sm_status st = SM_OK;
  for (int i0 = 0; i0 < n && st == SM_OK; i0 += kFillMax) {
    const int k = std::min(kFillMax, n - i0);
    FillTbl t;
    std::memset(&t, 0, sizeof(t));
    for (int q = 0; q < k; ++q) {
      const sm_param& p = params[i0 + q];
      t.e[q] = entry_of(p, M, h->fp8);
      t.first[q] = first;
      t.norm_first[q] = norm_first;
      first += step_items(t.e[q]);
      norm_first += norm_items(p.count);
      const double c = (double)p.count;
      h->grad_bytes += c * M * dt_size(p.gdt);
      if (norm_only(p)) {
        if (p.count > 0) h->update = false;
        continue;
      }
      h->step_bytes += c * (p.master ? 8.0 + dt_size(p.wdt) : 2.0 * dt_size(p.wdt));
      h->step_bytes += p.state == SM_STATE_FP8 ? 4.0 * c + 16.0 * state_blocks(p.count) : 16.0 * c;
    }
    st = launch_set_fill(t, k, i0, ents, wi, ni, h->dev.counter, s);
  }
  h->dev.nitems = (int)first;
  h->dev.norm_items = (int)norm_first;
  h->step_bytes += h->grad_bytes;
  if (st == SM_OK) {
    e = hipStreamSynchronize(s);
    if (e != hipSuccess) st = hip_fail(e);
  }
  if (st != SM_OK) {
    delete h;
    return st;
  }
  *out = h;
  return SM_OK;
}

sm_status sm_param_set_destroy(sm_param_set set) {
  delete set;
  return SM_OK;
}

sm_status sm_adamw(const sm_adamw_config* c, sm_param_set set, int64_t t, int64_t* step,
                   const float* gscale, const float* lr_scale, hipStream_t s) {
  if (!c || !set || !set->update) return SM_ERR_ARG;
  if (step ? t != 0 || !multiple_of(step, 8) : t < 1) return SM_ERR_ARG;
  if (!multiple_of(gscale, 4) || !multiple_of(lr_scale, 4)) return SM_ERR_ARG;
  if (!finite(c->lr) || c->lr < 0.f) return SM_ERR_ARG;
  if (!(c->beta1 >= 0.f && c->beta1 < 1.f) || !(c->beta2 >= 0.f && c->beta2 < 1.f))
    return SM_ERR_ARG;
  if (!finite(c->eps) || c->eps < 1e-15f) return SM_ERR_ARG;
  if (c->rounding != SM_ROUND_NEAREST && c->rounding != SM_ROUND_STOCHASTIC) return SM_ERR_ARG;
  if (set->fp8 && (c->beta1 > kBetaMost8 || c->beta2 > kBetaMost8)) return SM_ERR_UNSUPPORTED;
  AdamwScalars a;
  std::memset(&a, 0, sizeof(a));
  if (step) {
    SM_TRY(launch_adamw_prep(*c, step, gscale, lr_scale, set->dev.scalars, s));
  } else {
    a = adamw_scalars(*c, t);
  }
  return launch_adamw(set->dev, a, step != nullptr, gscale, lr_scale, set->fp8,
                      scaled_roots(*c), set->step_bytes, s);
}

sm_status sm_grad_norm(const sm_param_set* sets, int nsets, float scale, float max_norm,
                       float* out, hipStream_t s) {
  if (!sets || nsets < 1 || !out || !multiple_of(out, 4)) return SM_ERR_ARG;
  if (nsets > kNormSets) return SM_ERR_UNSUPPORTED;
  for (int i = 0; i < nsets; ++i) {
    if (!sets[i]) return SM_ERR_ARG;
    for (int k = 0; k < i; ++k)
      if (sets[k] == sets[i]) return SM_ERR_ARG;   // its scratch holds one set's sums
  }
  if (!finite(scale) || !(max_norm > 0.f)) return SM_ERR_ARG;
  NormJoin f;
  std::memset(&f, 0, sizeof(f));
  f.scale = scale;
  f.max_norm = max_norm;
  f.out = out;
  for (int i = 0; i < nsets; ++i) {
    f.parts[i] = sets[i]->dev.parts;
    f.n[i] = norm_set_parts(sets[i]->dev.norm_items, sets[i]->dev.M);
    if (i == nsets - 1) f.nsets = nsets;
    SM_TRY(launch_grad_norm(sets[i]->dev, f, sets[i]->grad_bytes, s));
  }
  return SM_OK;
}

static sm_status check_state8(const void* m, const void* v, int64_t count, const void* m8,
                              const void* v8, const void* ms, const void* vs, bool pack) {
  if (count < 0 || count > kMaxCount) return SM_ERR_SHAPE;
  if (count == 0) return SM_OK;
  if (!m || !v || !m8 || !v8 || !ms || !vs) return SM_ERR_ARG;
  if (!multiple_of(m, 4) || !multiple_of(v, 4) || !multiple_of(ms, 4) || !multiple_of(vs, 4))
    return SM_ERR_ARG;
  const size_t c = (size_t)count, sb = 4 * (size_t)state_blocks(count);
  try {
    std::vector<Range> r;
    add_range(r, m, 4 * c, !pack);
    add_range(r, v, 4 * c, !pack);
    add_range(r, m8, c, pack);
    add_range(r, v8, c, pack);
    add_range(r, ms, sb, pack);
    add_range(r, vs, sb, pack);
    return conflict(r) ? SM_ERR_ARG : SM_OK;
  } catch (const std::bad_alloc&) {
    return hip_fail(hipErrorOutOfMemory);
  }
}

sm_status sm_state8_pack(const float* m, const float* v, int64_t count, uint8_t* m8, uint8_t* v8,
                         float* m_scale, float* v_scale, hipStream_t s) {
  SM_TRY(check_state8(m, v, count, m8, v8, m_scale, v_scale, true));
  if (count == 0) return SM_OK;
  return launch_state8_pack(m, v, count, m8, v8, m_scale, v_scale, s);
}

sm_status sm_state8_unpack(const uint8_t* m8, const uint8_t* v8, const float* m_scale,
                           const float* v_scale, int64_t count, float* m, float* v,
                           hipStream_t s) {
  SM_TRY(check_state8(m, v, count, m8, v8, m_scale, v_scale, false));
  if (count == 0) return SM_OK;
  return launch_state8_unpack(m8, v8, m_scale, v_scale, count, m, v, s);
}

}  // extern "C"
