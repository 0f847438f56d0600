// C ABI of the packed-row operators.  Host side: argument checks and kernel launches.  The
// arithmetic is in packed_rows.hip, packed_act.hip and packed_products.hip.
#include <hip/hip_runtime.h>

#include <exception>
#include <string>

#include "packed.h"
#include "zs_host.h"

namespace {

using zs::set_error;

constexpr int64_t kMaxRows = (int64_t)1 << 30;    // of any matrix, and its columns
constexpr int64_t kMaxPitch = (int64_t)1 << 30;   // elements
constexpr int64_t kMaxPacked = (int64_t)1 << 20;  // columns of packed rows
constexpr int64_t kMaxQPitch = (int64_t)1 << 22;  // bytes: 256 rows lie within 32-bit offsets
constexpr int64_t kMaxSum = 131056;               // columns of a linear layer: k * 128 * 128 < 2^31

zero_status_t bad(const std::string& msg) { return set_error(ZERO_EINVAL, msg); }
zero_status_t done(const char* what, hipError_t e) {
  return e == hipSuccess ? ZERO_OK : set_error(ZERO_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}
int64_t esize(int32_t dt) { return dt == ZERO_F32 ? 4 : 2; }

// Memory that a matrix takes: `rows` runs of `bytes`, `pitch` bytes apart.
struct Span {
  uint64_t at;
  int64_t rows, bytes, pitch;
  uint64_t end() const { return at + (uint64_t)(rows - 1) * (uint64_t)pitch + (uint64_t)bytes; }
  bool empty() const { return rows == 0 || bytes == 0; }
};
Span span(const zero_matrix_t& a) {
  return {(uint64_t)(uintptr_t)a.data, a.rows, a.cols * esize(a.dtype), (a.rows > 1 ? a.pitch : a.cols) * esize(a.dtype)};
}
Span span(const zero_packed_t& p) {
  return {(uint64_t)(uintptr_t)p.q, p.rows, (p.cols + 15) / 16 * 16, p.pitch};
}
Span scales(const zero_packed_t& p) { return {(uint64_t)(uintptr_t)p.scale, 1, p.rows * 4, p.rows * 4}; }

// Whether two matrices share memory.  Columns of one wider matrix are told apart: at the same pitch,
// by where their rows lie in it.
bool meet(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  if ((a.rows == 1 && b.rows == 1) || pitch <= 0) return true;
  const Span& lo = a.at <= b.at ? a : b;
  const Span& hi = a.at <= b.at ? b : a;
  const uint64_t off = (hi.at - lo.at) % (uint64_t)pitch;
  return !(off >= (uint64_t)lo.bytes && off + (uint64_t)hi.bytes <= (uint64_t)pitch);
}

zero_status_t check(const zero_matrix_t* a, const char* name) {
  const std::string n(name);
  if (!a) return bad("null " + n);
  if (a->dtype != ZERO_F16 && a->dtype != ZERO_BF16 && a->dtype != ZERO_F32) return bad(n + ": dtype must be ZERO_F16, ZERO_BF16 or ZERO_F32");
  if (a->rows < 0 || a->cols < 0 || a->rows > kMaxRows || a->cols > kMaxRows) return bad(n + ": rows and cols must be >= 0 and <= 2^30");
  if (a->rows > 1 && (a->pitch < a->cols || a->pitch > kMaxPitch)) return bad(n + ": pitch must be >= cols and <= 2^30");
  if (a->rows * a->cols == 0) return ZERO_OK;
  if (!a->data) return bad(n + ": null address");
  if ((uintptr_t)a->data % (uintptr_t)esize(a->dtype)) return bad(n + ": address not aligned to its elements");
  return ZERO_OK;
}
zero_status_t check(const zero_packed_t* p, const char* name) {
  const std::string n(name);
  if (!p) return bad("null " + n);
  if (p->rule != ZERO_SCALE_POW2 && p->rule != ZERO_SCALE_MAX) return bad(n + ": rule must be ZERO_SCALE_POW2 or ZERO_SCALE_MAX");
  if (p->rows < 0 || p->cols < 0 || p->rows > kMaxRows || p->cols > kMaxPacked) return bad(n + ": rows must be >= 0 and <= 2^30, cols >= 0 and <= 2^20");
  if (p->pitch < p->cols || p->pitch > kMaxQPitch || p->pitch % 16) return bad(n + ": pitch must be a multiple of 16, >= cols and <= 2^22");
  if (p->rows == 0) return ZERO_OK;
  if (!p->scale) return bad(n + ": null address of the scales");
  if ((uintptr_t)p->scale % 4) return bad(n + ": scales not aligned to their elements");
  if (p->cols == 0) return ZERO_OK;
  if (!p->q) return bad(n + ": null address");
  if ((uintptr_t)p->q % 16) return bad(n + ": q must be 16-byte aligned");
  return ZERO_OK;
}
// Results must not share memory with what is read, nor with each other.
zero_status_t apart(const Span& out, const Span& in, const char* a, const char* b) {
  return meet(out, in) ? bad(std::string(a) + " shares memory with " + b) : ZERO_OK;
}

zs::MatArg arg(const zero_matrix_t& a) { return {a.data, a.rows > 1 ? a.pitch : a.cols, a.dtype}; }
zs::PackArg arg(const zero_packed_t& p) { return {p.q, p.scale, p.pitch, p.rule}; }

zero_status_t check_workspace(void* workspace, int64_t capacity, int64_t need, const Span* used, int n_used) {
  if (need == 0) return ZERO_OK;
  if (!workspace) return bad("workspace must be non-null");
  if ((uintptr_t)workspace & 255u) return bad("workspace must be 256-byte aligned");
  if (capacity < need) return bad("workspace_capacity " + std::to_string(capacity) + " < " + std::to_string(need) + " bytes needed");
  const Span ws = {(uint64_t)(uintptr_t)workspace, 1, need, need};
  for (int i = 0; i < n_used; ++i)
    if (meet(ws, used[i])) return bad("the workspace shares memory with a matrix of the call");
  return ZERO_OK;
}

// A launch has fewer than 2^32 threads, here in blocks of at most 512, two for each tile.
zero_status_t check_tiles(const zs::ProductPlan& p) {
  return p.tiles_i * p.tiles_j * p.splits < (int64_t)1 << 22 ? ZERO_OK : bad("a result of 2^22 tiles or more");
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

#define ZS_TRY(expr)                                \
  do {                                              \
    const zero_status_t try_status_ = (expr);       \
    if (try_status_ != ZERO_OK) return try_status_; \
  } while (0)

zero_status_t write(const zero_matrix_t* x, const zero_packed_t* p, void* stream) {
  ZS_TRY(check(x, "x"));
  ZS_TRY(check(p, "p"));
  if (x->rows != p->rows || x->cols != p->cols) return bad("x and p must have the same size");
  ZS_TRY(apart(span(*p), span(*x), "p", "x"));
  ZS_TRY(apart(scales(*p), span(*x), "p's scales", "x"));
  ZS_TRY(apart(scales(*p), span(*p), "p's scales", "its q"));
  if (p->rows == 0) return ZERO_OK;
  return done("write kernel", zs::launch_write(arg(*x), arg(*p), p->rows, p->cols, static_cast<hipStream_t>(stream)));
}

zero_status_t read(const zero_packed_t* p, const zero_matrix_t* out, void* stream) {
  ZS_TRY(check(p, "p"));
  ZS_TRY(check(out, "out"));
  if (out->rows != p->rows || out->cols != p->cols) return bad("p and out must have the same size");
  ZS_TRY(apart(span(*out), span(*p), "out", "p"));
  ZS_TRY(apart(span(*out), scales(*p), "out", "p's scales"));
  if (p->rows * p->cols == 0) return ZERO_OK;
  return done("read kernel", zs::launch_read(arg(*p), arg(*out), p->rows, p->cols, static_cast<hipStream_t>(stream)));
}

zero_status_t linear(const zero_packed_t* x, const zero_packed_t* w, const zero_matrix_t* bias, const zero_matrix_t* y,
                     void* workspace, int64_t capacity, void* stream) {
  ZS_TRY(check(x, "x"));
  ZS_TRY(check(w, "w"));
  ZS_TRY(check(y, "y"));
  if (bias) ZS_TRY(check(bias, "bias"));
  const int64_t m = x->rows, k = x->cols, n = w->rows;
  if (w->cols != k) return bad("x and w must have the same number of columns");
  if (k > kMaxSum) return bad("more than 131056 columns: their sum may leave 32 bits");
  if (y->rows != m || y->cols != n) return bad("y must be x's rows by w's rows");
  if (bias && (bias->rows != 1 || bias->cols != n)) return bad("bias must be one row of w's rows");
  Span used[6] = {span(*y), span(*x), scales(*x), span(*w), scales(*w), bias ? span(*bias) : Span{}};
  static const char* const names[6] = {"y", "x", "x's scales", "w", "w's scales", "bias"};
  for (int i = 1; i < 6; ++i) ZS_TRY(apart(used[0], used[i], "y", names[i]));
  if (m * n == 0) return ZERO_OK;
  const zs::ProductPlan p = zs::plan_linear(m, k, n);
  ZS_TRY(check_tiles(p));
  ZS_TRY(check_workspace(workspace, capacity, p.ws_bytes, used, 6));
  zs::LinearArgs a{};
  a.x = arg(*x);
  a.w = arg(*w);
  a.y = arg(*y);
  if (bias) a.bias = arg(*bias);
  a.m = m;
  a.n = n;
  a.k = k;
  a.n4 = (n + 3) / 4 * 4;
  a.part = p.ws_bytes ? static_cast<int32_t*>(workspace) : nullptr;
  return done("linear kernel", zs::launch_linear(a, p, static_cast<hipStream_t>(stream)));
}

// Weight gradient (trans) or input gradient: c [ni][nj] from dy and the packed rows q [nc][nj].
zero_status_t grad(const zero_matrix_t* dy, const zero_packed_t* q, const zero_matrix_t* c, const zero_matrix_t* db, bool trans,
                   int32_t accumulate, void* workspace, int64_t capacity, void* stream) {
  const char* const cn = trans ? "dw" : "dx";
  const char* const qn = trans ? "x" : "w";
  ZS_TRY(check(dy, "dy"));
  ZS_TRY(check(q, qn));
  ZS_TRY(check(c, cn));
  if (db) ZS_TRY(check(db, "db"));
  if (dy->dtype == ZERO_F32) return bad("dy must be ZERO_F16 or ZERO_BF16");
  const int64_t ni = trans ? dy->cols : dy->rows, nc = trans ? dy->rows : dy->cols, nj = q->cols;
  if (q->rows != nc) return bad(trans ? "dy and x must have the same number of rows" : "dy must have as many columns as w has rows");
  if (c->rows != ni || c->cols != nj) return bad(trans ? "dw must be dy's columns by x's columns" : "dx must be dy's rows by w's columns");
  if (db && (db->rows != 1 || db->cols != ni)) return bad("db must be one row of dy's columns");
  Span used[5] = {span(*c), span(*dy), span(*q), scales(*q), db ? span(*db) : Span{}};
  static const char* const names[5] = {"", "dy", "the packed rows", "their scales", "db"};
  for (int i = 1; i < 5; ++i) ZS_TRY(apart(used[0], used[i], cn, names[i]));
  if (db)
    for (int i = 1; i < 4; ++i) ZS_TRY(apart(used[4], used[i], "db", names[i]));
  if (ni == 0 || (nj == 0 && !db)) return ZERO_OK;
  const zs::ProductPlan p = zs::plan_grad(ni, nj, nc);
  const zs::ColumnsPlan cp = zs::plan_columns(nc, ni);
  ZS_TRY(check_tiles(p));
  const int64_t need = up256(p.ws_bytes) + (db ? up256(cp.ws_bytes) : 0);
  ZS_TRY(check_workspace(workspace, capacity, need, used, 5));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (nj > 0) {
    zs::GradArgs g{};
    g.a = arg(*dy);
    g.c = arg(*c);
    g.q = arg(*q);
    g.ni = ni;
    g.nj = nj;
    g.nc = nc;
    g.accumulate = accumulate != 0;
    g.nj4 = (nj + 3) / 4 * 4;
    g.part = p.ws_bytes ? static_cast<float*>(workspace) : nullptr;
    ZS_TRY(done(trans ? "weight gradient kernel" : "input gradient kernel", zs::launch_grad(g, trans, p, st)));
  }
  if (db) {
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(p.ws_bytes));
    ZS_TRY(done("bias gradient kernel", zs::launch_columns(arg(*dy), nc, ni, arg(*db), accumulate != 0, part, cp, st)));
  }
  return ZERO_OK;
}

zero_status_t check_act(int32_t kind) {
  return kind == ZERO_ACT_GELU || kind == ZERO_ACT_SILU ? ZERO_OK : bad("kind must be ZERO_ACT_GELU or ZERO_ACT_SILU");
}

zero_status_t act(int32_t kind, int32_t gated, const zero_matrix_t* x, const zero_packed_t* xp, const zero_matrix_t* y,
                  const zero_packed_t* yp, void* stream) {
  ZS_TRY(check_act(kind));
  ZS_TRY(check(x, "x"));
  if (!xp && !y && !yp) return bad("no result asked for");
  if (gated && x->cols % 2) return bad("x: a gated function takes an even number of columns");
  const int64_t m = x->rows, n = gated ? x->cols / 2 : x->cols;
  Span out[5] = {};
  static const char* const names[5] = {"xp", "xp's scales", "y", "yp", "yp's scales"};
  if (xp) {
    ZS_TRY(check(xp, "xp"));
    if (xp->rows != m || xp->cols != x->cols) return bad("xp must have x's size");
    out[0] = span(*xp);
    out[1] = scales(*xp);
  }
  if (y) {
    ZS_TRY(check(y, "y"));
    if (y->rows != m || y->cols != n) return bad("y must be x's rows by the function's columns");
    out[2] = span(*y);
  }
  if (yp) {
    ZS_TRY(check(yp, "yp"));
    if (yp->rows != m || yp->cols != n) return bad("yp must be x's rows by the function's columns");
    out[3] = span(*yp);
    out[4] = scales(*yp);
  }
  for (int i = 0; i < 5; ++i) {
    ZS_TRY(apart(out[i], span(*x), names[i], "x"));
    for (int j = 0; j < i; ++j) ZS_TRY(apart(out[i], out[j], names[i], names[j]));
  }
  if (m == 0 || (n == 0 && !xp && !yp)) return ZERO_OK;
  zs::PackArg none{};
  none.rule = ZERO_SCALE_POW2;
  return done("activation kernel",
              zs::launch_act(kind, gated != 0, arg(*x), xp ? arg(*xp) : none, y ? arg(*y) : zs::MatArg{}, yp ? arg(*yp) : none, m,
                             n, static_cast<hipStream_t>(stream)));
}

zero_status_t act_grad(int32_t kind, int32_t gated, const zero_packed_t* xp, const zero_matrix_t* dy, const zero_matrix_t* dx,
                       void* stream) {
  ZS_TRY(check_act(kind));
  ZS_TRY(check(xp, "xp"));
  ZS_TRY(check(dy, "dy"));
  ZS_TRY(check(dx, "dx"));
  if (gated && xp->cols % 2) return bad("xp: a gated function takes an even number of columns");
  const int64_t m = xp->rows, n = gated ? xp->cols / 2 : xp->cols;
  if (dy->rows != m || dy->cols != n) return bad("dy must be xp's rows by the function's columns");
  if (dx->rows != m || dx->cols != xp->cols) return bad("dx must have xp's size");
  ZS_TRY(apart(span(*dx), span(*xp), "dx", "xp"));
  ZS_TRY(apart(span(*dx), scales(*xp), "dx", "xp's scales"));
  const bool same = !gated && dx->data == dy->data && dx->dtype == dy->dtype && (m <= 1 || dx->pitch == dy->pitch);
  if (!same) ZS_TRY(apart(span(*dx), span(*dy), "dx", "dy"));
  if (m * n == 0) return ZERO_OK;
  return done("activation gradient kernel",
              zs::launch_act_grad(kind, gated != 0, arg(*xp), arg(*dy), arg(*dx), m, n, static_cast<hipStream_t>(stream)));
}

// No exception leaves the C ABI (messages are strings).
template <class F>
zero_status_t guarded(F fn) {
  try {
    return fn();
  } catch (const std::exception& e) {
    return set_error(ZERO_ENOMEM, std::string("host resources: ") + e.what());
  }
}

}  // namespace

extern "C" {

zero_status_t zero_packed_write(const zero_matrix_t* x, const zero_packed_t* p, void* stream) {
  return guarded([&] { return write(x, p, stream); });
}
zero_status_t zero_packed_read(const zero_packed_t* p, const zero_matrix_t* out, void* stream) {
  return guarded([&] { return read(p, out, stream); });
}

zero_status_t zero_packed_workspace(int32_t call, int64_t m, int64_t k, int64_t n, int64_t* bytes) {
  return guarded([&] {
    if (!bytes) return bad("null output");
    if (m < 0 || k < 0 || n < 0 || m > kMaxRows || n > kMaxRows || k > kMaxPacked)
      return bad("m and n must be >= 0 and <= 2^30, k >= 0 and <= 2^20");
    if (call == ZERO_PACKED_LINEAR) {
      *bytes = m * n ? zs::plan_linear(m, k, n).ws_bytes : 0;
    } else if (call == ZERO_PACKED_WEIGHT_GRAD) {
      *bytes = n ? up256(k ? zs::plan_grad(n, k, m).ws_bytes : 0) + up256(zs::plan_columns(m, n).ws_bytes) : 0;
    } else if (call == ZERO_PACKED_INPUT_GRAD) {
      *bytes = m * k ? up256(zs::plan_grad(m, k, n).ws_bytes) : 0;
    } else {
      return bad("call must be ZERO_PACKED_LINEAR, ZERO_PACKED_WEIGHT_GRAD or ZERO_PACKED_INPUT_GRAD");
    }
    return ZERO_OK;
  });
}

zero_status_t zero_packed_linear(const zero_packed_t* x, const zero_packed_t* w, const zero_matrix_t* bias,
                                 const zero_matrix_t* y, void* workspace, int64_t workspace_capacity, void* stream) {
  return guarded([&] { return linear(x, w, bias, y, workspace, workspace_capacity, stream); });
}
zero_status_t zero_packed_weight_grad(const zero_matrix_t* dy, const zero_packed_t* x, const zero_matrix_t* dw,
                                      const zero_matrix_t* db, int32_t accumulate, void* workspace,
                                      int64_t workspace_capacity, void* stream) {
  return guarded([&] { return grad(dy, x, dw, db, true, accumulate, workspace, workspace_capacity, stream); });
}
zero_status_t zero_packed_input_grad(const zero_matrix_t* dy, const zero_packed_t* w, const zero_matrix_t* dx,
                                     int32_t accumulate, void* workspace, int64_t workspace_capacity, void* stream) {
  return guarded([&] { return grad(dy, w, dx, nullptr, false, accumulate, workspace, workspace_capacity, stream); });
}
zero_status_t zero_packed_act(int32_t kind, int32_t gated, const zero_matrix_t* x, const zero_packed_t* xp,
                              const zero_matrix_t* y, const zero_packed_t* yp, void* stream) {
  return guarded([&] { return act(kind, gated, x, xp, y, yp, stream); });
}
zero_status_t zero_packed_act_grad(int32_t kind, int32_t gated, const zero_packed_t* xp, const zero_matrix_t* dy,
                                   const zero_matrix_t* dx, void* stream) {
  return guarded([&] { return act_grad(kind, gated, xp, dy, dx, stream); });
}

}  // extern "C"
