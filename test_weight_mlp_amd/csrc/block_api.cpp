// C ABI of the rest of the block: the norm and the projections.  Nothing is
// launched and nothing is written unless every argument checks out; nothing here
// allocates or throws.
#include <cmath>

#include "../../include/ipttt.h"
#include "block.h"

using ipttt::GemmArgs;
using ipttt::Rows;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 26) - 4;  // 2^20 tiles of 64 rows, which the plans count in int
constexpr int64_t kMaxStride = int64_t(1) << 22;
constexpr int64_t kMaxNorm = 16384;                   // elements of a row in one workgroup's registers
constexpr int64_t kMaxLinear = int64_t(1) << 20;
// Tiles of 128 x 128 of a product: there are four times as many of 64 x 64, and the plans
// and walks count those, and the parts of cut ones, in int.
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 1;

#define IPTTT_TRY(e)                         \
  do {                                       \
    const ipttt_status s_ = (e);             \
    if (s_ != IPTTT_OK) return s_;           \
  } while (0)

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
ipttt_status hip_status(hipError_t e) { return e == hipSuccess ? IPTTT_OK : IPTTT_ERR_HIP; }

// A [rows, columns] tensor; `may_miss`: it may be NULL.
ipttt_status view(const ipttt_rows* t, int64_t rows, int64_t columns, bool may_miss, Rows* v) {
  *v = Rows{nullptr, 0};
  if (t == nullptr) return may_miss ? IPTTT_OK : IPTTT_ERR_NULL;
  if (t->data == nullptr) return IPTTT_ERR_NULL;
  if (!aligned(t->data, 16)) return IPTTT_ERR_ALIGN;
  const int64_t ld = rows == 1 ? columns : t->row_stride;
  if (ld < columns || ld % 8 != 0 || ld > kMaxStride) return IPTTT_ERR_SHAPE;
  *v = Rows{t->data, ld};
  return IPTTT_OK;
}

ipttt_status vectors(const void* a, const void* b) { return aligned(a, 16) && aligned(b, 16) ? IPTTT_OK : IPTTT_ERR_ALIGN; }

// An output over an input has to be that input, row for row.
ipttt_status in_place(const Rows& out, const Rows& in) {
  return out.p != nullptr && out.p == in.p && out.ld != in.ld ? IPTTT_ERR_ARG : IPTTT_OK;
}
// An output that may not be an input.
ipttt_status apart(const void* out, const void* in) { return out != nullptr && out == in ? IPTTT_ERR_ARG : IPTTT_OK; }

ipttt_status workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return IPTTT_OK;
  if (ws == nullptr || have < need) return IPTTT_ERR_WORKSPACE;
  return aligned(ws, 256) ? IPTTT_OK : IPTTT_ERR_ALIGN;
}

// --------------------------------------------------------------------- norm

ipttt_status check_norm(const ipttt_norm_problem* p) {
  if (p == nullptr) return IPTTT_ERR_NULL;
  if (p->dtype != IPTTT_F32 && p->dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (p->rows < 1 || p->rows > kMaxRows) return IPTTT_ERR_SHAPE;
  if (p->dim < 8 || p->dim > kMaxNorm || p->dim % 8 != 0) return IPTTT_ERR_SHAPE;
  if (p->kind != IPTTT_NORM_RMS && p->kind != IPTTT_NORM_LAYER) return IPTTT_ERR_ARG;
  return std::isfinite(p->eps) && p->eps >= 0.0f ? IPTTT_OK : IPTTT_ERR_ARG;
}

ipttt::NormArgs norm_args(const ipttt_norm_problem* p) {
  ipttt::NormArgs a{};
  a.dtype = p->dtype;
  a.dim = (int)p->dim;
  a.rows = p->rows;
  a.center = p->kind == IPTTT_NORM_LAYER;
  a.eps = p->eps;
  return a;
}

size_t norm_bytes(const ipttt_norm_problem* p) {
  return align256((size_t)ipttt::norm_parts(p->dtype, p->rows, (int)p->dim) * 2 * (size_t)p->dim * sizeof(float));
}

// ------------------------------------------------------------------- linear

ipttt_status check_linear(const ipttt_linear_problem* p) {
  if (p == nullptr) return IPTTT_ERR_NULL;
  if (p->dtype != IPTTT_F32 && p->dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (p->grad_dtype != IPTTT_F32 && p->grad_dtype != p->dtype) return IPTTT_ERR_DTYPE;
  if (p->rows < 1 || p->rows > kMaxRows) return IPTTT_ERR_SHAPE;
  for (const int64_t n : {p->in_dim, p->out_dim})
    if (n < 8 || n > kMaxLinear || n % 8 != 0) return IPTTT_ERR_SHAPE;
  if (p->act < IPTTT_ACT_NONE || p->act > IPTTT_ACT_GELU) return IPTTT_ERR_ARG;
  // the products' tiles of 128 x 128
  const int64_t tm = (p->rows + 127) / 128, tk = (p->in_dim + 127) / 128, tn = (p->out_dim + 127) / 128;
  if (tm * tn > kMaxTiles || tm * tk > kMaxTiles || tn * tk > kMaxTiles) return IPTTT_ERR_SHAPE;
  return IPTTT_OK;
}

GemmArgs forward_args(const ipttt_linear_problem* p) {
  GemmArgs g{};
  g.dtype = p->dtype;
  g.M = p->rows;
  g.N = p->out_dim;
  g.K = p->in_dim;
  g.act = p->act;
  return g;
}

// dx = dp W and dW = dp^T x.
GemmArgs dx_args(const ipttt_linear_problem* p) {
  GemmArgs g{};
  g.dtype = p->dtype;
  g.M = p->rows;
  g.N = p->in_dim;
  g.K = p->out_dim;
  g.b_kmaj = 1;
  return g;
}
GemmArgs dw_args(const ipttt_linear_problem* p) {
  GemmArgs g{};
  g.dtype = p->dtype;
  g.M = p->out_dim;
  g.N = p->in_dim;
  g.K = p->rows;
  g.a_kmaj = g.b_kmaj = 1;
  g.c_f32 = p->grad_dtype == IPTTT_F32;
  return g;
}

// The backward's workspace: dp (where there is an activation) | partial column
// sums | partial products of dx | of dW.
struct BackwardLayout {
  size_t dp, db, part_x, part_w, total;
};
BackwardLayout backward_layout(const ipttt_linear_problem* p) {
  const size_t e = p->dtype == IPTTT_BF16 ? 2 : 4;
  BackwardLayout l;
  l.dp = 0;
  l.db = l.dp + (p->act != IPTTT_ACT_NONE ? align256((size_t)p->rows * (size_t)p->out_dim * e) : 0);
  l.part_x = l.db + align256((size_t)ipttt::act_grad_parts(p->rows, p->out_dim) * (size_t)p->out_dim * sizeof(float));
  size_t x, w;
  ipttt::gemm_pair_workspace(dx_args(p), dw_args(p), &x, &w);
  l.part_w = l.part_x + align256(x);
  l.total = l.part_w + align256(w);
  return l;
}

}  // namespace

extern "C" {

ipttt_status ipttt_norm(const ipttt_norm_problem* p, const ipttt_rows* x, const void* w, const void* b,
                        const ipttt_rows* y, void* stream) {
  IPTTT_TRY(check_norm(p));
  ipttt::NormArgs a = norm_args(p);
  IPTTT_TRY(view(x, p->rows, p->dim, false, &a.x));
  IPTTT_TRY(view(y, p->rows, p->dim, false, &a.y));
  IPTTT_TRY(vectors(w, b));
  IPTTT_TRY(in_place(a.y, a.x));
  IPTTT_TRY(apart(a.y.p, w));
  IPTTT_TRY(apart(a.y.p, b));
  a.w = w;
  a.b = b;
  (void)hipGetLastError();
  return hip_status(ipttt::launch_norm(a, static_cast<hipStream_t>(stream)));
}

size_t ipttt_norm_backward_workspace_bytes(const ipttt_norm_problem* p) {
  return check_norm(p) == IPTTT_OK ? norm_bytes(p) : 0;
}

ipttt_status ipttt_norm_backward(const ipttt_norm_problem* p, const ipttt_rows* x, const void* w,
                                 const ipttt_rows* dy, const ipttt_rows* dres, const ipttt_rows* dx, float* dw,
                                 float* db, void* ws, size_t ws_bytes, void* stream) {
  IPTTT_TRY(check_norm(p));
  ipttt::NormArgs a = norm_args(p);
  IPTTT_TRY(view(x, p->rows, p->dim, false, &a.x));
  IPTTT_TRY(view(dy, p->rows, p->dim, false, &a.dy));
  IPTTT_TRY(view(dres, p->rows, p->dim, true, &a.dres));
  IPTTT_TRY(view(dx, p->rows, p->dim, false, &a.dx));
  IPTTT_TRY(vectors(w, nullptr));
  IPTTT_TRY(vectors(dw, db));
  IPTTT_TRY(in_place(a.dx, a.x));
  IPTTT_TRY(in_place(a.dx, a.dy));
  IPTTT_TRY(in_place(a.dx, a.dres));
  IPTTT_TRY(apart(a.dx.p, w));
  IPTTT_TRY(apart(dw, db));
  for (const void* in : {static_cast<const void*>(a.x.p), w, static_cast<const void*>(a.dy.p),
                         static_cast<const void*>(a.dres.p), static_cast<const void*>(a.dx.p)}) {
    IPTTT_TRY(apart(dw, in));
    IPTTT_TRY(apart(db, in));
  }
  if (dw != nullptr || db != nullptr) IPTTT_TRY(workspace(ws, ws_bytes, norm_bytes(p)));
  a.w = w;
  a.dw = dw;
  a.db = db;
  a.part = static_cast<float*>(ws);
  (void)hipGetLastError();
  return hip_status(ipttt::launch_norm_backward(a, static_cast<hipStream_t>(stream)));
}

size_t ipttt_linear_workspace_bytes(const ipttt_linear_problem* p) {
  return check_linear(p) == IPTTT_OK ? ipttt::gemm_workspace(forward_args(p)) : 0;
}

ipttt_status ipttt_linear(const ipttt_linear_problem* p, const ipttt_rows* x, const void* W, const void* b,
                          const ipttt_rows* res, const ipttt_rows* y, const ipttt_rows* pre, void* ws,
                          size_t ws_bytes, void* stream) {
  IPTTT_TRY(check_linear(p));
  GemmArgs g = forward_args(p);
  IPTTT_TRY(view(x, p->rows, p->in_dim, false, &g.a));
  if (W == nullptr) return IPTTT_ERR_NULL;
  IPTTT_TRY(view(res, p->rows, p->out_dim, true, &g.res));
  IPTTT_TRY(view(y, p->rows, p->out_dim, false, &g.c));
  IPTTT_TRY(view(pre, p->rows, p->out_dim, true, &g.pre));
  IPTTT_TRY(vectors(W, b));
  IPTTT_TRY(in_place(g.c, g.res));
  for (const void* out : {g.c.p, g.pre.p})
    for (const void* in : {static_cast<const void*>(g.a.p), W, b}) IPTTT_TRY(apart(out, in));
  IPTTT_TRY(apart(g.pre.p, g.res.p));
  IPTTT_TRY(apart(g.pre.p, g.c.p));
  IPTTT_TRY(workspace(ws, ws_bytes, ipttt::gemm_workspace(g)));
  g.b = Rows{const_cast<void*>(W), p->in_dim};
  g.bias = b;
  g.part = static_cast<float*>(ws);
  (void)hipGetLastError();
  return hip_status(ipttt::launch_gemm(g, static_cast<hipStream_t>(stream)));
}

size_t ipttt_linear_backward_workspace_bytes(const ipttt_linear_problem* p) {
  return check_linear(p) == IPTTT_OK ? backward_layout(p).total : 0;
}

ipttt_status ipttt_linear_backward(const ipttt_linear_problem* p, const ipttt_rows* x, const void* W,
                                   const ipttt_rows* pre, const ipttt_rows* dy, const ipttt_rows* dx, void* dW,
                                   float* db, void* ws, size_t ws_bytes, void* stream) {
  IPTTT_TRY(check_linear(p));
  const bool act = p->act != IPTTT_ACT_NONE;
  Rows xv, prev, dyv, dxv;
  IPTTT_TRY(view(x, p->rows, p->in_dim, false, &xv));
  if (W == nullptr) return IPTTT_ERR_NULL;
  IPTTT_TRY(view(act ? pre : nullptr, p->rows, p->out_dim, !act, &prev));
  IPTTT_TRY(view(dy, p->rows, p->out_dim, false, &dyv));
  IPTTT_TRY(view(dx, p->rows, p->in_dim, true, &dxv));
  IPTTT_TRY(vectors(W, nullptr));
  IPTTT_TRY(vectors(dW, db));
  for (const void* out : {dxv.p, dW, static_cast<void*>(db)}) {
    for (const void* in : {static_cast<const void*>(xv.p), W, static_cast<const void*>(prev.p),
                           static_cast<const void*>(dyv.p)})
      IPTTT_TRY(apart(out, in));
  }
  IPTTT_TRY(apart(dW, dxv.p));
  IPTTT_TRY(apart(db, dxv.p));
  IPTTT_TRY(apart(db, dW));
  const BackwardLayout l = backward_layout(p);
  IPTTT_TRY(workspace(ws, ws_bytes, l.total));
  char* base = static_cast<char*>(ws);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  Rows dp = dyv;
  if (act) dp = Rows{base + l.dp, p->out_dim};
  if ((act && (dxv.p != nullptr || dW != nullptr)) || db != nullptr) {
    ipttt::ActGradArgs a{};
    a.dtype = p->dtype;
    a.act = p->act;
    a.rows = p->rows;
    a.dim = p->out_dim;
    a.dy = dyv;
    a.pre = prev;
    if (act) a.dp = dp;
    a.db = db;
    a.part = reinterpret_cast<float*>(base + l.db);
    IPTTT_TRY(hip_status(ipttt::launch_act_grad(a, st)));
  }
  GemmArgs gx = dx_args(p), gw = dw_args(p);
  gx.a = dp;
  gx.b = Rows{const_cast<void*>(W), p->in_dim};
  gx.c = dxv;
  gx.part = reinterpret_cast<float*>(base + l.part_x);
  gw.a = dp;
  gw.b = xv;
  gw.c = Rows{dW, p->in_dim};
  gw.part = reinterpret_cast<float*>(base + l.part_w);
  return hip_status(ipttt::launch_gemm_pair(gx, gw, st));
}

}  // extern "C"
