// C ABI of the loss over a vocabulary, its gradients and the orthogonalised adapter
// updates (declared in include/gptq_train.h).  Every argument is validated on the
// host before anything is enqueued.
#include <cmath>

#include "../../include/gptq_train.h"
#include "api.hpp"
#include "loss.hpp"
#include "orthogonal.hpp"

using namespace gptq::api;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 22) - 64;
constexpr int64_t kMaxMatrices = int64_t(1) << 20;

// Pieces of a workspace, each 256-byte aligned.
struct Carve {
  char* base;
  int64_t used;
  template <class T>
  T* take(int64_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += align256(count * (int64_t)sizeof(T));
    return p;
  }
};

// Arrays of a call; an output may overlap nothing else.
struct Span {
  const void* p;
  int64_t rows, ld, cols, elem;
  bool out;
};

template <int N>
gptq_status check_apart(const char* fn, const Span (&s)[N]) {
  int64_t bytes[N];
  for (int i = 0; i < N; ++i) {
    bytes[i] = s[i].p ? extent_bytes(s[i].rows, s[i].ld, s[i].cols, s[i].elem) : 0;
    if (bytes[i] < 0) return fail(GPTQ_EUNSUPPORTED, fn, "matrix extent exceeds 2^63 bytes");
  }
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if ((s[i].out || s[j].out) && bytes[i] > 0 && bytes[j] > 0 && overlaps(s[i].p, bytes[i], s[j].p, bytes[j]))
        return fail(GPTQ_EINVAL, fn, "an output overlaps another argument");
  return GPTQ_OK;
}

gptq_status check_loss_sizes(const char* fn, int64_t n, int64_t d, int64_t vocab, bool grad) {
  if (n < 0 || d < 0 || vocab < 0) return fail(GPTQ_EINVAL, fn, "negative size");
  if (vocab == 0) return fail(GPTQ_ESHAPE, fn, "vocab must be positive");
  if (d == 0 || d % 8 != 0) return fail(GPTQ_ESHAPE, fn, "d must be a positive multiple of 8");
  if (n > kMaxRows || vocab > kMaxRows || d > kMaxDim || !gptq::loss_fits(n, vocab, d, grad))
    return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  return GPTQ_OK;
}

gptq_status check_loss(const char* fn, const void* X, gptq_dtype xt, int64_t n, int64_t d, int64_t ldx, const void* W, int64_t ldw,
                       const int64_t* target) {
  if (!valid_dtype(xt)) return fail(GPTQ_EINVAL, fn, "xt must be a gptq_dtype value");
  if (xt == GPTQ_F32) return fail(GPTQ_EDTYPE, fn, "X and W must be GPTQ_BF16 or GPTQ_F16");
  if (n > 0) {
    if (ldx < d) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
    if (!X || !target) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
    if (!aligned(X, 2) || !aligned(target, 8)) return fail(GPTQ_EALIGN, fn, "misaligned pointer");
    if (ldw < d) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
    if (ldw >= (int64_t(1) << 22)) return fail(GPTQ_EUNSUPPORTED, fn, "ldw must be below 2^22");
    if (!W) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
    if (!aligned(W, 16) || ldw % 8 != 0) return fail(GPTQ_EALIGN, fn, "rows of W must start on 16 bytes");
  }
  return GPTQ_OK;
}

gptq::Kept take_kept(Carve& c, int64_t n, bool grad) {
  gptq::Kept k{};
  k.token = c.take<int32_t>(n);
  k.place_of = c.take<int32_t>(n);
  k.col = c.take<int32_t>(n);
  k.count = c.take<int32_t>(1);
  k.down = c.take<float>(1);
  k.splits = c.take<int32_t>(1);
  if (grad) {
    k.lse = c.take<float>(n);
    k.grad = c.take<float>(n);
    k.rest = c.take<float>(n);
  }
  return k;
}

struct LossBuffers {
  gptq::Kept k;
  uint16_t* rows;
  float2* part;
  float* at_target;
};
LossBuffers take_loss(Carve& c, int64_t n, int64_t d, int64_t vocab) {
  LossBuffers b;
  b.k = take_kept(c, n, false);
  b.rows = c.take<uint16_t>(n * gptq::gemm16_depth(d));
  b.part = c.take<float2>(n * gptq::loss_tiles(n, vocab));
  b.at_target = c.take<float>(n);
  return b;
}

struct GradBuffers {
  gptq::Kept k;
  uint16_t *rows, *P;
  float* part;
  int64_t piece, ldp;
};
GradBuffers take_grad(Carve& c, int64_t n, int64_t d, int64_t vocab, bool want_dx) {
  GradBuffers b;
  b.piece = gptq::loss_piece(n, vocab);
  b.ldp = gptq::gemm16_depth(b.piece);
  b.k = take_kept(c, n, true);
  b.rows = c.take<uint16_t>(n * gptq::gemm16_depth(d));
  b.P = c.take<uint16_t>(n * b.ldp);
  b.part = c.take<float>(want_dx ? gptq::grad_x_part_floats(n, d, b.piece < vocab) : 0);
  return b;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ loss
gptq_status gptq_linear_cross_entropy_workspace_size(int64_t n, int64_t d, int64_t vocab, size_t* bytes) {
  const char* fn = "gptq_linear_cross_entropy_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (gptq_status st = check_loss_sizes(fn, n, d, vocab, false)) return st;
  Carve c{nullptr, 0};
  if (n > 0) take_loss(c, n, d, vocab);
  *bytes = (size_t)c.used;
  return ok();
}

gptq_status gptq_linear_cross_entropy(const void* X, gptq_dtype xt, int64_t n, int64_t d, int64_t ldx, const void* W, int64_t vocab,
                                      int64_t ldw, const int64_t* target, float* loss, float* lse, void* ws, size_t ws_bytes,
                                      void* stream) {
  const char* fn = "gptq_linear_cross_entropy";
  if (gptq_status st = check_loss_sizes(fn, n, d, vocab, false)) return st;
  if (gptq_status st = check_loss(fn, X, xt, n, d, ldx, W, ldw, target)) return st;
  if (n == 0) return ok();
  if (!loss || !lse) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  if (!aligned(loss, 4) || !aligned(lse, 4)) return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  const Span spans[] = {{X, n, ldx, d, 2, false}, {W, vocab, ldw, d, 2, false}, {target, 1, n, n, 8, false},
                        {loss, 1, n, n, 4, true}, {lse, 1, n, n, 4, true}};
  if (gptq_status st = check_apart(fn, spans)) return st;
  Carve size{nullptr, 0};
  take_loss(size, n, d, vocab);
  if (gptq_status st = need_ws(fn, ws, ws_bytes, size.used)) return st;
  Carve c{static_cast<char*>(ws), 0};
  const LossBuffers b = take_loss(c, n, d, vocab);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int dt = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  gptq::LossArgs l{};
  l.W = static_cast<const uint16_t*>(W);
  l.ldw = ldw;
  l.vocab = l.width = vocab;
  l.n = n;
  l.d = d;
  l.part = b.part;
  l.at_target = b.at_target;
  if (gptq::loss_takes(X, n, d, ldx)) {
    l.rows = static_cast<const uint16_t*>(X);
    l.ldr = ldx;
    l.target = target;
  } else {
    gptq::KeepArgs k{};
    k.target = target;
    k.n = n;
    k.vocab = vocab;
    k.loss = loss;
    k.lse = lse;
    k.k = b.k;
    gptq::launch_keep(k, s);
    gptq::GatherArgs g{};
    g.X = static_cast<const uint16_t*>(X);
    g.n = n;
    g.d = d;
    g.ldx = ldx;
    g.kp = gptq::gemm16_depth(d);
    g.k = b.k;
    g.rows = b.rows;
    gptq::launch_gather_kept(g, s);
    l.rows = b.rows;
    l.ldr = g.kp;
    l.k = b.k;
  }
  gptq::launch_logits(l, dt, false, s);
  gptq::launch_loss_join(l, loss, lse, s);
  return check_launch(fn);
}

// ------------------------------------------------------------------ its gradients
gptq_status gptq_linear_cross_entropy_backward_workspace_size(int64_t n, int64_t d, int64_t vocab, int want_dx, int want_dw,
                                                              size_t* bytes) {
  const char* fn = "gptq_linear_cross_entropy_backward_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if ((want_dx != 0 && want_dx != 1) || (want_dw != 0 && want_dw != 1)) return fail(GPTQ_EINVAL, fn, "want_dx and want_dw must be 0 or 1");
  if (!want_dx && !want_dw) return fail(GPTQ_EINVAL, fn, "neither dX nor dW is wanted");
  if (gptq_status st = check_loss_sizes(fn, n, d, vocab, true)) return st;
  Carve c{nullptr, 0};
  take_grad(c, n, d, vocab, want_dx != 0);
  *bytes = (size_t)c.used;
  return ok();
}

gptq_status gptq_linear_cross_entropy_backward(const void* X, gptq_dtype xt, int64_t n, int64_t d, int64_t ldx, const void* W,
                                               int64_t vocab, int64_t ldw, const int64_t* target, const float* lse,
                                               const float* dloss, void* dX, int64_t lddx, void* dW, int64_t lddw, void* ws,
                                               size_t ws_bytes, void* stream) {
  const char* fn = "gptq_linear_cross_entropy_backward";
  if (gptq_status st = check_loss_sizes(fn, n, d, vocab, true)) return st;
  if (gptq_status st = check_loss(fn, X, xt, n, d, ldx, W, ldw, target)) return st;
  if (n == 0 && !dW) return ok();
  if (!dX && !dW) return fail(GPTQ_EINVAL, fn, "neither dX nor dW is given");
  if (n > 0 && !lse) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  if ((dX && lddx < d) || (dW && lddw < d)) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
  if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dX, 2) || !aligned(dW, 2)) return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  const Span spans[] = {{X, n, ldx, d, 2, false}, {W, n > 0 ? vocab : 0, ldw, d, 2, false}, {target, n > 0, n, n, 8, false},
                        {lse, n > 0, n, n, 4, false}, {dloss, n > 0, n, n, 4, false}, {dX, n, lddx, d, 2, true},
                        {dW, vocab, lddw, d, 2, true}};
  if (gptq_status st = check_apart(fn, spans)) return st;
  Carve size{nullptr, 0};
  take_grad(size, n, d, vocab, dX != nullptr);
  if (gptq_status st = need_ws(fn, ws, ws_bytes, size.used)) return st;
  Carve c{static_cast<char*>(ws), 0};
  const GradBuffers b = take_grad(c, n, d, vocab, dX != nullptr);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int dt = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  const int64_t kp = gptq::gemm16_depth(d);
  gptq::KeepArgs k{};
  k.target = target;
  k.n = n;
  k.vocab = vocab;
  k.grad = true;
  k.lse_in = lse;
  k.dloss = dloss;
  k.half = xt == GPTQ_F16;
  k.d = dX ? d : 0;
  k.width = b.piece;
  k.large = gptq::grad_x_large(n);
  k.k = b.k;
  gptq::launch_keep(k, s);
  gptq::GatherArgs g{};
  g.X = static_cast<const uint16_t*>(X);
  g.n = n;
  g.d = d;
  g.ldx = ldx;
  g.kp = kp;
  g.k = b.k;
  g.rows = b.rows;
  g.dX = static_cast<uint16_t*>(dX);
  g.ldd = lddx;
  if (n > 0) gptq::launch_gather_kept(g, s);
  gptq::LossArgs l{};
  l.ldw = ldw;
  l.vocab = vocab;
  l.n = n;
  l.d = d;
  l.rows = b.rows;
  l.ldr = kp;
  l.k = b.k;
  l.P = b.P;
  l.W = static_cast<const uint16_t*>(W);
  gptq::GradXArgs x{};
  x.P = b.P;
  x.ldw = ldw;
  x.n = n;
  x.d = d;
  x.k = b.k;
  x.W0 = static_cast<const uint16_t*>(W);
  x.pieces = b.piece < vocab;
  x.part = b.part;
  x.dX = static_cast<uint16_t*>(dX);
  x.ldd = lddx;
  x.vec = gptq::rows_on_16(dX, lddx, dt);
  gptq::GradWArgs w{};
  w.P = b.P;
  w.rows = b.rows;
  w.kp = kp;
  w.n = n;
  w.d = d;
  w.k = b.k;
  w.ldd = lddw;
  w.vec = gptq::rows_on_16(dW, lddw, dt);
  for (int64_t v0 = 0; v0 < vocab; v0 += b.piece) {
    const int64_t width = vocab - v0 < b.piece ? vocab - v0 : b.piece;
    const int64_t ldp = gptq::gemm16_depth(width);
    if (n > 0) {
      l.v0 = v0;
      l.width = width;
      l.ldp = ldp;
      gptq::launch_logits(l, dt, true, s);
    }
    if (n > 0 && dX) {
      x.W = static_cast<const uint16_t*>(W) + v0 * ldw;
      x.width = width;
      x.ldp = ldp;
      x.add = v0 > 0;
      gptq::launch_grad_x(x, dt, s);
    }
    if (dW) {
      w.v0 = v0;
      w.width = width;
      w.ldp = ldp;
      w.dW = static_cast<uint16_t*>(dW) + v0 * lddw;
      gptq::launch_grad_w(w, dt, s);
    }
  }
  if (n > 0 && dX) gptq::launch_join_x(x, dt, s);
  return check_launch(fn);
}

// ------------------------------------------------------------------ orthogonalised updates
namespace {

gptq_status check_ortho_sizes(const char* fn, int64_t m, int64_t rank, int64_t c, int64_t r, int steps) {
  if (m < 0 || rank < 0 || c < 0 || r < 0) return fail(GPTQ_EINVAL, fn, "negative size");
  if (steps < 1 || steps > 16) return fail(GPTQ_EUNSUPPORTED, fn, "steps must be 1 .. 16");
  if (rank == 0) return fail(GPTQ_ESHAPE, fn, "rank must be positive");
  if (c == 0 && r == 0) return fail(GPTQ_EINVAL, fn, "neither factor is wanted");
  if (m > kMaxMatrices || rank > kMaxRows || c > kMaxRows || r > kMaxRows) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  for (const int64_t other : {c, r}) {
    if (other == 0) continue;
    const int64_t p = rank < other ? rank : other, q = rank < other ? other : rank;
    if (p > gptq::kOrthoRank) return fail(GPTQ_EUNSUPPORTED, fn, "the shorter side of a matrix must be at most 128");
    if (!gptq::ortho_fits(m, q)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  }
  return GPTQ_OK;
}

// Longer sides of an adapter's matrices, together (0: not wanted).
int64_t long_sides(int64_t rank, int64_t c, int64_t r) { return (c > rank || c == 0 ? c : rank) + (r > rank || r == 0 ? r : rank); }

// The problem of m matrices of rows x cols; both: long_sides().
void take_ortho(Carve& ws, gptq::OrthoProblem& o, int64_t m, int64_t rows, int64_t cols, int64_t both) {
  o.rows = rows;
  o.cols = cols;
  o.tall = rows > cols;
  o.p = (int)(o.tall ? cols : rows);
  o.q = o.tall ? rows : cols;
  o.splits = gptq::ortho_splits(m, o.q, both);
  const int64_t tiles = gptq::ortho_tiles(o.p), pp = 16 * gptq::ortho_blocks(o.p);
  o.part = ws.take<double>(m * o.splits * tiles * 256);
  o.inv = ws.take<double>(m);
  o.wide = ws.take<double>(m * gptq::ortho_wide(o.p));
  o.R = o.wide;
  o.apart = gptq::ortho_wide(o.p);
  if (o.apart > 0) return;
  o.R = ws.take<double>(m * pp * pp);
  o.apart = pp * pp;
}

}  // namespace

gptq_status gptq_adapter_orthogonalize_workspace_size(int64_t m, int64_t rank, int64_t c, int64_t r, int steps, size_t* bytes) {
  const char* fn = "gptq_adapter_orthogonalize_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (gptq_status st = check_ortho_sizes(fn, m, rank, c, r, steps)) return st;
  Carve ws{nullptr, 0};
  gptq::OrthoProblem o{};
  if (c > 0) take_ortho(ws, o, m, rank, c, long_sides(rank, c, r));
  if (r > 0) take_ortho(ws, o, m, r, rank, long_sides(rank, c, r));
  *bytes = (size_t)ws.used;
  return ok();
}

gptq_status gptq_adapter_orthogonalize(const void* G_A, const void* G_B, gptq_dtype gt, int64_t m, int64_t rank, int64_t c, int64_t r,
                                       int steps, float a, float b, float c3, float eps, void* out_A, void* out_B, gptq_dtype ot,
                                       void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "gptq_adapter_orthogonalize";
  if (!G_A) c = 0;
  if (!G_B) r = 0;
  if (!valid_dtype(gt) || !valid_dtype(ot)) return fail(GPTQ_EINVAL, fn, "gt and ot must be gptq_dtype values");
  if (m == 0 && !G_A && !G_B) return ok();
  if (!G_A && !G_B) return fail(GPTQ_EINVAL, fn, "neither G_A nor G_B is given");
  if ((G_A && c == 0) || (G_B && r == 0)) return fail(GPTQ_ESHAPE, fn, "c and r must be positive");
  if (gptq_status st = check_ortho_sizes(fn, m, rank, c, r, steps)) return st;
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c3) || !std::isfinite(eps) || eps < 0)
    return fail(GPTQ_EINVAL, fn, "coefficients must be finite, eps finite and not negative");
  if (m == 0) return ok();
  if ((G_A && !out_A) || (G_B && !out_B)) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  const int64_t eg = (int64_t)elem_size(gt), eo = (int64_t)elem_size(ot);
  if (!aligned(G_A, eg) || !aligned(G_B, eg) || (G_A && !aligned(out_A, eo)) || (G_B && !aligned(out_B, eo)))
    return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  const Span spans[] = {{G_A, m * rank, c, c, eg, false}, {G_B, m * r, rank, rank, eg, false},
                        {G_A ? out_A : nullptr, m * rank, c, c, eo, true}, {G_B ? out_B : nullptr, m * r, rank, rank, eo, true}};
  if (gptq_status st = check_apart(fn, spans)) return st;
  gptq::OrthoArgs args{};
  for (int pass = 0; pass < 2; ++pass) {
    Carve carve{pass ? static_cast<char*>(ws) : nullptr, 0};
    int at = 0;
    if (G_A) {
      gptq::OrthoProblem& o = args.p[at++];
      o.G = G_A;
      o.out = out_A;
      take_ortho(carve, o, m, rank, c, long_sides(rank, c, r));
    }
    if (G_B) {
      gptq::OrthoProblem& o = args.p[at++];
      o.G = G_B;
      o.out = out_B;
      take_ortho(carve, o, m, r, rank, long_sides(rank, c, r));
    }
    if (pass == 0)
      if (gptq_status st = need_ws(fn, ws, ws_bytes, carve.used)) return st;
  }
  args.m = m;
  args.steps = steps;
  args.a = a;
  args.b = b;
  args.c = c3;
  args.eps = eps;
  gptq::launch_orthogonalize(args, (int)gt, (int)ot, reinterpret_cast<hipStream_t>(stream));
  return check_launch(fn);
}

}  // extern "C"
