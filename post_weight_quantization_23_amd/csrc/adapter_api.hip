// C ABI of the packed products for many tokens and of the low-rank adapters
// (declared in include/gptq_adapter.h).  As in gptq_api.hip every argument is
// validated on the host before anything is enqueued.
#include <utility>

#include "../../include/gptq_adapter.h"
#include "adapter.hpp"
#include "api.hpp"

using namespace gptq::api;

namespace {

constexpr int64_t kMaxCols = int64_t(1) << 30;
constexpr int64_t kMaxDepth = (int64_t(1) << 22) - 64;   // rows of the layer in the input gradient
constexpr int64_t kMaxAdapters = int64_t(1) << 20;

int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }

// Pieces of a workspace, each 256-byte aligned.
struct Carve {
  char* at;
  template <class T>
  T* take(int64_t bytes) {
    T* p = reinterpret_cast<T*>(at);
    at += align256(bytes);
    return p;
  }
};

// Sizes that every call shares; keeps products of them inside 63 bits.
gptq_status check_sizes(const char* fn, int64_t n, int64_t r, int64_t c, int64_t c_unit) {
  if (n < 0 || r < 0 || c < 0) return fail(GPTQ_EINVAL, fn, "negative size");
  if (n > kMaxRows || r > kMaxRows || c > kMaxCols) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (c == 0 || c % c_unit != 0)
    return fail(GPTQ_ESHAPE, fn, c_unit == 32 ? "c must be a positive multiple of 32" : "c must be a positive multiple of 8");
  return GPTQ_OK;
}

gptq_status check_rank(const char* fn, int64_t m, int64_t rank) {
  if (m < 1) return fail(GPTQ_EINVAL, fn, "n_adapters must be positive");
  if (m > kMaxAdapters) return fail(GPTQ_EUNSUPPORTED, fn, "too many adapters");
  if (rank < 8 || rank > 128 || rank % 8 != 0) return fail(GPTQ_EUNSUPPORTED, fn, "rank must be a multiple of 8 in 8 .. 128");
  return GPTQ_OK;
}

gptq_status check_adapters(const char* fn, const void* A, const void* B, const int32_t* index, const float* alpha) {
  if (!A || !B) return fail(GPTQ_EINVAL, fn, "A or B is NULL");
  if (!aligned(A, 16) || !aligned(B, 16)) return fail(GPTQ_EALIGN, fn, "A and B must be 16-byte aligned");
  if (!aligned(index, 4) || !aligned(alpha, 4)) return fail(GPTQ_EALIGN, fn, "misaligned index or alpha");
  return GPTQ_OK;
}

gptq::Adapters adapters(const void* A, const void* B, int64_t m, int64_t rank, const int32_t* index, const float* alpha) {
  gptq::Adapters ad{};
  if (A) {
    ad.A = static_cast<const uint16_t*>(A);
    ad.B = static_cast<const uint16_t*>(B);
    ad.alpha = alpha;
    ad.index = index;
    ad.m = (int)m;
    ad.rank = (int)rank;
  }
  return ad;
}

gptq_status check_packed(const char* fn, const uint32_t* packed, int64_t c, int bits, int64_t ld_words, const float* scales,
                         const int32_t* zeros, int64_t ld_groups, int64_t groupsize, const int32_t* perm) {
  if (bits != 3 && bits != 4) return fail(GPTQ_EUNSUPPORTED, fn, "bits must be 3 or 4");
  const bool grouped = groupsize > 0 && groupsize < c;
  if (grouped && groupsize % 32 != 0) return fail(GPTQ_EUNSUPPORTED, fn, "groupsize must be a multiple of 32");
  if (ld_words < c / 32 * bits) return fail(GPTQ_ESHAPE, fn, "ld_words < c * bits / 32");
  if (ld_groups < (grouped ? (c + groupsize - 1) / groupsize : 1)) return fail(GPTQ_ESHAPE, fn, "ld_groups < number of groups");
  if (!packed || !scales || !zeros) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  if (bits == 4 && (!aligned(packed, 16) || ld_words % 4 != 0))
    return fail(GPTQ_EALIGN, fn, "4-bit words need a 16-byte aligned base and ld_words % 4 == 0");
  if (!aligned(packed, 4) || !aligned(scales, 4) || !aligned(zeros, 4) || !aligned(perm, 4))
    return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  return GPTQ_OK;
}

gptq::PackedLayer layer(const uint32_t* packed, int64_t r, int64_t c, int bits, int64_t ld_words, const float* scales,
                        const int32_t* zeros, int64_t ld_groups, int64_t groupsize, const int32_t* perm) {
  gptq::PackedLayer w;
  w.words = packed;
  w.ldw = ld_words;
  w.scales = scales;
  w.zeros = zeros;
  w.ldg = ld_groups;
  w.perm = perm;
  w.bits = bits;
  w.r = (int)r;
  w.c = (int)c;
  w.cpg = groupsize > 0 && groupsize < c ? (int)(groupsize / 32) : (int)(c / 32);
  w.shift = w.cpg == c / 32 ? 31 : ((w.cpg & (w.cpg - 1)) == 0 ? __builtin_ctz((unsigned)w.cpg) : -1);
  return w;
}

// `out` against one input: -1 extent too large, 1 overlap, 0 apart.
int clash(const void* out, int64_t eo, const void* in, int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
  const int64_t e = extent_bytes(rows, ld, cols, elem);
  if (eo < 0 || e < 0) return -1;
  return eo > 0 && e > 0 && overlaps(out, eo, in, e) ? 1 : 0;
}

gptq_status check_clash(const char* fn, int c) {
  if (c < 0) return fail(GPTQ_EUNSUPPORTED, fn, "matrix extent exceeds 2^63 bytes");
  if (c > 0) return fail(GPTQ_EINVAL, fn, "an output overlaps an input");
  return GPTQ_OK;
}

// An output against the arrays of a packed layer, and against adapters.
gptq_status check_clashes(const char* fn, const void* out, int64_t eo, const uint32_t* packed, int64_t r, int64_t c, int bits,
                          int64_t ld_words, const float* scales, const int32_t* zeros, int64_t ld_groups, int64_t groupsize,
                          const int32_t* perm) {
  const int64_t groups = groupsize > 0 && groupsize < c ? (c + groupsize - 1) / groupsize : 1;
  if (gptq_status st = check_clash(fn, clash(out, eo, packed, r, ld_words, c / 32 * bits, 4))) return st;
  if (gptq_status st = check_clash(fn, clash(out, eo, scales, r, ld_groups, groups, 4))) return st;
  if (gptq_status st = check_clash(fn, clash(out, eo, zeros, r, ld_groups, groups, 4))) return st;
  return perm ? check_clash(fn, clash(out, eo, perm, 1, c, c, 4)) : GPTQ_OK;
}

gptq_status check_clashes(const char* fn, const void* out, int64_t eo, int64_t n, int64_t r, int64_t c, const void* A, const void* B,
                          int64_t m, int64_t rank, const int32_t* index, const float* alpha) {
  if (gptq_status st = check_clash(fn, clash(out, eo, A, m * rank, c, c, 2))) return st;
  if (gptq_status st = check_clash(fn, clash(out, eo, B, m * r, rank, rank, 2))) return st;
  if (index)
    if (gptq_status st = check_clash(fn, clash(out, eo, index, 1, n, n, 4))) return st;
  return alpha ? check_clash(fn, clash(out, eo, alpha, 1, m, m, 4)) : GPTQ_OK;
}

// What the packed product's kernels prepare: the gathered activations of a few
// tokens of an act-order layer, or what many tokens need.
int64_t forward_bytes(int64_t n, int64_t r, int64_t c, bool perm, int yt) {
  if (gptq::packed_tiles(n, r, c)) return gptq::packed_tiles_bytes(n, r, c, yt);
  return perm ? align256(n * c * 2) : 0;
}

// The rank values of n tokens of d features, with what computing them takes.
int64_t low_bytes(int64_t n, int64_t d, int64_t rank) { return rank > 0 ? align256(gptq::adapter_down_floats(n, d, rank) * 4) : 0; }
int64_t order_bytes(int64_t n, int64_t rank) { return rank > 0 ? align256(n * 4) : 0; }

// A padded copy of n rows of d values for the rank values' product, where the
// rows themselves will not do.
int64_t rows_bytes(int64_t n, int64_t d, int64_t rank) { return rank > 0 ? align256(n * gptq::gemm16_depth(d) * 2) : 0; }

// Lays out what the adapters need (g's other pieces with it) and sets their order.
void prepare(gptq::PrepareArgs& g, gptq::Adapters& ad, int32_t* order, hipStream_t s) {
  g.ad = ad;
  if (gptq::adapters_want_order(g.n, ad.m, ad.index)) g.order = order;
  gptq::launch_prepare_adapters(g, s);
  ad.order = g.order;
}

// One side of the rank values: rows of X or their padded copy.
gptq::DownProblem down_problem(const void* X, int64_t n, int64_t d, int64_t ldx, const uint16_t* A, int64_t lda, float* S,
                               uint16_t* rows, int m, gptq::PadArgs& pad) {
  gptq::DownProblem q{};
  q.X = static_cast<const uint16_t*>(X);
  q.d = d;
  q.ldx = ldx;
  if (!gptq::adapter_rows_direct(X, n, d, ldx, m)) {
    pad.src = q.X;
    pad.d = d;
    pad.lds = ldx;
    pad.dst = rows;
    q.X = rows;
    q.d = q.ldx = gptq::gemm16_depth(d);
  }
  q.A = A;
  q.lda = lda;
  q.S = S;
  return q;
}

// Whether every launch that a call makes at these sizes is one that the
// dispatcher takes.  up: outputs that a launch of its own adds the adapters to (0: the
// product does).
bool low_fits(int64_t n, int64_t d, int64_t rank, int64_t m, int64_t up, int64_t turned_r, int64_t turned_c) {
  if (rank == 0) return true;
  return gptq::prepare_adapters_fits(n, m, rank, turned_r, turned_c, gptq::gemm16_depth(d)) &&
         gptq::adapter_down_fits(n, (int)m, rank, 1) && gptq::adapter_up_fits(n, (int)m, up);
}

bool forward_fits(int64_t n, int64_t r, int64_t c, int yt, int64_t rank, int64_t m) {
  const bool tiles = gptq::packed_tiles(n, r, c);
  if (!(tiles ? gptq::packed_tiles_fits(n, r, c, yt) : gptq::packed_rows_fits(n, r, c))) return false;
  return low_fits(n, c, rank, m, tiles && !gptq::packed_tiles_copies(n, yt) ? r : 0, 0, 0);
}

bool backward_fits(int64_t n, int64_t r, int64_t c, int64_t rank, int64_t m) {
  return gptq::packed_backward_fits(n, r, c) && low_fits(n, r, rank, m, 0, pad8(r), c);
}

bool grads_fit(int64_t n, int64_t r, int64_t c, int64_t rank, int64_t m) {
  return gptq::prepare_adapters_fits(n, m, rank, pad8(r), c, gptq::gemm16_depth(r) + gptq::gemm16_depth(c)) &&
         gptq::adapter_down_fits(n, (int)m, rank, 2) && gptq::adapter_up_fits(n, (int)m, c) &&
         gptq::adapter_grads_fits(n, (int)m, r, c, (int)rank);
}

// The input gradient's dequantized weights and padded rows of dY.
int64_t backward_bytes(int64_t n, int64_t r, int64_t c, int xt, int ot) {
  const int64_t depth = gptq::gemm16_depth(r);
  return align256(gptq::gemm16_terms(xt, ot) * c * depth * 2) + align256(n * depth * 2) +
         align256(gptq::gemm16_part_floats(n, c, depth, xt, ot) * 4);
}

struct GradSizes {
  int64_t places, part, lists, terms, total;
};

GradSizes grad_sizes(int64_t n, int64_t r, int64_t c, int64_t m, int64_t rank) {
  GradSizes z;
  z.part = align256(gptq::adapter_grad_floats(n, (int)m, r, c, (int)rank) * 4);
  z.places = gptq::list_places(n, m);
  z.lists = align256(z.places * 4) + align256((m + 1) * 4) + align256(m * 4);
  z.terms = align256(3 * ((rank + 15) / 16 * 16) * z.places * 2);
  z.total = order_bytes(n, rank) + rows_bytes(n, r, rank) + rows_bytes(n, c, rank) + align256(m * rank * pad8(r) * 2) + align256(m * c * rank * 2) + low_bytes(n, c, rank) + low_bytes(n, r, rank) + z.lists + 2 * z.terms + z.part;
  return z;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ packed product
gptq_status gptq_packed_linear_workspace_size(int64_t n, int64_t r, int64_t c, gptq_dtype yt, int64_t rank, int has_perm,
                                              size_t* bytes) {
  const char* fn = "gptq_packed_linear_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (has_perm != 0 && has_perm != 1) return fail(GPTQ_EINVAL, fn, "has_perm must be 0 or 1");
  if (!valid_dtype(yt)) return fail(GPTQ_EINVAL, fn, "yt must be a gptq_dtype value");
  if (gptq_status st = check_sizes(fn, n, r, c, 32)) return st;
  if (rank != 0)
    if (gptq_status st = check_rank(fn, 1, rank)) return st;
  if (!forward_fits(n, r, c, (int)yt, rank, rank != 0)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  *bytes = (size_t)(forward_bytes(n, r, c, has_perm != 0, (int)yt) + low_bytes(n, c, rank) + order_bytes(n, rank) + rows_bytes(n, c, rank));
  return ok();
}

gptq_status gptq_packed_linear(const void* X, gptq_dtype xt, int64_t n, int64_t ldx, const uint32_t* packed, int64_t r,
                               int64_t c, int bits, int64_t ld_words, const float* scales, const int32_t* zeros,
                               int64_t ld_groups, int64_t groupsize, const int32_t* perm, const void* A, const void* B,
                               int64_t m, int64_t rank, const int32_t* index, const float* alpha, void* Y, gptq_dtype yt,
                               int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "gptq_packed_linear";
  const bool low = A || B;
  if (!low) m = rank = 0;
  if (gptq_status st = check_sizes(fn, n, r, c, 32)) return st;
  if (!valid_dtype(xt) || !valid_dtype(yt)) return fail(GPTQ_EINVAL, fn, "xt and yt must be gptq_dtype values");
  if (xt == GPTQ_F32) return fail(GPTQ_EDTYPE, fn, "X must be GPTQ_BF16 or GPTQ_F16");
  if (yt != GPTQ_F32 && yt != xt) return fail(GPTQ_EDTYPE, fn, "Y must be GPTQ_F32 or of X's type");
  if (low)
    if (gptq_status st = check_rank(fn, m, rank)) return st;
  if (!forward_fits(n, r, c, (int)yt, rank, m)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (n == 0 || r == 0) return ok();
  if (low)
    if (gptq_status st = check_adapters(fn, A, B, index, alpha)) return st;
  if (gptq_status st = check_packed(fn, packed, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm)) return st;
  if (ldx < c || ldy < r) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
  if (!X || !Y) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  if (perm ? !aligned(X, 2) : (!aligned(X, 16) || ldx % 8 != 0)) return fail(GPTQ_EALIGN, fn, "rows of X must start on 16 bytes");
  if (!aligned(Y, elem_size(yt))) return fail(GPTQ_EALIGN, fn, "Y misaligned");
  const int64_t ey = extent_bytes(n, ldy, r, (int64_t)elem_size(yt));
  if (gptq_status st = check_clash(fn, clash(Y, ey, X, n, ldx, c, 2))) return st;
  if (gptq_status st = check_clashes(fn, Y, ey, packed, r, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm)) return st;
  if (low)
    if (gptq_status st = check_clashes(fn, Y, ey, n, r, c, A, B, m, rank, index, alpha)) return st;
  if (gptq_status st = need_ws(fn, ws, ws_bytes, forward_bytes(n, r, c, perm != nullptr, (int)yt) + low_bytes(n, c, rank) + order_bytes(n, rank) + rows_bytes(n, c, rank))) return st;
  Carve carve{static_cast<char*>(ws)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const gptq::PackedLayer w = layer(packed, r, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm);
  gptq::Adapters ad = adapters(A, B, m, rank, index, alpha);
  const int xi = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  const int yi = yt == GPTQ_F32 ? 0 : xi;
  float* S = nullptr;
  if (low) {
    S = carve.take<float>(low_bytes(n, c, rank));
    int32_t* order = carve.take<int32_t>(n * 4);
    uint16_t* rows = carve.take<uint16_t>(rows_bytes(n, c, rank));
    gptq::PrepareArgs g{};
    g.n = n;
    gptq::DownArgs d{};
    d.n = n;
    d.p[0] = down_problem(X, n, c, ldx, ad.A, c, S, rows, ad.m, g.pad[0]);
    prepare(g, ad, order, s);
    d.ad = ad;
    gptq::launch_adapter_down(d, xi, true, s);
  }
  if (gptq::packed_tiles(n, r, c)) {
    gptq::launch_packed_tiles(X, xi, n, ldx, w, ad, S, Y, yi, ldy, carve.at, s);
  } else {
    const void* xp = X;
    if (perm) {
      uint16_t* g = carve.take<uint16_t>(n * c * 2);
      gptq::launch_gather_columns(X, n, c, ldx, perm, g, s);
      xp = g;
    }
    gptq::launch_packed_linear(xp, xi, n, perm ? c : ldx, w, ad, S, Y, yi, ldy, s);
  }
  return check_launch(fn);
}

// ------------------------------------------------------------------ its input gradient
gptq_status gptq_packed_linear_backward_workspace_size(int64_t n, int64_t r, int64_t c, gptq_dtype xt, gptq_dtype ot, int64_t m,
                                                       int64_t rank, size_t* bytes) {
  const char* fn = "gptq_packed_linear_backward_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (!valid_dtype(xt) || !valid_dtype(ot)) return fail(GPTQ_EINVAL, fn, "xt and ot must be gptq_dtype values");
  if (xt == GPTQ_F32 || (ot != GPTQ_F32 && ot != xt)) return fail(GPTQ_EDTYPE, fn, "xt must be 16-bit, ot GPTQ_F32 or xt");
  if (gptq_status st = check_sizes(fn, n, r, c, 32)) return st;
  if (m != 0 || rank != 0)
    if (gptq_status st = check_rank(fn, m, rank)) return st;
  if (!backward_fits(n, r, c, rank, m)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (r > kMaxDepth) return fail(GPTQ_EUNSUPPORTED, fn, "r too large");
  *bytes = (size_t)(backward_bytes(n, r, c, (int)xt, (int)ot) + align256(m * c * rank * 2) +
                    align256(m * rank * pad8(r) * 2) + low_bytes(n, r, rank) + order_bytes(n, rank) + rows_bytes(n, r, rank));
  return ok();
}

gptq_status gptq_packed_linear_backward(const void* dY, gptq_dtype xt, int64_t n, int64_t ldy, const uint32_t* packed,
                                        int64_t r, int64_t c, int bits, int64_t ld_words, const float* scales,
                                        const int32_t* zeros, int64_t ld_groups, int64_t groupsize, const int32_t* perm,
                                        const void* A, const void* B, int64_t m, int64_t rank, const int32_t* index,
                                        const float* alpha, void* dX, gptq_dtype ot, int64_t ldx, void* ws, size_t ws_bytes,
                                        void* stream) {
  const char* fn = "gptq_packed_linear_backward";
  const bool low = A || B;
  if (!low) m = rank = 0;
  if (gptq_status st = check_sizes(fn, n, r, c, 32)) return st;
  if (!valid_dtype(xt) || !valid_dtype(ot)) return fail(GPTQ_EINVAL, fn, "xt and ot must be gptq_dtype values");
  if (xt == GPTQ_F32) return fail(GPTQ_EDTYPE, fn, "dY must be GPTQ_BF16 or GPTQ_F16");
  if (ot != GPTQ_F32 && ot != xt) return fail(GPTQ_EDTYPE, fn, "dX must be GPTQ_F32 or of dY's type");
  if (low) {
    if (gptq_status st = check_rank(fn, m, rank)) return st;
    if (gptq_status st = check_adapters(fn, A, B, index, alpha)) return st;
  }
  if (!backward_fits(n, r, c, rank, m)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (r == 0) return fail(GPTQ_ESHAPE, fn, "r must be positive");
  if (r > kMaxDepth) return fail(GPTQ_EUNSUPPORTED, fn, "r too large");
  if (n == 0) return ok();
  if (gptq_status st = check_packed(fn, packed, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm)) return st;
  if (ldx < c || ldy < r) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
  if (!dY || !dX) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  if (!aligned(dY, 2) || !aligned(dX, elem_size(ot))) return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  const int64_t ex = extent_bytes(n, ldx, c, (int64_t)elem_size(ot));
  if (gptq_status st = check_clash(fn, clash(dX, ex, dY, n, ldy, r, 2))) return st;
  if (gptq_status st = check_clashes(fn, dX, ex, packed, r, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm)) return st;
  if (low)
    if (gptq_status st = check_clashes(fn, dX, ex, n, r, c, A, B, m, rank, index, alpha)) return st;
  const int terms = gptq::gemm16_terms((int)xt, (int)ot);
  const int64_t need = backward_bytes(n, r, c, (int)xt, (int)ot) + align256(m * c * rank * 2) + align256(m * rank * pad8(r) * 2) + low_bytes(n, r, rank) +
                       order_bytes(n, rank) + rows_bytes(n, r, rank);
  if (gptq_status st = need_ws(fn, ws, ws_bytes, need)) return st;
  Carve carve{static_cast<char*>(ws)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const gptq::PackedLayer w = layer(packed, r, c, bits, ld_words, scales, zeros, ld_groups, groupsize, perm);
  gptq::Adapters ad = adapters(A, B, m, rank, index, alpha);
  const int xi = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  uint16_t* Wt = carve.take<uint16_t>(terms * c * gptq::gemm16_depth(r) * 2);
  uint16_t* rows = carve.take<uint16_t>(n * gptq::gemm16_depth(r) * 2);
  float* part = carve.take<float>(gptq::gemm16_part_floats(n, c, gptq::gemm16_depth(r), (int)xt, (int)ot) * 4);
  uint16_t* At = nullptr;
  float* T = nullptr;
  if (low) {
    At = carve.take<uint16_t>(m * c * rank * 2);
    uint16_t* Bt = carve.take<uint16_t>(m * rank * pad8(r) * 2);
    T = carve.take<float>(low_bytes(n, r, rank));
    int32_t* order = carve.take<int32_t>(n * 4);
    uint16_t* padded = carve.take<uint16_t>(rows_bytes(n, r, rank));
    gptq::PrepareArgs g{};
    g.n = n;
    g.turn[0] = {ad.A, rank, c, At, rank, 0};
    g.turn[1] = {ad.B, r, rank, Bt, pad8(r), 0};
    gptq::DownArgs d{};
    d.n = n;
    d.p[0] = down_problem(dY, n, r, ldy, Bt, pad8(r), T, padded, ad.m, g.pad[0]);
    prepare(g, ad, order, s);
    d.ad = ad;
    gptq::launch_adapter_down(d, xi, true, s);
  }
  gptq::launch_packed_backward(dY, xi, n, ldy, w, ad, At, T, dX, ot == GPTQ_F32 ? 0 : xi, ldx, Wt, rows, part, s);
  return check_launch(fn);
}

// ------------------------------------------------------------------ adapters beside any projection
gptq_status gptq_adapter_add_workspace_size(int64_t n, int64_t c, int64_t rank, size_t* bytes) {
  const char* fn = "gptq_adapter_add_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (gptq_status st = check_sizes(fn, n, 0, c, 8)) return st;
  if (gptq_status st = check_rank(fn, 1, rank)) return st;
  *bytes = (size_t)(low_bytes(n, c, rank) + order_bytes(n, rank) + rows_bytes(n, c, rank));
  return ok();
}

gptq_status gptq_adapter_add(const void* X, gptq_dtype xt, int64_t n, int64_t c, int64_t ldx, const void* A, const void* B,
                             int64_t m, int64_t rank, int64_t r, const int32_t* index, const float* alpha, const void* Y,
                             gptq_dtype yt, int64_t ldy, void* out, int64_t ldo, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "gptq_adapter_add";
  if (gptq_status st = check_sizes(fn, n, r, c, 8)) return st;
  if (!valid_dtype(xt) || !valid_dtype(yt)) return fail(GPTQ_EINVAL, fn, "xt and yt must be gptq_dtype values");
  if (xt == GPTQ_F32) return fail(GPTQ_EDTYPE, fn, "X must be GPTQ_BF16 or GPTQ_F16");
  if (yt != GPTQ_F32 && yt != xt) return fail(GPTQ_EDTYPE, fn, "Y must be GPTQ_F32 or of X's type");
  if (gptq_status st = check_rank(fn, m, rank)) return st;
  if (!low_fits(n, c, rank, m, r, 0, 0)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (n == 0 || r == 0) return ok();
  if (gptq_status st = check_adapters(fn, A, B, index, alpha)) return st;
  if (ldx < c || ldy < r || ldo < r) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
  if (!X || !Y || !out) return fail(GPTQ_EINVAL, fn, "a required pointer is NULL");
  const int64_t el = (int64_t)elem_size(yt);
  if (!aligned(X, 2) || !aligned(Y, el) || !aligned(out, el)) return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  const int64_t eo = extent_bytes(n, ldo, r, el);
  if (gptq_status st = check_clash(fn, clash(out, eo, X, n, ldx, c, 2))) return st;
  if (gptq_status st = check_clashes(fn, out, eo, n, r, c, A, B, m, rank, index, alpha)) return st;
  if (!(out == Y && ldo == ldy))
    if (gptq_status st = check_clash(fn, clash(out, eo, Y, n, ldy, r, el))) return st;
  if (gptq_status st = need_ws(fn, ws, ws_bytes, low_bytes(n, c, rank) + order_bytes(n, rank) + rows_bytes(n, c, rank))) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  gptq::Adapters ad = adapters(A, B, m, rank, index, alpha);
  const int xi = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  Carve carve{static_cast<char*>(ws)};
  float* S = carve.take<float>(low_bytes(n, c, rank));
  int32_t* order = carve.take<int32_t>(n * 4);
  uint16_t* rows = carve.take<uint16_t>(rows_bytes(n, c, rank));
  gptq::PrepareArgs g{};
  g.n = n;
  gptq::DownArgs d{};
  d.n = n;
  d.p[0] = down_problem(X, n, c, ldx, ad.A, c, S, rows, ad.m, g.pad[0]);
  prepare(g, ad, order, s);
  d.ad = ad;
  gptq::launch_adapter_down(d, xi, true, s);
  gptq::UpArgs u{};
  u.S = S; u.n = n; u.rows = r; u.ad = ad; u.B = ad.B; u.base = Y; u.ldb = ldy; u.out = out; u.ldo = ldo;
  gptq::launch_adapter_up(u, xi, yt == GPTQ_F32 ? 0 : xi, s);
  return check_launch(fn);
}

// ------------------------------------------------------------------ their gradients
gptq_status gptq_adapter_backward_workspace_size(int64_t n, int64_t r, int64_t c, int64_t m, int64_t rank, size_t* bytes) {
  const char* fn = "gptq_adapter_backward_workspace_size";
  if (!bytes) return fail(GPTQ_EINVAL, fn, "bytes is NULL");
  if (gptq_status st = check_sizes(fn, n, r, c, 8)) return st;
  if (gptq_status st = check_rank(fn, m, rank)) return st;
  if (!grads_fit(n, r, c, rank, m)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  *bytes = (size_t)grad_sizes(n, r, c, m, rank).total;
  return ok();
}

gptq_status gptq_adapter_backward(const void* dY, int64_t ldy, const void* X, int64_t ldx, gptq_dtype xt, int64_t n,
                                  int64_t r, int64_t c, const void* A, const void* B, int64_t m, int64_t rank,
                                  const int32_t* index, const float* alpha, float* gA, float* gB, const void* base, void* dX,
                                  gptq_dtype ot, int64_t ldd, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "gptq_adapter_backward";
  if (gptq_status st = check_sizes(fn, n, r, c, 8)) return st;
  if (!valid_dtype(xt) || !valid_dtype(ot)) return fail(GPTQ_EINVAL, fn, "xt and ot must be gptq_dtype values");
  if (xt == GPTQ_F32) return fail(GPTQ_EDTYPE, fn, "dY and X must be GPTQ_BF16 or GPTQ_F16");
  if (ot != GPTQ_F32 && ot != xt) return fail(GPTQ_EDTYPE, fn, "dX must be GPTQ_F32 or of X's type");
  if (r == 0) return fail(GPTQ_ESHAPE, fn, "r must be positive");
  if (gptq_status st = check_rank(fn, m, rank)) return st;
  if (gptq_status st = check_adapters(fn, A, B, index, alpha)) return st;
  if (!grads_fit(n, r, c, rank, m)) return fail(GPTQ_EUNSUPPORTED, fn, "size too large");
  if (ldy < r || ldx < c || (dX && ldd < c)) return fail(GPTQ_ESHAPE, fn, "leading dimension too small");
  if (!gA || !gB) return fail(GPTQ_EINVAL, fn, "gA or gB is NULL");
  if (n > 0 && (!dY || !X)) return fail(GPTQ_EINVAL, fn, "dY or X is NULL");
  if (base && !dX) return fail(GPTQ_EINVAL, fn, "base without dX");
  const int64_t el = (int64_t)elem_size(ot);
  if (!aligned(dY, 2) || !aligned(X, 2) || !aligned(dX, el) || !aligned(base, el))
    return fail(GPTQ_EALIGN, fn, "misaligned pointer");
  if (!aligned(gA, 16) || !aligned(gB, 16)) return fail(GPTQ_EALIGN, fn, "gA and gB must be 16-byte aligned");
  const int64_t ea = extent_bytes(m * rank, c, c, 4), eb = extent_bytes(m * r, rank, rank, 4);
  const int64_t ed = dX ? extent_bytes(n, ldd, c, el) : 0;
  struct { const void* p; int64_t rows, ld, cols, elem; } in[] = {
      {dY, n, ldy, r, 2}, {X, n, ldx, c, 2}};
  for (const auto& v : in)
    for (const auto& o : {std::pair<const void*, int64_t>{gA, ea}, {gB, eb}, {dX, ed}})
      if (o.first)
        if (gptq_status st = check_clash(fn, clash(o.first, o.second, v.p, v.rows, v.ld, v.cols, v.elem))) return st;
  for (const auto& o : {std::pair<const void*, int64_t>{gA, ea}, {gB, eb}, {dX, ed}})
    if (o.first)
      if (gptq_status st = check_clashes(fn, o.first, o.second, n, r, c, A, B, m, rank, index, alpha)) return st;
  if (overlaps(gA, ea, gB, eb) || (dX && ed > 0 && (overlaps(dX, ed, gA, ea) || overlaps(dX, ed, gB, eb))))
    return fail(GPTQ_EINVAL, fn, "outputs overlap");
  if (base && base != dX)
    for (const auto& o : {std::pair<const void*, int64_t>{gA, ea}, {gB, eb}, {dX, ed}})
      if (gptq_status st = check_clash(fn, clash(o.first, o.second, base, n, ldd, c, el))) return st;
  const GradSizes z = grad_sizes(n, r, c, m, rank);
  if (gptq_status st = need_ws(fn, ws, ws_bytes, z.total)) return st;
  Carve carve{static_cast<char*>(ws)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  gptq::Adapters ad = adapters(A, B, m, rank, index, alpha);
  const int xi = xt == GPTQ_BF16 ? gptq::kBF16 : gptq::kF16;
  int32_t* by_adapter = carve.take<int32_t>(n * 4);
  uint16_t* rows_y = carve.take<uint16_t>(rows_bytes(n, r, rank));
  uint16_t* rows_x = carve.take<uint16_t>(rows_bytes(n, c, rank));
  uint16_t* Bt = carve.take<uint16_t>(m * rank * pad8(r) * 2);
  uint16_t* At = carve.take<uint16_t>(m * c * rank * 2);
  float* S = carve.take<float>(low_bytes(n, c, rank));
  float* T = carve.take<float>(low_bytes(n, r, rank));
  gptq::PrepareArgs g{};
  g.n = n;
  g.list = carve.take<int32_t>(z.places * 4);
  g.start = carve.take<int32_t>((m + 1) * 4);
  g.count = carve.take<int32_t>(m * 4);
  uint16_t* Sx = carve.take<uint16_t>(z.terms);
  uint16_t* Tx = carve.take<uint16_t>(z.terms);
  float* part = carve.take<float>(z.part);
  g.turn[0] = {ad.B, r, rank, Bt, pad8(r), 0};
  if (dX) g.turn[1] = {ad.A, rank, c, At, rank, 0};
  gptq::DownArgs d{};
  d.n = n;
  d.p[0] = down_problem(dY, n, r, ldy, Bt, pad8(r), T, rows_y, ad.m, g.pad[0]);
  d.p[1] = down_problem(X, n, c, ldx, ad.A, c, S, rows_x, ad.m, g.pad[1]);
  // the gradients read dY and X eight columns at a time in any case
  gptq::GradArgs w{};
  auto side = [&](gptq::GradProblem& q, const void* Z, int64_t cols, int64_t ldz, uint16_t* rows, gptq::PadArgs& pad,
                  const uint16_t* terms, int up) {
    q.cols = cols;
    q.up = up;
    q.terms = terms;
    if (aligned(Z, 16) && ldz % 8 == 0 && cols % 8 == 0) {
      q.Z = static_cast<const uint16_t*>(Z);
      q.ldz = ldz;
      q.width = cols;
    } else {
      pad.src = static_cast<const uint16_t*>(Z);
      pad.d = cols;
      pad.lds = ldz;
      pad.dst = rows;
      q.Z = rows;
      q.ldz = q.width = gptq::gemm16_depth(cols);
    }
  };
  side(w.p[0], X, c, ldx, rows_x, g.pad[1], Tx, 0);
  side(w.p[1], dY, r, ldy, rows_y, g.pad[0], Sx, 1);
  prepare(g, ad, by_adapter, s);
  w.ad = d.ad = ad;
  if (n > 0) gptq::launch_adapter_down(d, xi, false, s);
  gptq::TermsArgs v{};
  v.ad = ad;
  v.n = n;
  v.places = z.places;
  v.list = w.list = g.list;
  v.start = w.start = g.start;
  w.count = g.count;
  v.S[0] = T;
  v.S[1] = S;
  v.splits[0] = gptq::adapter_down_parts(n, ad.m, d.p[0].d);
  v.splits[1] = gptq::adapter_down_parts(n, ad.m, d.p[1].d);
  v.keep[0] = dX != nullptr;
  v.terms[0] = Tx;
  v.terms[1] = Sx;
  gptq::launch_adapter_grads(v, w, xi, gA, gB, part, s);
  if (dX && n > 0) {
    gptq::UpArgs u{};
    u.S = T; u.n = n; u.rows = c; u.ad = ad; u.B = At; u.base = base; u.ldb = ldd; u.out = dX; u.ldo = ldd;
    gptq::launch_adapter_up(u, xi, ot == GPTQ_F32 ? 0 : xi, s);
  }
  return check_launch(fn);
}

}  // extern "C"
