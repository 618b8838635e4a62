// Launch interfaces of the loss over a vocabulary and its gradients (loss.hip,
// loss_tiles.hip; internal to the library).
#pragma once
#include "adapter.hpp"

namespace gptq {

// Tiles of logits, entries of the vocabulary x tokens.
enum LossShape { k256x256, k128x128, k128x64, k128x32, kFew };   // kFew: 32 entries, up to 64 tokens
LossShape loss_shape(int64_t n, int64_t vocab);
inline int64_t loss_entries(LossShape s) { return s == k256x256 ? 256 : s == kFew ? 32 : 128; }
// Up to as many tokens one or two tiles hold them all, and leaving tokens out
// saves little work: they are taken as they lie (forward).
constexpr int64_t kFewTokens = 256;

// The tokens that have a target, in order: place p is token token[p] with target
// col[p]; place_of[t] is token t's place or -1.  count: how many there are.
struct Kept {
  int32_t* token;
  int32_t* place_of;
  int32_t* col;
  float* lse;       // of each place (backward), as grad: dloss, for fp16 times 1 / *down
  float* grad;
  int32_t* count;
  float* down;      // what results are multiplied by (a power of two, 1 for bf16)
  float* rest;      // what rounding took from the target's entry of D (backward), for dX and dW
  int32_t* splits;  // parts of the contraction that dX is computed in
};

struct KeepArgs {
  const int64_t* target;
  int64_t n, vocab;
  float *loss, *lse;              // forward: zeroed where there is no target
  bool grad;                      // backward (also without tokens, and so without pointers)
  const float *lse_in, *dloss;    // ... (dloss null: 1)
  bool half;                      // fp16 gradients
  int64_t d, width;               // dX: columns, and entries of a piece
  bool large;                     // ... in tiles of 256 x 256
  Kept k;
};
void launch_keep(const KeepArgs& a, hipStream_t s);

// Rows of X that have a target, in their order, each kp values with zeros past d;
// dX (nullable): rows without one are zeroed.
struct GatherArgs {
  const uint16_t* X;
  int64_t n, d, ldx, kp;
  bool vec;
  Kept k;
  uint16_t* rows;
  uint16_t* dX;
  int64_t ldd;
  bool vec_dx;
};
void launch_gather_kept(GatherArgs a, hipStream_t s);

constexpr float kLog2e = 1.4426950408889634f;

// The largest of two sets of values and the sum of exponentials against it.  A set
// that holds nothing is (-inf, 0).
GPTQ_DEV float2 join_sums(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), r = m == -INFINITY ? 0.f : m;
  return float2{m, a.y * __builtin_amdgcn_exp2f((a.x - r) * kLog2e) + b.y * __builtin_amdgcn_exp2f((b.x - r) * kLog2e)};
}

// v += much x eight 16-bit values (on 16 bytes).
template <int DT>
GPTQ_DEV void add_row(const uint16_t* row, float much, float (&v)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(row);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __builtin_fmaf(much, f16_to_f32<DT>(w[e] & 0xFFFFu), v[2 * e]);
    v[2 * e + 1] = __builtin_fmaf(much, f16_to_f32<DT>(w[e] >> 16), v[2 * e + 1]);
  }
}

// Logits of every kept token in tiles: of each tile the
// largest and the sum of exponentials against it, and the target's logit.
struct LossArgs {
  const uint16_t* W;
  int64_t ldw, vocab, n, d;
  const uint16_t* rows;    // [n][ldr], on 16 bytes
  int64_t ldr;
  const int64_t* target;   // not null: all n tokens as they lie, k unused (forward)
  Kept k;
  float2* part;            // [tiles][n]
  float* at_target;        // [n]
  int64_t v0, width;       // gradients: entries v0 .. v0 + width - 1
  uint16_t* P;             // [n][ldp]: dloss (softmax - onehot)
  int64_t ldp;
};
void launch_logits(const LossArgs& a, int dt, bool grad, hipStream_t s);

constexpr int kJoinTokens = 16;   // of a workgroup of the join, where there are enough of them
void launch_loss_join(const LossArgs& a, float* loss, float* lse, hipStream_t s);

// dX[place] = P W over one piece of the vocabulary, in *k.splits fp32 parts (added
// to what earlier pieces left), and their sum; at once where one piece and part are all.
struct GradXArgs {
  const uint16_t* P;
  int64_t ldp, width;
  const uint16_t* W;       // the piece's rows
  int64_t ldw, n, d;
  Kept k;
  const uint16_t* W0;      // all of W
  bool pieces, add;        // there are several pieces; this one adds to parts of an earlier one
  float* part;             // [splits][kept][d]
  uint16_t* dX;
  int64_t ldd;
  bool vec;
};
void launch_grad_x(const GradXArgs& a, int dt, hipStream_t s);
void launch_join_x(const GradXArgs& a, int dt, hipStream_t s);

// dW rows of one piece of the vocabulary = P^T rows, and what rounding took from the targets' entries.
struct GradWArgs {
  const uint16_t* P;
  int64_t ldp, v0, width;
  const uint16_t* rows;
  int64_t kp, n, d;
  Kept k;
  uint16_t* dW;
  int64_t ldd;
  bool vec;
};
void launch_grad_w(const GradWArgs& a, int dt, hipStream_t s);

// dX in tiles of 256 x 256, else 128 x 128, and workspace of its parts.
bool grad_x_large(int64_t n);
int64_t grad_x_part_floats(int64_t n, int64_t d, bool pieces);
constexpr int kMostSplits = 16;
constexpr int64_t kMostParts = 768;   // tiles times parts, where there are several parts
// Entries of a piece.
int64_t loss_piece(int64_t n, int64_t vocab);
inline int64_t loss_tiles(int64_t n, int64_t vocab) {
  const int64_t e = loss_entries(loss_shape(n, vocab));
  return (vocab + e - 1) / e;
}
// Whether rows of X can be taken as they lie.
bool loss_takes(const void* X, int64_t n, int64_t d, int64_t ldx);
bool loss_fits(int64_t n, int64_t vocab, int64_t d, bool grad);

}  // namespace gptq
