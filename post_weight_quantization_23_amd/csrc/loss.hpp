// Launch interfaces of the loss over a vocabulary and its gradients (loss.hip,
// loss_tiles.hip; internal to the library).
#pragma once
#include "adapter.hpp"

namespace gptq {

// Vocabulary entries of a tile of logits: its part of a token's sums.
constexpr int64_t kLossTile = 256, kFewTile = 128;
// Up to as many tokens the largest tiles hold them all, and leaving tokens out
// saves no work: they are taken as they lie (forward).
constexpr int64_t kFewTokens = 256;
// ... and up to as many tiles are of kFewTile entries.
constexpr int64_t kFewEntries = 128;
inline int64_t loss_tile(int64_t n) { return n <= kFewEntries ? kFewTile : kLossTile; }

// The tokens that have a target, in order: place p is token token[p] with target
// col[p]; place_of[t] is token t's place or -1.  count: how many there are.
struct Kept {
  int32_t* token;
  int32_t* place_of;
  int32_t* col;
  float* lse;       // of each place (backward), as grad: dloss, for fp16 times `up`
  float* grad;
  int32_t* count;
  float* down;      // what results are multiplied by (a power of two, 1 for bf16)
};

struct KeepArgs {
  const int64_t* target;
  int64_t n, vocab;
  float *loss, *lse;              // forward: zeroed where there is no target
  const float *lse_in, *dloss;    // backward (dloss null: 1)
  bool half;                      // fp16 gradients
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

// Logits of every kept token in tiles of loss_tile(n) entries: of each tile the
// largest and the sum of exponentials against it, and the target's logit.
struct LossArgs {
  const uint16_t* W;
  int64_t ldw, vocab, n, d;
  const uint16_t* rows;    // [n][ldr], zero past d up to a whole step, or d itself a whole number of them
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

void launch_loss_join(const LossArgs& a, float* loss, float* lse, hipStream_t s);

// dX[place] = P W over one piece of the vocabulary, in `splits` fp32 parts (added
// to what earlier pieces left), and their sum.
struct GradXArgs {
  const uint16_t* P;
  int64_t ldp, width;
  const uint16_t* W;       // the piece's rows
  int64_t ldw, n, d;
  Kept k;
  int splits;
  bool add;                // to parts of an earlier piece
  float* part;             // [splits][n][d]; null: dX is written at once
  uint16_t* dX;
  int64_t ldd;
  bool vec;
};
void launch_grad_x(const GradXArgs& a, int dt, hipStream_t s);
void launch_join_x(const GradXArgs& a, int dt, hipStream_t s);

// dW rows of one piece of the vocabulary = P^T rows.
struct GradWArgs {
  const uint16_t* P;
  int64_t ldp, width;
  const uint16_t* rows;
  int64_t kp, n, d;
  Kept k;
  uint16_t* dW;
  int64_t ldd;
  bool vec;
};
void launch_grad_w(const GradWArgs& a, int dt, hipStream_t s);

// The parts of the contraction that dX is computed in, at a piece of `width` entries.
int grad_x_splits(int64_t n, int64_t d, int64_t width);
// Entries of a piece.
int64_t loss_piece(int64_t n, int64_t vocab);
inline int64_t loss_tiles(int64_t n, int64_t vocab) { return (vocab + loss_tile(n) - 1) / loss_tile(n); }
// Whether rows of X can be taken as they lie.
bool loss_takes(const void* X, int64_t n, int64_t d, int64_t ldx);
bool loss_fits(int64_t n, int64_t vocab, int64_t d, bool grad);

}  // namespace gptq
