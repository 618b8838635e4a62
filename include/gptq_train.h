/*
 * gptq_train.h -- the two ends of training low-rank adapters beside frozen packed
 * layers, and of scoring a quantized model (part of the C ABI of the MI355X GPTQ
 * layer quantizer).
 *
 *   gptq_linear_cross_entropy            the loss of each token over a vocabulary
 *   gptq_linear_cross_entropy_backward   its gradient for the hidden states, with which
 *                                        gptq_packed_linear_backward goes on, and for
 *                                        the output head
 *   gptq_adapter_orthogonalize           what gptq_adapter_backward's gradients (or
 *                                        momenta of them) become as an update
 *
 * The conventions of gptq.h and gptq_adapter.h hold: device pointers, row-major
 * matrices with leading dimensions in elements, caller-owned workspaces
 * (256-byte aligned, sized by the query, free for other use once the stream
 * has passed the call), host-side validation before anything is enqueued, no
 * synchronisation, no allocation, bitwise reproducible results.  A call may be
 * captured into a HIP graph; calls that can run at the same time need workspaces
 * of their own.  Outputs overlap neither inputs nor each other (GPTQ_EINVAL).
 */
#ifndef GPTQ_TRAIN_MI355X_H
#define GPTQ_TRAIN_MI355X_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Softmax cross entropy of hidden states under an output head, the logits never
 * kept: with z = X W^T in fp32 (exact products, fp32 sums),
 *
 *   lse[t]  = log sum_v exp z[t, v]
 *   loss[t] = lse[t] - z[t, target[t]]
 *
 * A target outside 0 .. vocab-1 is none (a prompt's token, padding): the token's
 * loss and lse are 0, and what its hidden state holds reaches no result.  Such tokens are
 * left out of the products, but for the loss of up to 256 tokens whose rows start on
 * 16 bytes, which are multiplied as they lie.  A token whose own logits hold an infinity or NaN gives infinities or NaN;
 * the others are not touched.
 *
 * X      : n_tok x d of type xt (GPTQ_BF16 or GPTQ_F16), 2-byte aligned, ldx >= d
 *          (rows that start on 16 bytes take the fast load path).
 * W      : vocab x d of type xt, 16-byte aligned, ldw >= d, a multiple of 8 and below
 *          2^22.
 * d      : a positive multiple of 8; vocab at least 1.
 * target : int64[n_tok].
 * loss, lse : fp32[n_tok] out.
 * ws     : gptq_linear_cross_entropy_workspace_size() bytes.
 * n_tok = 0 is nothing to do.  Sizes of which a launch would pass 2^32 threads are
 * GPTQ_EUNSUPPORTED, here and below, as are d of 2^22 or more.
 * ------------------------------------------------------------------------ */
gptq_status gptq_linear_cross_entropy_workspace_size(int64_t n_tok, int64_t d, int64_t vocab, size_t* bytes);
gptq_status gptq_linear_cross_entropy(const void* X, gptq_dtype xt, int64_t n_tok, int64_t d, int64_t ldx,
                                      const void* W, int64_t vocab, int64_t ldw, const int64_t* target,
                                      float* loss, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Its gradients, with the logits computed again:
 *
 *   D[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v = target[t]]), 0 without a target
 *   dX = D W,   dW = D^T X
 *
 * D enters the products rounded once to xt (GPTQ_F16: scaled by a power of two, so
 * that entries down to 2^-28 of the largest dloss are normal numbers), the targets' entries
 * in fp32 for dX and as two values of xt for dW.  Hidden
 * states of tokens without a target enter nothing.  The vocabulary is taken in
 * pieces, so that D takes 512 MB or 512 bytes per token, whichever is more.
 *
 * lse    : fp32[n_tok] from gptq_linear_cross_entropy on the same inputs.
 * dloss  : fp32[n_tok], the gradient that arrives at each token's loss.  NULL: 1.
 * dX     : n_tok x d of type xt, 2-byte aligned, row stride lddx; NULL: not wanted.
 *          Rows of tokens without a target are written with zeros.
 * dW     : vocab x d of type xt, 2-byte aligned, row stride lddw; NULL: not wanted.
 *          Written whole, also for n_tok = 0.
 * ws     : gptq_linear_cross_entropy_backward_workspace_size() bytes.
 * At least one of dX and dW has to be given.
 * ------------------------------------------------------------------------ */
gptq_status gptq_linear_cross_entropy_backward_workspace_size(int64_t n_tok, int64_t d, int64_t vocab, int want_dx,
                                                              int want_dw, size_t* bytes);
gptq_status gptq_linear_cross_entropy_backward(const void* X, gptq_dtype xt, int64_t n_tok, int64_t d, int64_t ldx,
                                               const void* W, int64_t vocab, int64_t ldw, const int64_t* target,
                                               const float* lse, const float* dloss, void* dX, int64_t lddx, void* dW,
                                               int64_t lddw, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Orthogonalised updates of low-rank factors by Newton-Schulz products, as the Muon
 * optimiser has them.  Of each adapter's matrix G, one of G_A[i] (rank x c) and G_B[i]
 * (r x rank):
 *
 *   M_0 = G / (|G|_F + eps),   M_{k+1} = a M_k + (b S + c3 S S) M_k,  S = M_k M_k^T
 *
 * (for a matrix of more rows than columns S = M^T M, multiplied from the right,
 * which is the same), `steps` times; out = M_steps.  The singular vectors stay, the
 * singular values s become p(p(..p(s))), p(s) = a s + b s^3 + c3 s^5.
 * The iteration runs on S in 64 bits: S_{k+1} = S_k q(S_k)^2 with q(S) = a + b S + c3 S^2,
 * out = q(S_{steps-1}) .. q(S_0) M_0.  S is formed again from M_k, also in 64 bits, where an error of it
 * would have grown by more than 2^16, a^2 a step (after 5 steps of a = 3.4445), so that
 * matrices of less than full rank stay so.  Nothing is rounded to fewer bits but the result, once.
 *
 * G_A    : m x rank x c of type gt (GPTQ_F32, GPTQ_BF16 or GPTQ_F16), dense, aligned
 *          to its elements; NULL: not wanted (out_A is then ignored).
 * G_B    : m x r x rank, likewise.
 * out_A, out_B : the same shapes, of type ot (any of the three).
 * rank, c, r : positive; min(rank, c) and min(rank, r) at most 128.
 * steps  : 1 .. 16.  a, b, c3: finite.  eps: finite and not negative; a zero matrix gives
 *          zeros (with eps = 0 NaN).  A matrix that holds an infinity or NaN gives NaN, the
 *          others are not touched.
 * ws     : gptq_adapter_orthogonalize_workspace_size() bytes (c or r 0: that side is not
 *          wanted).
 * m = 0 is nothing to do.
 * ------------------------------------------------------------------------ */
gptq_status gptq_adapter_orthogonalize_workspace_size(int64_t m, int64_t rank, int64_t c, int64_t r, int steps,
                                                      size_t* bytes);
gptq_status gptq_adapter_orthogonalize(const void* G_A, const void* G_B, gptq_dtype gt, int64_t m, int64_t rank,
                                       int64_t c, int64_t r, int steps, float a, float b, float c3, float eps,
                                       void* out_A, void* out_B, gptq_dtype ot, void* ws, size_t ws_bytes,
                                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_TRAIN_MI355X_H */
