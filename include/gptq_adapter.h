/*
 * gptq_adapter.h -- packed layers with many tokens, and low-rank adapters
 * beside them (part of the C ABI of the MI355X GPTQ layer quantizer).
 *
 * gptq_dequant_gemv (gptq.h) multiplies a packed layer with one activation
 * vector.  The calls here take any number of tokens: the requests that decode
 * together, prompts, or a training batch.  Each request may bring its own
 * low-rank adapter beside the frozen packed projection; the adapters can be
 * trained through it.  With
 *
 *   W_hat[i, j] = scales[i, g(j)] * (q[i, j] - zeros[i, g(j)])      (gptq_dequant_gemv)
 *   a(t) = index[t], delta[t, :] = alpha[a] * B_a (A_a X[t, :])
 *
 *   gptq_packed_linear            Y   = X W_hat^T + delta
 *   gptq_packed_linear_backward   dX  = dY W_hat + alpha (dY B) A
 *   gptq_adapter_add              out = Y + delta             (any projection's Y)
 *   gptq_adapter_backward         gradients of A and B, and of X through them
 *
 * The conventions of gptq.h hold: device pointers, row-major matrices with
 * leading dimensions in elements, caller-owned workspaces (256-byte aligned,
 * sized by the query, free for other use once the stream has passed the call),
 * host-side validation before anything is enqueued, no synchronisation, no
 * allocation, bitwise reproducible results.  A call may be captured into a HIP
 * graph; calls that can run at the same time need workspaces of their own.
 *
 * Packed layer arguments (packed, r, c, bits, ld_words, scales, zeros,
 * ld_groups, groupsize, col_perm) are those of gptq_dequant_gemv, with its
 * requirements, except that c is a positive multiple of 32 of any size up to
 * 2^30, zeros lie in -1000 .. 1000 (a ruler's lie in 0 .. 2^bits - 1), and
 * col_perm has to be a permutation of 0 .. c-1 in the backward call (an input
 * column that it leaves out or names twice has no defined gradient; entries
 * outside the range are clamped; both stay inside the buffers).
 *
 * Adapter arguments:
 * A       : n_adapters x rank x c, B: n_adapters x r x rank, both dense, 16-byte
 *           aligned and of the activations' type.  A == B == NULL: no adapters
 *           (the packed calls only); the other adapter arguments are ignored.
 * rank    : a multiple of 8 in 8 .. 128 (adapters of a smaller rank are padded
 *           with zeros).
 * index   : int32[n_tok], the adapter of each token, in any order; a value
 *           outside 0 .. n_adapters-1 means none.  NULL: adapter 0 for all.
 * alpha   : fp32[n_adapters], the factor of each adapter.  NULL: 1.
 * A token's result never depends on other requests' tokens or adapters, not
 * even where those hold infinities or NaN.  A request's own infinities and NaN, in
 * its tokens, factors or alpha, give infinities or NaN in the results that they enter
 * (an infinity may come out as NaN: fp32 values go into the matrix cores in terms).
 *
 * Sizes: a launch holds fewer than 2^32 threads; a call one of whose launches
 * would pass that is GPTQ_EUNSUPPORTED (also in its query, as far as the query is
 * told of the adapters).  Fewer than 2^24 tokens and rows of the layer, activations
 * and results of up to 2^31 elements, layers of up to 2^37 and factors A and B of up
 * to 2^29 always fit; only where adapters have few tokens each (n_tok <= 4
 * n_adapters) n_tok rank has to stay below 2^25 besides.
 *
 * n_tok = 0, or r = 0 in the two forward calls, is nothing to do (pointers to what
 * has no elements may be NULL); gptq_adapter_backward still writes zeros.
 *
 * Types: activations and gradients are GPTQ_BF16 or GPTQ_F16; results are of
 * that type or GPTQ_F32, rounded once (round-to-nearest-even).
 */
#ifndef GPTQ_ADAPTER_MI355X_H
#define GPTQ_ADAPTER_MI355X_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Y[t, i] = round_yt( sum_j W_hat[i, j] X[t, src(j)] + delta[t, i] ),
 * src(j) = col_perm[j], or j.  Up to 1023 tokens, and for fp32 results of any
 * number, codes are multiplied as whole numbers and the rulers applied to each
 * group's fp32 sum, so the weights are not rounded: the fp32 result is within
 * about 2^-16 sum_j scale (2 * 2^bits + q + |zero|) |x_j| of the exact product (a
 * bound; usual errors are far smaller).  16-bit results of more tokens take
 * weights rounded once to X's type, as gptq_linear_forward does.  |X| must stay
 * below 2^115 (larger bf16 values can overflow a group's sum); a token that
 * holds an infinity or NaN gives infinities or NaN, the others are not touched.
 *
 * X  : n_tok x c of type xt, 16-byte aligned, ldx a multiple of 8 and >= c
 *      (2-byte alignment and any ldx >= c when col_perm is given).
 * Y  : n_tok x r of type yt (GPTQ_F32 or xt), row stride ldy; overlaps no input.
 * ws : gptq_packed_linear_workspace_size() bytes (rank 0 without adapters;
 *      NULL when that is 0).
 * ------------------------------------------------------------------------ */
gptq_status gptq_packed_linear_workspace_size(int64_t n_tok, int64_t r, int64_t c, gptq_dtype yt, int64_t rank,
                                              int has_perm, size_t* bytes);
gptq_status gptq_packed_linear(const void* X, gptq_dtype xt, int64_t n_tok, int64_t ldx, const uint32_t* packed,
                               int64_t r, int64_t c, int bits, int64_t ld_words, const float* scales,
                               const int32_t* zeros, int64_t ld_groups, int64_t groupsize, const int32_t* col_perm,
                               const void* A, const void* B, int64_t n_adapters, int64_t rank, const int32_t* index,
                               const float* alpha, void* Y, gptq_dtype yt, int64_t ldy, void* ws, size_t ws_bytes,
                               void* stream);

/* ------------------------------------------------------------------------
 * dX[t, src(j)] = round_ot( sum_i dY[t, i] W_hat[i, j]
 *                           + alpha sum_p (sum_i dY[t, i] B_a[i, p]) A_a[p, src(j)] ),
 * the gradient of gptq_packed_linear for its input.  W_hat is rounded once to
 * dY's type, as gptq_linear_forward does, when dX is of that type; with ot =
 * GPTQ_F32 it enters as a sum of such values that holds fp32's precision
 * (for GPTQ_F16: down to 2^-25).
 *
 * dY : n_tok x r of type xt, 2-byte aligned, ldy >= r (rows that start on 16
 *      bytes take the fast load path).
 * dX : n_tok x c of type ot (GPTQ_F32 or xt), row stride ldx; overlaps no input.
 * r  : 1 .. 2^22 - 64.
 * ws : gptq_packed_linear_backward_workspace_size() bytes (n_adapters = rank
 *      = 0 without adapters): it holds a dequantized copy of the layer, 2 r c
 *      bytes (4 r c or 6 r c for fp32 results), while the call runs.
 * ------------------------------------------------------------------------ */
gptq_status gptq_packed_linear_backward_workspace_size(int64_t n_tok, int64_t r, int64_t c, gptq_dtype xt,
                                                       gptq_dtype ot, int64_t n_adapters, int64_t rank,
                                                       size_t* bytes);
gptq_status gptq_packed_linear_backward(const void* dY, gptq_dtype xt, int64_t n_tok, int64_t ldy,
                                        const uint32_t* packed, int64_t r, int64_t c, int bits, int64_t ld_words,
                                        const float* scales, const int32_t* zeros, int64_t ld_groups,
                                        int64_t groupsize, const int32_t* col_perm, const void* A, const void* B,
                                        int64_t n_adapters, int64_t rank, const int32_t* index, const float* alpha,
                                        void* dX, gptq_dtype ot, int64_t ldx, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * out[t, i] = round_yt( Y[t, i] + delta[t, i] ): the adapters beside a
 * projection computed elsewhere, for instance by gptq_linear_forward.
 *
 * X   : n_tok x c of type xt, 2-byte aligned, ldx >= c; c a positive multiple
 *       of 8.
 * Y   : n_tok x r of type yt (GPTQ_F32 or xt), row stride ldy.
 * out : the same type and shape, row stride ldo; may be Y itself (same
 *       stride); any other overlap with Y or X is GPTQ_EINVAL.
 * ws  : gptq_adapter_add_workspace_size() bytes.
 * ------------------------------------------------------------------------ */
gptq_status gptq_adapter_add_workspace_size(int64_t n_tok, int64_t c, int64_t rank, size_t* bytes);
gptq_status gptq_adapter_add(const void* X, gptq_dtype xt, int64_t n_tok, int64_t c, int64_t ldx, const void* A,
                             const void* B, int64_t n_adapters, int64_t rank, int64_t r, const int32_t* index,
                             const float* alpha, const void* Y, gptq_dtype yt, int64_t ldy, void* out, int64_t ldo,
                             void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Gradients of the adapters (sums over each adapter's own tokens):
 *   gA[a, p, k] = alpha_a sum_t (sum_i dY[t, i] B_a[i, p]) X[t, k]     fp32 n_adapters x rank x c
 *   gB[a, i, p] = alpha_a sum_t dY[t, i] (sum_k A_a[p, k] X[t, k])     fp32 n_adapters x r x rank
 * both written whole (zero for an adapter without tokens), 16-byte aligned,
 * and, when dX is given, the gradient for the input through the adapters
 * alone, on top of what other paths contributed:
 *   dX[t, k] = round_ot( base[t, k] + alpha sum_p (dY B_a)[t, p] A_a[p, k] )
 *
 * dY   : n_tok x r, X: n_tok x c, both of type xt, 2-byte aligned, ldy >= r and
 *        ldx >= c (rows that start on 16 bytes take the fast load path); c a
 *        positive multiple of 8, r >= 1.
 * base : n_tok x c of type ot (GPTQ_F32 or xt), row stride ldd; NULL: zero.
 * dX   : the same type and stride ldd; may be base; NULL: not wanted.
 * ws   : gptq_adapter_backward_workspace_size() bytes.
 * ------------------------------------------------------------------------ */
gptq_status gptq_adapter_backward_workspace_size(int64_t n_tok, int64_t r, int64_t c, int64_t n_adapters,
                                                 int64_t rank, size_t* bytes);
gptq_status gptq_adapter_backward(const void* dY, int64_t ldy, const void* X, int64_t ldx, gptq_dtype xt,
                                  int64_t n_tok, int64_t r, int64_t c, const void* A, const void* B,
                                  int64_t n_adapters, int64_t rank, const int32_t* index, const float* alpha,
                                  float* gA, float* gB, const void* base, void* dX, gptq_dtype ot, int64_t ldd,
                                  void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_ADAPTER_MI355X_H */
