/*
 * experts_mi355x.h - C ABI of the MI355X (gfx950) operators of a mixture of
 * experts: tokens sorted by expert and back, the experts' matrix product with
 * its epilogue, and the AdamW step that trains their weights. Expert numbers
 * are the labels of kmeans_assign (a router by nearest centroid, one expert a
 * token) or any other int64 numbers, several a token.
 *
 * Common conventions (those of kmeans_mi355x.h, with strides)
 *   - Every array pointer is a DEVICE pointer owned by the caller; the library
 *     never allocates, frees or keeps device memory. A matrix is row-major;
 *     its rows are `ld` elements apart (ld >= the row length).
 *   - dtype is an experts_dtype and names the type of every `void *` matrix of
 *     the call. Sums are kept in float32 and rounded once where they are
 *     stored, except dz of experts_linear_backward (see there).
 *   - A pair is one (token, slot) of the (tokens, top) expert numbers: pair
 *     t * top + s. Pairs whose number lies outside [0, experts) are dropped:
 *     they reach no expert and add nothing to their token.
 *   - workspace is a caller-owned device buffer of at least the bytes that the
 *     matching *_workspace_bytes function gives, any alignment; its contents
 *     on entry do not matter. Two calls that may run at the same time need two.
 *     Where those bytes are 256 or fewer (slack for the alignment alone) the
 *     workspace may be NULL. 0 bytes mean that the shape is not supported.
 *   - stream is a hipStream_t (NULL = the default stream). Every call only
 *     enqueues kernels on it: no allocation, host wait, copy or memset, so it
 *     can be captured into a HIP graph and replayed.
 *   - Arguments are validated on the host before any HIP call; an invalid call
 *     returns a negative km_status (kmeans_mi355x.h) and enqueues nothing.
 *     Outputs must not overlap inputs, each other or the workspace.
 *   - No float atomics: the same inputs give the same bits.
 */
#ifndef EXPERTS_MI355X_H
#define EXPERTS_MI355X_H

#include <stddef.h>
#include <stdint.h>

#include "kmeans_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { EXPERTS_F32 = 0, EXPERTS_BF16 = 1, EXPERTS_F16 = 2 } experts_dtype;

/* Activations: z; max(z, 0); z * sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3)),
 * which is gelu in its tanh form; z * sigmoid(z). */
typedef enum {
    EXPERTS_ACT_NONE = 0,
    EXPERTS_ACT_RELU = 1,
    EXPERTS_ACT_GELU_TANH = 2,
    EXPERTS_ACT_SILU = 3
} experts_act;

/*
 * The plan of one batch: its pairs sorted by expert.
 *   ids      (tokens, top) int64 expert numbers, dense.
 *   order    (tokens * top) int32 output: the pair at each sorted place, pairs
 *            of one expert in increasing order; -1 at the places past the last
 *            pair that was not dropped.
 *   place    (tokens, top) int32 output: the sorted place of each pair, -1 for
 *            a dropped one (the inverse of order).
 *   offsets  (experts + 1) int32 output: expert e has the places
 *            [offsets[e], offsets[e + 1]).
 * 0 <= tokens, 1 <= top <= 64, tokens * top < 2^31, 1 <= experts <= 65536.
 */
size_t experts_plan_workspace_bytes(int64_t tokens, int64_t top, int64_t experts);
int experts_plan(const int64_t *ids, int64_t tokens, int64_t top, int64_t experts, int32_t *order,
                 int32_t *place, int32_t *offsets, void *workspace, size_t workspace_bytes,
                 void *stream);

/*
 * xs[p] = x[order[p] / top]: the token rows in sorted order (tokens * top rows
 * of xs; rows at places without a pair become zero).
 * Limits of this call, its gradient and experts_combine, tighter than the plan's:
 * tokens < 2^24 (a workgroup of 256 a token is one dispatch), 1 <= width < 2^31.
 */
int experts_dispatch(const void *x, int64_t ldx, int dtype, int64_t tokens, int64_t top,
                     int64_t width, const int32_t *order, const int32_t *place, void *xs,
                     int64_t ldxs, void *stream);

/* dx[t] = sum over the token's pairs, in slot order, of dxs[place]. */
int experts_dispatch_backward(const void *dxs, int64_t lddxs, int dtype, int64_t tokens,
                              int64_t top, int64_t width, const int32_t *place, void *dx,
                              int64_t lddx, void *stream);

/* y[t] = sum over the token's pairs, in slot order, of weights[t, s] *
 * ys[place[t, s]]; weights (tokens, top) float32, dense. */
int experts_combine(const void *ys, int64_t ldys, const float *weights, int dtype, int64_t tokens,
                    int64_t top, int64_t width, const int32_t *place, void *y, int64_t ldy,
                    void *stream);

/*
 * Gradients of experts_combine: dys[p] = weights[order[p]] * dy[token] (zero at
 * places without a pair) and dweights[t, s] = <dy[t], ys[place[t, s]]> (zero
 * for a dropped pair; float32, (tokens, top), dense). Either output may be
 * NULL; ys is read only for dweights. tokens * top < 2^26 - 4.
 */
int experts_combine_backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                             const float *weights, int dtype, int64_t tokens, int64_t top,
                             int64_t width, const int32_t *order, const int32_t *place, void *dys,
                             int64_t lddys, float *dweights, void *stream);

/*
 * The product with its epilogue: for every row r of x, with e its expert,
 *   pre[r] = x[r] w_e^T + bias_e,  out[r] = act(pre[r]) + residual[r].
 *   x         (rows, ins); out, residual, pre (rows, outs); each with its ld.
 *   w         (outs, ins), or (experts, outs, ins) with offsets; dense.
 *   bias      (outs) or (experts, outs), dense, or NULL.
 *   residual  or NULL. pre: output, or NULL.
 *   offsets   NULL (experts is then 1 and every row uses w), or the plan's
 *             (experts + 1) int32: offsets[0] is 0 and expert e has the rows
 *             [offsets[e], offsets[e + 1]). Rows from offsets[experts] on become
 *             zero in out and pre. (Other values leave rows unwritten, but make no
 *             call read or write outside its matrices.)
 * 0 <= rows < 2^31; 1 <= outs, ins <= 2^20; 1 <= experts <= 65536; ld <= 2^20;
 * and one dispatch has to hold the call: rows * outs < 2^35 - 2^12 (rows * ins too for
 * the gradient and the 16-bit types, for these also experts * outs * ins; outs and ins
 * rounded up to multiples of 8), and fewer than about 2^23 tiles of 64 x 64 to
 * 256 x 256 outputs.
 * float32 uses the float32 matrix instructions, the 16-bit types theirs; both
 * accumulate in float32.
 * Workspace: partial sums where the depth is split; and where 16-bit rows of x
 * or w do not lie on 4-byte boundaries (ins odd, or, with `unaligned` non-zero, an
 * odd ld or a pointer off 4 bytes) room for their copies on padded rows. The
 * size query's op: 0 for experts_linear, 1 for experts_linear_backward.
 */
size_t experts_linear_workspace_bytes(int64_t rows, int64_t outs, int64_t ins, int64_t experts,
                                      int dtype, int op, int unaligned);
int experts_linear(const void *x, int64_t ldx, const void *w, const void *bias,
                   const void *residual, int64_t ldr, const int32_t *offsets, int dtype, int act,
                   int64_t rows, int64_t outs, int64_t ins, int64_t experts, void *out,
                   int64_t ldo, void *pre, int64_t ldpre, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * Gradients of experts_linear (the residual's is dy itself):
 *   dz = dy * act'(pre)     (pre may be NULL with EXPERTS_ACT_NONE)
 *   dx = (dz w_e) * in_act'(in_pre)   in_pre NULL: no second factor. With the
 *        pre of the layer before, dx is that layer's dz.
 *   dw_e = sum over the expert's rows of dz[r]^T x[r], dbias_e = sum of dz[r].
 * dx, dw and dbias may be NULL, not all three; an expert without rows gets zero
 * dw and dbias; rows of dx from offsets[experts] on become zero. dbias sums dz
 * in float32; the products read dz rounded to dtype, which is what the 16-bit
 * matrix instructions take.
 */
int experts_linear_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                            const void *w, const void *pre, int64_t ldpre, const void *in_pre,
                            int64_t ldin, const int32_t *offsets, int dtype, int act, int in_act,
                            int64_t rows, int64_t outs, int64_t ins, int64_t experts, void *dx,
                            int64_t lddx, void *dw, void *dbias, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * One AdamW step (decoupled weight decay) over `count` tensors. With g the
 * gradient times *grad_scale (a device float, NULL for 1):
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m /
 *       (sqrt(v) / sqrt(1 - beta2^step) + eps),
 * all in float32; p is rounded once when its type is 16 bits wide.
 *   params, grads, copies  HOST arrays of `count` device pointers, read during
 *            the call; copies (or NULL) receives the new parameters in bfloat16.
 *            A bfloat16 parameter may be its own copy; else what is written
 *            overlaps nothing of the call (a tied weight is given once).
 *            Elements are dense. param_dtype and grad_dtype hold for all.
 *   numels   HOST array of the tensors' lengths (>= 0).
 *   m, v     device moments of all tensors in one array each: a tensor's start
 *            on the next multiple of 256 elements after the one before it
 *            (experts_adamw_state_elements in all). bits = 32: float32, the
 *            scales NULL. bits = 8: m int8, v uint8 and one float32 scale for
 *            every 256 elements: m = m_scale (q / 127) |q / 127|,
 *            v = v_scale (q / 255)^4, each scale the largest magnitude of its
 *            block. q is rounded to nearest, but a v above 0 never to 0: its
 *            m may still be above 0, and m / (0 + eps) would be a huge step.
 *            The step itself uses the moments before they are rounded. A block
 *            with a NaN or infinity in a moment gets a NaN scale.
 * step counts from 1.
 */
int64_t experts_adamw_state_elements(const int64_t *numels, int64_t count);
int experts_adamw_step(void *const *params, const void *const *grads, void *const *copies,
                       const int64_t *numels, int64_t count, int param_dtype, int grad_dtype,
                       void *m, void *v, float *m_scale, float *v_scale, int bits, double lr,
                       double beta1, double beta2, double eps, double weight_decay, int64_t step,
                       const float *grad_scale, void *stream);

/* The values that 8-bit moments stand for, in float32: elements a multiple of
 * 256. Either pair (q, out) may be NULL. */
int experts_adamw_moments(const int8_t *m, const uint8_t *v, const float *m_scale,
                          const float *v_scale, int64_t elements, float *m_out, float *v_out,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERTS_MI355X_H */
