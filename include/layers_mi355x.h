/*
 * layers_mi355x.h - C ABI of the MI355X (gfx950) operators around a mixture of
 * experts (experts_mi355x.h): rows of a table by number, layer norm, the choice of
 * experts from scores, and the softmax cross entropy of a product with a table. Numbers
 * are the labels of kmeans_assign (codes of centroids) or any other int64 numbers.
 *
 * Common conventions: those of experts_mi355x.h. Device pointers owned by the caller,
 * matrices of rows `ld` elements apart, a caller-owned workspace of the bytes that the
 * matching *_workspace_bytes function gives (256 or fewer: it may be NULL; 0: the shape
 * is not supported; two calls that may run at the same time need two), arguments checked on
 * the host before any HIP call, nothing but enqueued kernels (a call can be captured into a
 * HIP graph), outputs that overlap nothing of the call, no float atomics: equal calls
 * give equal bits. dtype is an experts_dtype and names the type of every `void *` matrix
 * unless the call says otherwise. Sums, means and softmax statistics are kept in float32
 * and rounded once where they are stored.
 */
#ifndef LAYERS_MI355X_H
#define LAYERS_MI355X_H

#include "experts_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * out[t] = scale * w[ids[t]]: rows of the dense table w (classes, width) by the int64
 * numbers ids (tokens). A number outside [0, classes) gives a zero row.
 * 0 <= tokens < 2^26 - 4, 1 <= classes, width <= 2^20.
 */
int layers_embed(const int64_t *ids, int64_t tokens, const void *w, int dtype, int64_t classes,
                 int64_t width, double scale, void *out, int64_t ldo, void *stream);

/*
 * The table's gradient: dw[v] = scale * sum over the tokens t with ids[t] = v, in an order
 * that the numbers alone settle, of dy[t]; zero where there is none. dw (classes, width), dense.
 * One dispatch has to hold the sums: (tokens / 16 to 64) * (width / 256) < 2^24.
 */
size_t layers_embed_backward_workspace_bytes(int64_t tokens, int64_t classes, int64_t width,
                                             int dtype);
int layers_embed_backward(const void *dy, int64_t lddy, const int64_t *ids, int64_t tokens,
                          int dtype, int64_t classes, int64_t width, double scale, void *dw,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * Layer norm of the rows of x (rows, width):
 *   h = (x - mean) * rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps), out = h * weight + bias.
 *   weight, bias  (width), dense, of weights_dtype (dtype, or EXPERTS_F32); NULL: ones, zeros.
 *   mean, rstd    (rows) float32 outputs for the gradient; both NULL or neither.
 * 0 <= rows < 2^24, 1 <= width <= 2^20, eps >= 0.
 */
int layers_norm(const void *x, int64_t ldx, const void *weight, const void *bias, int dtype,
                int weights_dtype, int64_t rows, int64_t width, double eps, void *out, int64_t ldo,
                float *mean, float *rstd, void *stream);

/*
 * Its gradients, with g = dy * weight (weight NULL: ones) and the forward call's mean and rstd:
 *   dx = rstd * (g - mean(g) - h * mean(g * h)),
 *   dweight = sum over rows of dy * h, dbias = sum over rows of dy (of weights_dtype).
 * dx, dweight and dbias may be NULL, not all three.
 */
size_t layers_norm_backward_workspace_bytes(int64_t rows, int64_t width, int dtype);
int layers_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                         const void *weight, const float *mean, const float *rstd, int dtype,
                         int weights_dtype, int64_t rows, int64_t width, void *dx, int64_t lddx,
                         void *dweight, void *dbias, void *workspace, size_t workspace_bytes,
                         void *stream);

typedef enum { LAYERS_SOFTMAX = 0, LAYERS_SIGMOID = 1 } layers_score;

/*
 * The experts of each token from their logits (tokens, experts), and the weights of
 * experts_combine:
 *   s = softmax of the row, or 1 / (1 + e^-logit); c = s + bias.
 *   With groups > 1 the experts are `groups` equal runs. A group's rank is its largest c, or,
 *   with group_best 2, the sum of its two largest; only the top_groups best groups stay
 *   (ties: the lower group).
 *   ids (tokens, top) int64: the numbers of the `top` largest c, the largest first (ties:
 *   the lower number).
 *   weights (tokens, top) float32: scale * s, with `renormalize` scale * s / (the sum of
 *   the chosen experts' s).
 * An expert whose c is -inf or NaN (a logit that a mask has set to -inf, a bias of -inf) is
 * never chosen; where fewer than `top` are left, the ids after them are -1 (experts_plan drops
 * such pairs) and their weights 0. Without bias and with group_best 1 or one group the choice goes
 * by the logits themselves, whose order s keeps. Otherwise it is that of the formulas in float64.
 * A softmax row with a NaN or +inf has no s. With bias, or group_best 2 of several groups, it
 * has no c either: ids -1, weights 0. By the logits its other experts (and +inf, the first) are
 * chosen all the same; their weights are the shares among them with `renormalize` (NaN with a
 * chosen +inf), else NaN. A sigmoid's NaN takes out its own expert alone.
 *   bias      (experts) float32, dense, or NULL.
 * 0 <= tokens < 2^26 - 16, 1 <= top <= 64, top <= experts, groups a divisor of experts,
 * groups <= 64, experts / groups <= 32 * (64 / groups rounded down): up to 2048 experts.
 */
int layers_route(const void *logits, int64_t ld, int dtype, int64_t tokens, int64_t experts,
                 int64_t top, int score, const float *bias, int64_t groups, int64_t top_groups,
                 int64_t group_best, int renormalize, double scale, int64_t *ids, float *weights,
                 void *stream);

/*
 * The logits' gradient (tokens, experts) for dweights (tokens, top), the ids as layers_route
 * gave them: that of the weights with the choice fixed. A number outside [0, experts) has no
 * weight, and its dweights are not read. The bias has no gradient: it moves no weight.
 */
int layers_route_backward(const float *dweights, const void *logits, int64_t ld,
                          const int64_t *ids, int dtype, int64_t tokens, int64_t experts,
                          int64_t top, int score, int renormalize, double scale, void *dlogits,
                          int64_t lddl, void *stream);

/*
 * Softmax cross entropy of z = x w^T, z not kept: for every row r of x (rows, width)
 *   lse[r] = log sum_j e^z[r, j], loss[r] = lse[r] - z[r, targets[r]].
 *   w        (classes, width), dense; targets (rows) int64; loss, lse (rows) float32.
 * A target outside [0, classes) is ignored: its loss is 0 (lse is still given). Logits have to
 * stay below 2^127 in magnitude, or they leave float32 in units of log 2.
 * 0 <= rows < 2^31, 1 <= classes, width, ld <= 2^20, and fewer than about 2^23 tiles of
 * 64 x 64 to 256 x 256 logits. float32 uses the float32 matrix instructions, the 16-bit types
 * theirs; both accumulate in float32. Workspace: 8 bytes for 16 to 256 logits of a row (small
 * products of a long width: their logits' partial sums, at most 1024 tiles), and where more
 * than 32 16-bit rows do not lie on 4-byte boundaries (width odd, or, with `unaligned` non-zero,
 * an odd ld or a pointer off 4 bytes) room for their copies on padded rows, w's too.
 */
size_t layers_cross_entropy_workspace_bytes(int64_t rows, int64_t classes, int64_t width,
                                            int dtype, int unaligned);
int layers_cross_entropy(const void *x, int64_t ldx, const void *w, const int64_t *targets,
                         int dtype, int64_t rows, int64_t classes, int64_t width, float *loss,
                         float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Its gradients for dloss (rows) and dlse (rows, or NULL for zeros), float32, with the
 * forward call's lse:
 *   dz = (dloss + dlse) e^(z - lse) - dloss [j = target], without dloss in ignored rows,
 *   dx = dz w, dw = dz^T x.
 * dlse makes any function of lse a part of the loss (for c lse^2: 2 c lse). dx or dw may be
 * NULL, not both. z is computed again, in pieces of the classes whose dz takes 512 MiB of the
 * workspace at most, or, past 2^20 16-bit rows (2^19 of float32), 256 classes of all rows; the
 * products read dz rounded to dtype, which is what the 16-bit matrix instructions take, divided
 * by the largest |dloss + dlse| or |dloss| of a row (for float16 times 2^14, which keeps it in
 * range). dx is summed over the pieces in float32. An ignored row
 * without dlse has dz 0 and dx 0; its x is read by dw's product all the same and has to be
 * finite.
 */
size_t layers_cross_entropy_backward_workspace_bytes(int64_t rows, int64_t classes, int64_t width,
                                                     int dtype, int unaligned);
int layers_cross_entropy_backward(const float *dloss, const float *dlse, const void *x,
                                  int64_t ldx, const void *w, const int64_t *targets,
                                  const float *lse, int dtype, int64_t rows, int64_t classes,
                                  int64_t width, void *dx, int64_t lddx, void *dw, void *workspace,
                                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYERS_MI355X_H */
