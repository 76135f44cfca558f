// layers.h - internal launchers of the operators around the experts (embed.hip,
// norm.hip, route.hip, entropy*.hip), used by layers_api.hip. Not part of the public
// interface.
#pragma once

#include "experts.h"

namespace kx {

// ------------------------------------------------------------------ embed
hipError_t launch_embed(const int64_t *ids, int64_t tokens, const void *w, int dtype,
                        int64_t classes, int64_t width, float scale, void *out, int64_t ldo,
                        hipStream_t s);

// Classes up to this many are sorted by the plan; more of them first by their
// number modulo kEmbedBuckets. (us of the gradient, plan / buckets: 65536 x 512 bf16 of 2000 62 /
// 100, of 500 x 128 33 / 86 before the buckets' sort had no barriers; 65536 x 64 of 2500 36 / 35,
// frequent as 1 / number 44 / 56, of 10000 45 / 37 and 52 / 57, of 50000 94 / 46 and 96 / 59.)
constexpr int64_t kEmbedDirect = 2048;
constexpr int64_t kEmbedBuckets = 1024;
struct EmbedScratch {
    int64_t *bucket;          // tokens, with buckets
    int *order, *place;       // tokens
    int *sorted;              // tokens, with buckets
    int *offsets;             // classes or kEmbedBuckets, and 1
    int *lo, *hi;             // classes, with buckets
    float *partial;           // embed_chunks() x 2 x width
    PlanScratch plan;
};
// Sorted places that one wave or block sums.
int64_t embed_chunk(int64_t tokens);
hipError_t launch_embed_backward(const void *dy, int64_t lddy, const int64_t *ids, int64_t tokens,
                                 int dtype, int64_t classes, int64_t width, float scale, void *dw,
                                 const EmbedScratch &ws, hipStream_t s);
// False when a launch's grid would not fit.
bool embed_grid_ok(int dtype, int64_t tokens, int64_t classes, int64_t width);

// ------------------------------------------------------------------- norm
struct NormProblem {
    const void *x, *weight, *bias, *dy;
    int64_t ldx, lddy, ldo, rows, width;
    float eps;
    void *out;             // y or dx (NULL: not computed)
    float *mean, *rstd;    // read by the gradient, written by the forward call (or NULL)
    void *dweight, *dbias; // or NULL
    float *partial;        // norm_parts() x 2 x width
};
// weights_dtype: that of weight, bias, dweight and dbias, dtype or float32.
hipError_t launch_norm(int dtype, int weights_dtype, const NormProblem &pr, hipStream_t s);
hipError_t launch_norm_backward(int dtype, int weights_dtype, const NormProblem &pr, hipStream_t s);
int64_t norm_parts(int dtype, int64_t rows, int64_t width);
bool norm_grid_ok(int dtype, int64_t rows, int64_t width);

// ------------------------------------------------------------------ route
struct RouteProblem {
    const void *logits;
    int64_t ld, tokens;
    int experts, top, groups, kept, best;  // best: choices that a group's rank sums
    bool sigmoid, renormalize;
    const float *bias;
    float scale;
    int64_t *ids;
    float *weights;
    const int64_t *chosen;   // the gradient's ids
    const float *dweights;
    void *dlogits;
    int64_t lddl;
};
// Whether a kernel holds `groups` groups of `experts / groups`.
bool route_fits(int64_t experts, int64_t groups, int64_t top);
hipError_t launch_route(int dtype, const RouteProblem &pr, hipStream_t s);
hipError_t launch_route_backward(int dtype, const RouteProblem &pr, hipStream_t s);

// ---------------------------------------------------------------- entropy
struct EntropyProblem {
    const void *x, *w;        // rows x width, classes x width, on 4-byte boundaries
    int64_t ldx, ldw, rows, classes, width;
    const int64_t *targets;
    int tile, thin;           // entropy_plan's tile, and with its `thin` its splits
    // The sums of each row over one column tile, and the target's logit.
    float2 *part;             // column tiles x rows
    float *hit;               // rows
    float *loss, *lse;        // outputs; lse is read by the gradient
    // The gradient.
    const float *dloss, *dlse;
    float *scale;             // dz's factor and its inverse (NULL: 1)
    float most_dz;            // of scaled rows; 0: scale is given, else the dz kernel finds it
    // A product cut in depth: float32 parts of the logits, rows x count each (parts 1: none).
    int parts;
    float *logits;
    int64_t first, count;     // classes of this piece
    void *dz;                 // rows x lddz
    int64_t lddz;
};
// With `thin` (few rows, the forward call), tile rows and 16 * splits columns a block, and any
// rows are read in place; else in `splits` parts of the depth (logits, above).
Cut entropy_plan(int dtype, int64_t rows, int64_t classes, int64_t width, bool grad);
int entropy_columns(const Cut &cut);  // of a tile
hipError_t launch_entropy(int dtype, const EntropyProblem &pr, hipStream_t s);
hipError_t launch_entropy_dz(int dtype, const EntropyProblem &pr, hipStream_t s);
// The factor of a 16-bit dz and its inverse, where the rows are too many for every block of the
// dz kernel to look at them.
hipError_t launch_entropy_scale(const EntropyProblem &pr, hipStream_t s);
// (dx and dw of 64 x 8192 x 512 bf16 21.5 us, with a launch for the scale 23.0; 2048 x 2048 x 512
// 37.5 and 39; 8192 x 8192 x 512 253 and 240. The launch is one block: 4 to 7 us for 8192 rows, 15
// for 65536, 440 for 2^20, 10700 for 2^24.)
constexpr int64_t kOwnScale = 1024;  // rows

// dx (first and last piece, sums between them) and dw of a piece.
struct EntropyGrad {
    const void *dz, *x, *w;   // w, dw: the piece's first row
    int64_t lddz, ldx, ldw;
    int64_t x_cols, w_cols;   // readable columns (a pad is zero)
    int64_t rows, count, width;
    const float *scale;
    void *dx;                 // NULL: not computed
    int64_t lddx;
    float *sum;               // rows x width, between pieces
    bool first, last;
    void *dw;                 // NULL: not computed
    Cut dx_cut, dw_cut;
    bool together;            // one launch, both with dx_cut's tile and neither split
    float *partial;
};
hipError_t launch_entropy_grad(int dtype, const EntropyGrad &g, hipStream_t s);

}  // namespace kx
