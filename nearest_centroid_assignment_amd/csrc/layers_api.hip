// layers_api.hip - the C ABI declared in include/layers_mi355x.h.
//
// Every entry point validates its arguments on the host before the first HIP
// call, carves its sections out of the caller's workspace and enqueues the
// kernels on the caller's stream. Nothing here allocates, waits or keeps state.
#include <math.h>

#include "../../include/layers_mi355x.h"
#include "api_checks.h"
#include "layers.h"

namespace {

// The sections of a workspace, one after another.
struct Sections {
    size_t total = 0;
    size_t add(size_t bytes) {
        const size_t at = total;
        total += round_up(bytes);
        return at;
    }
    size_t with_slack() const { return total + kAlign; }
};

// ------------------------------------------------------------------ embed

bool embed_shape_ok(int64_t tokens, int64_t classes, int64_t width) {
    return tokens >= 0 && tokens <= kMaxRows && tokens * 64 <= kMaxGridThreads - 256 &&
           classes >= 1 && classes <= kMaxWidth && width >= 1 && width <= kMaxWidth;
}
struct EmbedLayout {
    size_t bucket = 0, order = 0, place = 0, sorted = 0, offsets = 0, lo = 0, hi = 0, partial = 0, plan = 0;
    PlanLayout sort;
    size_t total = 0;
};
EmbedLayout embed_layout(int64_t tokens, int64_t classes, int64_t width) {
    EmbedLayout L;
    Sections s;
    const bool direct = classes <= kx::kEmbedDirect;
    const int64_t bins = direct ? classes : kx::kEmbedBuckets;
    L.order = s.add((size_t)tokens * 4);
    L.place = s.add((size_t)tokens * 4);
    L.offsets = s.add((size_t)(bins + 1) * 4);
    if (!direct) {
        L.bucket = s.add((size_t)tokens * 8);
        L.sorted = s.add((size_t)tokens * 4);
        L.lo = s.add((size_t)classes * 4);
        L.hi = s.add((size_t)classes * 4);
    }
    L.partial = s.add((size_t)cdiv(tokens, kx::embed_chunk(tokens)) * 2 * (size_t)width * 4);
    L.sort = plan_layout(tokens, bins);
    L.plan = s.add(L.sort.total);
    L.total = s.with_slack();
    return L;
}

// ------------------------------------------------------------------- norm

bool norm_shape_ok(int dtype, int64_t rows, int64_t width) {
    return rows >= 0 && width >= 1 && width <= kMaxWidth && kx::norm_grid_ok(dtype, rows, width);
}
bool weights_ok(int dtype, int weights_dtype) {
    return dtype_ok(dtype) && (weights_dtype == dtype || weights_dtype == EXPERTS_F32);
}

// ------------------------------------------------------------------ route

bool route_shape_ok(int64_t tokens, int64_t experts, int64_t top) {
    return tokens >= 0 && tokens <= kMaxRows && tokens * 64 <= kMaxGridThreads - 1024 && top >= 1 && top <= kMaxTop &&
           experts >= top && experts <= 2048;
}

// ---------------------------------------------------------------- entropy

constexpr size_t kPiece = (size_t)1 << 29;  // bytes of dz at a time, but for piece_of's least

bool entropy_shape_ok(int dtype, int64_t rows, int64_t classes, int64_t width) {
    if (rows < 0 || rows > kMaxRows || classes < 1 || classes > kMaxWidth || width < 1 || width > kMaxWidth)
        return false;
    // The padded copies take a thread for every eight values.
    if (dtype != EXPERTS_F32 && (rows * cdiv(width, 8) + 256 > kMaxGridThreads ||
                                 classes * cdiv(width, 8) + 256 > kMaxGridThreads))
        return false;
    for (bool grad : {false, true}) {
        const kx::Cut cut = kx::entropy_plan(dtype, rows, classes, width, grad);
        const int64_t m = cut.tile == 129 ? 128 : cut.tile, n = kx::entropy_columns(cut);
        if (cdiv(rows, m) * cdiv(classes, n) * (cut.thin ? 1 : cut.splits) + 8 > kMaxGridThreads / 512) return false;
    }
    return true;
}
// The classes of a piece: equal pieces, of whole tiles, 256 at least (dx's float32 sums are read
// and written once a piece).
int64_t piece_of(int64_t rows, int64_t classes, int dtype) {
    const int64_t row = (int64_t)(kPiece / size_of(dtype)) / (rows < 1 ? 1 : rows);
    const int64_t most = row < 512 ? 256 : row / 256 * 256;
    if (classes <= most) return classes;
    const int64_t pieces = cdiv(classes, most);
    return cdiv(cdiv(classes, pieces), 256) * 256;
}
// Few rows or classes leave few tiles of a deep product: up to 64 parts of it.
constexpr int kMostParts = 64;
kx::Cut dx_cut(int dtype, int64_t rows, int64_t count, int64_t width) {
    return kx::plan_in_parts(dtype, rows, width, count, kMostParts);
}
kx::Cut dw_cut(int dtype, int64_t rows, int64_t count, int64_t width) {
    return kx::plan_in_parts(dtype, count, width, rows, kMostParts);
}
bool cut_fits(const kx::Cut &c, int64_t m, int64_t n) {
    const int64_t tm = c.tile == 129 ? 128 : c.tile, tn = c.tile == 32 ? 64 : tm;
    return cdiv(m, tm) * cdiv(n, tn) * c.splits + 8 <= kMaxGridThreads / 512 &&
           cdiv(m * cdiv(n, 8), 256) <= kMaxGridThreads / 256;
}
bool entropy_grad_ok(int dtype, int64_t rows, int64_t classes, int64_t width) {
    const int64_t count = piece_of(rows, classes, dtype);
    const int64_t last = classes - (classes - 1) / count * count;
    for (int64_t n : {count, last})
        if (!cut_fits(dx_cut(dtype, rows, n, width), rows, width) ||
            !cut_fits(dw_cut(dtype, rows, n, width), n, width))
            return false;
    return true;
}

struct EntropyLayout {
    size_t x = 0, w = 0, part = 0, hit = 0, logits = 0, dz = 0, sum = 0, partial = 0, scale = 0, total = 0;
};
EntropyLayout entropy_layout(int64_t rows, int64_t classes, int64_t width, int dtype, bool grad,
                             bool pads) {
    EntropyLayout L;
    Sections s;
    if (pads) {
        L.x = s.add((size_t)rows * pad8(width) * 2);
        L.w = s.add((size_t)classes * pad8(width) * 2);
    }
    if (!grad) {
        const kx::Cut cut = kx::entropy_plan(dtype, rows, classes, width, false);
        if (cut.thin || cut.splits == 1) {
            L.part = s.add((size_t)cdiv(classes, kx::entropy_columns(cut)) * rows * 8);
            L.hit = s.add((size_t)rows * 4);
        } else {
            L.logits = s.add((size_t)cut.splits * rows * classes * 4);
        }
    } else {
        const int64_t count = piece_of(rows, classes, dtype);
        const int64_t last = classes - (classes - 1) / count * count;
        L.dz = s.add((size_t)rows * pad8(count) * size_of(dtype));
        if (count < classes) L.sum = s.add((size_t)rows * width * 4);
        size_t partial = 0, logits = 0;
        for (int64_t n : {count, last}) {
            const int z = kx::entropy_plan(dtype, rows, n, width, true).splits;
            const size_t c = z > 1 ? (size_t)z * rows * n * 4 : 0;
            logits = c > logits ? c : logits;
            const int dx = dx_cut(dtype, rows, n, width).splits;
            const int dw = dw_cut(dtype, rows, n, width).splits;
            const size_t a = dx > 1 ? (size_t)dx * rows * width * 4 : 0;
            const size_t b = dw > 1 ? (size_t)dw * n * width * 4 : 0;
            partial = a > partial ? a : partial;
            partial = b > partial ? b : partial;
        }
        // (The logits' parts are done with before the products' parts are made.)
        L.partial = L.logits = s.add(partial > logits ? partial : logits);
        if (dtype != EXPERTS_F32) L.scale = s.add(8);
    }
    L.total = s.with_slack();
    return L;
}

}  // namespace

extern "C" {

int layers_embed(const int64_t *ids, int64_t tokens, const void *w, int dtype, int64_t classes,
                 int64_t width, double scale, void *out, int64_t ldo, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!embed_shape_ok(tokens, classes, width) || ldo < width) return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!ids || !w || !out) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(ids, 8) || !aligned(w, b) || !aligned(out, b)) return KM_ERR_ALIGN;
    const Span outs[] = {{out, tokens, ldo, width, b}};
    const Span ins[] = {{ids, 1, 0, tokens, 8}, {w, 1, 0, classes * width, b}};
    if (int rc = check_alias(outs, 1, ins, 2)) return rc;
    return status(kx::launch_embed(ids, tokens, w, dtype, classes, width, (float)scale, out, ldo,
                                   (hipStream_t)stream));
}

size_t layers_embed_backward_workspace_bytes(int64_t tokens, int64_t classes, int64_t width,
                                             int dtype) {
    if (!dtype_ok(dtype) || !embed_shape_ok(tokens, classes, width) ||
        !kx::embed_grid_ok(dtype, tokens, classes, width))
        return 0;
    return embed_layout(tokens, classes, width).total;
}

int layers_embed_backward(const void *dy, int64_t lddy, const int64_t *ids, int64_t tokens,
                          int dtype, int64_t classes, int64_t width, double scale, void *dw,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!embed_shape_ok(tokens, classes, width) || lddy < width ||
        !kx::embed_grid_ok(dtype, tokens, classes, width))
        return KM_ERR_SHAPE;
    if (!dw || (tokens > 0 && (!dy || !ids))) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(dy, b) || !aligned(ids, 8) || !aligned(dw, b)) return KM_ERR_ALIGN;
    const EmbedLayout L = embed_layout(tokens, classes, width);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span outs[] = {{dw, 1, 0, classes * width, b}, {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span ins[] = {{dy, tokens, lddy, width, b}, {ids, 1, 0, tokens, 8}};
    if (int rc = check_alias(outs, 2, ins, 2)) return rc;
    char *base = ws_base(workspace);
    kx::EmbedScratch ws = {};
    ws.bucket = (int64_t *)(base + L.bucket);
    ws.order = (int *)(base + L.order);
    ws.place = (int *)(base + L.place);
    ws.sorted = (int *)(base + L.sorted);
    ws.offsets = (int *)(base + L.offsets);
    ws.lo = (int *)(base + L.lo);
    ws.hi = (int *)(base + L.hi);
    ws.partial = (float *)(base + L.partial);
    ws.plan.tile_hist = (int *)(base + L.plan + L.sort.hist);
    ws.plan.count = (int *)(base + L.plan + L.sort.count);
    ws.plan.rank = (unsigned short *)(base + L.plan + L.sort.rank);
    ws.plan.tiles = cdiv(tokens, km::kSortTileRows);
    return status(kx::launch_embed_backward(dy, lddy, ids, tokens, dtype, classes, width, (float)scale,
                                            dw, ws, (hipStream_t)stream));
}

int layers_norm(const void *x, int64_t ldx, const void *weight, const void *bias, int dtype,
                int weights_dtype, int64_t rows, int64_t width, double eps, void *out, int64_t ldo,
                float *mean, float *rstd, void *stream) {
    if (!weights_ok(dtype, weights_dtype) || !(eps >= 0)) return KM_ERR_OP;
    if (!norm_shape_ok(dtype, rows, width) || ldx < width || ldo < width) return KM_ERR_SHAPE;
    if (!mean != !rstd) return KM_ERR_NULL;
    if (rows == 0) return KM_OK;
    if (!x || !out) return KM_ERR_NULL;
    const size_t b = size_of(dtype), wb = size_of(weights_dtype);
    if (!aligned(x, b) || !aligned(out, b) || !aligned(weight, wb) || !aligned(bias, wb) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return KM_ERR_ALIGN;
    const Span outs[] = {{out, rows, ldo, width, b}, {mean, 1, 0, rows, 4}, {rstd, 1, 0, rows, 4}};
    const Span ins[] = {{x, rows, ldx, width, b}, {weight, 1, 0, width, wb}, {bias, 1, 0, width, wb}};
    if (int rc = check_alias(outs, 3, ins, 3)) return rc;
    kx::NormProblem pr = {};
    pr.x = x;
    pr.ldx = ldx;
    pr.weight = weight;
    pr.bias = bias;
    pr.rows = rows;
    pr.width = width;
    pr.eps = (float)eps;
    pr.out = out;
    pr.ldo = ldo;
    pr.mean = mean;
    pr.rstd = rstd;
    return status(kx::launch_norm(dtype, weights_dtype, pr, (hipStream_t)stream));
}

size_t layers_norm_backward_workspace_bytes(int64_t rows, int64_t width, int dtype) {
    if (!dtype_ok(dtype) || !norm_shape_ok(dtype, rows, width)) return 0;
    return round_up((size_t)kx::norm_parts(dtype, rows, width) * 2 * width * 4) + kAlign;
}

int layers_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                         const void *weight, const float *mean, const float *rstd, int dtype,
                         int weights_dtype, int64_t rows, int64_t width, void *dx, int64_t lddx,
                         void *dweight, void *dbias, void *workspace, size_t workspace_bytes,
                         void *stream) {
    if (!weights_ok(dtype, weights_dtype)) return KM_ERR_OP;
    if (!norm_shape_ok(dtype, rows, width) || lddy < width || ldx < width || (dx && lddx < width))
        return KM_ERR_SHAPE;
    if (!dx && !dweight && !dbias) return KM_ERR_NULL;
    if (rows > 0 && (!dy || !x || !mean || !rstd)) return KM_ERR_NULL;
    const size_t b = size_of(dtype), wb = size_of(weights_dtype);
    if (!aligned(dy, b) || !aligned(x, b) || !aligned(weight, wb) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dx, b) || !aligned(dweight, wb) || !aligned(dbias, wb))
        return KM_ERR_ALIGN;
    const bool sums = dweight || dbias;
    if (sums && !ws_ok(workspace, workspace_bytes, layers_norm_backward_workspace_bytes(rows, width, dtype)))
        return KM_ERR_WORKSPACE;
    const Span outs[] = {{dx, rows, lddx, width, b},
                         {dweight, 1, 0, width, wb},
                         {dbias, 1, 0, width, wb},
                         {sums ? workspace : nullptr, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span ins[] = {{dy, rows, lddy, width, b},
                        {x, rows, ldx, width, b},
                        {weight, 1, 0, width, wb},
                        {mean, 1, 0, rows, 4},
                        {rstd, 1, 0, rows, 4}};
    if (int rc = check_alias(outs, 4, ins, 5)) return rc;
    if (rows == 0 && !sums) return KM_OK;
    kx::NormProblem pr = {};
    pr.x = x;
    pr.ldx = ldx;
    pr.dy = dy;
    pr.lddy = lddy;
    pr.weight = weight;
    pr.mean = const_cast<float *>(mean);
    pr.rstd = const_cast<float *>(rstd);
    pr.rows = rows;
    pr.width = width;
    pr.out = dx;
    pr.ldo = lddx;
    pr.dweight = dweight;
    pr.dbias = dbias;
    pr.partial = (float *)ws_base(workspace);
    return status(kx::launch_norm_backward(dtype, weights_dtype, pr, (hipStream_t)stream));
}

int layers_route(const void *logits, int64_t ld, int dtype, int64_t tokens, int64_t experts,
                 int64_t top, int score, const float *bias, int64_t groups, int64_t top_groups,
                 int64_t group_best, int renormalize, double scale, int64_t *ids, float *weights,
                 void *stream) {
    if (!dtype_ok(dtype) || (score != LAYERS_SOFTMAX && score != LAYERS_SIGMOID) || group_best < 1 ||
        group_best > 2)
        return KM_ERR_OP;
    if (!route_shape_ok(tokens, experts, top) || ld < experts || groups < 1 || experts % groups != 0 ||
        top_groups < 1 || top_groups > groups || !kx::route_fits(experts, groups, top))
        return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!logits || !ids || !weights) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(logits, b) || !aligned(bias, 4) || !aligned(ids, 8) || !aligned(weights, 4))
        return KM_ERR_ALIGN;
    const Span outs[] = {{ids, 1, 0, tokens * top, 8}, {weights, 1, 0, tokens * top, 4}};
    const Span ins[] = {{logits, tokens, ld, experts, b}, {bias, 1, 0, experts, 4}};
    if (int rc = check_alias(outs, 2, ins, 2)) return rc;
    kx::RouteProblem pr = {};
    pr.logits = logits;
    pr.ld = ld;
    pr.tokens = tokens;
    pr.experts = (int)experts;
    pr.top = (int)top;
    pr.groups = (int)groups;
    pr.kept = (int)top_groups;
    pr.best = (int)group_best;
    pr.sigmoid = score == LAYERS_SIGMOID;
    pr.renormalize = renormalize != 0;
    pr.bias = bias;
    pr.scale = (float)scale;
    pr.ids = ids;
    pr.weights = weights;
    return status(kx::launch_route(dtype, pr, (hipStream_t)stream));
}

int layers_route_backward(const float *dweights, const void *logits, int64_t ld,
                          const int64_t *ids, int dtype, int64_t tokens, int64_t experts,
                          int64_t top, int score, int renormalize, double scale, void *dlogits,
                          int64_t lddl, void *stream) {
    if (!dtype_ok(dtype) || (score != LAYERS_SOFTMAX && score != LAYERS_SIGMOID)) return KM_ERR_OP;
    if (!route_shape_ok(tokens, experts, top) || ld < experts || lddl < experts) return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!dweights || !logits || !ids || !dlogits) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(logits, b) || !aligned(dlogits, b) || !aligned(ids, 8) || !aligned(dweights, 4))
        return KM_ERR_ALIGN;
    const Span outs[] = {{dlogits, tokens, lddl, experts, b}};
    const Span ins[] = {{logits, tokens, ld, experts, b},
                        {ids, 1, 0, tokens * top, 8},
                        {dweights, 1, 0, tokens * top, 4}};
    if (int rc = check_alias(outs, 1, ins, 3)) return rc;
    kx::RouteProblem pr = {};
    pr.logits = logits;
    pr.ld = ld;
    pr.tokens = tokens;
    pr.experts = (int)experts;
    pr.top = (int)top;
    pr.sigmoid = score == LAYERS_SIGMOID;
    pr.renormalize = renormalize != 0;
    pr.scale = (float)scale;
    pr.chosen = ids;
    pr.dweights = dweights;
    pr.dlogits = dlogits;
    pr.lddl = lddl;
    return status(kx::launch_route_backward(dtype, pr, (hipStream_t)stream));
}

size_t layers_cross_entropy_workspace_bytes(int64_t rows, int64_t classes, int64_t width,
                                            int dtype, int unaligned) {
    if (!dtype_ok(dtype) || !entropy_shape_ok(dtype, rows, classes, width)) return 0;
    const bool pads = dtype != EXPERTS_F32 && (unaligned || width % 2 != 0) &&
                      !kx::entropy_plan(dtype, rows, classes, width, false).thin;
    return entropy_layout(rows, classes, width, dtype, false, pads).total;
}

int layers_cross_entropy(const void *x, int64_t ldx, const void *w, const int64_t *targets,
                         int dtype, int64_t rows, int64_t classes, int64_t width, float *loss,
                         float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!entropy_shape_ok(dtype, rows, classes, width)) return KM_ERR_SHAPE;
    if (rows == 0) return KM_OK;
    if (!x || !w || !targets || !loss || !lse) return KM_ERR_NULL;
    if (!ld_ok(x, ldx, width)) return KM_ERR_SHAPE;
    const size_t b = size_of(dtype);
    if (!aligned(x, b) || !aligned(w, b) || !aligned(targets, 8) || !aligned(loss, 4) || !aligned(lse, 4))
        return KM_ERR_ALIGN;
    const kx::Cut cut = kx::entropy_plan(dtype, rows, classes, width, false);
    const bool pads = dtype != EXPERTS_F32 && !cut.thin &&
                      !(in_place(x, ldx, width) && in_place(w, width, width));
    const EntropyLayout L = entropy_layout(rows, classes, width, dtype, false, pads);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span outs[] = {{loss, 1, 0, rows, 4},
                         {lse, 1, 0, rows, 4},
                         {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span ins[] = {{x, rows, ldx, width, b}, {w, 1, 0, classes * width, b}, {targets, 1, 0, rows, 8}};
    if (int rc = check_alias(outs, 3, ins, 3)) return rc;
    const hipStream_t s = (hipStream_t)stream;
    char *base = ws_base(workspace);
    Operand xq = {x, ldx, width, hipSuccess}, wp = {w, width, width, hipSuccess};
    if (pads) {
        xq = operand(x, ldx, rows, width, dtype, base + L.x, s);
        if (xq.e != hipSuccess) return KM_ERR_HIP;
        wp = operand(w, width, classes, width, dtype, base + L.w, s);
        if (wp.e != hipSuccess) return KM_ERR_HIP;
    }
    kx::EntropyProblem pr = {};
    pr.x = xq.p;
    pr.ldx = xq.ld;
    pr.w = wp.p;
    pr.ldw = wp.ld;
    pr.rows = rows;
    pr.classes = classes;
    pr.width = width;
    pr.targets = targets;
    pr.tile = cut.tile;
    pr.thin = cut.thin ? cut.splits : 0;
    pr.parts = cut.thin ? 1 : cut.splits;
    pr.logits = (float *)(base + L.logits);
    pr.part = (float2 *)(base + L.part);
    pr.hit = (float *)(base + L.hit);
    pr.loss = loss;
    pr.lse = lse;
    pr.first = 0;
    pr.count = classes;
    return status(kx::launch_entropy(dtype, pr, s));
}

size_t layers_cross_entropy_backward_workspace_bytes(int64_t rows, int64_t classes, int64_t width,
                                                     int dtype, int unaligned) {
    if (!dtype_ok(dtype) || !entropy_shape_ok(dtype, rows, classes, width) ||
        !entropy_grad_ok(dtype, rows, classes, width))
        return 0;
    const bool pads = dtype != EXPERTS_F32 && (unaligned || width % 2 != 0);
    return entropy_layout(rows, classes, width, dtype, true, pads).total;
}

int layers_cross_entropy_backward(const float *dloss, const float *dlse, const void *x,
                                  int64_t ldx, const void *w, const int64_t *targets,
                                  const float *lse, int dtype, int64_t rows, int64_t classes,
                                  int64_t width, void *dx, int64_t lddx, void *dw, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!entropy_shape_ok(dtype, rows, classes, width) || !entropy_grad_ok(dtype, rows, classes, width))
        return KM_ERR_SHAPE;
    if (!dx && !dw) return KM_ERR_NULL;
    if (rows > 0 && (!dloss || !x || !w || !targets || !lse)) return KM_ERR_NULL;
    if (!ld_ok(x, ldx, width) || !ld_ok(dx, lddx, width)) return KM_ERR_SHAPE;
    const size_t b = size_of(dtype);
    if (!aligned(dloss, 4) || !aligned(dlse, 4) || !aligned(x, b) || !aligned(w, b) ||
        !aligned(targets, 8) || !aligned(lse, 4) || !aligned(dx, b) || !aligned(dw, b))
        return KM_ERR_ALIGN;
    const bool pads = dtype != EXPERTS_F32 && !(in_place(x, ldx, width) && in_place(w, width, width));
    const EntropyLayout L = entropy_layout(rows, classes, width, dtype, true, pads);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span outs[] = {{dx, rows, lddx, width, b},
                         {dw, 1, 0, classes * width, b},
                         {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span ins[] = {{dloss, 1, 0, rows, 4}, {dlse, 1, 0, rows, 4},    {x, rows, ldx, width, b},
                        {w, 1, 0, classes * width, b}, {targets, 1, 0, rows, 8}, {lse, 1, 0, rows, 4}};
    if (int rc = check_alias(outs, 3, ins, 6)) return rc;
    if (rows == 0 && !dw) return KM_OK;
    const hipStream_t s = (hipStream_t)stream;
    char *base = ws_base(workspace);
    Operand xq = {x, ldx, width, hipSuccess}, wp = {w, width, width, hipSuccess};
    if (rows > 0) xq = operand(x, ldx, rows, width, dtype, base + L.x, s);  // (else w may be NULL)
    if (xq.e != hipSuccess) return KM_ERR_HIP;
    if (rows > 0) wp = operand(w, width, classes, width, dtype, base + L.w, s);
    if (wp.e != hipSuccess) return KM_ERR_HIP;
    kx::EntropyProblem pr = {};
    pr.x = xq.p;
    pr.ldx = xq.ld;
    pr.w = wp.p;
    pr.ldw = wp.ld;
    pr.rows = rows;
    pr.classes = classes;
    pr.width = width;
    pr.targets = targets;
    pr.lse = const_cast<float *>(lse);
    pr.dloss = dloss;
    pr.dlse = dlse;
    pr.dz = base + L.dz;
    pr.logits = (float *)(base + L.logits);
    if (dtype != EXPERTS_F32 && rows > 0) {
        pr.scale = (float *)(base + L.scale);
        pr.most_dz = dtype == EXPERTS_F16 ? 16384.0f : 1.0f;
        if (rows > kx::kOwnScale) {
            if (kx::launch_entropy_scale(pr, s) != hipSuccess) return KM_ERR_HIP;
            pr.most_dz = 0.0f;
        }
    }
    kx::EntropyGrad g = {};
    g.dz = pr.dz;
    g.x = xq.p;
    g.ldx = xq.ld;
    g.x_cols = xq.cols;
    g.ldw = wp.ld;
    g.w_cols = wp.cols;
    g.rows = rows;
    g.width = width;
    g.scale = pr.scale;
    g.dx = rows > 0 ? dx : nullptr;
    g.lddx = lddx;
    g.sum = (float *)(base + L.sum);
    g.partial = (float *)(base + L.partial);
    const int64_t piece = piece_of(rows, classes, dtype);
    for (int64_t first = 0; first < classes; first += piece) {
        const int64_t count = classes - first < piece ? classes - first : piece;
        pr.first = first;
        pr.count = count;
        pr.lddz = pad8(count);
        const kx::Cut cut = kx::entropy_plan(dtype, rows, count, width, true);
        pr.tile = cut.tile;
        pr.parts = cut.splits;
        if (rows > 0 && kx::launch_entropy_dz(dtype, pr, s) != hipSuccess) return KM_ERR_HIP;
        g.w = (const char *)wp.p + (size_t)first * wp.ld * b;
        g.lddz = pr.lddz;
        g.count = count;
        g.first = first == 0;
        g.last = first + count == classes;
        g.dw = dw ? (char *)dw + (size_t)first * width * b : nullptr;
        g.dx_cut = dx_cut(dtype, rows, count, width);
        g.dw_cut = dw_cut(dtype, rows, count, width);
        const int tile = g.dx && g.dw ? kx::both_plan(dtype, rows, count, width, false, 1, g.dx_cut, g.dw_cut) : 0;
        g.together = tile != 0;
        if (tile) {
            g.dx_cut.tile = g.dw_cut.tile = tile;
            g.dx_cut.splits = g.dw_cut.splits = 1;
        }
        if (kx::launch_entropy_grad(dtype, g, s) != hipSuccess) return KM_ERR_HIP;
    }
    return KM_OK;
}

}  // extern "C"
