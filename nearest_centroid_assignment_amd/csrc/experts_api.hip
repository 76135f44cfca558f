// experts_api.hip - the C ABI declared in include/experts_mi355x.h.
//
// Every entry point validates its arguments on the host before the first HIP
// call, carves its sections out of the caller's workspace and enqueues the
// kernels on the caller's stream. Nothing here allocates, waits or keeps state.
#include <math.h>

#include <algorithm>
#include <new>

#include "api_checks.h"

namespace {

bool act_ok(int a) { return a >= EXPERTS_ACT_NONE && a <= EXPERTS_ACT_SILU; }

// Whether a range that is written overlaps any other range. Sorts them.
struct Range {
    uintptr_t lo, hi;
    bool written;
};
bool any_overlap(Range *r, int64_t n) {
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t written_to = 0, to = 0;  // ends of the ranges so far
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].lo < (r[i].written ? to : written_to)) return true;
        to = std::max(to, r[i].hi);
        if (r[i].written) written_to = std::max(written_to, r[i].hi);
    }
    return false;
}

// ------------------------------------------------------------------ tokens

bool tokens_shape_ok(int64_t tokens, int64_t top) {
    return tokens >= 0 && tokens <= kMaxRows && top >= 1 && top <= kMaxTop &&
           tokens <= kMaxRows / top;
}
// A block of 256 threads a token at most.
bool rows_shape_ok(int64_t tokens, int64_t top, int64_t width) {
    return tokens_shape_ok(tokens, top) && width >= 1 && width <= kMaxRows;
}

// ------------------------------------------------------------------ linear

bool linear_shape_ok(int64_t rows, int64_t outs, int64_t ins, int64_t experts) {
    return rows >= 0 && rows <= kMaxRows && outs >= 1 && outs <= kMaxWidth && ins >= 1 &&
           ins <= kMaxWidth && experts >= 1 && experts <= kMaxExperts;
}
bool linear_grid_ok(int dtype, int op, int64_t rows, int64_t outs, int64_t ins, bool grouped,
                    int64_t experts) {
    // The padded copies take a thread for every eight values.
    if (dtype != EXPERTS_F32 && (rows * cdiv(ins, 8) + 256 > kMaxGridThreads ||
                                 experts * outs * cdiv(ins, 8) + 256 > kMaxGridThreads))
        return false;
    if (op == 0) return kx::rows_grid_ok(dtype, rows, outs, ins, grouped, experts, false);
    return kx::rows_grid_ok(dtype, rows, ins, outs, grouped, experts, true) &&
           kx::grad_grid_ok(dtype, rows, outs, ins, experts) &&
           cdiv(outs + 8, 256) * experts * kx::slope_splits(rows, outs, experts) <= kMaxGridThreads / 512;
}

// Sections of the workspace. Every one that a call of this shape may need;
// those for rows that do not lie on 4-byte boundaries only with `pads`.
struct LinearLayout {
    size_t x = 0, w = 0, dz = 0, partial = 0, total = 0;
};
LinearLayout linear_layout(int64_t rows, int64_t outs, int64_t ins, int64_t experts, bool grouped,
                           int dtype, int op, bool pads) {
    LinearLayout L;
    size_t off = 0;
    if (pads) {
        L.x = off;
        off += round_up((size_t)rows * pad8(ins) * 2);
        L.w = off;
        off += round_up((size_t)experts * outs * pad8(ins) * 2);
    }
    // Partial sums of one kernel after another: the largest.
    size_t partial = 0;
    auto most = [&](int64_t parts, int64_t n) {
        const size_t bytes = parts > 1 ? (size_t)parts * (size_t)n * 4 : 0;
        partial = bytes > partial ? bytes : partial;
    };
    if (op == 0) {
        most(kx::rows_plan(dtype, rows, outs, ins, grouped, experts, false).splits, rows * outs);
    } else {
        L.dz = off;
        off += round_up((size_t)rows * pad8(outs) * size_of(dtype));
        most(kx::slope_splits(rows, outs, experts), experts * outs);
        most(kx::rows_plan(dtype, rows, ins, outs, grouped, experts, true).splits, rows * ins);
        most(kx::grad_plan(dtype, rows, outs, ins, experts).splits, experts * outs * ins);
    }
    L.partial = off;
    off += round_up(partial);
    L.total = off + kAlign;
    return L;
}

}  // namespace

extern "C" {

size_t experts_plan_workspace_bytes(int64_t tokens, int64_t top, int64_t experts) {
    if (!tokens_shape_ok(tokens, top) || experts < 1 || experts > kMaxExperts) return 0;
    return plan_layout(tokens * top, experts).total;
}

int experts_plan(const int64_t *ids, int64_t tokens, int64_t top, int64_t experts, int32_t *order,
                 int32_t *place, int32_t *offsets, void *workspace, size_t workspace_bytes,
                 void *stream) {
    if (!tokens_shape_ok(tokens, top) || experts < 1 || experts > kMaxExperts) return KM_ERR_SHAPE;
    const int64_t pairs = tokens * top;
    if (!offsets || (pairs > 0 && (!ids || !order || !place))) return KM_ERR_NULL;
    if (!aligned(ids, 8) || !aligned(order, 4) || !aligned(place, 4) || !aligned(offsets, 4))
        return KM_ERR_ALIGN;
    const PlanLayout L = plan_layout(pairs, experts);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span outs[] = {{order, 1, 0, pairs, 4},
                         {place, 1, 0, pairs, 4},
                         {offsets, 1, 0, experts + 1, 4},
                         {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span ins[] = {{ids, 1, 0, pairs, 8}};
    if (int rc = check_alias(outs, 4, ins, 1)) return rc;
    char *base = ws_base(workspace);
    kx::PlanScratch ws;
    ws.tile_hist = (int *)(base + L.hist);
    ws.count = (int *)(base + L.count);
    ws.rank = (unsigned short *)(base + L.rank);
    ws.tiles = cdiv(pairs, km::kSortTileRows);
    return status(kx::launch_plan(ids, pairs, experts, order, place, offsets, ws,
                                  (hipStream_t)stream));
}

int experts_dispatch(const void *x, int64_t ldx, int dtype, int64_t tokens, int64_t top,
                     int64_t width, const int32_t *order, const int32_t *place, void *xs,
                     int64_t ldxs, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!rows_shape_ok(tokens, top, width) || ldx < width || ldxs < width ||
        tokens * 256 > kMaxGridThreads)
        return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!x || !order || !place || !xs) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(x, b) || !aligned(xs, b) || !aligned(order, 4) || !aligned(place, 4))
        return KM_ERR_ALIGN;
    const int64_t pairs = tokens * top;
    const Span outs[] = {{xs, pairs, ldxs, width, b}};
    const Span ins[] = {{x, tokens, ldx, width, b}, {order, 1, 0, pairs, 4}, {place, 1, 0, pairs, 4}};
    if (int rc = check_alias(outs, 1, ins, 3)) return rc;
    return status(kx::launch_dispatch(x, ldx, dtype, tokens, top, width, order, place, xs, ldxs,
                                      (hipStream_t)stream));
}

int experts_dispatch_backward(const void *dxs, int64_t lddxs, int dtype, int64_t tokens,
                              int64_t top, int64_t width, const int32_t *place, void *dx,
                              int64_t lddx, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!rows_shape_ok(tokens, top, width) || lddxs < width || lddx < width ||
        tokens * 256 > kMaxGridThreads)
        return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!dxs || !place || !dx) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(dxs, b) || !aligned(dx, b) || !aligned(place, 4)) return KM_ERR_ALIGN;
    const Span outs[] = {{dx, tokens, lddx, width, b}};
    const Span ins[] = {{dxs, tokens * top, lddxs, width, b}, {place, 1, 0, tokens * top, 4}};
    if (int rc = check_alias(outs, 1, ins, 2)) return rc;
    return status(kx::launch_combine(dxs, lddxs, nullptr, dtype, tokens, top, width, place, dx,
                                     lddx, (hipStream_t)stream));
}

int experts_combine(const void *ys, int64_t ldys, const float *weights, int dtype, int64_t tokens,
                    int64_t top, int64_t width, const int32_t *place, void *y, int64_t ldy,
                    void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!rows_shape_ok(tokens, top, width) || ldys < width || ldy < width ||
        tokens * 256 > kMaxGridThreads)
        return KM_ERR_SHAPE;
    if (tokens == 0) return KM_OK;
    if (!ys || !weights || !place || !y) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(ys, b) || !aligned(y, b) || !aligned(weights, 4) || !aligned(place, 4))
        return KM_ERR_ALIGN;
    const int64_t pairs = tokens * top;
    const Span outs[] = {{y, tokens, ldy, width, b}};
    const Span ins[] = {{ys, pairs, ldys, width, b}, {weights, 1, 0, pairs, 4}, {place, 1, 0, pairs, 4}};
    if (int rc = check_alias(outs, 1, ins, 3)) return rc;
    return status(kx::launch_combine(ys, ldys, weights, dtype, tokens, top, width, place, y, ldy,
                                     (hipStream_t)stream));
}

int experts_combine_backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                             const float *weights, int dtype, int64_t tokens, int64_t top,
                             int64_t width, const int32_t *order, const int32_t *place, void *dys,
                             int64_t lddys, float *dweights, void *stream) {
    if (!dtype_ok(dtype)) return KM_ERR_OP;
    if (!rows_shape_ok(tokens, top, width) || lddy < width || (dweights && ldys < width) ||
        (dys && lddys < width) || tokens * top * 64 > kMaxGridThreads - 256)
        return KM_ERR_SHAPE;
    if (!dys && !dweights) return KM_ERR_NULL;
    if (tokens == 0) return KM_OK;
    if (!dy || !place || !order || (dys && !weights) || (dweights && !ys)) return KM_ERR_NULL;
    const size_t b = size_of(dtype);
    if (!aligned(dy, b) || !aligned(ys, b) || !aligned(weights, 4) || !aligned(dys, b) ||
        !aligned(dweights, 4) || !aligned(order, 4) || !aligned(place, 4))
        return KM_ERR_ALIGN;
    const int64_t pairs = tokens * top;
    const Span outs[] = {{dys, pairs, lddys, width, b}, {dweights, 1, 0, pairs, 4}};
    const Span ins[] = {{dy, tokens, lddy, width, b},
                        {dweights ? ys : nullptr, pairs, ldys, width, b},
                        {weights, 1, 0, pairs, 4},
                        {order, 1, 0, pairs, 4},
                        {place, 1, 0, pairs, 4}};
    if (int rc = check_alias(outs, 2, ins, 5)) return rc;
    return status(kx::launch_combine_backward(dy, lddy, ys, ldys, weights, dtype, tokens, top,
                                              width, order, place, dys, lddys, dweights,
                                              (hipStream_t)stream));
}

size_t experts_linear_workspace_bytes(int64_t rows, int64_t outs, int64_t ins, int64_t experts,
                                      int dtype, int op, int unaligned) {
    if (!linear_shape_ok(rows, outs, ins, experts) || !dtype_ok(dtype) || op < 0 || op > 1 ||
        !linear_grid_ok(dtype, op, rows, outs, ins, true, experts))
        return 0;
    auto bytes = [&](bool grouped) {
        // (The kernel for few rows reads any rows in place.)
        const bool pads = dtype != EXPERTS_F32 && (unaligned || ins % 2 != 0) &&
                          !(op == 0 && kx::rows_plan(dtype, rows, outs, ins, grouped, experts, false).thin);
        return linear_layout(rows, outs, ins, experts, grouped, dtype, op, pads).total;
    };
    // Without offsets a single expert may be cut differently; both fit.
    const size_t grouped = bytes(true), dense = experts == 1 ? bytes(false) : 0;
    return dense > grouped ? dense : grouped;
}

int experts_linear(const void *x, int64_t ldx, const void *w, const void *bias,
                   const void *residual, int64_t ldr, const int32_t *offsets, int dtype, int act,
                   int64_t rows, int64_t outs, int64_t ins, int64_t experts, void *out,
                   int64_t ldo, void *pre, int64_t ldpre, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype) || !act_ok(act)) return KM_ERR_OP;
    if (!linear_shape_ok(rows, outs, ins, experts) || (!offsets && experts != 1) ||
        !linear_grid_ok(dtype, 0, rows, outs, ins, offsets != nullptr, experts))
        return KM_ERR_SHAPE;
    if (!w || (rows > 0 && (!x || !out))) return KM_ERR_NULL;
    if (!ld_ok(x, ldx, ins) || !ld_ok(out, ldo, outs) || !ld_ok(residual, ldr, outs) ||
        !ld_ok(pre, ldpre, outs))
        return KM_ERR_SHAPE;
    const size_t b = size_of(dtype);
    if (!aligned(x, b) || !aligned(w, b) || !aligned(bias, b) || !aligned(residual, b) ||
        !aligned(out, b) || !aligned(pre, b) || !aligned(offsets, 4))
        return KM_ERR_ALIGN;
    const kx::Cut cut = kx::rows_plan(dtype, rows, outs, ins, offsets != nullptr, experts, false);
    const bool pads = dtype != EXPERTS_F32 && !cut.thin &&
                      !(in_place(x, ldx, ins) && in_place(w, ins, ins));
    const LinearLayout L =
        linear_layout(rows, outs, ins, experts, offsets != nullptr, dtype, 0, pads);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span os[] = {{out, rows, ldo, outs, b},
                       {pre, rows, ldpre, outs, b},
                       {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span is[] = {{x, rows, ldx, ins, b},
                       {w, 1, 0, experts * outs * ins, b},
                       {bias, 1, 0, experts * outs, b},
                       {residual, rows, ldr, outs, b},
                       {offsets, 1, 0, experts + 1, 4}};
    if (int rc = check_alias(os, 3, is, 5)) return rc;
    if (rows == 0) return KM_OK;
    const hipStream_t s = (hipStream_t)stream;
    char *base = ws_base(workspace);
    Operand xq = {x, ldx, ins, hipSuccess}, wp = {w, ins, ins, hipSuccess};
    if (pads) {
        xq = operand(x, ldx, rows, ins, dtype, base + L.x, s);
        if (xq.e != hipSuccess) return KM_ERR_HIP;
        wp = operand(w, ins, experts * outs, ins, dtype, base + L.w, s);
        if (wp.e != hipSuccess) return KM_ERR_HIP;
    }
    kx::RowsProblem pr = {};
    pr.tile = cut.tile;
    pr.splits = cut.splits;
    pr.partial = (float *)(base + L.partial);
    pr.q = xq.p;
    pr.ldq = xq.ld;
    pr.p = wp.p;
    pr.ldp = wp.ld;
    pr.p_expert = outs * wp.ld;
    pr.rows = rows;
    pr.cols = outs;
    pr.depth = ins;
    pr.p_rows = false;
    pr.offsets = offsets;
    pr.experts = (int)experts;
    pr.bias = bias;
    pr.residual = residual;
    pr.ldr = ldr;
    pr.out = out;
    pr.ldo = ldo;
    pr.pre = pre;
    pr.ldpre = ldpre;
    pr.act = act;
    return status(kx::launch_rows(dtype, pr, cut.thin, s));
}

int experts_linear_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                            const void *w, const void *pre, int64_t ldpre, const void *in_pre,
                            int64_t ldin, const int32_t *offsets, int dtype, int act, int in_act,
                            int64_t rows, int64_t outs, int64_t ins, int64_t experts, void *dx,
                            int64_t lddx, void *dw, void *dbias, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype) || !act_ok(act) || !act_ok(in_act)) return KM_ERR_OP;
    if (!linear_shape_ok(rows, outs, ins, experts) || (!offsets && experts != 1) ||
        !linear_grid_ok(dtype, 1, rows, outs, ins, offsets != nullptr, experts))
        return KM_ERR_SHAPE;
    if (!dx && !dw && !dbias) return KM_ERR_NULL;
    if (rows > 0 && (!dy || (act != EXPERTS_ACT_NONE && !pre) || (dx && !w) || (dw && !x)))
        return KM_ERR_NULL;
    if (!ld_ok(dy, lddy, outs) || (dw && !ld_ok(x, ldx, ins)) ||
        (act != EXPERTS_ACT_NONE && !ld_ok(pre, ldpre, outs)) || !ld_ok(dx, lddx, ins) ||
        (dx && !ld_ok(in_pre, ldin, ins)))
        return KM_ERR_SHAPE;
    const size_t b = size_of(dtype);
    if (!aligned(dy, b) || !aligned(x, b) || !aligned(w, b) || !aligned(pre, b) ||
        !aligned(in_pre, b) || !aligned(dx, b) || !aligned(dw, b) || !aligned(dbias, b) ||
        !aligned(offsets, 4))
        return KM_ERR_ALIGN;
    const bool half = dtype != EXPERTS_F32;
    const bool pads = half && ((dw && !in_place(x, ldx, ins)) || (dx && !in_place(w, ins, ins)));
    const bool grouped = offsets != nullptr;
    const LinearLayout L = linear_layout(rows, outs, ins, experts, grouped, dtype, 1, pads);
    if (!ws_ok(workspace, workspace_bytes, L.total)) return KM_ERR_WORKSPACE;
    const Span os[] = {{dx, rows, lddx, ins, b},
                       {dw, 1, 0, experts * outs * ins, b},
                       {dbias, 1, 0, experts * outs, b},
                       {workspace, 1, 0, (int64_t)workspace_bytes, 1}};
    const Span is[] = {{dy, rows, lddy, outs, b},
                       {dw ? x : nullptr, rows, ldx, ins, b},
                       {dx ? w : nullptr, 1, 0, experts * outs * ins, b},
                       {act != EXPERTS_ACT_NONE ? pre : nullptr, rows, ldpre, outs, b},
                       {dx ? in_pre : nullptr, rows, ldin, ins, b},
                       {offsets, 1, 0, experts + 1, 4}};
    if (int rc = check_alias(os, 4, is, 6)) return rc;
    const hipStream_t s = (hipStream_t)stream;
    char *base = ws_base(workspace);
    // dz: dy itself, or its product with act', or dy on 4-byte boundaries.
    const bool products = dx || dw;
    const bool copy = products && (act != EXPERTS_ACT_NONE || (half && !in_place(dy, lddy, outs)));
    const void *dz = dy;
    int64_t lddz = lddy, dz_cols = outs;
    if (copy) {
        dz = base + L.dz;
        lddz = dz_cols = half ? pad8(outs) : outs;
    }
    const bool dx_runs = dx && rows > 0;
    kx::Cut rcut = {}, gcut = {};
    if (dx_runs) rcut = kx::rows_plan(dtype, rows, ins, outs, grouped, experts, true);
    if (dw) gcut = kx::grad_plan(dtype, rows, outs, ins, experts);
    const int tile =
        dx_runs && dw ? kx::both_plan(dtype, rows, outs, ins, grouped, experts, rcut, gcut) : 0;
    kx::SlopeSum sum = {};
    if (copy || dbias) {
        const hipError_t e = kx::launch_slope(dtype, dy, lddy, pre, ldpre, act, offsets,
                                              (int)experts, rows, outs, copy ? (void *)dz : nullptr,
                                              lddz, dbias, (float *)(base + L.partial),
                                              tile ? &sum : nullptr, s);
        if (e != hipSuccess) return KM_ERR_HIP;
    }
    kx::RowsProblem r = {};
    kx::GradProblem g = {};
    if (dx_runs) {
        const Operand wp = operand(w, ins, experts * outs, ins, dtype, base + L.w, s);
        if (wp.e != hipSuccess) return KM_ERR_HIP;
        r.tile = tile ? tile : rcut.tile;
        r.splits = tile ? 1 : rcut.splits;
        r.partial = (float *)(base + L.partial);
        r.q = dz;
        r.ldq = lddz;
        r.p = wp.p;
        r.ldp = wp.ld;
        r.p_expert = outs * wp.ld;
        r.rows = rows;
        r.cols = ins;
        r.depth = outs;
        r.p_cols = wp.cols;
        r.p_rows = true;
        r.offsets = offsets;
        r.experts = (int)experts;
        r.in_pre = in_pre;
        r.ldin = ldin;
        r.in_act = in_act;
        r.out = dx;
        r.ldo = lddx;
    }
    if (dw) {
        const Operand xp = operand(x, ldx, rows, ins, dtype, base + L.x, s);
        if (xp.e != hipSuccess) return KM_ERR_HIP;
        g.tile = tile ? tile : gcut.tile;
        g.splits = tile ? 1 : gcut.splits;
        g.partial = (float *)(base + L.partial);
        g.x = xp.p;
        g.ldx = xp.ld;
        g.x_cols = xp.cols;
        g.dz = dz;
        g.lddz = lddz;
        g.dz_cols = dz_cols;
        g.rows = rows;
        g.m_cols = outs;
        g.n_cols = ins;
        g.offsets = offsets;
        g.experts = (int)experts;
        g.out = dw;
    }
    if (tile) return status(kx::launch_both(dtype, r, g, sum, s));
    if (dx_runs && kx::launch_rows(dtype, r, rcut.thin, s) != hipSuccess) return KM_ERR_HIP;
    if (dw && kx::launch_grad(dtype, g, s) != hipSuccess) return KM_ERR_HIP;
    return KM_OK;
}

int64_t experts_adamw_state_elements(const int64_t *numels, int64_t count) {
    if (count < 0 || (count > 0 && !numels)) return -1;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (numels[i] < 0 || numels[i] > ((int64_t)1 << 44)) return -1;
        total += cdiv(numels[i], 256) * 256;
        if (total > ((int64_t)1 << 44)) return -1;
    }
    return total;
}

int experts_adamw_step(void *const *params, const void *const *grads, void *const *copies,
                       const int64_t *numels, int64_t count, int param_dtype, int grad_dtype,
                       void *m, void *v, float *m_scale, float *v_scale, int bits, double lr,
                       double beta1, double beta2, double eps, double weight_decay, int64_t step,
                       const float *grad_scale, void *stream) {
    if (!dtype_ok(param_dtype) || !dtype_ok(grad_dtype) || (bits != 8 && bits != 32))
        return KM_ERR_OP;
    // The negated forms also refuse NaN.
    if (!(lr >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
        !(weight_decay >= 0) || step < 1)
        return KM_ERR_OP;
    const int64_t total = experts_adamw_state_elements(numels, count);
    if (total < 0) return KM_ERR_SHAPE;
    if (total == 0) return KM_OK;
    if (!params || !grads || !m || !v || (bits == 8 && (!m_scale || !v_scale))) return KM_ERR_NULL;
    const size_t ps = size_of(param_dtype), gs = size_of(grad_dtype), ms = bits == 8 ? 1 : 4;
    if (!aligned(m, ms) || !aligned(v, ms) || !aligned(m_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(grad_scale, 4))
        return KM_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        if (numels[i] == 0) continue;
        if (!params[i] || !grads[i] || (copies && !copies[i])) return KM_ERR_NULL;
        if (!aligned(params[i], ps) || !aligned(grads[i], gs) || (copies && !aligned(copies[i], 2)))
            return KM_ERR_ALIGN;
    }
    // The ranges of all tensors: a tensor given twice would be stepped by two workgroups
    // at once. (Up to 32 tensors on the stack.)
    const int64_t scales = bits == 8 ? total / 256 : 0;
    constexpr int64_t kOwn = 101;
    Range own[kOwn], *ranges = own;
    if (count > (kOwn - 5) / 3) ranges = new (std::nothrow) Range[3 * count + 5];
    if (!ranges) return KM_ERR_HIP;  // no host memory left
    int64_t n = 0;
    auto add = [&](const void *p, int64_t len, size_t size, bool written) {
        if (p && len > 0) ranges[n++] = {(uintptr_t)p, (uintptr_t)p + (size_t)len * size, written};
    };
    add(m, total, ms, true);
    add(v, total, ms, true);
    add(m_scale, scales, 4, true);
    add(v_scale, scales, 4, true);
    add(grad_scale, 1, 4, false);
    for (int64_t i = 0; i < count; ++i) {
        add(params[i], numels[i], ps, true);
        add(grads[i], numels[i], gs, false);
        // A bfloat16 parameter may be its own copy.
        if (copies && !(copies[i] == params[i] && param_dtype == EXPERTS_BF16))
            add(copies[i], numels[i], 2, true);
    }
    const bool overlapping = any_overlap(ranges, n);
    if (ranges != own) delete[] ranges;
    if (overlapping) return KM_ERR_ALIAS;
    kx::AdamwStep st;
    st.beta1 = (float)beta1;
    st.one_minus_beta1 = (float)(1.0 - beta1);
    st.beta2 = (float)beta2;
    st.one_minus_beta2 = (float)(1.0 - beta2);
    st.keep = (float)(1.0 - lr * weight_decay);
    st.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    st.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    st.eps = (float)eps;
    st.grad_scale = grad_scale;
    st.m = m;
    st.v = v;
    st.m_scale = m_scale;
    st.v_scale = v_scale;
    st.param_dtype = param_dtype;
    st.grad_dtype = grad_dtype;
    st.bits = bits;
    return status(kx::launch_adamw(params, grads, copies, numels, count, st, (hipStream_t)stream));
}

int experts_adamw_moments(const int8_t *m, const uint8_t *v, const float *m_scale,
                          const float *v_scale, int64_t elements, float *m_out, float *v_out,
                          void *stream) {
    if (elements < 0 || elements % 256 != 0 || elements / 4 > kMaxGridThreads) return KM_ERR_SHAPE;
    if (!m_out && !v_out) return KM_ERR_NULL;
    if (elements == 0) return KM_OK;
    if ((m_out && (!m || !m_scale)) || (v_out && (!v || !v_scale))) return KM_ERR_NULL;
    if (!aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(m_out, 4) || !aligned(v_out, 4))
        return KM_ERR_ALIGN;
    const Span outs[] = {{m_out, 1, 0, elements, 4}, {v_out, 1, 0, elements, 4}};
    const Span ins[] = {{m_out ? m : nullptr, 1, 0, elements, 1},
                        {v_out ? v : nullptr, 1, 0, elements, 1},
                        {m_out ? m_scale : nullptr, 1, 0, elements / 256, 4},
                        {v_out ? v_scale : nullptr, 1, 0, elements / 256, 4}};
    if (int rc = check_alias(outs, 2, ins, 4)) return rc;
    return status(kx::launch_moments(m, v, m_scale, v_scale, elements, m_out, v_out,
                                     (hipStream_t)stream));
}

}  // extern "C"
