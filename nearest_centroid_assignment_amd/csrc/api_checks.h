// api_checks.h - what the entry points of experts_api.hip and layers_api.hip check and
// carve on the host.
#pragma once

#include "../../include/experts_mi355x.h"
#include "experts.h"
#include "kernels.h"

namespace {

constexpr int64_t kMaxRows = 2147483647;      // rows, pairs < 2^31
constexpr int64_t kMaxWidth = 1 << 20;        // outs, ins, ld of the products: a tile of 256
                                              // rows stays below 2^31 bytes
constexpr int64_t kMaxExperts = 65536;
constexpr int64_t kMaxTop = 64;
constexpr size_t kAlign = 256;
constexpr int64_t kMaxGridThreads = 4294967295LL;  // one dispatch dimension, in work-items

size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool dtype_ok(int d) { return d >= EXPERTS_F32 && d <= EXPERTS_F16; }
size_t size_of(int dtype) { return dtype == EXPERTS_F32 ? 4 : 2; }
bool aligned(const void *p, size_t a) { return (uintptr_t)p % a == 0; }

char *ws_base(void *workspace) {
    return (char *)(((uintptr_t)workspace + kAlign - 1) / kAlign * kAlign);
}

// Whether the workspace holds `total` bytes; one that holds slack alone (no
// section) may be left out.
bool ws_ok(const void *workspace, size_t bytes, size_t total) {
    return total <= kAlign || (workspace && bytes >= total);
}

// An array of rows (ld apart) of len elements.
struct Span {
    const void *p;
    int64_t rows, ld, len;
    size_t elem;
};
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.len <= 0 || b.len <= 0) return false;
    const uintptr_t alo = (uintptr_t)a.p, blo = (uintptr_t)b.p;
    const uintptr_t ahi = alo + ((uintptr_t)(a.rows - 1) * a.ld + a.len) * a.elem;
    const uintptr_t bhi = blo + ((uintptr_t)(b.rows - 1) * b.ld + b.len) * b.elem;
    if (alo >= bhi || blo >= ahi) return false;
    // Rows equally far apart: b's start `at` bytes into a's, and where they lie past a's
    // end and end before a's next row (columns of one buffer), no two rows meet.
    const uintptr_t step = (uintptr_t)a.ld * a.elem;
    if (a.rows > 1 && b.rows > 1 && step == (uintptr_t)b.ld * b.elem) {
        const uintptr_t at = blo >= alo ? (blo - alo) % step : (step - (alo - blo) % step) % step;
        if (at >= a.len * a.elem && at + b.len * b.elem <= step) return false;
    }
    return true;
}
int check_alias(const Span *outs, int n_outs, const Span *ins, int n_ins) {
    for (int i = 0; i < n_outs; ++i) {
        for (int j = 0; j < n_ins; ++j)
            if (overlap(outs[i], ins[j])) return KM_ERR_ALIAS;
        for (int j = i + 1; j < n_outs; ++j)
            if (overlap(outs[i], outs[j])) return KM_ERR_ALIAS;
    }
    return KM_OK;
}
int status(hipError_t e) { return e == hipSuccess ? KM_OK : KM_ERR_HIP; }

struct PlanLayout {
    size_t hist, count, rank, total;
};
PlanLayout plan_layout(int64_t pairs, int64_t experts) {
    PlanLayout L = {0, 0, 0, kAlign};
    if (kx::plan_is_small(pairs, experts)) return L;
    const int64_t tiles = cdiv(pairs, km::kSortTileRows);
    size_t off = 0;
    L.hist = off;
    off += round_up((size_t)tiles * (size_t)experts * sizeof(int));
    L.count = off;
    off += round_up((size_t)experts * sizeof(int));
    L.rank = off;
    off += round_up((size_t)pairs * sizeof(unsigned short));
    L.total = off + kAlign;
    return L;
}

int64_t pad8(int64_t n) { return cdiv(n, 8) * 8; }
bool ld_ok(const void *p, int64_t ld, int64_t len) {
    return p == nullptr || (ld >= len && ld <= kMaxWidth);
}
// Whether the 16-bit products can read rows of `len` in place.
bool in_place(const void *p, int64_t ld, int64_t len) {
    return aligned(p, 4) && ld % 2 == 0 && len % 2 == 0;
}

struct Operand {
    const void *p;
    int64_t ld, cols;  // cols: readable columns
    hipError_t e;
};
// The rows in place, or their padded copy.
Operand operand(const void *p, int64_t ld, int64_t rows, int64_t len, int dtype, void *pad,
                hipStream_t s) {
    if (dtype == EXPERTS_F32 || in_place(p, ld, len)) return {p, ld, len, hipSuccess};
    const int64_t n = pad8(len);
    return {pad, n, n, kx::launch_pad_rows(p, ld, rows, len, pad, n, s)};
}

}  // namespace
