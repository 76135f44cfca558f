// entropy.hip - what surrounds the products of entropy.h: the choice of the type, the
// joins of the rows' sums and of split depths, and dz's scale.
#include "entropy_rows.h"

namespace kx {

template <typename T>
hipError_t launch_rows_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_entropy_t(const EntropyProblem &pr, bool dz, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dx_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dw_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_both_t(const EntropyGrad &e, hipStream_t s);

namespace {

// R rows a block from row `start` on, 256 / R threads to a row, each joining every (256 / R)-th of
// the column tiles' sums (the largest first, then the sums relative to it).
template <int R>
__global__ __launch_bounds__(256) void entropy_join_kernel(EntropyProblem pr, int tiles, int64_t start) {
    constexpr int kSlices = 256 / R;
    __shared__ float most[kSlices][R + 1], sums[kSlices][R + 1];
    const int r = threadIdx.x % R, slice = threadIdx.x / R;
    const int64_t row = start + (int64_t)blockIdx.x * R + r;
    const bool there = row < pr.rows;
    const float2 *part = pr.part + (there ? row : pr.rows - 1);
    // (Nothing times an overflowing factor would be a NaN.)
    auto scaled = [&](float s, float m, float from) {
        return s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((finite_or_0(m) - from) * kLog2e);
    };
    float m = -INFINITY, s = 0.0f;
    for (int k0 = slice; k0 < tiles; k0 += kSlices * 8) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = k0 + kSlices * u;
            v[u] = part[(int64_t)(k < tiles ? k : k0) * pr.rows];
            if (k >= tiles) v[u] = make_float2(-INFINITY, 0.0f);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) top = fmaxf(top, v[u].x);
        const float from = finite_or_0(top);
        s = scaled(s, m, from);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += scaled(v[u].y, v[u].x, from);
        m = top;
    }
    most[slice][r] = m;
    sums[slice][r] = s;
    __syncthreads();
    // Halves join until 16 slices are left, which one thread a row adds.
    for (int half = kSlices / 2; half >= 16; half /= 2) {
        if (slice < half) {
            const float other = most[slice + half][r], top = fmaxf(m, other), from = finite_or_0(top);
            s = scaled(s, m, from) + scaled(sums[slice + half][r], other, from);
            m = top;
            most[slice][r] = m;
            sums[slice][r] = s;
        }
        __syncthreads();
    }
    if (slice != 0 || !there) return;
    for (int k = 1; k < 16; ++k) m = fmaxf(m, most[k][r]);
    const float from = finite_or_0(m);
    float sum = 0.0f;
    for (int k = 0; k < 16; ++k) sum += scaled(sums[k][r], most[k][r], from);
    const float lse = from + logf(sum);
    const int64_t t = pr.targets[row];
    pr.lse[row] = lse;
    pr.loss[row] = t >= 0 && t < pr.classes ? lse - pr.hit[row] : 0.0f;
}

__global__ __launch_bounds__(1024) void entropy_scale_kernel(EntropyProblem pr) {
    __shared__ float memory[16];
    float inverse;
    const float scale = scale_from(largest_factor(pr, threadIdx.x, 1024), pr.most_dz, memory, inverse);
    if (threadIdx.x != 0) return;
    pr.scale[0] = scale;
    pr.scale[1] = inverse;
}

// Logits left in parts by a product whose depth was cut (few tiles of it): eight columns of a row.
__device__ __forceinline__ void logits_of(const EntropyProblem &pr, int64_t row, int64_t n, float (&z)[8]) {
    const int valid = (int)(pr.count - n < 8 ? pr.count - n : 8);
    load_row(pr.logits + row * pr.count + n, valid, z);
#pragma unroll 4
    for (int k = 1; k < pr.parts; ++k) {
        float x[8];
        load_row(pr.logits + ((int64_t)k * pr.rows + row) * pr.count + n, valid, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += x[i];
    }
}

// One wave to a row: its loss and lse.
__global__ __launch_bounds__(256) void entropy_row_kernel(EntropyProblem pr) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= pr.rows) return;
    const int lane = threadIdx.x & 63;
    const int target = class_of(pr.targets[row], pr.classes);
    RowSum sum = {-INFINITY, 0.0f};
    float hit = 0.0f;
    for (int64_t n = lane * 8; n < pr.count; n += 512) {
        float z[8], m = -INFINITY, s = 0.0f;
        logits_of(pr, row, n, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (n + i >= pr.count) z[i] = -INFINITY;
            if (n + i == target) hit = z[i];
            m = fmaxf(m, z[i]);
        }
        const float from = finite_or_0(m);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += __builtin_amdgcn_exp2f((z[i] - from) * kLog2e);
        sum.add(m, s);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        sum.add(__shfl_xor(sum.m, d), __shfl_xor(sum.s, d));
        hit += __shfl_xor(hit, d);  // zeros, but for one lane
    }
    if (lane != 0) return;
    const float lse = finite_or_0(sum.m) + logf(sum.s);
    pr.lse[row] = lse;
    pr.loss[row] = target >= 0 ? lse - hit : 0.0f;
}

// dz: eight columns of a row a thread.
template <typename T>
__global__ __launch_bounds__(256) void entropy_dz_rows_kernel(EntropyProblem pr) {
    __shared__ float memory[4];
    const float scale = scale_of(pr, memory);
    const int64_t chunks = pr.lddz / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = id / chunks, n = (id - row * chunks) * 8;
    if (row >= pr.rows) return;
    float z[8];
    logits_of(pr, row, n, z);
    dz_of(z, (int)n, terms_of(pr, row, scale));
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = n + i < pr.count ? z[i] : 0.0f;
    store_row((T *)pr.dz + row * pr.lddz + n, z, 8);
}

template <typename T>
hipError_t launch_parts(const EntropyProblem &pr, hipStream_t s) {
    RowsProblem r = {};
    r.q = pr.x;
    r.ldq = pr.ldx;
    r.p = (const T *)pr.w + pr.first * pr.ldw;
    r.ldp = pr.ldw;
    r.rows = pr.rows;
    r.cols = pr.count;
    r.depth = pr.width;
    r.experts = 1;
    r.tile = pr.tile;
    r.splits = pr.parts;
    r.partial = pr.logits;
    return launch_rows_t<T>(r, s);
}
template <typename T>
hipError_t entropy_t(const EntropyProblem &pr, hipStream_t s) {
    if (pr.parts > 1) {
        const hipError_t e = launch_parts<T>(pr, s);
        return e != hipSuccess ? e : launch(entropy_row_kernel, cdiv(pr.rows, 4), 256, 0, s, pr);
    }
    const hipError_t e = launch_entropy_t<T>(pr, false, s);
    if (e != hipSuccess) return e;
    const Cut cut = {pr.tile, pr.thin, pr.thin != 0, 0.0};
    // A block to a row of many tiles: 2 rows of 1079 tiles 10.9 us with 16 threads to a row, 4.7.
    const int tiles = (int)cdiv(pr.count, entropy_columns(cut));
    if (pr.rows <= 512 && tiles > 64)
        return launch(entropy_join_kernel<1>, pr.rows, 256, 0, s, pr, tiles, (int64_t)0);
    // (One dispatch holds less than 2^32 work-items, 16 of them a row.)
    constexpr int64_t kMost = 1 << 27;
    hipError_t done = hipSuccess;
    for (int64_t start = 0; start < pr.rows && done == hipSuccess; start += kMost) {
        const int64_t rows = pr.rows - start < kMost ? pr.rows - start : kMost;
        done = launch(entropy_join_kernel<16>, cdiv(rows, 16), 256, 0, s, pr, tiles, start);
    }
    return done;
}
template <typename T>
hipError_t dz_t(const EntropyProblem &pr, hipStream_t s) {
    if (pr.parts <= 1) return launch_entropy_t<T>(pr, true, s);
    const hipError_t e = launch_parts<T>(pr, s);
    if (e != hipSuccess) return e;
    return launch(entropy_dz_rows_kernel<T>, cdiv(pr.rows * (pr.lddz / 8), 256), 256, 0, s, pr);
}

// A product whose depth was split: eight columns of a row to S threads of the block, each of
// which adds every S-th part; their sums in order, then the piece before.
// (64 parts of 2 x 498 with one thread 23.5 us.)
template <typename T, int S>
__global__ __launch_bounds__(256) void entropy_parts_kernel(const float *__restrict__ partial,
                                                            int splits, int64_t rows, int64_t cols,
                                                            float *__restrict__ sum, bool first,
                                                            bool last, const float *__restrict__ scale,
                                                            T *__restrict__ out, int64_t ldo) {
    constexpr int kOwn = 256 / S;
    __shared__ float sums[S > 1 ? S : 1][kOwn][8];
    const int64_t chunks = (cols + 7) / 8;
    const int own = threadIdx.x % kOwn, slice = threadIdx.x / kOwn;
    const int64_t id = (int64_t)blockIdx.x * kOwn + own;
    const int64_t m = id / chunks, n = (id - m * chunks) * 8;
    const bool there = m < rows;
    const int valid = there ? (int)(cols - n < 8 ? cols - n : 8) : 0;
    float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
    for (int k = slice; k < splits; k += S) {
        float x[8];
        load_row(partial + ((int64_t)k * rows + m) * cols + n, valid, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += x[i];
    }
    if (S > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[slice][own][i] = z[i];
        __syncthreads();
        if (slice != 0) return;
#pragma unroll
        for (int k = 1; k < S; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] += sums[k][own][i];
    }
    if (!there) return;
    if (!first) {
        float x[8];
        load_row(sum + m * cols + n, valid, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += x[i];
    }
    if (!last) {
        store_row(sum + m * cols + n, z, valid);
        return;
    }
    const float alpha = scale ? scale[1] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= alpha;
    store_row(out + m * ldo + n, z, valid);
}
template <typename T>
hipError_t join_parts(const float *partial, int splits, int64_t rows, int64_t cols, float *sum, bool first,
                      bool last, const float *scale, void *out, int64_t ldo, hipStream_t s) {
    const int64_t own = rows * cdiv(cols, 8);
    if (splits > 8)
        return launch(entropy_parts_kernel<T, 8>, cdiv(own, 32), 256, 0, s, partial, splits, rows, cols, sum,
                      first, last, scale, (T *)out, ldo);
    return launch(entropy_parts_kernel<T, 1>, cdiv(own, 256), 256, 0, s, partial, splits, rows, cols, sum, first,
                  last, scale, (T *)out, ldo);
}

template <typename T>
hipError_t grad_t(const EntropyGrad &g, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (g.rows == 0)  // a sum of no parts
        return join_parts<T>(nullptr, 0, g.count, g.width, nullptr, true, true, nullptr, g.dw, g.width, s);
    if (g.together) return launch_entropy_both_t<T>(g, s);
    if (g.dx) {
        e = launch_entropy_dx_t<T>(g, s);
        if (e == hipSuccess && g.dx_cut.splits > 1)
            e = join_parts<T>(g.partial, g.dx_cut.splits, g.rows, g.width, g.sum, g.first, g.last, g.scale,
                              g.dx, g.lddx, s);
    }
    if (e != hipSuccess || !g.dw) return e;
    e = launch_entropy_dw_t<T>(g, s);
    if (e == hipSuccess && g.dw_cut.splits > 1)
        e = join_parts<T>(g.partial, g.dw_cut.splits, g.count, g.width, nullptr, true, true, g.scale, g.dw,
                          g.width, s);
    return e;
}

}  // namespace

Cut entropy_plan(int dtype, int64_t rows, int64_t classes, int64_t width, bool grad) {
    if (!grad && rows <= 32) {
        const int groups = classes >= 16384 ? 4 : classes >= 8192 ? 2 : 1;  // a block a compute unit
        return {rows <= 16 ? 16 : 32, groups, true, 0.0};
    }
    return plan_in_parts(dtype, rows, classes, width, 8);
}
int entropy_columns(const Cut &cut) {
    if (cut.thin) return 16 * cut.splits;
    return cut.tile == 129 ? 128 : cut.tile == 32 ? 64 : cut.tile;
}

hipError_t launch_entropy(int dtype, const EntropyProblem &pr, hipStream_t s) {
    if (dtype == 0) return entropy_t<float>(pr, s);
    return dtype == 1 ? entropy_t<bf16>(pr, s) : entropy_t<f16>(pr, s);
}
hipError_t launch_entropy_dz(int dtype, const EntropyProblem &pr, hipStream_t s) {
    if (dtype == 0) return dz_t<float>(pr, s);
    return dtype == 1 ? dz_t<bf16>(pr, s) : dz_t<f16>(pr, s);
}
hipError_t launch_entropy_scale(const EntropyProblem &pr, hipStream_t s) {
    return launch(entropy_scale_kernel, 1, 1024, 0, s, pr);
}
hipError_t launch_entropy_grad(int dtype, const EntropyGrad &g, hipStream_t s) {
    if (dtype == 0) return grad_t<float>(g, s);
    return dtype == 1 ? grad_t<bf16>(g, s) : grad_t<f16>(g, s);
}

}  // namespace kx
