// linear.hip - what surrounds the tiled products (linear.h): the choice of the
// type, padded copies of 16-bit rows, and dz = dy * act'(pre) with its column
// sums.
#include "experts.h"

namespace kx {

template <typename T>
hipError_t launch_rows_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_grad_t(const GradProblem &pr, hipStream_t s);

namespace {

constexpr int64_t kMaxGridThreads = 4294967295LL;  // one dispatch dimension, in work-items

// dst[r][c] = src[r][c], c < cols, and 0 for cols <= c < ldd: eight values a
// thread, so that a row starts on 16 bytes. Bound by memory; it runs only where
// the products could not read the rows in place.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t *__restrict__ src,
                                                       int64_t lds, int64_t rows, int64_t cols,
                                                       uint16_t *__restrict__ dst, int64_t ldd) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t chunks = ldd / 8;
    const int64_t r = i / chunks, c = (i - r * chunks) * 8;
    if (r >= rows) return;
    uint16_t v[8];
    const uint16_t *p = src + r * lds + c;
    if (c + 8 <= cols) {
        load_vec(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? p[j] : (uint16_t)0;
    }
    store_vec(dst + r * ldd + c, v);
}

// One block: 64 * V columns (a lane has V of them) of the rows of part s of
// expert e, its four waves taking every fourth row. Each column's partial sum is
// a float32 sum in a fixed order: a wave's rows in turn, the four waves, and
// then (slope_sum_kernel) the parts.
template <typename T, int V>
__global__ __launch_bounds__(256) void slope_kernel(const T *__restrict__ dy, int64_t lddy,
                                                    const T *__restrict__ pre, int64_t ldpre,
                                                    int act, const int *__restrict__ offsets,
                                                    int experts, int64_t rows, int64_t outs,
                                                    T *__restrict__ dz, int64_t lddz,
                                                    T *__restrict__ dbias,
                                                    float *__restrict__ partial, int splits,
                                                    int col_blocks) {
    __shared__ float part[4][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = ((int64_t)(blockIdx.x % col_blocks) * 64 + lane) * V;
    const int64_t es = blockIdx.x / col_blocks;
    const int s = (int)(es % splits), e = (int)(es / splits);
    int64_t lo = 0, hi = rows;
    if (offsets) {
        lo = offsets[e];
        hi = offsets[e + 1];
        lo = lo < 0 ? 0 : lo > rows ? rows : lo;
        hi = hi < lo ? lo : hi > rows ? rows : hi;
    }
    const int64_t n = hi - lo;
    const int64_t r0 = lo + n * s / splits, r1 = lo + n * (s + 1) / splits;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    const bool full = c + V <= outs;
    // kRows rows of a wave at a time, all their loads in flight together.
    constexpr int kRows = 4;
    for (int64_t rr = r0 + wave; rr < r1; rr += 4 * kRows) {
        T y[kRows][V], z[kRows][V];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = rr + 4 * u < r1 ? rr + 4 * u : rr;  // no condition on the loads
            if (full) {
                load_vec(dy + r * lddy + c, y[u]);
                if (pre) load_vec(pre + r * ldpre + c, z[u]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    y[u][j] = c + j < outs ? dy[r * lddy + c + j] : (T)0.0f;
                    z[u][j] = pre && c + j < outs ? pre[r * ldpre + c + j] : (T)0.0f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int64_t r = rr + 4 * u;
            if (r >= r1) break;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = (float)y[u][j];
                if (pre) v *= act_slope((float)z[u][j], act);
                sum[j] += v;
                y[u][j] = (T)v;
            }
            if (dz) {
                if (c + V <= lddz) {
                    store_vec(dz + r * lddz + c, y[u]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (c + j < lddz) dz[r * lddz + c + j] = y[u][j];
                }
            }
        }
    }
    if (!dbias) return;
#pragma unroll
    for (int j = 0; j < V; ++j) part[wave][lane * V + j] = sum[j];
    __syncthreads();
    for (int j = threadIdx.x; j < 64 * V; j += 256) {
        const int64_t col = (int64_t)(blockIdx.x % col_blocks) * 64 * V + j;
        if (col >= outs) continue;
        const float v = ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j];
        if (splits == 1)
            dbias[(int64_t)e * outs + col] = (T)v;
        else
            partial[((int64_t)s * experts + e) * outs + col] = v;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void slope_sum_kernel(const float *__restrict__ partial,
                                                        int splits, int64_t n,
                                                        T *__restrict__ dbias) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.0f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += partial[s * n + i];
    dbias[i] = (T)v;
}

template <typename T>
hipError_t slope_t(const void *dy, int64_t lddy, const void *pre, int64_t ldpre, int act,
                   const int *offsets, int experts, int64_t rows, int64_t outs, void *dz,
                   int64_t lddz, void *dbias, float *partial, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int splits = (int)slope_splits(rows, outs, experts);
    const int64_t width = dz && lddz > outs ? lddz : outs;
    const int64_t cb = cdiv(width, 64 * V);
    slope_kernel<T, V><<<(unsigned)(cb * splits * experts), 256, 0, s>>>(
        (const T *)dy, lddy, act == kActNone ? nullptr : (const T *)pre, ldpre, act, offsets,
        experts, rows, outs, (T *)dz, lddz, (T *)dbias, partial, splits, (int)cb);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !dbias || splits == 1) return e;
    const int64_t n = (int64_t)experts * outs;
    slope_sum_kernel<T><<<(unsigned)cdiv(n, 256), 256, 0, s>>>(partial, splits, n, (T *)dbias);
    return hipGetLastError();
}

}  // namespace

// The smallest tile is 64 x 64 with 256 threads; larger ones need fewer.
bool rows_grid_ok(int dtype, int64_t rows, int64_t cols, int64_t depth, int experts) {
    (void)dtype;
    (void)depth;
    const int64_t tiles = (rows / 64 + experts + 1) * cdiv(cols, 64);
    return tiles <= kMaxGridThreads / 1024;
}
bool grad_grid_ok(int dtype, int64_t m_cols, int64_t n_cols, int experts) {
    (void)dtype;
    return cdiv(m_cols, 64) * cdiv(n_cols, 64) * experts <= kMaxGridThreads / 1024;
}

hipError_t launch_rows(int dtype, const RowsProblem &pr, hipStream_t s) {
    if (pr.rows == 0) return hipSuccess;
    if (dtype == 0) return launch_rows_t<float>(pr, s);
    return dtype == 1 ? launch_rows_t<bf16>(pr, s) : launch_rows_t<f16>(pr, s);
}
hipError_t launch_grad(int dtype, const GradProblem &pr, hipStream_t s) {
    if (dtype == 0) return launch_grad_t<float>(pr, s);
    return dtype == 1 ? launch_grad_t<bf16>(pr, s) : launch_grad_t<f16>(pr, s);
}

hipError_t launch_pad_rows(const void *src, int64_t lds, int64_t rows, int64_t cols, void *dst,
                           int64_t ldd, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    pad_rows_kernel<<<(unsigned)cdiv(rows * (ldd / 8), 256), 256, 0, s>>>(
        (const uint16_t *)src, lds, rows, cols, (uint16_t *)dst, ldd);
    return hipGetLastError();
}

// Parts of an expert's rows: about 4096 blocks in all, 64 rows a part at least.
int64_t slope_splits(int64_t rows, int64_t outs, int64_t experts) {
    const int64_t blocks = cdiv(outs, 256) * experts;
    int64_t n = 4096 / blocks;
    const int64_t most = rows / experts / 64;
    n = n > most ? most : n;
    return n < 1 ? 1 : n > 128 ? 128 : n;
}

hipError_t launch_slope(int dtype, const void *dy, int64_t lddy, const void *pre, int64_t ldpre,
                        int act, const int *offsets, int experts, int64_t rows, int64_t outs,
                        void *dz, int64_t lddz, void *dbias, float *partial, hipStream_t s) {
    if (dtype == 0)
        return slope_t<float>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz,
                              dbias, partial, s);
    if (dtype == 1)
        return slope_t<bf16>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz,
                             dbias, partial, s);
    return slope_t<f16>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz, dbias,
                        partial, s);
}

}  // namespace kx
