// linear.hip - what surrounds the tiled products (linear.h): the choice of the
// type, padded copies of 16-bit rows, and dz = dy * act'(pre) with its column
// sums.
#include "experts.h"

namespace kx {

template <typename T>
hipError_t launch_rows_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_thin_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_grad_t(const GradProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_both_t(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                         hipStream_t s);

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

// The join of a product whose depth was split: eight columns of a row a thread,
// the parts added in order, then the epilogue.
template <typename T>
__global__ __launch_bounds__(256) void join_rows_kernel(RowsProblem pr) {
    const int64_t chunks = (pr.cols + 7) / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = id / chunks;
    const int n = (int)(id - m * chunks) * 8;
    if (m >= pr.rows) return;
    const int valid = (int)pr.cols - n < 8 ? (int)pr.cols - n : 8;
    int expert = 0;
    if (pr.offsets) {  // the first expert whose rows end past m
        int lo = 0, hi = pr.experts;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pr.offsets[mid + 1] > m)
                hi = mid;
            else
                lo = mid + 1;
        }
        expert = lo;
    }
    const bool tail = expert == pr.experts && pr.offsets;
    const int64_t part = pr.rows * pr.cols;
    const float *p = pr.partial + m * pr.cols + n;
    float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (!tail) {
#pragma unroll 4
        for (int s = 0; s < pr.splits; ++s) {
            if (valid == 8) {
                float x[8];
                load_vec(p + s * part, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += x[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < valid) z[i] += p[s * part + i];
            }
        }
    }
    const T *bias = (const T *)pr.bias, *res = (const T *)pr.residual, *in = (const T *)pr.in_pre;
    T x[8];
    if (bias && !tail) {
        load_row(bias + (int64_t)expert * pr.cols + n, valid, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += (float)x[i];
    }
    if (pr.pre) store_row((T *)pr.pre + m * pr.ldpre + n, z, valid);
    apply_act(z, pr.act);
    if (res && !tail) {
        load_row(res + m * pr.ldr + n, valid, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += (float)x[i];
    }
    if (in && !tail) {
        load_row(in + m * pr.ldin + n, valid, x);
        apply_slope(z, x, pr.in_act);
    }
    store_row((T *)pr.out + m * pr.ldo + n, z, valid);
}

template <typename T>
__global__ __launch_bounds__(256) void join_grad_kernel(const float *__restrict__ partial,
                                                        int splits, int64_t n, T *__restrict__ out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    if (i + 4 <= n) {
        float z[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            float x[4];
            load_vec(partial + s * n + i, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] += x[j];
        }
        T r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = (T)z[j];
        store_vec(out + i, r);
    } else {
        for (int64_t j = i; j < n; ++j) {
            float z = 0.0f;
            for (int s = 0; s < splits; ++s) z += partial[s * n + j];
            out[j] = (T)z;
        }
    }
}

template <typename T>
hipError_t rows_t(const RowsProblem &pr, bool thin, hipStream_t s) {
    const hipError_t e = thin ? launch_thin_t<T>(pr, s) : launch_rows_t<T>(pr, s);
    if (e != hipSuccess || pr.splits == 1) return e;
    return launch(join_rows_kernel<T>, cdiv(pr.rows * cdiv(pr.cols, 8), 256), 256, 0, s, pr);
}
template <typename T>
hipError_t grad_t(const GradProblem &pr, hipStream_t s) {
    const hipError_t e = launch_grad_t<T>(pr, s);
    if (e != hipSuccess || pr.splits == 1) return e;
    const int64_t n = pr.m_cols * pr.n_cols * pr.experts;
    return launch(join_grad_kernel<T>, cdiv(n, 1024), 256, 0, s, pr.partial, pr.splits, n, (T *)pr.out);
}

// dz = dy * act'(pre) is rounded to T for the products, the one rounding here that torch's
// own float32 forms do not have: the 16-bit matrix instructions take nothing wider. It adds
// an error as large as that of rounding dx and dw (8192 x 8192 x 2048 bf16 with gelu, norm of
// the error against 64 bits over the norm: 0.0017 -> 0.0024); a second product with what the
// rounding leaves would double both products. float32 tensors keep dz in float32, and dbias
// sums dz before it is rounded.
//
// One block: 64 * V columns (a lane has V of them) of the rows of part s of
// expert e, its four waves taking every fourth row. Each column's partial sum is
// a float32 sum in a fixed order: a wave's rows in turn, the four waves, and
// then (slope_sum_kernel) the parts.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(256) void slope_kernel(const T *__restrict__ dy, int64_t lddy,
                                                    const T *__restrict__ pre, int64_t ldpre,
                                                    const int *__restrict__ offsets,
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
                if (ACT != kActNone) {  // the products read dz, not these
                    load_once(dy + r * lddy + c, y[u]);
                    load_once(pre + r * ldpre + c, z[u]);
                } else {
                    load_vec(dy + r * lddy + c, y[u]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    y[u][j] = c + j < outs ? dy[r * lddy + c + j] : (T)0.0f;
                    z[u][j] = ACT != kActNone && c + j < outs ? pre[r * ldpre + c + j] : (T)0.0f;
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
                if (ACT != kActNone) v *= slope_of<ACT>((float)z[u][j]);
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
__global__ __launch_bounds__(256) void slope_sum_kernel(SlopeSum sum) {
    __shared__ float quarter[256];
    slope_sum<T>(sum, blockIdx.x, quarter);
}

template <typename T>
hipError_t slope_t(const void *dy, int64_t lddy, const void *pre, int64_t ldpre, int act,
                   const int *offsets, int experts, int64_t rows, int64_t outs, void *dz,
                   int64_t lddz, void *dbias, float *partial, SlopeSum *later, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int splits = (int)slope_splits(rows, outs, experts);
    const int64_t width = dz && lddz > outs ? lddz : outs;
    const int64_t cb = cdiv(width, 64 * V);
    hipError_t e = hipSuccess;
    with_act(act, [&](auto tag) {
        e = launch(slope_kernel<T, V, decltype(tag)::value>, cb * splits * experts, 256, 0, s,
                   (const T *)dy, lddy, (const T *)pre, ldpre, offsets, experts, rows, outs, (T *)dz,
                   lddz, (T *)dbias, partial, splits, (int)cb);
    });
    if (e != hipSuccess || !dbias || splits == 1) return e;
    const SlopeSum sum = {partial, splits, (int64_t)experts * outs, dbias};
    if (later) {
        *later = sum;
        return e;
    }
    return launch(slope_sum_kernel<T>, cdiv(sum.n, 64), 256, 0, s, sum);
}

}  // namespace

namespace {

// What a cut costs, in microseconds: a tile's stage costs `each` on a compute unit that
// is kept busy by its tiles (`apart` times that where rows do not start on lines of 128
// bytes, and a stage's rows touch two), and `wait` on top per stage for latency that
// nothing hides; a round of tiles costs `edge` for its first loads and its epilogue;
// joining split depths writes and reads the sums. The constants are fitted to 354 sizes
// (64 to 8192 a side, up to 16 experts), each in every tile and in 1 to 8 parts: what the
// model takes is 2.6 % (16 bits) and 3.2 % (float32) slower than the best of them in the
// geometric mean. Longer sides and more experts are extrapolated.
//   (bf16: 512 x 1024 with depth 4096 37 us in 128 tiles of 64, 20 in four parts; 188 x
//   4096 with depth 776 8 us in 64s, 15 in two parts or in 128s; 8192 x 4098 with
//   depth 2050 312 us in 64s, 215 in 256s.)
struct TileCost {
    int tile, rows, cols;
    double each, wait, edge, apart;
};
constexpr TileCost kHalf[] = {{256, 256, 256, 1.30, 0.10, 10.0, 1.2},
                              {128, 128, 128, 0.50, 0.35, 2.5, 1.0},
                              {64, 64, 64, 0.14, 0.40, 0.9, 1.5}};
constexpr TileCost kFloat[] = {{128, 128, 128, 2.25, 0.10, 7.5, 1.0},
                               {64, 64, 64, 0.42, 0.20, 2.0, 1.0},
                               {32, 32, 64, 0.23, 0.20, 1.4, 1.0}};
constexpr double kBytes = 6.0e6;  // that operands pass at, a microsecond
constexpr double kSetup = 0.8;    // what a round costs more where its blocks look their rows up

bool lines(int64_t len, int64_t size) { return len * size % 128 == 0; }

// tiles_of(rows, cols): the number of tiles of that size; bytes: of the operands;
// sums: values to join.
template <class F>
Cut best_cut(int dtype, int64_t stages, int64_t bytes, int64_t sums, bool grouped,
             bool on_lines, F tiles_of, int most_parts = 8) {
    Cut best = {64, 1, false, 0.0};
    double least = 1e300;
    for (const TileCost &c : dtype == 0 ? kFloat : kHalf) {
        const int64_t tiles = tiles_of(c.rows, c.cols);
        for (int parts = 1; parts <= most_parts; parts *= 2) {
            if (parts > 1 && (stages / parts < 4 || tiles * parts > 1024)) break;
            const double rounds = (double)cdiv(tiles * parts, 256);
            const double each = c.each * (on_lines ? 1.0 : c.apart);
            const double edge = c.edge + (grouped ? kSetup : 0.0);
            const double memory = (double)bytes / kBytes + edge;
            double t = (double)cdiv(stages, parts) * (rounds * each + c.wait) + rounds * edge;
            if (t < memory) t = memory;
            if (parts > 1) t += 4.0 + (double)parts * (double)sums * 8.0 / 3e6;
            if (t < least) {
                least = t;
                best = {c.tile, parts, false, t};
            }
        }
    }
    return best;
}

// Groups that may have rows, and the row tiles to expect: half a tile lost per group,
// and one to each at least.
int64_t groups_of(int64_t rows, bool grouped, int64_t experts) {
    const int64_t groups = grouped ? (experts < rows ? experts : rows) : 1;
    return groups < 1 ? 1 : groups;
}
int64_t row_tiles(int64_t rows, int64_t bm, bool grouped, int64_t experts) {
    if (!grouped) return cdiv(rows, bm);
    const int64_t groups = groups_of(rows, grouped, experts), n = rows / bm + groups / 2;
    return n < groups ? groups : n;
}
}  // namespace

Cut rows_plan(int dtype, int64_t rows, int64_t cols, int64_t depth, bool grouped, int64_t experts,
              bool p_rows) {
    const int64_t groups = groups_of(rows, grouped, experts), each = rows / groups;
    auto tiles = [&](int64_t m, int64_t n) {
        return row_tiles(rows, m, grouped, experts) * cdiv(cols, n);
    };
    // Few rows and too few tiles to stream w with: 16 x 4096 with depth 4096 10 us
    // against 15 in eight parts of 64s; but 16 x 4096 of 16 experts 45 against 43.
    if (!p_rows && each <= 32 && groups * cdiv(cols, 64) < 256) return {each <= 16 ? 16 : 32, 1, true, 0.0};
    const int64_t size = dtype == 0 ? 4 : 2;
    Cut c = best_cut(dtype, cdiv(depth * size, 128), (rows + groups * cols) * depth * size, rows * cols,
                     grouped, lines(depth, size) && (!p_rows || lines(cols, size)), tiles);
    // Three stages in LDS where a compute unit has one tile at most anyhow (two stages leave
    // room for two tiles). bf16, two / three stages: 2374 x 1164 with depth 3133 49.7 / 44.2
    // us, 545 x 2880 with depth 7872 in two parts 50.4 / 43.0, 2000 x 2048 with depth 1024
    // 14.3 / 14.5; dx and dw within 5 % either way. Past 256 tiles: dw of 826 x 743 x 914, 16
    // experts, 25.7 / 27.8, of 6932 x 1068 x 3888, 4 experts, 82 / 134.
    const int64_t most = most_row_tiles(rows, 128, grouped, experts) * cdiv(cols, 128);
    if (c.tile == 128 && dtype != 0 && most <= 256) c.tile = 129;
    return c;
}

Cut plan_in_parts(int dtype, int64_t rows, int64_t cols, int64_t depth, int most_parts) {
    auto tiles = [&](int64_t m, int64_t n) { return cdiv(rows, m) * cdiv(cols, n); };
    const int64_t size = dtype == 0 ? 4 : 2;
    Cut c = best_cut(dtype, cdiv(depth * size, 128), (rows + cols) * depth * size, rows * cols, false,
                     lines(depth, size), tiles, most_parts);
    if (c.tile == 128 && dtype != 0 && tiles(128, 128) <= 256) c.tile = 129;
    return c;
}

Cut grad_plan(int dtype, int64_t rows, int64_t m_cols, int64_t n_cols, int64_t experts) {
    auto tiles = [&](int64_t m, int64_t n) { return cdiv(m_cols, m) * cdiv(n_cols, n) * experts; };
    const int64_t size = dtype == 0 ? 4 : 2;
    Cut c = best_cut(dtype, cdiv(rows / experts * size, 128), rows * (m_cols + n_cols) * size,
                     m_cols * n_cols * experts, false, lines(m_cols, size) && lines(n_cols, size),
                     tiles);
    if (c.tile == 128 && dtype != 0 && tiles(128, 128) <= 256) c.tile = 129;
    return c;
}

// One launch leaves no compute unit idle between the two and saves a launch. Blocks
// that all run at once meet the compute units in turn, the longer ones first; more of
// them even out.
//   (dx and dw, two launches -> one: 1000 x 1111 x 777 float32 54 us -> 45, bf16 1024^3
//   17 -> 12, 2048^3 60 -> 39, 256 x 2048 x 2048 20 -> 17, 16 experts 8192 x 4096 x 1024
//   220 -> 163; but 512 x 2048 x 1000 float32, dx four times as long as dw, 51 -> 57.)
int both_plan(int dtype, int64_t rows, int64_t outs, int64_t ins, bool grouped, int64_t experts,
              const Cut &dx, const Cut &dw) {
    const int64_t size = dtype == 0 ? 4 : 2;
    const double depth_dx = (double)cdiv(outs * size, 128);
    const double depth_dw = (double)cdiv(rows / experts * size, 128);
    const bool on_lines = lines(outs, size) && lines(ins, size);
    const double bytes = (double)(2 * rows * (outs + ins) + 2 * experts * outs * ins) * size;
    double least = dx.cost + dw.cost + 2.0;
    int best = 0;
    for (const TileCost &c : dtype == 0 ? kFloat : kHalf) {
        if (c.tile == 32) continue;
        const int64_t ndx = row_tiles(rows, c.rows, grouped, experts) * cdiv(ins, c.cols);
        const int64_t ndw = cdiv(outs, c.rows) * cdiv(ins, c.cols) * experts;
        const int64_t most = most_row_tiles(rows, c.rows, grouped, experts) * cdiv(ins, c.cols) + ndw;
        if (most + 256 + cdiv(experts * outs, 64) > kMaxGridThreads / 512) continue;
        const double each = c.each * (on_lines ? 1.0 : c.apart);
        const double tdx = depth_dx * each + c.edge + (grouped ? kSetup : 0.0);
        const double tdw = depth_dw * each + c.edge;
        const bool dx_long = tdx >= tdw;
        const double tl = dx_long ? tdx : tdw, ts = dx_long ? tdw : tdx;
        const int64_t nl = dx_long ? ndx : ndw, n = ndx + ndw;
        // Bound by memory past the caches, nothing idles: 16 rows of 16 experts, 4096 x
        // 2048, 84 us -> 90.
        const double busy = ((double)ndx * depth_dx + (double)ndw * depth_dw) * each / 256;
        if (bytes > 256 << 20 && busy < bytes / kBytes) continue;
        const int together = c.tile == 256 ? 1 : c.tile == 128 ? 2 : 4;  // blocks on a compute unit
        double t;
        if (n <= 256 * together)
            t = (double)cdiv(nl, 256) * tl + (double)(cdiv(n, 256) - cdiv(nl, 256)) * ts;
        else
            t = ((double)ndx * tdx + (double)ndw * tdw) / 256;
        if (t < tl) t = tl;
        if (n > 256 * together) t += 0.5 * ts;
        t += (depth_dx > depth_dw ? depth_dx : depth_dw) * c.wait;
        if (t < least) {
            least = t;
            best = c.tile;
        }
    }
    return best;
}

bool rows_grid_ok(int dtype, int64_t rows, int64_t cols, int64_t depth, bool grouped,
                  int64_t experts, bool p_rows) {
    const Cut c = rows_plan(dtype, rows, cols, depth, grouped, experts, p_rows);
    const int64_t m = c.tile == 129 ? 128 : c.tile, n = c.thin ? 16 : c.tile == 32 ? 64 : m;
    const int64_t blocks = most_row_tiles(rows, m, grouped, experts) * cdiv(cols, n) * c.splits;
    return blocks + 8 <= kMaxGridThreads / 512 && cdiv(rows * cdiv(cols, 8), 256) <= kMaxGridThreads / 256;
}
bool grad_grid_ok(int dtype, int64_t rows, int64_t m_cols, int64_t n_cols, int64_t experts) {
    const Cut c = grad_plan(dtype, rows, m_cols, n_cols, experts);
    const int64_t m = c.tile == 129 ? 128 : c.tile, n = c.tile == 32 ? 64 : m;
    const int64_t blocks = cdiv(m_cols, m) * cdiv(n_cols, n) * experts * c.splits;
    return blocks + 128 <= kMaxGridThreads / 512;
}

hipError_t launch_rows(int dtype, const RowsProblem &pr, bool thin, hipStream_t s) {
    if (pr.rows == 0) return hipSuccess;
    if (dtype == 0) return rows_t<float>(pr, thin, s);
    return dtype == 1 ? rows_t<bf16>(pr, thin, s) : rows_t<f16>(pr, thin, s);
}
hipError_t launch_grad(int dtype, const GradProblem &pr, hipStream_t s) {
    if (dtype == 0) return grad_t<float>(pr, s);
    return dtype == 1 ? grad_t<bf16>(pr, s) : grad_t<f16>(pr, s);
}
hipError_t launch_both(int dtype, const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                       hipStream_t s) {
    if (dtype == 0) return launch_both_t<float>(r, g, sum, s);
    return dtype == 1 ? launch_both_t<bf16>(r, g, sum, s) : launch_both_t<f16>(r, g, sum, s);
}

hipError_t launch_pad_rows(const void *src, int64_t lds, int64_t rows, int64_t cols, void *dst,
                           int64_t ldd, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    return launch(pad_rows_kernel, cdiv(rows * (ldd / 8), 256), 256, 0, s, (const uint16_t *)src, lds,
                  rows, cols, (uint16_t *)dst, ldd);
}

// Parts of an expert's rows: about 4096 blocks in all, 16 rows a part at least (one
// group of loads a wave).
int64_t slope_splits(int64_t rows, int64_t outs, int64_t experts) {
    const int64_t blocks = cdiv(outs, 256) * experts;
    int64_t n = 4096 / blocks;
    const int64_t most = rows / experts / 16;
    n = n > most ? most : n;
    return n < 1 ? 1 : n > 128 ? 128 : n;
}

hipError_t launch_slope(int dtype, const void *dy, int64_t lddy, const void *pre, int64_t ldpre,
                        int act, const int *offsets, int experts, int64_t rows, int64_t outs,
                        void *dz, int64_t lddz, void *dbias, float *partial, SlopeSum *later,
                        hipStream_t s) {
    if (dtype == 0)
        return slope_t<float>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz,
                              dbias, partial, later, s);
    if (dtype == 1)
        return slope_t<bf16>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz,
                             dbias, partial, later, s);
    return slope_t<f16>(dy, lddy, pre, ldpre, act, offsets, experts, rows, outs, dz, lddz, dbias,
                        partial, later, s);
}

}  // namespace kx
