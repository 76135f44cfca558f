// entropy.h - softmax cross entropy of x w^T against one class a row, without the
// logits in memory; instantiated per type by entropy_f32.hip, entropy_bf16.hip,
// entropy_f16.hip.
//
//   z = x w^T,  lse = log sum_j e^z_j,  loss = lse - z_target
//   a = dloss + dlse, b = dloss (both without dloss where the target is no class)
//   dz_j = a e^(z_j - lse) - b [j = target],  dx = dz w,  dw = dz^T x
//
// Bound by the matrix units: 2 rows classes width operations for the loss, three times
// that with the gradient, which computes z once more (the price of not keeping it: a
// fourth product). The tiles are those of linear.h. Forward: the epilogue of a tile
// leaves, for each of its rows, the largest logit and the sum of e^(z - largest) over its
// columns (8 bytes for 64 to 256 logits), from the accumulators; a second kernel joins
// them. Gradient, for one piece of the classes after another: dz of the piece (in the
// operands' type) is the epilogue of z's product; then dw of the piece, and dx summed
// over the pieces in float32.
#pragma once

#include "entropy_rows.h"
#include "linear.h"

namespace kx {
namespace {

// acc = the tile (mt, nt) of x w^T over the piece's classes.
template <class S>
__device__ __forceinline__ void entropy_tile(const EntropyProblem &pr, int m0, int n0, lds_char *smem,
                                             int wave, int lane, f32x4 (&acc)[S::TM][S::TN]) {
    typedef typename S::type T;
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    const char *q = (const char *)pr.x + (int64_t)m0 * pr.ldx * sizeof(T);
    const char *p = (const char *)pr.w + (pr.first + n0) * pr.ldw * sizeof(T);
    typename S::TileP tp;
    typename S::TileQ tq;
    tp.init(p, pr.ldw, pr.count - n0, (int)pr.width, wave, lane);
    tq.init(q, pr.ldx, pr.rows - m0, (int)pr.width, wave, lane);
    run_product<S>(smem, tp, tq, (int)pr.width, wave, lane, acc);
}

// The block's tile of the piece's; false: none.
template <class S>
__device__ __forceinline__ bool entropy_place(const EntropyProblem &pr, int block, int &mt, int &nt) {
    const int tiles_m = (int)((pr.rows + S::BM - 1) / S::BM);
    const int tiles_n = (int)((pr.count + S::BN - 1) / S::BN);
    const int id = xcd_tile(block, tiles_m * tiles_n, 0);
    if (id < 0) return false;
    walk(id, tiles_m, tiles_n, kWalk, mt, nt);
    return true;
}

// 8192 x 65536 x 2048 bf16, tiles of 256 x 256: 1.73 ms, 1270 TFLOP/s, matrix units busy 58 % of
// the cycles (a plain product of the library at 8192^3: 1418).
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_kernel(EntropyProblem pr) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    __shared__ int targets[S::BM];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    if (!entropy_place<S>(pr, blockIdx.x, mt, nt)) return;
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    // Read before the product, which has barriers enough between this and their use.
    if (threadIdx.x < S::BM)
        targets[threadIdx.x] = m0 + (int)threadIdx.x < pr.rows ? class_of(pr.targets[m0 + threadIdx.x], pr.classes) : -1;
    f32x4 acc[S::TM][S::TN];
    entropy_tile<S>(pr, m0, n0, (lds_char *)memory, wave, lane, acc);
    // A lane has row lane % 16 of each block of 16, columns 4 (lane / 16) .. + 3 of each.
    const int i = lane & 15, g = lane >> 4;
    const int wm = (wave / S::WN) * (S::BM / S::WM), wn = (wave % S::WN) * (S::BN / S::WN);
    const int left = (int)pr.count - n0 - wn - g * 4;  // valid columns from the lane's first on
    typedef RowSum Sums[S::BM];
    Sums *sums = (Sums *)memory;  // by the waves that share rows
    static_assert(sizeof(Sums) * S::WN <= sizeof(memory), "the stages' memory");
    if (n0 + S::BN > pr.count) {
#pragma unroll
        for (int tm = 0; tm < S::TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (tn * 16 + r >= left) acc[tm][tn][r] = -INFINITY;
    }
#pragma unroll
    for (int tm = 0; tm < S::TM; ++tm) {
        const int row = m0 + wm + tm * 16 + i;
        const int t = targets[wm + tm * 16 + i];
        float m = -INFINITY;
#pragma unroll
        for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
            for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[tm][tn][r]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float from = finite_or_0(m) * kLog2e;
        float s = 0.0f;
#pragma unroll
        for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s += __builtin_amdgcn_exp2f(fmaf(acc[tm][tn][r], kLog2e, -from));
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (g == 0) sums[wave % S::WN][wm + tm * 16 + i] = {m, s};
        const int at = t - (int)pr.first - n0 - wn;  // the target among the wave's columns
        const bool here = t >= 0 && at >= 0 && at < S::BN / S::WN;
        if (__any(here)) {
#pragma unroll
            for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (here && at == tn * 16 + g * 4 + r) pr.hit[row] = acc[tm][tn][r];
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < S::BM && m0 + r < pr.rows; r += S::NW * 64) {
        RowSum a = sums[0][r];
#pragma unroll
        for (int w = 1; w < S::WN; ++w) a.add(sums[w][r].m, sums[w][r].s);
        pr.part[(int64_t)nt * pr.rows + m0 + r] = make_float2(a.m, a.s);
    }
}

// The same for few rows (16 MT at most), which is bound by reading w once: nothing is
// shared through LDS. A block has 16 CG columns, and each group of 16 of them 8 / CG waves
// that take a part of the depth, every lane loading its fragments straight from memory, 16
// bytes at any alignment, a batch of them in flight (thin_kernel's loop). The logits meet in
// LDS. Rows and columns past the end are read at the last valid one.
// 16 rows of 16384 classes x 2048 bf16: 18.5 us, 3.6 TB/s (tiles of 64 x 64: 19.2; the join
// after it takes 4.4 behind 64 columns a block, 6.4 behind 32 and 10.3 behind 16).
template <typename T, int MT, int CG>
__global__ __launch_bounds__(512) void entropy_thin_kernel(EntropyProblem pr) {
    typedef typename Frag<T>::type frag;
    constexpr int kWaves = 8, kParts = kWaves / CG, kLane = 16 / (int)sizeof(T), kStep = 4 * kLane;
    constexpr int kBatch = MT == 1 ? 8 : 6;
    __shared__ float logits[kWaves][MT][64][4];
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)pr.rows, cols = (int)pr.classes, depth = (int)pr.width;
    const int first_col = blockIdx.x * 16 * CG;
    const int n0 = first_col + wave % CG * 16;
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    {
        const int steps = (depth + kStep - 1) / kStep;
        int first, count;
        part_of(steps, kParts, wave / CG, first, count);
        const int n = n0 + i < cols ? n0 + i : cols - 1;
        const T *p = (const T *)pr.w + n * pr.ldw + g * kLane;
        const T *q[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = 16 * t + i < rows ? 16 * t + i : rows - 1;
            q[t] = (const T *)pr.x + (int64_t)m * pr.ldx + g * kLane;
        }
        int s = first;
        const int whole = depth / kStep < first + count ? depth / kStep : first + count;
        union Chunk {
            T v[kLane];
            frag f;
        };
        for (; s + kBatch <= whole; s += kBatch) {
            Chunk a[kBatch], b[kBatch][MT];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                load_vec(p + (s + u) * kStep, a[u].v);
#pragma unroll
                for (int t = 0; t < MT; ++t) load_vec(q[t] + (s + u) * kStep, b[u][t].v);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < Frag<T>::kSteps; ++j)
                        acc[t] = Frag<T>::mma(a[u].f, b[u][t].f, acc[t], j);
        }
        for (; s < first + count; ++s) {
            // One step at a time, the last of them possibly past the depth's end.
            const int left = depth - s * kStep - g * kLane;
            Chunk a, b;
            auto some = [&](const T *x, Chunk &c) {
                if (left >= kLane) {
                    load_vec(x + s * kStep, c.v);
                } else {
#pragma unroll
                    for (int j = 0; j < kLane; ++j) c.v[j] = j < left ? x[s * kStep + j] : (T)0.0f;
                }
            };
            some(p, a);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                some(q[t], b);
#pragma unroll
                for (int j = 0; j < Frag<T>::kSteps; ++j) acc[t] = Frag<T>::mma(a.f, b.f, acc[t], j);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) logits[wave][t][lane][r] = acc[t][r];
    __syncthreads();
    // 512 / (16 MT) threads to a row, CG MT / 2 columns to each at most. (Lane l of a tile holds
    // columns 4 (l / 16) .. + 3 of row l % 16.)
    constexpr int kEach = 32 / MT;
    const int row = threadIdx.x / kEach, t = row >> 4;
    const int target = row < rows ? class_of(pr.targets[row], pr.classes) : -1;
    constexpr int kCols = (16 * CG + kEach - 1) / kEach;
    float z[kCols], m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
        const int c = threadIdx.x % kEach + k * kEach, col = c & 15;
        z[k] = -INFINITY;
        if (c < 16 * CG && first_col + c < cols) {
            z[k] = 0.0f;
#pragma unroll
            for (int part = 0; part < kParts; ++part)
                z[k] += logits[part * CG + (c >> 4)][t][(col >> 2) * 16 + (row & 15)][col & 3];
            if (first_col + c == target) pr.hit[row] = z[k];
        }
        m = fmaxf(m, z[k]);
    }
#pragma unroll
    for (int d = kEach / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float from = finite_or_0(m);
#pragma unroll
    for (int k = 0; k < kCols; ++k) s += __builtin_amdgcn_exp2f((z[k] - from) * kLog2e);
#pragma unroll
    for (int d = kEach / 2; d >= 1; d >>= 1) s += __shfl_xor(s, d);
    if (threadIdx.x % kEach == 0 && row < rows) pr.part[(int64_t)blockIdx.x * rows + row] = make_float2(m, s);
}

// At that size, in two pieces: 1.03 ms each, 1070 TFLOP/s; the epilogue and its 512 MiB take what
// dx's product, 0.80 ms, does not.
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dz_kernel(EntropyProblem pr) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    __shared__ RowTerms terms[S::BM];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    if (!entropy_place<S>(pr, blockIdx.x, mt, nt)) return;
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    const int rows = (int)pr.rows, count = (int)pr.count;
    // Read before the product, which has barriers enough between this and their use.
    const float scale = scale_of(pr, (float *)memory);
    if (threadIdx.x < S::BM)
        terms[threadIdx.x] = terms_of(pr, m0 + (int)threadIdx.x < rows ? m0 + threadIdx.x : rows - 1, scale);
    f32x4 acc[S::TM][S::TN];
    entropy_tile<S>(pr, m0, n0, (lds_char *)memory, wave, lane, acc);
    const int wm = (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    T *dz = (T *)pr.dz + (int64_t)m0 * pr.lddz;
    auto write = [&](auto is_whole) {
        constexpr bool kWhole = decltype(is_whole)::value != 0;
        by_rows<S, RowTerms>(
            (lds_char *)memory, wave, lane, acc, [&](int row, int) { return terms[wm + row]; },
            [&](int row, int col, float (&z)[8], const RowTerms &x) {
                const int64_t m = wm + row;
                const int n = wn + col;
                if (!kWhole && (m0 + m >= rows || n >= pr.lddz)) return;
                dz_of(z, n, x);
                if (!kWhole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = n + i < count ? z[i] : 0.0f;  // pads whole vectors
                }
                if (kWhole)
                    store_whole<S::kOnce>(dz + m * pr.lddz + n, z);
                else
                    store_row(dz + m * pr.lddz + n, z, (int)(pr.lddz - n));
            });
    };
    if (m0 + S::BM <= rows && n0 + S::BN <= count)
        write(ActTag<1>{});
    else
        write(ActTag<0>{});
}

// dx's tile, its depth (the piece's classes) whole or in parts. (0.80 ms a piece, 1370 TFLOP/s.)
template <class S>
__device__ __forceinline__ void entropy_dx_block(const EntropyGrad &e, int block, lds_char *smem) {
    typedef typename S::type T;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)e.rows, cols = (int)e.width;
    const int tiles_m = (rows + S::BM - 1) / S::BM, tiles_n = (cols + S::BN - 1) / S::BN;
    const int tiles = tiles_m * tiles_n;
    int id = xcd_tile(block, tiles * e.dx_cut.splits, 0);
    if (id < 0) return;
    const int part = __builtin_amdgcn_readfirstlane(id / tiles);
    id -= part * tiles;
    int mt, nt;
    walk(id, tiles_m, tiles_n, kWalk, mt, nt);
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    {
        constexpr int kDepth = S::TileP::kDepth;
        const int depth = (int)e.count;
        int first, count;
        part_of((depth + kDepth - 1) / kDepth, e.dx_cut.splits, part, first, count);
        const int k0 = __builtin_amdgcn_readfirstlane(first * kDepth);
        const int len = depth - k0 < count * kDepth ? depth - k0 : count * kDepth;
        const char *q = (const char *)e.dz + ((int64_t)m0 * e.lddz + k0) * sizeof(T);
        const char *p = (const char *)e.w + (k0 * e.ldw + n0) * sizeof(T);
        typename S::TileP tp;
        typename S::TileQ tq;
        tp.init(p, e.ldw, e.w_cols - n0, len, wave, lane);
        tq.init(q, e.lddz, rows - m0, len, wave, lane);
        run_product<S>(smem, tp, tq, len, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    const bool split = e.dx_cut.splits > 1, add = !split && !e.first, write = !split && e.last;
    float *to = split ? e.partial + (int64_t)part * rows * cols : e.sum;
    const float alpha = e.scale ? e.scale[1] : 1.0f;
    struct Aux {
        float v[8];
    };
    auto finish = [&](auto is_whole) {
        constexpr bool kWhole = decltype(is_whole)::value != 0;
        by_rows<S, Aux>(
            smem, wave, lane, acc,
            [&](int row, int col) {
                Aux x;
                const int64_t m = wm + row;
                const int n = wn + col;
                if (kWhole && add)
                    load_vec(e.sum + m * cols + n, x.v);
                else
                    load_row(e.sum + m * cols + n, !kWhole && add && m < rows ? cols - n : 0, x.v);
                return x;
            },
            [&](int row, int col, float (&z)[8], const Aux &x) {
                const int64_t m = wm + row;
                const int n = wn + col, valid = kWhole ? 8 : cols - n;
                if (!kWhole && (m >= rows || valid <= 0)) return;
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += x.v[i];
                if (!write) {
                    store_row(to + m * cols + n, z, valid);
                    return;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= alpha;
                store_row((T *)e.dx + m * e.lddx + n, z, valid);
            });
    };
    if (m0 + S::BM <= rows && n0 + S::BN <= cols)
        finish(ActTag<1>{});
    else
        finish(ActTag<0>{});
}

// dw's tile of the piece, its depth (the rows) whole or in parts. (0.95 ms a piece, 1160 TFLOP/s:
// both operands come out of LDS transposed.)
template <class S>
__device__ __forceinline__ void entropy_dw_block(const EntropyGrad &e, int block, lds_char *smem) {
    typedef typename S::type T;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mc = (int)e.count, nc = (int)e.width;
    const int tiles_m = (mc + S::BM - 1) / S::BM, tiles_n = (nc + S::BN - 1) / S::BN;
    const int tiles = tiles_m * tiles_n;
    int id = xcd_tile(block, tiles * e.dw_cut.splits, 0);
    if (id < 0) return;
    const int part = __builtin_amdgcn_readfirstlane(id / tiles);
    id -= part * tiles;
    int mt, nt;
    walk(id, tiles_m, tiles_n, 4, mt, nt);
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    {
        constexpr int kDepth = S::TileP::kDepth;
        const int depth = (int)e.rows;
        int first, count;
        part_of((depth + kDepth - 1) / kDepth, e.dw_cut.splits, part, first, count);
        const int64_t k0 = __builtin_amdgcn_readfirstlane(first * kDepth);
        const int len = (int)(depth - k0 < count * kDepth ? depth - k0 : count * kDepth);
        typename S::TileP tp;
        typename S::TileQ tq;
        tp.init((const char *)e.x + (k0 * e.ldx + n0) * sizeof(T), e.ldx, e.x_cols - n0, len, wave, lane);
        tq.init((const char *)e.dz + (k0 * e.lddz + m0) * sizeof(T), e.lddz, e.lddz - m0, len, wave, lane);
        run_product<S>(smem, tp, tq, len, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    const bool split = e.dw_cut.splits > 1;
    float *to = e.partial + (int64_t)part * mc * nc;
    const float alpha = e.scale ? e.scale[1] : 1.0f;
    struct None {};
    auto write = [&](auto is_whole) {
        constexpr bool kWhole = decltype(is_whole)::value != 0;
        by_rows<S, None>(
            smem, wave, lane, acc, [](int, int) { return None{}; },
            [&](int row, int col, float (&z)[8], const None &) {
                const int64_t m = wm + row;
                const int n = wn + col, valid = nc - n;
                if (!kWhole && (m >= mc || valid <= 0)) return;
                if (!kWhole && split) {
                    store_row(to + m * nc + n, z, valid);
                    return;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= alpha;
                if (kWhole)
                    store_whole<S::kOnce>((T *)e.dw + m * nc + n, z);
                else
                    store_row((T *)e.dw + m * nc + n, z, valid);
            });
    };
    if (!split && m0 + S::BM <= mc && n0 + S::BN <= nc)
        write(ActTag<1>{});
    else
        write(ActTag<0>{});
}

template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dx_kernel(EntropyGrad e) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    entropy_dx_block<S>(e, blockIdx.x, (lds_char *)memory);
}
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dw_kernel(EntropyGrad e) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    entropy_dw_block<S>(e, blockIdx.x, (lds_char *)memory);
}
// dx and dw in one launch, where both_plan finds it better: the deeper (longer) blocks first.
template <class SX, class SW>
__global__ __launch_bounds__(SX::NW * 64, 2) void entropy_both_kernel(EntropyGrad e, int first, bool dx_first) {
    static_assert(SX::NW == SW::NW, "one block size");
    constexpr int kBytes = SX::NS * SX::kStage > SW::NS * SW::kStage ? SX::NS * SX::kStage : SW::NS * SW::kStage;
    __shared__ __align__(1024) char memory[kBytes];
    const int b = blockIdx.x, in = b < first ? b : b - first;
    if ((b < first) == dx_first)
        entropy_dx_block<SX>(e, in, (lds_char *)memory);
    else
        entropy_dw_block<SW>(e, in, (lds_char *)memory);
}

template <class S>
int64_t entropy_blocks(int64_t m, int64_t n, int splits) {
    return cdiv(cdiv(m, S::BM) * cdiv(n, S::BN) * splits, 8) * 8;
}
template <class S>
hipError_t run_entropy(const EntropyProblem &pr, bool dz, hipStream_t s) {
    return launch(dz ? entropy_dz_kernel<S> : entropy_kernel<S>, entropy_blocks<S>(pr.rows, pr.count, 1),
                  S::NW * 64, 0, s, pr);
}
template <class S>
hipError_t run_dx(const EntropyGrad &e, hipStream_t s) {
    return launch(entropy_dx_kernel<S>, entropy_blocks<S>(e.rows, e.width, e.dx_cut.splits), S::NW * 64,
                  0, s, e);
}
template <class S>
hipError_t run_dw(const EntropyGrad &e, hipStream_t s) {
    return launch(entropy_dw_kernel<S>, entropy_blocks<S>(e.count, e.width, e.dw_cut.splits), S::NW * 64,
                  0, s, e);
}

template <class SX, class SW>
hipError_t run_both(const EntropyGrad &e, hipStream_t s) {
    const int64_t nx = entropy_blocks<SX>(e.rows, e.width, 1), nw = entropy_blocks<SW>(e.count, e.width, 1);
    const bool dx_first = e.count >= e.rows;
    return launch(entropy_both_kernel<SX, SW>, nx + nw, SX::NW * 64, 0, s, e, (int)(dx_first ? nx : nw),
                  dx_first);
}

template <typename T, int MT>
hipError_t run_thin_entropy(const EntropyProblem &pr, hipStream_t s) {
    const int64_t blocks = cdiv(pr.classes, 16 * pr.thin);
    if (pr.thin == 4) return launch(entropy_thin_kernel<T, MT, 4>, blocks, 512, 0, s, pr);
    if (pr.thin == 2) return launch(entropy_thin_kernel<T, MT, 2>, blocks, 512, 0, s, pr);
    return launch(entropy_thin_kernel<T, MT, 1>, blocks, 512, 0, s, pr);
}
template <typename T>
hipError_t pick_entropy(const EntropyProblem &pr, bool dz, hipStream_t s) {
    if (pr.thin) return pr.tile == 16 ? run_thin_entropy<T, 1>(pr, s) : run_thin_entropy<T, 2>(pr, s);
    if constexpr (sizeof(T) == 2) {
        if (pr.tile == 256) return run_entropy<Rows256<T, false>>(pr, dz, s);
        if (pr.tile == 129) return run_entropy<Rows129<T, false>>(pr, dz, s);
    } else {
        if (pr.tile == 32) return run_entropy<Rows32<T, false>>(pr, dz, s);
    }
    if (pr.tile == 128) return run_entropy<Rows128<T, false>>(pr, dz, s);
    return run_entropy<Rows64<T, false>>(pr, dz, s);
}
template <typename T>
hipError_t pick_dx(const EntropyGrad &e, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (e.dx_cut.tile == 256) return run_dx<Rows256<T, true>>(e, s);
        if (e.dx_cut.tile == 129) return run_dx<Rows129<T, true>>(e, s);
    } else {
        if (e.dx_cut.tile == 32) return run_dx<Rows32<T, true>>(e, s);
    }
    if (e.dx_cut.tile == 128) return run_dx<Rows128<T, true>>(e, s);
    return run_dx<Rows64<T, true>>(e, s);
}
template <typename T>
hipError_t pick_dw(const EntropyGrad &e, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (e.dw_cut.tile == 256) return run_dw<Grad256<T>>(e, s);
        if (e.dw_cut.tile == 129) return run_dw<Grad129<T>>(e, s);
    } else {
        if (e.dw_cut.tile == 32) return run_dw<Grad32<T>>(e, s);
    }
    if (e.dw_cut.tile == 128) return run_dw<Grad128<T>>(e, s);
    return run_dw<Grad64<T>>(e, s);
}

template <typename T>
hipError_t pick_entropy_both(const EntropyGrad &e, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (e.dx_cut.tile == 256) return run_both<Rows256<T, true>, Grad256<T>>(e, s);
    }
    if (e.dx_cut.tile == 128) return run_both<Rows128<T, true>, Grad128<T>>(e, s);
    return run_both<Rows64<T, true>, Grad64<T>>(e, s);
}

}  // namespace

template <typename T>
hipError_t launch_entropy_t(const EntropyProblem &pr, bool dz, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dx_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dw_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_both_t(const EntropyGrad &e, hipStream_t s);

}  // namespace kx
