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

#include "layers.h"
#include "linear.h"

namespace kx {
namespace {

constexpr float kLog2e = 1.44269504088896f;

__device__ __forceinline__ float finite_or_0(float m) {
    return fabsf(m) < INFINITY ? m : 0.0f;
}

// A row's largest logit m and its sum of e^(z - m) (of e^z where m is not finite), and
// another's added to it.
struct RowSum {
    float m, s;
    __device__ __forceinline__ void add(float m2, float s2) {
        const float most = fmaxf(m, m2), from = finite_or_0(most);
        // (Nothing times an overflowing factor would be a NaN.)
        const float own = s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((finite_or_0(m) - from) * kLog2e);
        const float other = s2 == 0.0f ? 0.0f : s2 * __builtin_amdgcn_exp2f((finite_or_0(m2) - from) * kLog2e);
        m = most;
        s = own + other;
    }
};

// Whether target t is a class, and its number.
__device__ __forceinline__ int class_of(int64_t t, int64_t classes) {
    return t >= 0 && t < classes ? (int)t : -1;
}

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

template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_kernel(EntropyProblem pr) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    if (!entropy_place<S>(pr, blockIdx.x, mt, nt)) return;
    const int m0 = mt * S::BM, n0 = nt * S::BN;
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
        const int t = row < pr.rows ? class_of(pr.targets[row], pr.classes) : -1;
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

template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dz_kernel(EntropyProblem pr) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    if (!entropy_place<S>(pr, blockIdx.x, mt, nt)) return;
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    f32x4 acc[S::TM][S::TN];
    entropy_tile<S>(pr, m0, n0, (lds_char *)memory, wave, lane, acc);
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    const float scale = pr.scale ? *pr.scale : 1.0f;
    const int rows = (int)pr.rows, count = (int)pr.count;
    T *dz = (T *)pr.dz;
    struct Aux {
        float lse, a, b;
        int t;  // the target in the piece
    };
    by_rows<S, Aux>(
        (lds_char *)memory, wave, lane, acc,
        [&](int row, int) {
            const int m = wm + row < rows ? wm + row : rows - 1;
            const int t = class_of(pr.targets[m], pr.classes);
            Aux x;
            x.lse = pr.lse[m] * kLog2e;
            x.b = t >= 0 ? pr.dloss[m] * scale : 0.0f;
            x.a = x.b + (pr.dlse ? pr.dlse[m] * scale : 0.0f);
            x.t = t >= 0 ? t - (int)pr.first : -1;
            return x;
        },
        [&](int row, int col, float (&z)[8], const Aux &x) {
            const int64_t m = wm + row;
            const int n = wn + col;
            if (m >= rows || n >= pr.lddz) return;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // Nothing weighs an ignored row, whatever it holds.
                z[i] = x.a == 0.0f ? 0.0f : x.a * __builtin_amdgcn_exp2f(fmaf(z[i], kLog2e, -x.lse));
                if (n + i == x.t) z[i] -= x.b;
                if (n + i >= count) z[i] = 0.0f;  // what pads the row to whole vectors
            }
            store_row(dz + m * pr.lddz + n, z, (int)(pr.lddz - n));
        });
}

// dx's tile, its depth (the piece's classes) whole or in parts.
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dx_kernel(EntropyGrad e) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)e.rows, cols = (int)e.width;
    const int tiles_m = (rows + S::BM - 1) / S::BM, tiles_n = (cols + S::BN - 1) / S::BN;
    const int tiles = tiles_m * tiles_n;
    int id = xcd_tile(blockIdx.x, tiles * e.dx_cut.splits, 0);
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
        run_product<S>((lds_char *)memory, tp, tq, len, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    const bool split = e.dx_cut.splits > 1, add = !split && !e.first, write = !split && e.last;
    float *to = split ? e.partial + (int64_t)part * rows * cols : e.sum;
    const float alpha = e.scale ? e.scale[1] : 1.0f;
    struct Aux {
        float v[8];
    };
    by_rows<S, Aux>(
        (lds_char *)memory, wave, lane, acc,
        [&](int row, int col) {
            Aux x;
            const int64_t m = wm + row;
            const int n = wn + col;
            load_row(e.sum + m * cols + n, add && m < rows ? cols - n : 0, x.v);
            return x;
        },
        [&](int row, int col, float (&z)[8], const Aux &x) {
            const int64_t m = wm + row;
            const int n = wn + col, valid = cols - n;
            if (m >= rows || valid <= 0) return;
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
}

// dw's tile of the piece, its depth (the rows) whole or in parts.
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void entropy_dw_kernel(EntropyGrad e) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mc = (int)e.count, nc = (int)e.width;
    const int tiles_m = (mc + S::BM - 1) / S::BM, tiles_n = (nc + S::BN - 1) / S::BN;
    const int tiles = tiles_m * tiles_n;
    int id = xcd_tile(blockIdx.x, tiles * e.dw_cut.splits, 0);
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
        run_product<S>((lds_char *)memory, tp, tq, len, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    const bool split = e.dw_cut.splits > 1;
    float *to = e.partial + (int64_t)part * mc * nc;
    const float alpha = e.scale ? e.scale[1] : 1.0f;
    struct None {};
    by_rows<S, None>(
        (lds_char *)memory, wave, lane, acc, [](int, int) { return None{}; },
        [&](int row, int col, float (&z)[8], const None &) {
            const int64_t m = wm + row;
            const int n = wn + col, valid = nc - n;
            if (m >= mc || valid <= 0) return;
            if (split) {
                store_row(to + m * nc + n, z, valid);
                return;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] *= alpha;
            store_row((T *)e.dw + m * nc + n, z, valid);
        });
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

template <typename T>
hipError_t pick_entropy(const EntropyProblem &pr, bool dz, hipStream_t s) {
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

}  // namespace

template <typename T>
hipError_t launch_entropy_t(const EntropyProblem &pr, bool dz, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dx_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dw_t(const EntropyGrad &e, hipStream_t s);

}  // namespace kx
