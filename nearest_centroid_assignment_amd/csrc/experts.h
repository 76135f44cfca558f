// experts.h - internal launchers and device helpers of the expert operators
// (tokens.hip, linear*.hip, adamw.hip), used by experts_api.hip. Not part of
// the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace kx {

using km::launch;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef _Float16 f16;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Inclusive prefix sum over the 64 lanes of a wave (all active) with DPP
// moves: inside each row of 16 lanes, then row totals to the rows above.
__device__ __forceinline__ int wave_incl_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);   // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);   // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);   // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31
    return x;
}

// V elements of T at any element-aligned address, one access (global memory
// takes any alignment; a vector type keeps the compiler from splitting it).
template <typename T, int V>
struct Unaligned {
    typedef T type __attribute__((ext_vector_type(V), aligned(alignof(T))));
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, T (&out)[V]) {
    const auto x = *reinterpret_cast<const typename Unaligned<T, V>::type *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = x[i];
}
// The same past the caches' replacement order: for what this kernel touches once.
template <typename T, int V>
__device__ __forceinline__ void load_once(const T *p, T (&out)[V]) {
    const auto x = __builtin_nontemporal_load(reinterpret_cast<const typename Unaligned<T, V>::type *>(p));
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = x[i];
}
template <typename T, int V>
__device__ __forceinline__ void store_once(T *p, const T (&in)[V]) {
    typename Unaligned<T, V>::type x;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = in[i];
    __builtin_nontemporal_store(x, reinterpret_cast<typename Unaligned<T, V>::type *>(p));
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const T (&in)[V]) {
    typename Unaligned<T, V>::type x;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = in[i];
    *reinterpret_cast<typename Unaligned<T, V>::type *>(p) = x;
}

// V values of one row, `valid` of them inside it, at any alignment.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T *p, int valid, T (&x)[V]) {
    if (valid >= V) {
        load_vec(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < valid ? p[i] : (T)0.0f;
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_row(T *p, const float (&v)[V], int valid) {
    T x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (T)v[i];
    if (valid >= V) {
        store_vec(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < valid) p[i] = x[i];
    }
}

// ------------------------------------------------------------ activations
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

// 1 / (1 + e^-x) from the hardware's 2^x and reciprocal (about 1 ulp each).
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896f * x));
}
constexpr float kGelu1 = 1.59576912160573f;   // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.0713548162726f;    // 0.044715 * 2 sqrt(2/pi)

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // keeps NaN
    if (ACT == kActGelu) return z * sigmoid(z * (kGelu1 + kGelu3 * z * z));
    if (ACT == kActSilu) return z * sigmoid(z);
    return z;
}
// act'(z). With s = sigmoid(u(z)): (z s)' = s + z s (1 - s) u'. Where s (1 - s) rounds to
// 0 the slope is s, 0 or 1: the other factors may be infinite there (u' from 2e19 on, z
// where a 16-bit pre was too large for its type), and 0 times them a NaN.
__device__ __forceinline__ float slope_from(float z, float s, float du) {
    const float bend = s * (1.0f - s);
    return bend == 0.0f ? s : s + z * bend * du;
}
template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
    if (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (ACT == kActGelu) {
        const float s = sigmoid(z * (kGelu1 + kGelu3 * z * z));
        return slope_from(z, s, kGelu1 + 3.0f * kGelu3 * z * z);
    }
    if (ACT == kActSilu) return slope_from(z, sigmoid(z), 1.0f);
    return 1.0f;
}
template <int ACT>
struct ActTag {
    static constexpr int value = ACT;
};
// f(tag of act): the choice is made once, around the loops that use it. (Made for
// each value inside them, it left the products' epilogue with 2500 branches.)
template <class F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case kActRelu: f(ActTag<kActRelu>{}); break;
        case kActGelu: f(ActTag<kActGelu>{}); break;
        case kActSilu: f(ActTag<kActSilu>{}); break;
        default: f(ActTag<kActNone>{}); break;
    }
}
template <int V>
__device__ __forceinline__ void apply_act(float (&z)[V], int act) {
    with_act(act, [&](auto tag) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = act_of<decltype(tag)::value>(z[i]);
    });
}
// z *= act'(x)
template <typename T, int V>
__device__ __forceinline__ void apply_slope(float (&z)[V], const T (&x)[V], int act) {
    with_act(act, [&](auto tag) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= slope_of<decltype(tag)::value>((float)x[i]);
    });
}

// ----------------------------------------------------------------- tokens
struct PlanScratch {
    int *tile_hist;        // tiles x experts
    int *count;            // experts
    unsigned short *rank;  // pairs
    int64_t tiles;
};
// Whether one block sorts the pairs (then the scratch is not used).
bool plan_is_small(int64_t pairs, int64_t experts);
hipError_t launch_plan(const int64_t *ids, int64_t pairs, int64_t experts, int *order, int *place,
                       int *offsets, const PlanScratch &ws, hipStream_t s);
hipError_t launch_dispatch(const void *x, int64_t ldx, int dtype, int64_t tokens, int64_t top,
                           int64_t width, const int *order, const int *place, void *xs,
                           int64_t ldxs, hipStream_t s);
// weights == NULL: all ones (the gradient of dispatch).
hipError_t launch_combine(const void *ys, int64_t ldys, const float *weights, int dtype,
                          int64_t tokens, int64_t top, int64_t width, const int *place, void *y,
                          int64_t ldy, hipStream_t s);
hipError_t launch_combine_backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                                   const float *weights, int dtype, int64_t tokens, int64_t top,
                                   int64_t width, const int *order, const int *place, void *dys,
                                   int64_t lddys, float *dweights, hipStream_t s);

// ----------------------------------------------------------------- linear
// out = act(q p_e^T + bias_e) + residual, or (with in_pre) (q p_e) *
// in_act'(in_pre). q: rows x contraction. p: per expert cols x contraction
// (p_rows false) or contraction x cols (p_rows true), dense rows of ldp.
struct RowsProblem {
    const void *q, *p;
    int64_t ldq, ldp, p_expert;  // elements
    int64_t rows, cols, depth;   // depth: the contraction
    int64_t p_cols;              // with p_rows: readable columns of p (>= cols; a pad is zero)
    bool p_rows;
    const int *offsets;          // NULL: one expert, no tail
    int experts;
    const void *bias, *residual, *in_pre;
    int64_t ldr, ldin;
    void *out, *pre;
    int64_t ldo, ldpre;
    int act, in_act;
    int tile, splits;            // rows_plan's
    float *partial;              // splits x rows x cols when splits > 1
};
// out[e] (m_cols x n_cols, dense) = dz[rows of e]^T x[rows of e].
struct GradProblem {
    const void *x, *dz;
    int64_t ldx, lddz;
    int64_t rows, m_cols, n_cols;  // m: columns of dz, n: columns of x
    int64_t x_cols, dz_cols;       // readable columns (a pad is zero)
    const int *offsets;
    int experts;
    void *out;
    int tile, splits;              // grad_plan's
    float *partial;                // splits x experts x m_cols x n_cols when splits > 1
};
// How a product is cut: tiles of tile x tile (32: 32 x 64; 129: 128 x 128 with three
// stages in flight; with `thin`, blocks of `tile` rows by 16 columns), its depth in
// `splits` parts whose sums are joined by a second kernel.
struct Cut {
    int tile, splits;
    bool thin;
    double cost;  // microseconds, by the cost model
};
Cut rows_plan(int dtype, int64_t rows, int64_t cols, int64_t depth, bool grouped, int64_t experts,
              bool p_rows);
Cut grad_plan(int dtype, int64_t rows, int64_t m_cols, int64_t n_cols, int64_t experts);
// The tile of dx and dw in one launch, 0 where the two launches are better.
int both_plan(int dtype, int64_t rows, int64_t outs, int64_t ins, bool grouped, int64_t experts,
              const Cut &dx, const Cut &dw);

// Row tiles of all groups at most: every group that has a row may end in a
// partial tile, and the rows past the last expert's are one more group.
inline int64_t most_row_tiles(int64_t rows, int64_t bm, bool grouped, int64_t experts) {
    if (!grouped) return cdiv(rows, bm);
    return rows / bm + (experts + 1 < rows ? experts + 1 : rows);
}

// dtype: 0 float, 1 bf16, 2 f16. False when a launch's grid would not fit.
bool rows_grid_ok(int dtype, int64_t rows, int64_t cols, int64_t depth, bool grouped,
                  int64_t experts, bool p_rows);
bool grad_grid_ok(int dtype, int64_t rows, int64_t m_cols, int64_t n_cols, int64_t experts);
hipError_t launch_rows(int dtype, const RowsProblem &pr, bool thin, hipStream_t s);
hipError_t launch_grad(int dtype, const GradProblem &pr, hipStream_t s);
// The parts of dbias still to be added: out[i] = sum over s of partial[s * n + i].
struct SlopeSum {
    const float *partial;
    int splits;  // 0: none
    int64_t n;
    void *out;
};
// 64 columns a block; each of its first four waves adds a quarter of the parts.
// `quarter`: 256 floats of LDS.
template <typename T>
__device__ __forceinline__ void slope_sum(const SlopeSum &sum, int block, float *quarter) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = (int64_t)block * 64 + lane;
    if (wave < 4) {
        const int per = (sum.splits + 3) / 4;
        const int end = (wave + 1) * per < sum.splits ? (wave + 1) * per : sum.splits;
        float v = 0.0f;
        if (i < sum.n) {
#pragma unroll 8
            for (int s = wave * per; s < end; ++s) v += sum.partial[s * sum.n + i];
        }
        quarter[threadIdx.x] = v;
    }
    __syncthreads();
    if (wave == 0 && i < sum.n)
        ((T *)sum.out)[i] = (T)((quarter[lane] + quarter[64 + lane]) +
                                (quarter[128 + lane] + quarter[192 + lane]));
}

// dx and dw in one launch, with both_plan's tile in both and neither split, and `sum`.
hipError_t launch_both(int dtype, const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                       hipStream_t s);

// dst rows of ldd elements (a multiple of 8) = src rows with zeros from cols on.
hipError_t launch_pad_rows(const void *src, int64_t lds, int64_t rows, int64_t cols, void *dst,
                           int64_t ldd, hipStream_t s);

// dz = dy * act'(pre) rounded to dtype into dz (NULL: not written; rows of
// lddz, zeros from outs to lddz), dbias[e] = column sums of the float32 dz
// (NULL: not computed) with `partial` of slope_splits() x experts x outs floats. With
// `later`, parts that have to be added are left there to launch_both.
int64_t slope_splits(int64_t rows, int64_t outs, int64_t experts);
hipError_t launch_slope(int dtype, const void *dy, int64_t lddy, const void *pre, int64_t ldpre,
                        int act, const int *offsets, int experts, int64_t rows, int64_t outs,
                        void *dz, int64_t lddz, void *dbias, float *partial, SlopeSum *later,
                        hipStream_t s);

// ------------------------------------------------------------------ adamw
struct AdamwStep {
    float beta1, one_minus_beta1, beta2, one_minus_beta2, keep, rate, root, eps;
    const float *grad_scale;
    void *m, *v;
    float *m_scale, *v_scale;
    int param_dtype, grad_dtype, bits;
};
hipError_t launch_adamw(void *const *params, const void *const *grads, void *const *copies,
                        const int64_t *numels, int64_t count, const AdamwStep &st, hipStream_t s);
hipError_t launch_moments(const int8_t *m, const uint8_t *v, const float *m_scale,
                          const float *v_scale, int64_t elements, float *m_out, float *v_out,
                          hipStream_t s);

}  // namespace kx
