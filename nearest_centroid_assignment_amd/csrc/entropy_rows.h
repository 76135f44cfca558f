// entropy_rows.h - what a row's cross entropy and dz are made of (entropy.h, entropy.hip).
#pragma once

#include "layers.h"

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

// What a row gives dz: its factors without the common scale (both 0: nothing weighs it).
struct Factors {
    float a, b;
};
__device__ __forceinline__ Factors factors_of(const EntropyProblem &pr, int64_t row) {
    const float b = class_of(pr.targets[row], pr.classes) >= 0 ? pr.dloss[row] : 0.0f;
    return {b + (pr.dlse ? pr.dlse[row] : 0.0f), b};
}

// The products take dz rounded to 16 bits. It is kept divided by the largest of its rows'
// factors: with one factor for all rows, as of a mean, the target's place holds p - 1 and
// loses nothing where p is small (rounded as it is, 1 / rows makes every such place off by the
// same part, and with them all of dx and dw: a mean of 300 rows of 513 classes bf16, norm of
// dx's error against 64 bits over its norm 0.0024 -> 0.0018, where rounding dx alone leaves
// 0.0017; factors that differ from row to row keep more of dz's own rounding: with a dlse of each
// row's own 0.0026 for 83 rows of 12416 classes, 0.0020 for 2394 of 5046). float16 holds 2^-24 to
// 65504: there it is multiplied by 2^14 (most_dz) as well, or most of a large softmax would be
// zeros. dx and dw are multiplied by the inverse. scale: the factor, and its inverse.
//
// The largest factor of the rows that this thread looks at, every `step`-th; infinity where one
// is not finite.
__device__ __forceinline__ float largest_factor(const EntropyProblem &pr, int64_t first, int64_t step) {
    float m = 0.0f;
#pragma unroll 4
    for (int64_t r = first; r < pr.rows; r += step) {
        const Factors f = factors_of(pr, r);
        const float most = fmaxf(fabsf(f.a), fabsf(f.b));
        m = fabsf(f.a) < INFINITY ? fmaxf(m, most) : INFINITY;
    }
    return m;
}
// Of the block's threads, in `memory` (a float for each of its waves), and the scale it makes.
__device__ __forceinline__ float scale_from(float m, float most_dz, float *memory, float &inverse) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0) memory[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 64; ++w) m = fmaxf(m, memory[w]);
    __syncthreads();
    const bool scaled = m > 0.0f && m < INFINITY;
    m = m < 0x1p-100f ? 0x1p-100f : m;
    inverse = scaled ? m / most_dz : 1.0f;
    return scaled ? most_dz / m : 1.0f;
}
// The scale: given, or found by every block, the first of which leaves it to dx and dw. (For few
// rows: a launch of its own takes 2 to 5 us.)
__device__ __forceinline__ float scale_of(const EntropyProblem &pr, float *memory) {
    if (!pr.scale) return 1.0f;
    if (pr.most_dz == 0.0f) return *pr.scale;
    float inverse;
    const float scale = scale_from(largest_factor(pr, threadIdx.x, blockDim.x), pr.most_dz, memory, inverse);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        pr.scale[0] = scale;
        pr.scale[1] = inverse;
    }
    return scale;
}

// What dz of a row needs.
struct RowTerms {
    float lse, a, b;  // lse in units of log 2
    int target;       // in the piece
};
__device__ __forceinline__ RowTerms terms_of(const EntropyProblem &pr, int64_t row, float scale) {
    const Factors f = factors_of(pr, row);
    const int t = class_of(pr.targets[row], pr.classes);
    return {pr.lse[row] * kLog2e, f.a * scale, f.b * scale, t >= 0 ? t - (int)pr.first : -1};
}
// z = dz of eight logits from column n of the piece on.
__device__ __forceinline__ void dz_of(float (&z)[8], int n, const RowTerms &x) {
    if (x.a == 0.0f) {  // nothing weighs an ignored row, whatever it holds
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = x.a * __builtin_amdgcn_exp2f(fmaf(z[i], kLog2e, -x.lse));
    }
    if ((unsigned)(x.target - n) < 8u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] -= n + i == x.target ? x.b : 0.0f;
    }
}

}  // namespace
}  // namespace kx
