// entropy.hip - what surrounds the products of entropy.h: the choice of the type, the
// joins of the rows' sums and of split depths, and dz's scale.
#include "layers.h"

namespace kx {

template <typename T>
hipError_t launch_entropy_t(const EntropyProblem &pr, bool dz, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dx_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_dw_t(const EntropyGrad &e, hipStream_t s);
template <typename T>
hipError_t launch_entropy_both_t(const EntropyGrad &e, hipStream_t s);

namespace {

// 16 rows a block, 16 threads to a row, each joining every 16th of the column tiles' sums
// (the largest first, then the sums relative to it).
__global__ __launch_bounds__(256) void entropy_join_kernel(EntropyProblem pr, int tiles) {
    __shared__ float most[16][17], sums[16][17];
    const int r = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int64_t row = (int64_t)blockIdx.x * 16 + r;
    const bool there = row < pr.rows;
    const float2 *part = pr.part + (there ? row : pr.rows - 1);
    constexpr float kLog2e = 1.44269504088896f;
    auto finite_or_0 = [](float m) { return fabsf(m) < INFINITY ? m : 0.0f; };
    float m = -INFINITY, s = 0.0f;
    for (int k0 = slice; k0 < tiles; k0 += 16 * 8) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = k0 + 16 * u;
            v[u] = part[(int64_t)(k < tiles ? k : k0) * pr.rows];
            if (k >= tiles) v[u] = make_float2(-INFINITY, 0.0f);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) top = fmaxf(top, v[u].x);
        const float from = finite_or_0(top);
        // (Nothing times an overflowing factor would be a NaN.)
        s = s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((finite_or_0(m) - from) * kLog2e);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            s += v[u].y == 0.0f ? 0.0f
                                : v[u].y * __builtin_amdgcn_exp2f((finite_or_0(v[u].x) - from) * kLog2e);
        m = top;
    }
    most[slice][r] = m;
    sums[slice][r] = s;
    __syncthreads();
    if (slice != 0 || !there) return;
    for (int k = 1; k < 16; ++k) m = fmaxf(m, most[k][r]);
    const float from = finite_or_0(m);
    float sum = 0.0f;
    for (int k = 0; k < 16; ++k)
        sum += sums[k][r] == 0.0f
                   ? 0.0f
                   : sums[k][r] * __builtin_amdgcn_exp2f((finite_or_0(most[k][r]) - from) * kLog2e);
    const float lse = from + logf(sum);
    const int64_t t = pr.targets[row];
    pr.lse[row] = lse;
    pr.loss[row] = t >= 0 && t < pr.classes ? lse - pr.hit[row] : 0.0f;
}

// The products take dz rounded to 16 bits. It is kept divided by the largest of its rows'
// factors: with one factor for all rows, as of a mean, the target's place holds p - 1 and
// loses nothing where p is small (rounded as it is, 1 / rows makes every such place off by the
// same part, and with them all of dx and dw: a mean of 300 rows of 513 classes bf16, norm of
// dx's error against 64 bits over its norm 0.0024 -> 0.0018, where rounding dx alone leaves
// 0.0017). float16 holds 2^-24 to 65504: there
// it is multiplied by 2^14 as well, or most of a large softmax would be zeros. dx and dw are
// multiplied by the inverse. scale: the factor, and its inverse.
__global__ __launch_bounds__(1024) void entropy_scale_kernel(EntropyProblem pr, float most_dz,
                                                             float *scale) {
    __shared__ float most[16];
    float m = 0.0f;
    bool odd = false;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < pr.rows; r += 1024) {
        const int64_t t = pr.targets[r];
        const float b = t >= 0 && t < pr.classes ? pr.dloss[r] : 0.0f;
        const float a = b + (pr.dlse ? pr.dlse[r] : 0.0f);
        odd |= !(fabsf(a) < INFINITY);
        m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
    }
    if (__any(odd)) m = INFINITY;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) m = fmaxf(m, most[w]);
    const bool scaled = m > 0.0f && m < INFINITY;
    m = m < 0x1p-100f ? 0x1p-100f : m;
    scale[0] = scaled ? most_dz / m : 1.0f;
    scale[1] = scaled ? m / most_dz : 1.0f;
}

// A product whose depth was split: eight columns of a row a thread, the parts added in
// order, then the piece before.
template <typename T>
__global__ __launch_bounds__(256) void entropy_parts_kernel(const float *__restrict__ partial,
                                                            int splits, int64_t rows, int64_t cols,
                                                            float *__restrict__ sum, bool first,
                                                            bool last, const float *__restrict__ scale,
                                                            T *__restrict__ out, int64_t ldo) {
    const int64_t chunks = (cols + 7) / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = id / chunks, n = (id - m * chunks) * 8;
    if (m >= rows) return;
    const int valid = (int)(cols - n < 8 ? cols - n : 8);
    float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (!first) load_row(sum + m * cols + n, valid, z);
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
        float x[8];
        load_row(partial + ((int64_t)k * rows + m) * cols + n, valid, x);
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
hipError_t grad_t(const EntropyGrad &g, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (g.together) return launch_entropy_both_t<T>(g, s);
    if (g.dx) {
        e = launch_entropy_dx_t<T>(g, s);
        if (e == hipSuccess && g.dx_cut.splits > 1)
            e = launch(entropy_parts_kernel<T>, cdiv(g.rows * cdiv(g.width, 8), 256), 256, 0, s, g.partial,
                       g.dx_cut.splits, g.rows, g.width, g.sum, g.first, g.last, g.scale, (T *)g.dx, g.lddx);
    }
    if (e != hipSuccess || !g.dw) return e;
    e = launch_entropy_dw_t<T>(g, s);
    if (e == hipSuccess && g.dw_cut.splits > 1)
        e = launch(entropy_parts_kernel<T>, cdiv(g.count * cdiv(g.width, 8), 256), 256, 0, s, g.partial,
                   g.dw_cut.splits, g.count, g.width, (float *)nullptr, true, true, g.scale, (T *)g.dw,
                   g.width);
    return e;
}

}  // namespace

Cut entropy_plan(int dtype, int64_t rows, int64_t classes, int64_t width, bool grad) {
    if (!grad && rows <= 32) {
        const int groups = classes >= 16384 ? 4 : classes >= 8192 ? 2 : 1;  // a block a compute unit
        return {rows <= 16 ? 16 : 32, groups, true, 0.0};
    }
    return whole_plan(dtype, rows, classes, width);
}
int entropy_columns(int, const Cut &cut) {
    if (cut.thin) return 16 * cut.splits;
    return cut.tile == 129 ? 128 : cut.tile == 32 ? 64 : cut.tile;
}

hipError_t launch_entropy(int dtype, const EntropyProblem &pr, hipStream_t s) {
    hipError_t e;
    if (dtype == 0)
        e = launch_entropy_t<float>(pr, false, s);
    else
        e = dtype == 1 ? launch_entropy_t<bf16>(pr, false, s) : launch_entropy_t<f16>(pr, false, s);
    if (e != hipSuccess) return e;
    const Cut cut = {pr.tile, pr.thin, pr.thin != 0, 0.0};
    return launch(entropy_join_kernel, cdiv(pr.rows, 16), 256, 0, s, pr,
                  (int)cdiv(pr.count, entropy_columns(dtype, cut)));
}
hipError_t launch_entropy_dz(int dtype, const EntropyProblem &pr, hipStream_t s) {
    if (dtype == 0) return launch_entropy_t<float>(pr, true, s);
    return dtype == 1 ? launch_entropy_t<bf16>(pr, true, s) : launch_entropy_t<f16>(pr, true, s);
}
hipError_t launch_entropy_scale(int dtype, const EntropyProblem &pr, float *scale, hipStream_t s) {
    return launch(entropy_scale_kernel, 1, 1024, 0, s, pr, dtype == 2 ? 16384.0f : 1.0f, scale);
}
hipError_t launch_entropy_grad(int dtype, const EntropyGrad &g, hipStream_t s) {
    if (dtype == 0) return grad_t<float>(g, s);
    return dtype == 1 ? grad_t<bf16>(g, s) : grad_t<f16>(g, s);
}

}  // namespace kx
