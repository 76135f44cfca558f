// rows.h - device helpers of the kernels that give a wave or a block to a row
// (tokens.hip, embed.hip, norm.hip, route.hip).
#pragma once

#include "experts.h"

namespace kx {
namespace {

// Rank of the lane's expert among the wave's lanes with the same one and a lower
// index, and how many have it; both 0 where expert < 0. `bits`: of the largest expert.
__device__ __forceinline__ void wave_rank(int expert, int bits, int &rank, int &count) {
    const int lane = threadIdx.x & 63;
    unsigned long long same = __ballot(expert >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool set = (expert >> b) & 1;
        const unsigned long long with = __ballot(set);
        same &= set ? with : ~with;
    }
    rank = expert < 0 ? 0 : __popcll(same & ((1ull << lane) - 1ull));
    count = expert < 0 ? 0 : __popcll(same);
}
// The wave's accesses to LDS before this one, by any of its lanes, come before those after it.
__device__ __forceinline__ void in_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// x of another of the 16 lanes (CTRL 0x120 + n: n places on).
template <int CTRL>
__device__ __forceinline__ float rotated(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <typename T>
constexpr int vec() {
    return 16 / (int)sizeof(T);
}

template <bool ONCE, typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int64_t left, T (&v)[V]) {
    if (left >= V) {
        if (ONCE)
            load_once(p, v);
        else
            load_vec(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < left ? p[j] : (T)0.0f;
    }
}
template <bool ONCE, typename T, int V>
__device__ __forceinline__ void store_part(T *p, int64_t left, const T (&v)[V]) {
    if (left >= V) {
        if (ONCE)
            store_once(p, v);
        else
            store_vec(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) p[j] = v[j];
    }
}

// Where the chunk of V values at c is read and written: the last one, where it would
// leave the row, over the end of the one before (1001-wide rows, against one lane
// going value by value: 15009 f16 rows, all five operators 65 us).
template <int V>
__device__ __forceinline__ int64_t chunk_at(int64_t c, int64_t width) {
    return width >= V && c + V > width ? width - V : c;
}

// The token, or place, of this wave (NT = 64) or block.
template <int NT>
__device__ __forceinline__ int64_t own_token() {
    const int64_t t = (int64_t)blockIdx.x * (256 / NT) + (NT == 64 ? threadIdx.x >> 6 : 0);
    return ((int64_t)__builtin_amdgcn_readfirstlane((int)(t >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
}

// Sum over the NT threads of a token, in a fixed order, to all of them.
template <int NT>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    if (NT == 256) {
        __shared__ float part[4];
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return v;
}

}  // namespace
}  // namespace kx
