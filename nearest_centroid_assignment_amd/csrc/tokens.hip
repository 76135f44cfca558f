// tokens.hip - pairs of (token, slot) sorted by expert, the token rows gathered
// in that order, the experts' rows summed back with weights, and gradients.
//
// The sort is the counting sort of the centroid update (a stable rank per tile
// of 1024 pairs and that tile's histogram, launch_rank_hist), then a prefix over
// the tiles per expert, a prefix over the experts, and a scatter that writes
// both the order and its inverse. At most kSmallPairs pairs are sorted by one
// block in one launch.
//
// The row kernels give one wave (or, with few tokens, one block) to a token: its
// own row is read once, and the rows of its `top` pairs are reached through the
// inverse permutation, so every row is moved once and no sum needs an atomic.
#include "experts.h"
#include "kernels.h"

namespace kx {
namespace {

constexpr int kTile = (int)km::kSortTileRows;
constexpr int kSmallTiles = 4;                     // tiles that the one-block sort takes
constexpr int kSmallPairs = kSmallTiles * 1024;
constexpr int kSmallExperts = 4096;

// Per expert (a thread): the exclusive prefix of its tile counts, in place, and
// its size. Loads of 16 tiles are in flight before the first store.
__global__ __launch_bounds__(64) void plan_tiles_kernel(int *__restrict__ tile_hist,
                                                        int64_t experts, int64_t tiles,
                                                        int *__restrict__ count) {
    const int64_t e = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (e >= experts) return;
    constexpr int U = 16;
    int run = 0;
    for (int64_t b = 0; b < tiles; b += U) {
        int v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = b + u < tiles ? tile_hist[(b + u) * experts + e] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b + u < tiles) tile_hist[(b + u) * experts + e] = run;
            run += v[u];
        }
    }
    count[e] = run;
}

// Exclusive prefix of x over the 1024 threads of the block; total = the sum.
__device__ __forceinline__ int block_scan(int x, int &total) {
    __shared__ int wave_sum[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int incl = wave_incl_scan(x);
    __syncthreads();  // wave_sum of a call before is read by now
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        before += w < wave ? wave_sum[w] : 0;
        total += wave_sum[w];
    }
    return before + incl - x;
}

__global__ __launch_bounds__(1024) void plan_scan_kernel(const int *__restrict__ count,
                                                         int64_t experts,
                                                         int *__restrict__ offsets) {
    int carry = 0;
    for (int64_t e0 = 0; e0 < experts; e0 += 1024) {
        const int64_t e = e0 + threadIdx.x;
        int total;
        const int at = block_scan(e < experts ? count[e] : 0, total);
        if (e < experts) offsets[e] = carry + at;
        carry += total;
    }
    if (threadIdx.x == 0) offsets[experts] = carry;
}

__global__ __launch_bounds__(256) void plan_scatter_kernel(
    const int64_t *__restrict__ ids, int64_t pairs, int64_t experts,
    const int *__restrict__ tile_prefix, const unsigned short *__restrict__ rank,
    const int *__restrict__ offsets, int *__restrict__ order, int *__restrict__ place) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pairs) return;
    const int64_t e = ids[i];
    int at = -1;
    if (e >= 0 && e < experts) {
        at = offsets[e] + tile_prefix[(i / kTile) * experts + e] + rank[i];
        order[at] = (int)i;
    }
    place[i] = at;
    if (i >= offsets[experts]) order[i] = -1;
}

// The whole sort in one block. Waves rank their own 64 pairs (the lanes with an
// equal expert, found by ballots) and take turns, in pair order, to add the
// expert's count so far; the counts become starts by one block scan.
__global__ __launch_bounds__(1024) void plan_small_kernel(const int64_t *__restrict__ ids, int pairs,
                                                          int experts, int *__restrict__ order,
                                                          int *__restrict__ place,
                                                          int *__restrict__ offsets) {
    __shared__ int table[kSmallExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < experts; e += 1024) table[e] = 0;
    int expert[kSmallTiles], rank[kSmallTiles];
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t) {
        const int i = t * 1024 + tid;
        expert[t] = -1;
        rank[t] = 0;
        if (i < pairs) {
            const int64_t e = ids[i];
            if (e >= 0 && e < experts) expert[t] = (int)e;
        }
    }
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t) {
        if (t * 1024 >= pairs) break;
        unsigned long long todo = __ballot(expert[t] >= 0);
        int count = 0;
        while (todo) {
            const int e = __builtin_amdgcn_readlane(expert[t], __builtin_ctzll(todo));
            const unsigned long long same = __ballot(expert[t] == e);
            if (expert[t] == e) {
                rank[t] = __popcll(same & ((1ull << lane) - 1ull));
                count = __popcll(same);
            }
            todo &= ~same;
        }
        const int left = pairs - t * 1024;
        const int waves = left < 1024 ? (left + 63) / 64 : 16;
        for (int w = 0; w < waves; ++w) {
            __syncthreads();
            if (wave == w && expert[t] >= 0) {
                const int before = table[expert[t]];
                if (rank[t] == count - 1) table[expert[t]] = before + count;
                rank[t] += before;
            }
        }
    }
    __syncthreads();
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += 1024) {
        const int e = e0 + tid;
        int total;
        const int at = carry + block_scan(e < experts ? table[e] : 0, total);
        if (e < experts) {
            table[e] = at;
            offsets[e] = at;
        }
        carry += total;
    }
    if (tid == 0) offsets[experts] = carry;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t) {
        const int i = t * 1024 + tid;
        if (i >= pairs) break;
        int at = -1;
        if (expert[t] >= 0) {
            at = table[expert[t]] + rank[t];
            order[at] = i;
        }
        place[i] = at;
        if (i >= carry) order[i] = -1;
    }
}

// ------------------------------------------------------------------- rows
//
// A row is moved 16 bytes a thread; NT threads (64 or 256) walk a token's row.
// `width` need not be a multiple of the vector, nor the rows be aligned to it.

template <typename T>
constexpr int vec() {
    return 16 / (int)sizeof(T);
}

template <typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int64_t left, T (&v)[V]) {
    if (left >= V) {
        load_vec(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < left ? p[j] : (T)0.0f;
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, int64_t left, const T (&v)[V]) {
    if (left >= V) {
        store_vec(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) p[j] = v[j];
    }
}

template <int NT>
__device__ __forceinline__ int64_t own_token() {
    const int64_t t = (int64_t)blockIdx.x * (256 / NT) + (NT == 64 ? threadIdx.x >> 6 : 0);
    return ((int64_t)__builtin_amdgcn_readfirstlane((int)(t >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
}

// Zero the rows among places [t * top, t * top + top) that hold no pair.
template <typename T, int NT>
__device__ __forceinline__ void clear_empty(const int *order, int64_t t, int64_t top, T *rows,
                                            int64_t ld, int64_t width) {
    constexpr int V = vec<T>();
    T zero[V];
#pragma unroll
    for (int j = 0; j < V; ++j) zero[j] = (T)0.0f;
    for (int64_t s = t * top; s < t * top + top; ++s) {
        if (order[s] >= 0) continue;
        for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V)
            store_part<T, V>(rows + s * ld + c, width - c, zero);
    }
}

template <typename T, int NT>
__global__ __launch_bounds__(256) void dispatch_kernel(const T *__restrict__ x, int64_t ldx,
                                                       int64_t tokens, int64_t top, int64_t width,
                                                       const int *__restrict__ order,
                                                       const int *__restrict__ place,
                                                       T *__restrict__ xs, int64_t ldxs) {
    constexpr int V = vec<T>();
    const int64_t t = own_token<NT>();
    if (t >= tokens) return;
    const int64_t pairs = tokens * top;
    for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V) {
        T v[V];
        load_part<T, V>(x + t * ldx + c, width - c, v);
        for (int64_t s = 0; s < top; ++s) {
            const int64_t p = place[t * top + s];
            if (p >= 0 && p < pairs) store_part<T, V>(xs + p * ldxs + c, width - c, v);
        }
    }
    clear_empty<T, NT>(order, t, top, xs, ldxs, width);
}

template <typename T, int NT, bool WEIGHTS>
__global__ __launch_bounds__(256) void combine_kernel(const T *__restrict__ ys, int64_t ldys,
                                                      const float *__restrict__ weights,
                                                      int64_t tokens, int64_t top, int64_t width,
                                                      const int *__restrict__ place,
                                                      T *__restrict__ y, int64_t ldy) {
    constexpr int V = vec<T>();
    const int64_t t = own_token<NT>();
    if (t >= tokens) return;
    const int64_t pairs = tokens * top;
    for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V) {
        float sum[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
#pragma unroll 2
        for (int64_t s = 0; s < top; ++s) {
            const int64_t p = place[t * top + s];
            if (p < 0 || p >= pairs) continue;
            const float w = WEIGHTS ? weights[t * top + s] : 1.0f;
            T v[V];
            load_part<T, V>(ys + p * ldys + c, width - c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += w * (float)v[j];
        }
        T r[V];
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = (T)sum[j];
        store_part<T, V>(y + t * ldy + c, width - c, r);
    }
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

template <typename T, int NT>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const T *__restrict__ dy, int64_t lddy, const T *__restrict__ ys, int64_t ldys,
    const float *__restrict__ weights, int64_t tokens, int64_t top, int64_t width,
    const int *__restrict__ order, const int *__restrict__ place, T *__restrict__ dys,
    int64_t lddys, float *__restrict__ dweights) {
    constexpr int V = vec<T>();
    const int64_t t = own_token<NT>();
    if (t >= tokens) return;
    const int64_t pairs = tokens * top;
    for (int64_t s = 0; s < top; ++s) {
        const int64_t p = place[t * top + s];
        const bool live = p >= 0 && p < pairs;
        float dot = 0.0f;
        if (live) {
            const float w = dys ? weights[t * top + s] : 0.0f;
#pragma unroll 2
            for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V) {
                T g[V], v[V];
                load_part<T, V>(dy + t * lddy + c, width - c, g);
                if (dweights) {
                    load_part<T, V>(ys + p * ldys + c, width - c, v);
#pragma unroll
                    for (int j = 0; j < V; ++j) dot += (float)g[j] * (float)v[j];
                }
                if (dys) {
#pragma unroll
                    for (int j = 0; j < V; ++j) g[j] = (T)(w * (float)g[j]);
                    store_part<T, V>(dys + p * lddys + c, width - c, g);
                }
            }
        }
        if (dweights) {
            dot = token_sum<NT>(dot);
            if (threadIdx.x % NT == 0) dweights[t * top + s] = dot;
        }
    }
    if (dys) clear_empty<T, NT>(order, t, top, dys, lddys, width);
}

// A wave a token once the tokens fill the chip, a block before that.
inline bool wave_per_token(int64_t tokens) { return tokens >= 4096; }

template <typename T>
struct Rows {
    static hipError_t dispatch(const void *x, int64_t ldx, int64_t tokens, int64_t top,
                               int64_t width, const int *order, const int *place, void *xs,
                               int64_t ldxs, hipStream_t s) {
        if (wave_per_token(tokens))
            dispatch_kernel<T, 64><<<(unsigned)cdiv(tokens, 4), 256, 0, s>>>(
                (const T *)x, ldx, tokens, top, width, order, place, (T *)xs, ldxs);
        else
            dispatch_kernel<T, 256><<<(unsigned)tokens, 256, 0, s>>>(
                (const T *)x, ldx, tokens, top, width, order, place, (T *)xs, ldxs);
        return hipGetLastError();
    }
    template <bool W>
    static hipError_t combine_w(const void *ys, int64_t ldys, const float *weights, int64_t tokens,
                                int64_t top, int64_t width, const int *place, void *y, int64_t ldy,
                                hipStream_t s) {
        if (wave_per_token(tokens))
            combine_kernel<T, 64, W><<<(unsigned)cdiv(tokens, 4), 256, 0, s>>>(
                (const T *)ys, ldys, weights, tokens, top, width, place, (T *)y, ldy);
        else
            combine_kernel<T, 256, W><<<(unsigned)tokens, 256, 0, s>>>(
                (const T *)ys, ldys, weights, tokens, top, width, place, (T *)y, ldy);
        return hipGetLastError();
    }
    static hipError_t combine(const void *ys, int64_t ldys, const float *weights, int64_t tokens,
                              int64_t top, int64_t width, const int *place, void *y, int64_t ldy,
                              hipStream_t s) {
        return weights ? combine_w<true>(ys, ldys, weights, tokens, top, width, place, y, ldy, s)
                       : combine_w<false>(ys, ldys, weights, tokens, top, width, place, y, ldy, s);
    }
    static hipError_t backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                               const float *weights, int64_t tokens, int64_t top, int64_t width,
                               const int *order, const int *place, void *dys, int64_t lddys,
                               float *dweights, hipStream_t s) {
        if (wave_per_token(tokens))
            combine_backward_kernel<T, 64><<<(unsigned)cdiv(tokens, 4), 256, 0, s>>>(
                (const T *)dy, lddy, (const T *)ys, ldys, weights, tokens, top, width, order, place,
                (T *)dys, lddys, dweights);
        else
            combine_backward_kernel<T, 256><<<(unsigned)tokens, 256, 0, s>>>(
                (const T *)dy, lddy, (const T *)ys, ldys, weights, tokens, top, width, order, place,
                (T *)dys, lddys, dweights);
        return hipGetLastError();
    }
};

}  // namespace

bool plan_is_small(int64_t pairs, int64_t experts) {
    return pairs <= kSmallPairs && experts <= kSmallExperts;
}

hipError_t launch_plan(const int64_t *ids, int64_t pairs, int64_t experts, int *order, int *place,
                       int *offsets, const PlanScratch &ws, hipStream_t s) {
    if (plan_is_small(pairs, experts)) {
        plan_small_kernel<<<1, 1024, 0, s>>>(ids, (int)pairs, (int)experts, order, place, offsets);
        return hipGetLastError();
    }
    km::UpdateScratch us = {};
    us.tile_hist = ws.tile_hist;
    us.rank = ws.rank;
    us.n_tiles = ws.tiles;
    const hipError_t e = km::launch_rank_hist(ids, pairs, experts, us, km::Gate{}, s);
    if (e != hipSuccess) return e;
    plan_tiles_kernel<<<(unsigned)cdiv(experts, 64), 64, 0, s>>>(ws.tile_hist, experts, ws.tiles,
                                                                 ws.count);
    plan_scan_kernel<<<1, 1024, 0, s>>>(ws.count, experts, offsets);
    if (pairs > 0)
        plan_scatter_kernel<<<(unsigned)cdiv(pairs, 256), 256, 0, s>>>(
            ids, pairs, experts, ws.tile_hist, ws.rank, offsets, order, place);
    return hipGetLastError();
}

#define KX_BY_TYPE(call)                        \
    if (tokens == 0) return hipSuccess;         \
    if (dtype == 0) return Rows<float>::call;   \
    if (dtype == 1) return Rows<bf16>::call;    \
    return Rows<f16>::call

hipError_t launch_dispatch(const void *x, int64_t ldx, int dtype, int64_t tokens, int64_t top,
                           int64_t width, const int *order, const int *place, void *xs,
                           int64_t ldxs, hipStream_t s) {
    KX_BY_TYPE(dispatch(x, ldx, tokens, top, width, order, place, xs, ldxs, s));
}
hipError_t launch_combine(const void *ys, int64_t ldys, const float *weights, int dtype,
                          int64_t tokens, int64_t top, int64_t width, const int *place, void *y,
                          int64_t ldy, hipStream_t s) {
    KX_BY_TYPE(combine(ys, ldys, weights, tokens, top, width, place, y, ldy, s));
}
hipError_t launch_combine_backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                                   const float *weights, int dtype, int64_t tokens, int64_t top,
                                   int64_t width, const int *order, const int *place, void *dys,
                                   int64_t lddys, float *dweights, hipStream_t s) {
    KX_BY_TYPE(backward(dy, lddy, ys, ldys, weights, tokens, top, width, order, place, dys, lddys,
                        dweights, s));
}

}  // namespace kx
