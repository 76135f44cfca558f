// tokens.hip - pairs of (token, slot) sorted by expert, the token rows gathered
// in that order, the experts' rows summed back with weights, and gradients.
//
// The sort is a stable counting sort. A wave ranks its 64 pairs among themselves
// by ballots over the bits of the expert numbers, leaves its count of each expert in
// LDS, and the ranks of a whole block follow from a prefix over its waves; then a
// prefix over blocks and experts gives the places. One block in one launch, two
// launches (the second sums the blocks' counts in every block) or four: see
// plan_is_small and plan_in_two.
//
// The row kernels give one wave or one block to a token (see how()): its own row is read
// once, and the rows of its `top` pairs are reached through the inverse permutation, so
// every row is moved once and no sum needs an atomic. The gradient of combine, whose rows
// are all the pairs', goes by place instead.
#include "experts.h"
#include "kernels.h"

namespace kx {
namespace {

constexpr int kTile = (int)km::kSortTileRows;
constexpr int kSmallTiles = 2;                     // tiles that the one-block sort takes
constexpr int kSmallPairs = kSmallTiles * 1024;
constexpr int kWaveCounts = 65536;                 // counts of (wave, expert) in LDS: 128 KB
constexpr int kPlaceTiles = 256, kPlaceExperts = 2048;  // most of the two-launch sort

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
__device__ __forceinline__ int bits_of(int64_t experts) { return 64 - __clzll((unsigned long long)experts); }

__device__ __forceinline__ int expert_of(const int64_t *ids, int64_t i, int64_t pairs, int64_t experts) {
    if (i >= pairs) return -1;
    const int64_t e = ids[i];
    return e >= 0 && e < experts ? (int)e : -1;
}

// One block per tile of 1024 pairs: rank of every pair in its tile, and the
// tile's count of every expert.
__global__ __launch_bounds__(1024) void plan_rank_kernel(const int64_t *__restrict__ ids,
                                                         int64_t pairs, int experts,
                                                         int *__restrict__ tile_hist,
                                                         unsigned short *__restrict__ rank_out) {
    extern __shared__ unsigned short counts[];  // 16 x experts, by wave
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t i = (int64_t)blockIdx.x * 1024 + tid;
    const int expert = expert_of(ids, i, pairs, experts);
    for (int j = tid; j < 16 * experts; j += 1024) counts[j] = 0;
    int rank, count;
    wave_rank(expert, bits_of(experts), rank, count);
    __syncthreads();
    if (expert >= 0 && rank == 0) counts[wave * experts + expert] = (unsigned short)count;
    __syncthreads();
    for (int e = tid; e < experts; e += 1024) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int c = counts[w * experts + e];
            counts[w * experts + e] = (unsigned short)run;
            run += c;
        }
        tile_hist[(int64_t)blockIdx.x * experts + e] = run;
    }
    __syncthreads();
    if (expert >= 0) rank_out[i] = (unsigned short)(rank + counts[wave * experts + expert]);
}

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

// One block per tile: every expert's count in all tiles and in the tiles before
// this one, a prefix over the experts, and the tile's pairs put in their places.
// The sums are the same in every block; block 0 writes the offsets.
__global__ __launch_bounds__(1024) void plan_place_kernel(
    const int64_t *__restrict__ ids, int64_t pairs, int experts, int tiles,
    const int *__restrict__ tile_hist, const unsigned short *__restrict__ rank,
    int *__restrict__ order, int *__restrict__ place, int *__restrict__ offsets) {
    __shared__ int base[kPlaceExperts];
    const int tid = threadIdx.x, b = blockIdx.x;
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += 1024) {
        const int e = e0 + tid;
        int before = 0, all = 0;
        if (e < experts) {
            constexpr int U = 32;  // counts in flight
            for (int t0 = 0; t0 < tiles; t0 += U) {
                int v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    v[u] = tile_hist[(int64_t)(t0 + u < tiles ? t0 + u : tiles - 1) * experts + e];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = t0 + u < tiles ? v[u] : 0;
                    before += t0 + u < b ? c : 0;
                    all += c;
                }
            }
        }
        int total;
        const int at = carry + block_scan(all, total);
        if (e < experts) {
            base[e] = at + before;
            if (b == 0) offsets[e] = at;
        }
        carry += total;
    }
    if (b == 0 && tid == 0) offsets[experts] = carry;
    __syncthreads();
    const int64_t i = (int64_t)b * 1024 + tid;
    if (i >= pairs) return;
    const int expert = expert_of(ids, i, pairs, experts);
    int at = -1;
    if (expert >= 0) {
        at = base[expert] + rank[i];
        order[at] = (int)i;
    }
    place[i] = at;
    if (i >= carry) order[i] = -1;
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

// The whole sort in one block, `tiles` rounds of 1024 pairs.
__global__ __launch_bounds__(1024) void plan_small_kernel(const int64_t *__restrict__ ids, int pairs,
                                                          int experts, int *__restrict__ order,
                                                          int *__restrict__ place,
                                                          int *__restrict__ offsets) {
    extern __shared__ unsigned short counts[];  // waves x experts
    const int tid = threadIdx.x, wave = tid >> 6;
    const int waves = (pairs + 63) / 64;  // of pairs, 16 to a round
    for (int j = tid; j < waves * experts; j += 1024) counts[j] = 0;
    int expert[kSmallTiles], rank[kSmallTiles], count[kSmallTiles];
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t) expert[t] = expert_of(ids, t * 1024 + tid, pairs, experts);
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t) {
        rank[t] = count[t] = 0;
        if (t * 1024 < pairs) wave_rank(expert[t], bits_of(experts), rank[t], count[t]);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kSmallTiles; ++t)
        if (expert[t] >= 0 && rank[t] == 0)
            counts[(t * 16 + wave) * experts + expert[t]] = (unsigned short)count[t];
    __syncthreads();
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += 1024) {
        const int e = e0 + tid;
        int all = 0;
        if (e < experts)
            for (int w = 0; w < waves; ++w) all += counts[w * experts + e];
        int total;
        int at = carry + block_scan(all, total);
        if (e < experts) {
            offsets[e] = at;
            for (int w = 0; w < waves; ++w) {  // (places are below 2048)
                const int c = counts[w * experts + e];
                counts[w * experts + e] = (unsigned short)at;
                at += c;
            }
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
            at = counts[(t * 16 + wave) * experts + expert[t]] + rank[t];
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
        for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V) {
            const int64_t a = chunk_at<V>(c, width);
            store_part<false, T, V>(rows + s * ld + a, width - a, zero);
        }
    }
}

template <typename T, int NT, bool ONCE>
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
        const int64_t a = chunk_at<V>(c, width);
        T v[V];
        load_part<false, T, V>(x + t * ldx + a, width - a, v);
        for (int64_t s = 0; s < top; ++s) {
            const int64_t p = place[t * top + s];
            if (p >= 0 && p < pairs) store_part<ONCE, T, V>(xs + p * ldxs + a, width - a, v);
        }
    }
    clear_empty<T, NT>(order, t, top, xs, ldxs, width);
}

template <typename T, int NT, bool ONCE, bool WEIGHTS>
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
        const int64_t a = chunk_at<V>(c, width);
        float sum[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.0f;
#pragma unroll 2
        for (int64_t s = 0; s < top; ++s) {
            const int64_t p = place[t * top + s];
            if (p < 0 || p >= pairs) continue;
            const float w = WEIGHTS ? weights[t * top + s] : 1.0f;
            T v[V];
            load_part<ONCE, T, V>(ys + p * ldys + a, width - a, v);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += w * (float)v[j];
        }
        T r[V];
#pragma unroll
        for (int j = 0; j < V; ++j) r[j] = (T)sum[j];
        store_part<false, T, V>(y + t * ldy + a, width - a, r);
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

// One place a wave (or block): its row of ys is read and its row of dys written in
// sorted order, the token's row of dy gathered (a token's rows again, from the
// caches). By token, with dys scattered, a wave each: 131072 x 2048 bf16 rows 281 us, by
// place 251 (this call alone; between the other operators of a pass 282).
template <typename T, int NT, bool ONCE>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const T *__restrict__ dy, int64_t lddy, const T *__restrict__ ys, int64_t ldys,
    const float *__restrict__ weights, int64_t pairs, int64_t top, int64_t width,
    const int *__restrict__ order, const int *__restrict__ place, T *__restrict__ dys,
    int64_t lddys, float *__restrict__ dweights) {
    constexpr int V = vec<T>();
    const int64_t p = own_token<NT>();
    if (p >= pairs) return;
    const int first = (threadIdx.x % NT) * V;
    if (dweights && threadIdx.x % NT == 0) {
        const int64_t at = place[p];  // of pair p: a dropped one has no row
        if (at < 0 || at >= pairs) dweights[p] = 0.0f;
    }
    const int64_t pair = order[p];
    if (pair < 0 || pair >= pairs) {
        if (!dys) return;
        T zero[V];
#pragma unroll
        for (int j = 0; j < V; ++j) zero[j] = (T)0.0f;
        for (int64_t c = first; c < width; c += NT * V) {
            const int64_t a = chunk_at<V>(c, width);
            store_part<false, T, V>(dys + p * lddys + a, width - a, zero);
        }
        return;
    }
    const T *g_row = dy + pair / top * lddy;
    const float w = dys ? weights[pair] : 0.0f;
    float dot = 0.0f;
#pragma unroll 4
    for (int64_t c = first; c < width; c += NT * V) {
        const int64_t a = chunk_at<V>(c, width);
        const int again = (int)(c - a);  // values that the chunk before has counted
        T g[V], v[V];
        load_part<false, T, V>(g_row + a, width - a, g);
        if (dweights) {
            load_part<ONCE, T, V>(ys + p * ldys + a, width - a, v);
#pragma unroll
            for (int j = 0; j < V; ++j) dot += j < again ? 0.0f : (float)g[j] * (float)v[j];
        }
        if (dys) {
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = (T)(w * (float)g[j]);
            store_part<ONCE, T, V>(dys + p * lddys + a, width - a, g);
        }
    }
    if (!dweights) return;
    dot = token_sum<NT>(dot);
    if (threadIdx.x % NT == 0) dweights[pair] = dot;
}

// `wave`: a wave or a block of four to each of `own` rows. A wave moves 1 KB of a row at a
// time, so longer rows have more in flight with a block; short ones leave most of a block
// idle, which counts once there are enough of them to fill the chip. us, wave / block, of
// dispatch, combine (two slots a token; bf16 or float32) and combine's gradient:
//   1024 rows of 1 KB  2.9 2.8 3.6 / 2.9 2.8 4.3     8192 of 1 KB  5.6 5.1 12 / 7.2 6.0 21
//   1024 of 2 KB  3.5 3.3 4.2 / 3.2 3.1 4.5          8192 of 2 KB  9.8 9.0 18 / 11 10 22
//   4096 of 3 KB  8.5 8.6 14 / 9.0 8.8 16            80000 of 3 KB  144 118 224 / 135 118 278
//   4096 of 3.5 KB  9.5 10 18 / 9.9 9.8 17           80000 of 3.5 KB  168 154 308 / 157 154 295
//   256 of 4 KB  4.1 4.9 4.9 / 2.8 2.8 3.6           65536 of 4 KB  171 143 246 / 149 124 252
//   256 of 16 KB  10 14 12 / 4.9 5.4 5.8             20000 of 16 KB  201 206 320 / 193 184 305
//
// `once`: rows of the pairs that are more than the 256 MB of the memory-side cache pass
// the caches by, where they are whole lines of 128 bytes. 65536 x 2 rows of 4 KB, all five
// operators 770 -> 673 us: combine and dispatch's gradient 156 -> 124 (their loads),
// combine's gradient 281 -> 252 (its stores); dispatch's stores are as fast either way
// there (147, 149) and faster this way in shorter rows (360000 of 0.9 KB 73 -> 69). Smaller
// sets are read from the cache: 15009 x 1001 f16 (30 MB), the gradient 18 -> 25.
struct How {
    bool wave, once;
};
constexpr int64_t kMostBlocks = 1 << 24;  // of 256 threads: one dispatch
template <typename T>
How how(int64_t own, int64_t pairs, int64_t width, int64_t ld) {
    const int64_t bytes = width * (int64_t)sizeof(T);
    const bool lines = bytes % 128 == 0 && ld * (int64_t)sizeof(T) % 128 == 0;
    return {own >= kMostBlocks || (own >= 2048 && bytes <= 3 << 10), lines && pairs * bytes > 256 << 20};
}

#define KX_ROWS(kernel, rows, ...)                                                             \
    do {                                                                                       \
        if (h.wave)                                                                            \
            return launch(h.once ? kernel<T, 64, true __VA_ARGS__>                             \
                                 : kernel<T, 64, false __VA_ARGS__>,                           \
                          cdiv(rows, 4), 256, 0, s, KX_ARGS);                                  \
        return launch(h.once ? kernel<T, 256, true __VA_ARGS__>                                \
                             : kernel<T, 256, false __VA_ARGS__>,                              \
                      rows, 256, 0, s, KX_ARGS);                                               \
    } while (0)

template <typename T>
struct Rows {
    static hipError_t dispatch(const void *x, int64_t ldx, int64_t tokens, int64_t top,
                               int64_t width, const int *order, const int *place, void *xs,
                               int64_t ldxs, hipStream_t s) {
        const How h = how<T>(tokens, tokens * top, width, ldxs);
#define KX_ARGS (const T *)x, ldx, tokens, top, width, order, place, (T *)xs, ldxs
        KX_ROWS(dispatch_kernel, tokens);
#undef KX_ARGS
    }
    static hipError_t combine(const void *ys, int64_t ldys, const float *weights, int64_t tokens,
                              int64_t top, int64_t width, const int *place, void *y, int64_t ldy,
                              hipStream_t s) {
        const How h = how<T>(tokens, tokens * top, width, ldys);
#define KX_ARGS (const T *)ys, ldys, weights, tokens, top, width, place, (T *)y, ldy
        if (weights)
            KX_ROWS(combine_kernel, tokens, , true);
        else
            KX_ROWS(combine_kernel, tokens, , false);
#undef KX_ARGS
    }
    static hipError_t backward(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                               const float *weights, int64_t tokens, int64_t top, int64_t width,
                               const int *order, const int *place, void *dys, int64_t lddys,
                               float *dweights, hipStream_t s) {
        const int64_t pairs = tokens * top;
        const How h = how<T>(pairs, pairs, width, dys ? lddys : ldys);
#define KX_ARGS                                                                                 \
    (const T *)dy, lddy, (const T *)ys, ldys, weights, pairs, top, width, order, place, (T *)dys, \
        lddys, dweights
        KX_ROWS(combine_backward_kernel, pairs);
#undef KX_ARGS
    }
};

}  // namespace

// One block in one launch, as far as it is the fastest (its counts of (wave, expert) have
// to fit LDS). us, one block / two launches: 2048 pairs of 8 experts 5.2 / 6.5, of 256
// 6.3 / 7.0, of 1024 8.4 / 10.1; 2500 pairs 6.1 / 6.4, 7.6 / 7.1 and 10.3 / 10.4; 4096
// pairs 7.8 / 6.5, 10.2 / 7.1, 14.5 / 10.3.
bool plan_is_small(int64_t pairs, int64_t experts) {
    return pairs <= kSmallPairs && cdiv(pairs, 64) * experts <= kWaveCounts;
}
// In the two-launch sort every block sums the counts of all tiles, 1024 experts at a time.
// us, two / four launches: 256 tiles of 17 experts 15.1 / 23.9, of 768 27.7 / 31.6, 293
// tiles (blocks that no longer all run at once) 28.3 / 27.6 and 55.7 / 39.0; 1024 experts,
// 128 tiles 20.5 / 22.6, 157 23.6 / 25.1, 196 29.8 / 28.0; 1100 experts, 64 tiles 16.3 /
// 19.2, 128 24.9 / 23.4; 2048 experts, 32 tiles 15.5 / 17.4, 64 21.7 / 19.7; 2500
// experts, 3 tiles 17.1 / 16.8.
static bool plan_in_two(int64_t tiles, int64_t experts) {
    return tiles <= kPlaceTiles && experts <= kPlaceExperts &&
           tiles * experts * cdiv(experts, 1024) <= 160 * 1024;
}

hipError_t launch_plan(const int64_t *ids, int64_t pairs, int64_t experts, int *order, int *place,
                       int *offsets, const PlanScratch &ws, hipStream_t s) {
    if (plan_is_small(pairs, experts)) {
        const size_t lds = (size_t)cdiv(pairs, 64) * experts * sizeof(unsigned short);
        return launch(plan_small_kernel, 1, 1024, lds, s, ids, (int)pairs, (int)experts, order, place,
                      offsets);
    }
    if (plan_in_two(ws.tiles, experts)) {
        const size_t lds = (size_t)16 * experts * sizeof(unsigned short);
        const hipError_t e = launch(plan_rank_kernel, ws.tiles, 1024, lds, s, ids, pairs, (int)experts,
                                    ws.tile_hist, ws.rank);
        if (e != hipSuccess) return e;
        return launch(plan_place_kernel, ws.tiles, 1024, 0, s, ids, pairs, (int)experts, (int)ws.tiles,
                      ws.tile_hist, ws.rank, order, place, offsets);
    }
    km::UpdateScratch us = {};
    us.tile_hist = ws.tile_hist;
    us.rank = ws.rank;
    us.n_tiles = ws.tiles;
    hipError_t e = km::launch_rank_hist(ids, pairs, experts, us, km::Gate{}, s);
    if (e == hipSuccess)
        e = launch(plan_tiles_kernel, cdiv(experts, 64), 64, 0, s, ws.tile_hist, experts, ws.tiles,
                   ws.count);
    if (e == hipSuccess) e = launch(plan_scan_kernel, 1, 1024, 0, s, ws.count, experts, offsets);
    if (e != hipSuccess || pairs == 0) return e;
    return launch(plan_scatter_kernel, cdiv(pairs, 256), 256, 0, s, ids, pairs, experts, ws.tile_hist,
                  ws.rank, offsets, order, place);
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
