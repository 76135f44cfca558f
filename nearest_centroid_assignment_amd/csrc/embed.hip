// embed.hip - rows of a table by number, scaled, and the table's gradient.
//
//   y[t] = scale * w[ids[t]]          dw[v] = scale * sum over t with ids[t] = v of dy[t]
//
// Bound by memory: the lookup reads the rows that come up and writes y; the gradient
// reads dy once and writes every row of dw once. The gradient sorts the tokens by number
// (stable, so the sums have one order and no atomic), cuts the sorted places into chunks
// of equal length, whatever the numbers' frequencies, and gives a wave or a block to each
// chunk: a row whose tokens all lie in one chunk is written by it; of the others each
// chunk leaves a float32 part, and a second kernel adds a row's parts in order and clears
// the rows that no token has.
#include "layers.h"
#include "kernels.h"
#include "rows.h"

namespace kx {
namespace {

// (65536 rows of 50000 x 2048 bf16: 81 us, 3.3 TB/s written beside what the caches do not hold of
// as much read.)
template <typename T, int NT, bool ONCE>
__global__ __launch_bounds__(256) void embed_kernel(const int64_t *__restrict__ ids, int64_t tokens,
                                                    const T *__restrict__ w, int64_t classes,
                                                    int64_t width, float scale, T *__restrict__ out,
                                                    int64_t ldo) {
    constexpr int V = vec<T>();
    const int64_t t = NT == 16 ? (int64_t)blockIdx.x * 16 + threadIdx.x / 16 : own_token<NT>();
    if (t >= tokens) return;
    const int64_t id = ids[t];
    const bool live = id >= 0 && id < classes;
    const T *p = w + (live ? id : 0) * width;
#pragma unroll 4
    for (int64_t c = (threadIdx.x % NT) * V; c < width; c += NT * V) {
        const int64_t a = chunk_at<V>(c, width);
        T v[V];
        if (live) {
            load_part<false, T, V>(p + a, width - a, v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = (T)(scale * (float)v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = (T)0.0f;
        }
        store_part<ONCE, T, V>(out + t * ldo + a, width - a, v);
    }
}

// The bucket of every token: its number modulo kEmbedBuckets, which spreads numbers that
// lie together (frequent ones often do).
__global__ __launch_bounds__(256) void bucket_kernel(const int64_t *__restrict__ ids,
                                                     int64_t tokens, int64_t classes,
                                                     int64_t *__restrict__ bucket) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= tokens) return;
    const int64_t id = ids[t];
    bucket[t] = id >= 0 && id < classes ? id & (kEmbedBuckets - 1) : -1;
}

// One block sorts one bucket's tokens by their number, stably: each wave counts a run of them,
// a prefix over the bucket's numbers (at most `locals`) and the waves, and each wave places its
// run. (A frequent number's bucket holds a good part of all tokens, and no barrier is in its
// way. us of the gradient of 64 columns, 65536 tokens of 50000 numbers, frequent as 1 / number,
// and as often as each other: eight waves 59 and 46, sixteen 54 and 49; four in rounds of 256
// tokens with three barriers each 75 and 45.)
constexpr int kRefineWaves = 8;

__global__ __launch_bounds__(kRefineWaves * 64) void refine_kernel(
    const int64_t *__restrict__ ids, int64_t classes, const int *__restrict__ order,
    const int *__restrict__ offsets, int locals, int *__restrict__ sorted, int *__restrict__ lo,
    int *__restrict__ hi) {
    constexpr int kAhead = 4;
    extern __shared__ int count[];  // kRefineWaves x locals
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.x;
    const int first = offsets[b], members = offsets[b + 1] - first;
    const int bits = 32 - __clz(locals);
    const int run = (members + kRefineWaves * 64 - 1) / (kRefineWaves * 64) * 64;
    const int from = wave * run, to = from + run < members ? from + run : members;
    int *own = count + wave * locals;
    for (int j = tid; j < kRefineWaves * locals; j += kRefineWaves * 64) count[j] = 0;
    __syncthreads();
    // `place`: where they go; else they are counted.
    auto sweep = [&](bool place) {
        for (int r = from; r < to; r += kAhead * 64) {
            int token[kAhead], l[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = r + u * 64 + lane;
                token[u] = i < to ? order[first + i] : -1;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                l[u] = token[u] >= 0 ? (int)(ids[token[u]] / kEmbedBuckets) : -1;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (r + u * 64 >= to) break;
                int rank, same;
                wave_rank(l[u], bits, rank, same);
                in_order();
                const int before = l[u] >= 0 ? own[l[u]] : 0;
                in_order();
                if (l[u] >= 0 && rank == 0) own[l[u]] = before + same;
                if (place && l[u] >= 0) sorted[before + rank] = token[u];
            }
        }
    };
    sweep(false);
    __syncthreads();
    if (wave == 0) {
        int start = first;
        for (int l0 = 0; l0 < locals; l0 += 64) {
            const int l = l0 + lane;
            int n[kRefineWaves], all = 0;
#pragma unroll
            for (int w = 0; w < kRefineWaves; ++w) {
                n[w] = l < locals ? count[w * locals + l] : 0;
                all += n[w];
            }
            const int incl = wave_incl_scan(all);
            int at = start + incl - all;
            const int64_t v = (int64_t)l * kEmbedBuckets + b;
            if (l < locals) {
                if (v < classes) {
                    lo[v] = at;
                    hi[v] = at + all;
                }
#pragma unroll
                for (int w = 0; w < kRefineWaves; ++w) {
                    count[w * locals + l] = at;
                    at += n[w];
                }
            }
            start += __builtin_amdgcn_readlane(incl, 63);
        }
    }
    __syncthreads();
    sweep(true);
}

struct SumArgs {
    int64_t lddy, width;
    const int64_t *ids;
    const int *order, *total, *lo, *hi;  // total: places with a token
    int64_t classes;
    int chunk, col_blocks;
    float scale;
    float *partial;
};

// Chunk c's part of a row whose tokens start at `lo`: a row that starts inside the chunk
// has the second of its two slots, the one that starts before it, or with it, the first (as
// sum_kernel leaves them).
__device__ __forceinline__ int64_t slot_of(int64_t c, int chunk, int lo) {
    return 2 * c + (lo > c * chunk ? 1 : 0);
}

// A chunk's tokens and their numbers lie in the lanes of the wave (kChunk at most), and its rows
// come in groups of eight, the next group on its way while one is added. Which rows end
// inside the chunk shows in the numbers themselves; only the first row may have begun before
// it and the last go on after it. (65536 x 2048 bf16 of 50000: 72 us, 3.7 TB/s of dy read beside
// the rows written.)
constexpr int kChunk = 64;

template <typename T, int V, int NT, bool ONCE>
__global__ __launch_bounds__(256) void sum_kernel(SumArgs a, const T *__restrict__ dy,
                                                  T *__restrict__ dw) {
    constexpr int kAhead = 8;
    const int64_t unit = own_token<NT>();
    const int64_t c = unit / a.col_blocks;
    const int64_t col = ((unit - c * a.col_blocks) * NT + threadIdx.x % NT) * V;
    const int64_t p0 = c * a.chunk, total = *a.total;
    if (p0 >= total) return;
    const int n = (int)(total - p0 < a.chunk ? total - p0 : a.chunk);
    const int lane = threadIdx.x & 63;
    const int token = a.order[p0 + (lane < n ? lane : n - 1)];
    const int number = (int)a.ids[token];
    const int first_lo = a.lo[__builtin_amdgcn_readlane(number, 0)];
    const int last_hi = a.hi[__builtin_amdgcn_readlane(number, n - 1)];
    const bool active = col < a.width;
    const int64_t at = active ? chunk_at<V>(col, a.width) : 0;
    const int64_t left = active ? a.width - at : 0;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
    T v[kAhead][V], next[kAhead][V];
    auto fetch = [&](int p, T (&to)[kAhead][V]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t t = __builtin_amdgcn_readlane(token, p + u < n ? p + u : n - 1);
            load_part<ONCE, T, V>(dy + t * a.lddy + at, left, to[u]);
        }
    };
    int id = __builtin_amdgcn_readlane(number, 0), start = 0;
    auto flush = [&](int end) {
        const bool whole = (start > 0 || first_lo >= p0) && (end < n || last_hi <= p0 + n);
        if (whole) {
            T r[V];
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] = (T)(a.scale * sum[j]);
            store_part<false, T, V>(dw + (int64_t)id * a.width + at, left, r);
        } else {
            float *to = a.partial + (2 * c + (start > 0 ? 1 : 0)) * a.width;
            store_part<false, float, V>(to + at, left, sum);
        }
    };
    fetch(0, next);
    for (int p = 0; p < n; p += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j) v[u][j] = next[u][j];
        if (p + kAhead < n) fetch(p + kAhead, next);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (p + u >= n) break;
            const int now = __builtin_amdgcn_readlane(number, p + u);
            if (now != id) {
                flush(p + u);
                id = now;
                start = p + u;
#pragma unroll
                for (int j = 0; j < V; ++j) sum[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += (float)v[u][j];
        }
    }
    flush(n);
}

// The first `joins` blocks: chunk c and 256 columns; the row that starts in chunk c and
// goes on past it, if there is one, is the sum of its chunks' parts (four waves, each
// every fourth part). The blocks after them clear the rows without a token, a wave each. (34 us
// at that size, most of it zeros.)
template <typename T>
__global__ __launch_bounds__(256) void finish_kernel(SumArgs a, int64_t joins, T *__restrict__ dw) {
    constexpr int V = vec<T>();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (blockIdx.x >= joins) {
        const int64_t v = (int64_t)(blockIdx.x - joins) * 4 + wave;
        if (v >= a.classes || a.lo[v] < a.hi[v]) return;
        T zero[V];
#pragma unroll
        for (int j = 0; j < V; ++j) zero[j] = (T)0.0f;
        for (int64_t col = lane * V; col < a.width; col += 64 * V) {
            const int64_t at = chunk_at<V>(col, a.width);
            store_part<true, T, V>(dw + v * a.width + at, a.width - at, zero);
        }
        return;
    }
    __shared__ float part[4][256];
    const int64_t cols = (a.width + 255) / 256;
    const int64_t c = blockIdx.x / cols;
    const int64_t p0 = c * a.chunk, p1 = p0 + a.chunk;
    if (p1 >= *a.total) return;  // the last chunk: nothing goes on
    const int64_t id = a.ids[a.order[p1 - 1]];
    const int lo = a.lo[id], hi = a.hi[id];
    if (lo < p0 || hi <= p1) return;
    const int64_t col = (blockIdx.x - c * cols) * 256 + lane * 4;
    float sum[4] = {0, 0, 0, 0};
    const int64_t left = a.width - col, last = (hi - 1) / a.chunk;
    if (left > 0) {
#pragma unroll 8
        for (int64_t k = c + wave; k <= last; k += 4) {
            float v[4];
            load_part<false, float, 4>(a.partial + slot_of(k, a.chunk, lo) * a.width + col, left, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][lane * 4 + j] = sum[j];
    __syncthreads();
    const int64_t out = (blockIdx.x - c * cols) * 256 + threadIdx.x;
    if (out < a.width) {
        const int i = threadIdx.x;
        dw[id * a.width + out] =
            (T)(a.scale * ((part[0][i] + part[1][i]) + (part[2][i] + part[3][i])));
    }
}

// A wave to a token's row where there are enough of them and they are short, else a block
// (the rule of the token rows in tokens.hip); 16 lanes where they hold it in one access each.
// (Four rows a wave, their loads in flight together: 65536 x 4 KB of 50000 84 us, a block to
// each 78.)
constexpr int64_t kMostBlocks = 1 << 24;
bool by_wave(int64_t rows, int64_t bytes) {
    return rows >= kMostBlocks || (rows >= 2048 && bytes <= 3 << 10);
}

// Rows that are more than the 256 MB of the memory-side cache pass the caches by, where they
// are whole lines of 128 bytes (the same rule's other half).
template <typename T>
bool passes_by(int64_t rows, int64_t width, int64_t ld) {
    const int64_t size = sizeof(T);
    return width * size % 128 == 0 && ld * size % 128 == 0 && rows * width * size >= 256 << 20;
}

template <typename T>
hipError_t embed_t(const int64_t *ids, int64_t tokens, const void *w, int64_t classes, int64_t width,
                   float scale, void *out, int64_t ldo, hipStream_t s) {
    const int64_t bytes = width * (int64_t)sizeof(T);
    const bool once = passes_by<T>(tokens, width, ldo);
    if (width <= 16 * vec<T>() && tokens < kMostBlocks * 16)
        return launch(once ? embed_kernel<T, 16, true> : embed_kernel<T, 16, false>, cdiv(tokens, 16), 256, 0,
                      s, ids, tokens, (const T *)w, classes, width, scale, (T *)out, ldo);
    if (by_wave(tokens, bytes))
        return launch(once ? embed_kernel<T, 64, true> : embed_kernel<T, 64, false>, cdiv(tokens, 4),
                      256, 0, s, ids, tokens, (const T *)w, classes, width, scale, (T *)out, ldo);
    return launch(once ? embed_kernel<T, 256, true> : embed_kernel<T, 256, false>, tokens, 256, 0, s,
                  ids, tokens, (const T *)w, classes, width, scale, (T *)out, ldo);
}

// Threads and values a thread that a chunk's rows take: as many lanes busy as there are (65536 x 64
// bf16 of 1000: by 8 values 59 us, by 2 36).
template <typename T, class F>
hipError_t with_rows(int64_t width, F f) {
    constexpr int V = vec<T>();
    if (width <= 64 * V / 4) return f(ActTag<V / 4>{}, ActTag<64>{});
    if (width <= 64 * V) return f(ActTag<V>{}, ActTag<64>{});
    return f(ActTag<V>{}, ActTag<256>{});
}

template <typename T>
hipError_t backward_t(SumArgs a, int64_t tokens, const void *dy, void *dw, hipStream_t s) {
    const int64_t chunks = cdiv(tokens, a.chunk);
    const bool once = passes_by<T>(tokens, a.width, a.lddy);
    hipError_t e = hipSuccess;
    if (tokens > 0)
        e = with_rows<T>(a.width, [&](auto v, auto nt) {
            constexpr int V = decltype(v)::value, NT = decltype(nt)::value;
            a.col_blocks = (int)cdiv(a.width, V * NT);
            return launch(once ? sum_kernel<T, V, NT, true> : sum_kernel<T, V, NT, false>,
                          cdiv(chunks * a.col_blocks, 256 / NT), 256, 0, s, a, (const T *)dy, (T *)dw);
        });
    if (e != hipSuccess) return e;
    const int64_t joins = chunks * cdiv(a.width, 256);
    return launch(finish_kernel<T>, joins + cdiv(a.classes, 4), 256, 0, s, a, joins, (T *)dw);
}

}  // namespace

// Long chunks leave few parts to join, short ones more blocks. us of the gradient with chunks of
// 16 / 32 / 64: 5000 x 777 float32 of 1111 27 / 28 / 34, 20000 x 1024 bf16 of 500 43 / 37 / 45,
// 65536 x 2048 bf16 of 50000 185 / 166 / 158; bf16 of 5000, frequent as 1 / number: 65536 x 64 36 /
// 35 / 37, x 256 46 / 51 / 64, x 777 87 / 78 / 74; 131072 x 256 69 / 63 / 75; 40000 x 2048 82 / 74 /
// 67; 10000 x 5632 66 / 58 / 64. Over 160 sizes (1000 to 131072 tokens, 64 to 5632 columns, 500
// to 50000 numbers) the rule is 3.5 % slower than the best of the three in the geometric mean, and
// 42 % at most: it goes by the tokens alone, and the width counts as well, most of all for rows
// that leave half of a wave's lanes idle. (The order of the sums, and so their last bits, hang on
// it.)
int64_t embed_chunk(int64_t tokens) { return tokens >= 65536 ? kChunk : tokens >= 16384 ? kChunk / 2 : kChunk / 4; }

bool embed_grid_ok(int dtype, int64_t tokens, int64_t classes, int64_t width) {
    const int64_t chunks = cdiv(tokens, embed_chunk(tokens));
    const int64_t v = dtype == 0 ? 4 : 8;
    return chunks * cdiv(width, 64 * v) + 4 < kMostBlocks &&
           chunks * cdiv(width, 256) + cdiv(classes, 4) < kMostBlocks;
}

hipError_t launch_embed(const int64_t *ids, int64_t tokens, const void *w, int dtype,
                        int64_t classes, int64_t width, float scale, void *out, int64_t ldo,
                        hipStream_t s) {
    if (tokens == 0) return hipSuccess;
    if (dtype == 0) return embed_t<float>(ids, tokens, w, classes, width, scale, out, ldo, s);
    if (dtype == 1) return embed_t<bf16>(ids, tokens, w, classes, width, scale, out, ldo, s);
    return embed_t<f16>(ids, tokens, w, classes, width, scale, out, ldo, s);
}

hipError_t launch_embed_backward(const void *dy, int64_t lddy, const int64_t *ids, int64_t tokens,
                                 int dtype, int64_t classes, int64_t width, float scale, void *dw,
                                 const EmbedScratch &ws, hipStream_t s) {
    SumArgs a = {lddy, width, ids, ws.order, nullptr, ws.offsets, ws.offsets + 1, classes,
                 (int)embed_chunk(tokens), 1, scale, ws.partial};
    hipError_t e;
    if (classes <= kEmbedDirect) {
        e = launch_plan(ids, tokens, classes, ws.order, ws.place, ws.offsets, ws.plan, s);
        a.total = ws.offsets + classes;
    } else {
        e = tokens ? launch(bucket_kernel, cdiv(tokens, 256), 256, 0, s, ids, tokens, classes, ws.bucket)
                   : hipSuccess;
        if (e == hipSuccess)
            e = launch_plan(ws.bucket, tokens, kEmbedBuckets, ws.order, ws.place, ws.offsets, ws.plan, s);
        const int locals = (int)cdiv(classes, kEmbedBuckets);
        if (e == hipSuccess)
            e = launch(refine_kernel, kEmbedBuckets, kRefineWaves * 64,
                       (size_t)kRefineWaves * locals * sizeof(int), s, ids, classes, ws.order,
                       ws.offsets, locals, ws.sorted, ws.lo, ws.hi);
        a.total = ws.offsets + kEmbedBuckets;
        a.order = ws.sorted;
        a.lo = ws.lo;
        a.hi = ws.hi;
    }
    if (e != hipSuccess) return e;
    if (dtype == 0) return backward_t<float>(a, tokens, dy, dw, s);
    if (dtype == 1) return backward_t<bf16>(a, tokens, dy, dw, s);
    return backward_t<f16>(a, tokens, dy, dw, s);
}

}  // namespace kx
