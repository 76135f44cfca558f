// norm.hip - layer norm over the rows of a matrix, and its gradients.
//
//   h = (x - mean) rstd,  rstd = 1 / sqrt(mean of (x - mean)^2 + eps),  y = h weight + bias
//   g = dy weight,  dx = rstd (g - mean(g) - h mean(g h)),
//   dweight = sum over rows of dy h,  dbias = sum over rows of dy
//
// Bound by memory: x is read and y written once; the gradient reads x and dy and
// writes dx once. A row lives in the registers of a few lanes, a wave or a block, so that the
// variance is the mean square of what is left after the mean is taken off (two passes
// over registers: no cancellation), and the columns' sums of the gradient stay in
// registers over all rows that they take; the blocks' sums are added in order
// by a second kernel. Rows longer than four accesses of 512 threads are read again from the caches.
#include "layers.h"
#include "rows.h"

namespace kx {
namespace {

// A row's threads: 16 or 32 lanes, a wave, or a block of 128, 256 or 512.
template <int NT>
constexpr int kThreads = NT > 64 ? NT : 256;
template <int NT>
constexpr int kRowWaves = NT > 64 ? NT / 64 : 1;
template <int NT>
__device__ __forceinline__ int64_t own_row() {
    if (NT > 64) return blockIdx.x;
    return NT < 64 ? (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT : own_token<NT>();
}

// Sum of each of v over the NT threads of a row, in a fixed order, to all of them.
// `turn`: two calls in a row use the two halves of the memory, so one barrier is enough.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[kRowWaves<NT>][N], int turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] += rotated<0x128>(v[i]);
        v[i] += rotated<0x124>(v[i]);
        v[i] += rotated<0x122>(v[i]);
        v[i] += rotated<0x121>(v[i]);
        if (NT > 16) v[i] += __shfl_xor(v[i], 16);
        if (NT > 32) v[i] += __shfl_xor(v[i], 32);
    }
    if constexpr (NT > 64) {
        float(*p)[N] = part[turn & 1];
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) p[threadIdx.x >> 6][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = p[0][i] + p[1][i];
            if (NT > 128) v[i] += p[2][i] + p[3][i];
#pragma unroll
            for (int w = 4; w < kRowWaves<NT>; w += 4)
                v[i] += (p[w][i] + p[w + 1][i]) + (p[w + 2][i] + p[w + 3][i]);
        }
    }
}

// The thread's values of a row: C chunks of V, the last of the row moved back where it
// would leave it. again(i): how many of chunk i's first values the chunk before holds too
// (V: all, the chunk lies past the row).
// EVEN: the row is whole chunks, so again is 0 or V.
template <int V, int C, int NT, bool EVEN>
struct Chunks {
    int64_t at[C];
    int again[C];
    // Whether value j of chunk i counts here. (A comparison in the loop over rows: kept over
    // all of it, the answers were more than the scalar registers.)
    __device__ __forceinline__ bool counts(int i, int j) const {
        int n = again[i];
        if (!EVEN) asm volatile("" : "+v"(n));
        return EVEN ? n != V : j >= n;
    }
    __device__ __forceinline__ bool there(int i) const { return again[i] != V; }
    __device__ __forceinline__ void init(int64_t width) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int64_t c = ((int64_t)i * NT + threadIdx.x % NT) * V;
            at[i] = c < width ? chunk_at<V>(c, width) : 0;  // (width >= V)
            again[i] = c < width ? (int)(c - at[i]) : V;
        }
    }
};

template <bool ONCE, typename T, int V, int C, int NT, bool EVEN>
__device__ __forceinline__ void load_chunks(const Chunks<V, C, NT, EVEN> &ch, const T *row, T (&v)[C][V]) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (ch.there(i)) {
            if (ONCE)
                load_once(row + ch.at[i], v[i]);
            else
                load_vec(row + ch.at[i], v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = (T)0.0f;
        }
    }
}
template <bool ONCE, typename T, int V>
__device__ __forceinline__ void store_chunk(T *p, const T (&v)[V]) {
    if (ONCE)
        store_once(p, v);
    else
        store_vec(p, v);
}

// Every `step`-th row a few lanes, a wave or a block, the next one on its way meanwhile. ONCE:
// rows that no cache holds pass the caches by (see once_of).
// 65536 x 2048 bf16: 104 us, 5.2 TB/s.
template <typename T, typename W, int NT, int C, bool ONCE, bool EVEN>
__global__ __launch_bounds__(kThreads<NT>) void norm_kernel(NormProblem pr, int64_t step) {
    constexpr int V = vec<T>();
    __shared__ float part[2][kRowWaves<NT>][1];
    int64_t r = own_row<NT>();
    if (r >= pr.rows) return;
    const int64_t width = pr.width;
    Chunks<V, C, NT, EVEN> ch;
    ch.init(width);
    const W *weight = (const W *)pr.weight, *bias = (const W *)pr.bias;
    T next[C][V];
    load_chunks<ONCE>(ch, (const T *)pr.x + r * pr.ldx, next);
    for (; r < pr.rows; r += step) {
        T v[C][V];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = next[i][j];
        if (r + step < pr.rows) load_chunks<ONCE>(ch, (const T *)pr.x + (r + step) * pr.ldx, next);
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) sum[0] += ch.counts(i, j) ? (float)v[i][j] : 0.0f;
        row_sums<NT>(sum, part, 0);
        const float mean = sum[0] / (float)width;
        sum[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = (float)v[i][j] - mean;
                sum[0] += ch.counts(i, j) ? d * d : 0.0f;
            }
        row_sums<NT>(sum, part, 1);
        const float rstd = 1.0f / sqrtf(sum[0] / (float)width + pr.eps);
        T *out = (T *)pr.out + r * pr.ldo;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!ch.there(i)) continue;
            W w[V], b[V];
            if (weight) load_vec(weight + ch.at[i], w);
            if (bias) load_vec(bias + ch.at[i], b);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float h = ((float)v[i][j] - mean) * rstd;
                if (weight) h *= (float)w[j];
                if (bias) h += (float)b[j];
                v[i][j] = (T)h;
            }
            store_chunk<ONCE>(out + ch.at[i], v[i]);
        }
        if (threadIdx.x % NT == 0 && pr.mean) {
            pr.mean[r] = mean;
            pr.rstd[r] = rstd;
        }
    }
}

// Rows of any length: a block reads its row three times.
template <typename T, typename W>
__global__ __launch_bounds__(256) void norm_long_kernel(NormProblem pr) {
    constexpr int V = vec<T>();
    __shared__ float part[2][4][1];
    const int64_t r = blockIdx.x, width = pr.width;
    const T *x = (const T *)pr.x + r * pr.ldx;
    const W *weight = (const W *)pr.weight, *bias = (const W *)pr.bias;
    T *out = (T *)pr.out + r * pr.ldo;
    float sum[1] = {0.0f};
    for (int64_t c = threadIdx.x * V; c < width; c += 256 * V) {
        T v[V];
        load_part<false, T, V>(x + c, width - c, v);  // zeros past the end
#pragma unroll
        for (int j = 0; j < V; ++j) sum[0] += (float)v[j];
    }
    row_sums<256>(sum, part, 0);
    const float mean = sum[0] / (float)width;
    sum[0] = 0.0f;
    for (int64_t c = threadIdx.x * V; c < width; c += 256 * V) {
        T v[V];
        load_part<false, T, V>(x + c, width - c, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float d = (float)v[j] - mean;
            sum[0] += c + j < width ? d * d : 0.0f;
        }
    }
    row_sums<256>(sum, part, 1);
    const float rstd = 1.0f / sqrtf(sum[0] / (float)width + pr.eps);
    for (int64_t c = threadIdx.x * V; c < width; c += 256 * V) {
        const int64_t left = width - c;
        T v[V];
        W w[V], b[V];
        load_part<false, T, V>(x + c, left, v);
        if (weight) load_part<false, W, V>(weight + c, left, w);
        if (bias) load_part<false, W, V>(bias + c, left, b);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float h = ((float)v[j] - mean) * rstd;
            if (weight) h *= (float)w[j];
            if (bias) h += (float)b[j];
            v[j] = (T)h;
        }
        store_part<false, T, V>(out + c, left, v);
    }
    if (threadIdx.x == 0 && pr.mean) {
        pr.mean[r] = mean;
        pr.rstd[r] = rstd;
    }
}

// dx, and the columns' sums over the rows that the lanes, the wave or the block take: every
// `step`-th. A block leaves one part of the sums. 65536 x 2048 bf16: 137 us, 5.9 TB/s, and 5 for
// the join.
template <typename T, typename W, int NT, int C, bool ONCE, bool EVEN>
__global__ __launch_bounds__(kThreads<NT>) void norm_backward_kernel(NormProblem pr, int64_t step) {
    constexpr int V = vec<T>();
    __shared__ float part[2][kRowWaves<NT>][2];
    __shared__ float columns[NT <= 64 ? C * 64 * V : 1];
    const int64_t width = pr.width;
    Chunks<V, C, NT, EVEN> ch;
    ch.init(width);
    const W *weight = (const W *)pr.weight;
    W w[C][V];
    float dw[C][V], db[C][V];
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = (W)1.0f;
            dw[i][j] = db[i][j] = 0.0f;
        }
        if (weight && ch.there(i)) load_vec(weight + ch.at[i], w[i]);
    }
    const float each = 1.0f / (float)width;
    int turn = 0;
    int64_t r = own_row<NT>();
    T nv[C][V], nd[C][V];
    float mean_of_next = 0.0f, rstd_of_next = 0.0f;
    auto fetch = [&](int64_t r) {
        load_chunks<ONCE>(ch, (const T *)pr.x + r * pr.ldx, nv);
        load_chunks<ONCE>(ch, (const T *)pr.dy + r * pr.lddy, nd);
        mean_of_next = pr.mean[r];
        rstd_of_next = pr.rstd[r];
    };
    if (r < pr.rows) fetch(r);
    for (; r < pr.rows; r += step, ++turn) {
        T v[C][V], d[C][V];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] = nv[i][j];
                d[i][j] = nd[i][j];
            }
        const float mean = mean_of_next, rstd = rstd_of_next;
        if (r + step < pr.rows) fetch(r + step);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = ((float)v[i][j] - mean) * rstd, y = (float)d[i][j];
                const float g = ch.counts(i, j) ? y * (float)w[i][j] : 0.0f;
                dw[i][j] += y * h;
                db[i][j] += y;
                sum[0] += g;
                sum[1] += g * h;
            }
        if (!pr.out) continue;
        row_sums<NT>(sum, part, turn);
        const float m = sum[0] * each, mh = sum[1] * each;
        T *out = (T *)pr.out + r * pr.ldo;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!ch.there(i)) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = ((float)v[i][j] - mean) * rstd;
                v[i][j] = (T)(rstd * ((float)d[i][j] * (float)w[i][j] - m - h * mh));
            }
            store_chunk<ONCE>(out + ch.at[i], v[i]);
        }
    }
    if (!pr.partial) return;
    float *to = pr.partial + (int64_t)blockIdx.x * 2 * width;
    const bool only = gridDim.x == 1;  // then there is nothing to join
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        auto &own = k == 0 ? dw : db;
        if (NT < 64) {  // the wave's rows
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (NT == 16) own[i][j] += __shfl_xor(own[i][j], 16);
                    own[i][j] += __shfl_xor(own[i][j], 32);
                }
        }
        if (NT <= 64) {  // the four waves' sums, one after another
            for (int q = 0; q < 4; ++q) {
                __syncthreads();
                if ((int)(threadIdx.x >> 6) != q) continue;
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int at = (i * V + j) * 64 + (threadIdx.x & 63);
                        if (q > 0) own[i][j] += columns[at];
                        if (q < 3) columns[at] = own[i][j];
                    }
            }
            if (threadIdx.x < 192 || threadIdx.x >= 192 + NT) continue;
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (ch.there(i)) {
                W *out = (W *)(k == 0 ? pr.dweight : pr.dbias);
                if (!only) {
                    store_vec(to + k * width + ch.at[i], own[i]);
                } else if (out) {
                    W r[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) r[j] = (W)own[i][j];
                    store_vec(out + ch.at[i], r);
                }
            }
    }
}

// dx of rows of any length: a block reads its row twice.
template <typename T, typename W>
__global__ __launch_bounds__(256) void norm_long_dx_kernel(NormProblem pr) {
    constexpr int V = vec<T>();
    __shared__ float part[2][4][2];
    const int64_t r = blockIdx.x, width = pr.width;
    const T *x = (const T *)pr.x + r * pr.ldx, *dy = (const T *)pr.dy + r * pr.lddy;
    const W *weight = (const W *)pr.weight;
    T *out = (T *)pr.out + r * pr.ldo;
    const float mean = pr.mean[r], rstd = pr.rstd[r];
    float sum[2] = {0.0f, 0.0f}, m = 0.0f, mh = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t c = threadIdx.x * V; c < width; c += 256 * V) {
            const int64_t left = width - c;
            T v[V], d[V];
            W w[V];
            load_part<false, T, V>(x + c, left, v);
            load_part<false, T, V>(dy + c, left, d);  // zeros past the end
            if (weight) load_part<false, W, V>(weight + c, left, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = ((float)v[j] - mean) * rstd;
                const float g = weight ? (float)d[j] * (float)w[j] : (float)d[j];
                if (pass == 0) {
                    sum[0] += c + j < width ? g : 0.0f;
                    sum[1] += c + j < width ? g * h : 0.0f;
                } else {
                    v[j] = (T)(rstd * (g - m - h * mh));
                }
            }
            if (pass == 1) store_part<false, T, V>(out + c, left, v);
        }
        if (pass == 0) {
            row_sums<256>(sum, part, 0);
            m = sum[0] / (float)width;
            mh = sum[1] / (float)width;
        }
    }
}

// The columns' sums of long rows: 64 V columns and every `parts`-th row a wave.
template <typename T>
__global__ __launch_bounds__(256) void norm_long_sums_kernel(NormProblem pr, int64_t parts) {
    constexpr int V = vec<T>();
    const int64_t unit = own_token<64>();
    const int64_t col_blocks = (pr.width + 64 * V - 1) / (64 * V);
    const int64_t k = unit / col_blocks;
    const int64_t c = ((unit - k * col_blocks) * 64 + (threadIdx.x & 63)) * V;
    if (k >= parts || c >= pr.width) return;
    const int64_t left = pr.width - c;
    float dw[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
    for (int64_t r = k; r < pr.rows; r += parts) {
        T v[V], d[V];
        load_part<false, T, V>((const T *)pr.x + r * pr.ldx + c, left, v);
        load_part<false, T, V>((const T *)pr.dy + r * pr.lddy + c, left, d);
        const float mean = pr.mean[r], rstd = pr.rstd[r];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            dw[j] += (float)d[j] * (((float)v[j] - mean) * rstd);
            db[j] += (float)d[j];
        }
    }
    float *to = pr.partial + k * 2 * pr.width + c;
    store_part<false, float, V>(to, left, dw);
    store_part<false, float, V>(to + pr.width, left, db);
}

// dweight and dbias: the parts of 64 columns, added by 16 waves that each take a run of them.
template <typename W>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormProblem pr, int64_t parts) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 64 + lane, n = 2 * pr.width;
    const int64_t per = (parts + 15) / 16;
    const int64_t end = (wave + 1) * per < parts ? (wave + 1) * per : parts;
    float v = 0.0f;
    if (i < n) {
#pragma unroll 8
        for (int64_t p = wave * per; p < end; ++p) v += pr.partial[p * n + i];
    }
    sums[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || i >= n) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) v += sums[w][lane];
    W *to = (W *)(i < pr.width ? pr.dweight : pr.dbias);
    if (to) to[i < pr.width ? i : i - pr.width] = (W)v;
}

// How rows are held, in chunks of 16 bytes a thread: by 16 lanes up to two, by 32 up to four (a
// quarter of them idle), by a wave up to four, by two waves up to four where a block of 256 would
// leave more idle, by a block of 256 or 512 up to four; else not (nor are rows shorter than
// one access). The fewer threads, the more rows share a reduction; few rows want more threads.
// bf16, forward and backward, us: 262144 x 64 by a wave 86 and 113, by 16 lanes 24 and 28; 65536 x
// 257 by a wave 31 and 39, by 32 lanes 25 and 31, x 520 47 and 65, 36 and 57, but 16384 x 1001 18
// and 26, 16 and 34; 16384 x 2051 by a block 48 and 73, by two waves 42 and 66 (1100 rows: 7 and
// 16, 6 and 21). float32: 16384 x 4097 not held 147 and 413, by 512 threads 116 and 165.
enum { kLanes, kWave, kPair, kBlock, kWide, kLong };
template <typename T>
int how_held(int64_t rows, int64_t width) {
    const int64_t wave = 64 * vec<T>();
    if (width < vec<T>()) return kLong;
    if (2 * width <= wave || (2 * width <= 3 * wave && rows >= 1024)) return kLanes;
    if (width <= 4 * wave && (rows >= 1024 || width <= wave)) return kWave;
    if (width > 4 * wave && width <= 6 * wave && rows >= 4096) return kPair;
    return width <= 16 * wave ? kBlock : width <= 32 * wave ? kWide : kLong;
}
constexpr int64_t kParts = 512;
constexpr int64_t kBlocks = 1024;

// Rows that are more than the 256 MB of the memory-side cache pass the caches by, where they
// are whole lines of 128 bytes (the rule of the token rows in tokens.hip).
template <typename T>
bool once_of(const NormProblem &pr, int64_t tensors) {
    const int64_t size = sizeof(T);
    return tensors * pr.rows * pr.width * size > 256 << 20 && pr.width * size % 128 == 0 &&
           pr.ldx * size % 128 == 0 && pr.ldo * size % 128 == 0;
}

template <typename T, class F>
hipError_t by_size(int64_t rows, int64_t width, F f) {
    constexpr int V = vec<T>();
    const int how = how_held<T>(rows, width);
    if (how == kLanes) {
        if (width <= 16 * V) return f(ActTag<16>{}, ActTag<1>{});
        if (width <= 32 * V) return f(ActTag<16>{}, ActTag<2>{});
        return width <= 64 * V ? f(ActTag<32>{}, ActTag<2>{}) : f(ActTag<32>{}, ActTag<4>{});
    }
    if (how == kPair) return f(ActTag<128>{}, ActTag<4>{});
    if (how == kWide) return f(ActTag<512>{}, ActTag<4>{});
    if (how == kWave) {
        if (width <= 64 * V) return f(ActTag<64>{}, ActTag<1>{});
        return width <= 128 * V ? f(ActTag<64>{}, ActTag<2>{}) : f(ActTag<64>{}, ActTag<4>{});
    }
    if (width <= 256 * V) return f(ActTag<256>{}, ActTag<1>{});
    if (width <= 512 * V) return f(ActTag<256>{}, ActTag<2>{});
    return f(ActTag<256>{}, ActTag<4>{});
}

template <typename T, typename W>
hipError_t norm_t(const NormProblem &pr, hipStream_t s) {
    if (how_held<T>(pr.rows, pr.width) == kLong)
        return launch(norm_long_kernel<T, W>, pr.rows, 256, 0, s, pr);
    return by_size<T>(pr.rows, pr.width, [&](auto nt, auto c) {
        constexpr int NT = decltype(nt)::value, C = decltype(c)::value;
        // As many blocks as run at once.
        constexpr int kRows = kThreads<NT> / NT;
        const int64_t all = cdiv(pr.rows, kRows), most = NT == 128 ? 2 * kBlocks : kBlocks;
        const int64_t blocks = all < most ? all : most;
        const auto kernel = pr.width % vec<T>()  ? norm_kernel<T, W, NT, C, false, false>
                            : once_of<T>(pr, 2) ? norm_kernel<T, W, NT, C, true, true>
                                                : norm_kernel<T, W, NT, C, false, true>;
        return launch(kernel, blocks, kThreads<NT>, 0, s, pr, blocks * kRows);
    });
}

template <typename T, typename W>
hipError_t backward_t(NormProblem pr, int64_t parts, hipStream_t s) {
    const bool sums = pr.dweight || pr.dbias;
    if (!sums) pr.partial = nullptr;
    hipError_t e = hipSuccess;
    if (how_held<T>(pr.rows, pr.width) == kLong) {
        if (pr.out && pr.rows) e = launch(norm_long_dx_kernel<T, W>, pr.rows, 256, 0, s, pr);
        if (e == hipSuccess && sums)
            e = launch(norm_long_sums_kernel<T>, cdiv(parts * cdiv(pr.width, 64 * vec<T>()), 4), 256, 0, s,
                       pr, parts);
    } else {
        e = by_size<T>(pr.rows, pr.width, [&](auto nt, auto c) {
            constexpr int NT = decltype(nt)::value, C = decltype(c)::value;
            const auto kernel = pr.width % vec<T>()  ? norm_backward_kernel<T, W, NT, C, false, false>
                                : once_of<T>(pr, 3) ? norm_backward_kernel<T, W, NT, C, true, true>
                                                    : norm_backward_kernel<T, W, NT, C, false, true>;
            return launch(kernel, parts, kThreads<NT>, 0, s, pr, parts * (kThreads<NT> / NT));
        });
    }
    if (e != hipSuccess || !sums || (parts == 1 && how_held<T>(pr.rows, pr.width) != kLong)) return e;
    return launch(norm_join_kernel<W>, cdiv(2 * pr.width, 64), 1024, 0, s, pr, parts);
}

template <typename T>
int64_t parts_of(int64_t rows, int64_t width) {
    const int how = how_held<T>(rows, width);
    // A few rows in one block save the launch that joins the parts: 12 x 56 bf16 4.8 us against
    // 3.8 + 2.0; but 64 x 512 13.7 against 4.0 + 3.7.
    const int64_t most = how == kLong || how == kLanes ? cdiv(rows, width <= 32 * vec<T>() ? 16 : 8)
                         : how == kWave                ? cdiv(rows, rows <= 16 ? 16 : 4)
                                                       : rows;
    const int64_t parts = how == kLong ? 64 : how == kPair ? 2 * kParts : kParts;
    return most < 1 ? 1 : most < parts ? most : parts;
}

}  // namespace

int64_t norm_parts(int dtype, int64_t rows, int64_t width) {
    return dtype == 0 ? parts_of<float>(rows, width) : parts_of<bf16>(rows, width);
}
bool norm_grid_ok(int, int64_t rows, int64_t) { return rows < 1 << 24; }  // a block of 256 each

#define KX_NORM(call)                                                                         \
    if (dtype == 0) return call(float, float);                                                \
    if (dtype == 1) return weights_dtype == 0 ? call(bf16, float) : call(bf16, bf16);         \
    return weights_dtype == 0 ? call(f16, float) : call(f16, f16)

hipError_t launch_norm(int dtype, int weights_dtype, const NormProblem &pr, hipStream_t s) {
    if (pr.rows == 0) return hipSuccess;
#define KX_CALL(T, W) norm_t<T, W>(pr, s)
    KX_NORM(KX_CALL);
#undef KX_CALL
}

hipError_t launch_norm_backward(int dtype, int weights_dtype, const NormProblem &pr, hipStream_t s) {
    const int64_t parts = norm_parts(dtype, pr.rows, pr.width);
#define KX_CALL(T, W) backward_t<T, W>(pr, parts, s)
    KX_NORM(KX_CALL);
#undef KX_CALL
}

}  // namespace kx
