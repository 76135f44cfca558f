// linear.h - the tiled matrix-product kernels of the experts' layers,
// instantiated per type by linear_f32.hip, linear_bf16.hip, linear_f16.hip.
//
// One kernel computes D[m][n] = sum_k Q[m][k] P[n][k] over BM x BN tiles, each
// operand read in one of two layouts:
//   by depth  (KC)  rows of the output dimension, k contiguous (x and w of the
//                   forward product, dz of dx)
//   by column (MC)  rows of k, the output dimension contiguous (w of dx; x and
//                   dz of dw)
// so no operand is ever transposed in memory. A stage is 128 bytes of k per
// output row or column (64 16-bit values, 32 floats), moved from global memory
// straight into LDS (buffer_load ... lds); whatever lies outside an operand is
// dropped by the buffer's range check and reads as zero.
//
// The matrix instruction's row operand is P and its column operand Q: a lane
// then holds four consecutive output columns of one output row, so bias,
// activation, residual and stores are vectors along the row.
//
// LDS layouts (64 banks of 4 bytes; 16-byte chunks):
//   KC  rows of 128 bytes, chunk c of row r at c ^ ((r / 2) % 8): the 16 rows of
//       a fragment read at one chunk fall in 16 different 16-byte bank groups.
//   MC  rows of R values. 16 bits: granules of 32 bytes (16 values), granule g
//       of row k at g ^ ((k % 4) + 4 (k / 8 % 2)): the transposing read
//       (ds_read_b64_tr_b16: 16 lanes take 4 rows of 16 values and return each
//       lane 4 values of one column) touches rows 8 a + b, b < 4, together.
//       float: granules of 64 bytes at g ^ (k / 4 % 4), read 4 bytes a lane.
#pragma once

#include "experts.h"

namespace kx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kRow = 128;                // bytes of k per stage
constexpr uint32_t kNowhere = 1u << 31;  // an offset past every buffer (records < 2^31)

template <typename T>
struct Frag;  // 16 bytes of k per lane
template <>
struct Frag<bf16> {
    typedef bf16x8 type;
    static __device__ __forceinline__ f32x4 mma(bf16x8 p, bf16x8 q, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
    }
};
template <>
struct Frag<f16> {
    typedef f16x8 type;
    static __device__ __forceinline__ f32x4 mma(f16x8 p, f16x8 q, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, c, 0, 0, 0);
    }
};
template <>
struct Frag<float> {
    typedef f32x4 type;
    // Lane group g holds k = 4 g .. 4 g + 3 of both operands; instruction j
    // takes element j of each lane, so its four k are j, 4 + j, 8 + j, 12 + j.
    static __device__ __forceinline__ f32x4 mma(f32x4 p, f32x4 q, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], c, 0, 0, 0);
        return c;
    }
};

// One operand's stage: R output rows (or columns) x 128 bytes of k, moved by
// NW waves with DW bytes (16 or 4) a lane and instruction.
template <typename T, bool MC, int R, int NW, int DW>
struct Tile {
    static constexpr int kSize = (int)sizeof(T);
    static constexpr int kBytes = R * kRow;
    static constexpr int kDepth = kRow / kSize;  // k per stage
    static constexpr int kIssues = kBytes / (64 * DW * NW);
    static_assert(kIssues >= 1 && kIssues * 64 * DW * NW == kBytes, "tile and waves");

    uint32_t off[kIssues];
    const char *base;
    uint32_t ld;      // bytes
    uint32_t extent;  // KC: valid rows; MC: valid bytes of a row
    int64_t depth;

    static __device__ __forceinline__ int swizzle(int k) {  // MC, in 16-byte chunks
        if (kSize == 2) return (((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1)) << 1;
        return ((k >> 2) & 3) << 2;
    }
    // Byte q of the stage in LDS: its byte of the row in memory (KC).
    static __device__ __forceinline__ int kc_byte(int q) {
        return ((((q & (kRow - 1)) >> 4) ^ ((q >> 8) & 7)) << 4) | (q & 15);
    }
    static __device__ __forceinline__ int lds_byte(int wave, int lane, int i) {
        return ((wave * kIssues + i) * 64 + lane) * DW;
    }

    // p: the tile's first row (KC) or column (MC) at k = 0; valid: rows or columns.
    __device__ __forceinline__ void init(const char *p, int64_t ld_elems, int64_t valid,
                                         int64_t depth_, int wave, int lane) {
        base = p;
        ld = (uint32_t)(ld_elems * kSize);
        depth = depth_;
        const uint32_t n = (uint32_t)(valid < 0 ? 0 : valid > R ? R : valid);
        extent = __builtin_amdgcn_readfirstlane(MC ? n * kSize : n);
#pragma unroll
        for (int i = 0; i < kIssues; ++i) {
            const int q = lds_byte(wave, lane, i);
            if (MC) {
                constexpr int kRowBytes = R * kSize;
                const int k = q / kRowBytes, c = q % kRowBytes;
                const uint32_t src = (((c >> 4) ^ swizzle(k)) << 4) | (c & 15);
                off[i] = src < extent ? k * ld + src : kNowhere;
            } else {
                off[i] = (q >> 7) * ld + kc_byte(q);
            }
        }
    }

    __device__ __forceinline__ void issue(char *lds, int stage, int wave, int lane) const {
        const char *at;
        int64_t records;
        uint32_t left = kRow;  // KC: bytes of k from this stage on
        if (MC) {
            const int64_t k = depth - (int64_t)stage * kDepth;
            const int64_t rows = k < kDepth ? k : kDepth;
            at = base + (int64_t)stage * kDepth * ld;
            records = (rows - 1) * ld + extent;
            if (extent == 0) records = 0;
        } else {
            // 16-bit rows are padded with zeros to whole 16 bytes; the range check
            // drops a 4-byte word that the records end inside of.
            const int64_t all = kSize == 2 ? (depth + 7) / 8 * 16 : depth * kSize;
            const int64_t bytes = all - (int64_t)stage * kRow;
            at = base + (int64_t)stage * kRow;
            records = extent ? (int64_t)(extent - 1) * ld + bytes : 0;
            left = bytes < kRow ? (uint32_t)bytes : kRow;
        }
        const uint64_t a = (uint64_t)at;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
        const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
        const uint32_t rec = __builtin_amdgcn_readfirstlane((uint32_t)records);
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(((uint64_t)hi << 32) | lo), 0, (int)rec, 0x00020000);
#pragma unroll
        for (int i = 0; i < kIssues; ++i) {
            uint32_t o = off[i];
            if (!MC && left < kRow && (uint32_t)kc_byte(lds_byte(wave, lane, i)) >= left)
                o = kNowhere;
            lds_void *to = (lds_void *)(lds + (wave * kIssues + i) * 64 * DW);
            if constexpr (DW == 16)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16, (int)o, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, (int)o, 0, 0, 0);
        }
    }
};

// Fragment reads of one operand: `first` = the wave's first output row/column.
template <typename T, bool MC, int R, int N>
struct Reader {
    typedef typename Frag<T>::type frag;
    int at[N];

    __device__ __forceinline__ void init(int first, int lane) {
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < N; ++t) {
            if (!MC) {
                at[t] = (first + 16 * t + i) * kRow + ((g ^ (i >> 1)) << 4);
            } else if (sizeof(T) == 2) {
                const int k = 8 * g + (i >> 2);
                const int key = ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
                at[t] = k * (R * 2) + (((first / 16 + t) ^ key) << 5) + (i & 3) * 8;
            } else {
                at[t] = 4 * g * (R * 4) + (((first / 16 + t) ^ g) << 6) + i * 4;
            }
        }
    }
    // Half `s` of the stage (64 of its 128 bytes of k), block t.
    __device__ __forceinline__ frag read(const char *lds, int t, int s) const {
        if (!MC) return *reinterpret_cast<const frag *>(lds + (at[t] ^ (s << 6)));
        if constexpr (sizeof(T) == 2) {
            const char *p = lds + at[t] + s * 32 * (R * 2);
            union {
                s16x4 h[2];
                frag f;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (R * 2)));
            return u.f;
        } else {
            frag f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = *reinterpret_cast<const float *>(lds + at[t] + (s * 16 + j) * (R * 4));
            return f;
        }
    }
};

template <typename T, bool PMC, bool QMC, int BM_, int BN_, int WM_, int WN_, int DW_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, DW = DW_;
    static constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr int kStage = (BM + BN) * kRow;
    typedef T type;
    typedef Tile<T, PMC, BN, NW, DW> TileP;
    typedef Tile<T, QMC, BM, NW, DW> TileQ;
    typedef Reader<T, PMC, BN, TN> ReadP;
    typedef Reader<T, QMC, BM, TM> ReadQ;
    static constexpr bool p_mc = PMC;
};

// acc[tm][tn] += the tile's product over the whole depth. Two stages in LDS:
// the next one is in flight while this one is multiplied.
template <class S>
__device__ __forceinline__ void product(char *smem, typename S::TileP &tp, typename S::TileQ &tq,
                                        int64_t depth, int wave, int lane,
                                        f32x4 (&acc)[S::TM][S::TN]) {
    typedef typename S::type T;
    typedef typename Frag<T>::type frag;
    typename S::ReadP rp;
    typename S::ReadQ rq;
    rp.init((wave % S::WN) * (S::BN / S::WN), lane);
    rq.init((wave / S::WN) * (S::BM / S::WM), lane);
    const int stages = (int)((depth + S::TileP::kDepth - 1) / S::TileP::kDepth);
    if (stages == 0) return;
    tp.issue(smem, 0, wave, lane);
    tq.issue(smem + S::BN * kRow, 0, wave, lane);
    for (int it = 0; it < stages; ++it) {
        char *cur = smem + (it & 1) * S::kStage;
        char *nxt = smem + ((it & 1) ^ 1) * S::kStage;
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();  // this stage has landed; every wave is done with the one before
        if (it + 1 < stages) {
            tp.issue(nxt, it + 1, wave, lane);
            tq.issue(nxt + S::BN * kRow, it + 1, wave, lane);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            frag p[S::TN], q[S::TM];
#pragma unroll
            for (int t = 0; t < S::TN; ++t) p[t] = rp.read(cur, t, s);
#pragma unroll
            for (int t = 0; t < S::TM; ++t) q[t] = rq.read(cur + S::BN * kRow, t, s);
#pragma unroll
            for (int m = 0; m < S::TM; ++m)
#pragma unroll
                for (int n = 0; n < S::TN; ++n) acc[m][n] = Frag<T>::mma(p[n], q[m], acc[m][n]);
        }
    }
}

// Block b of a grid of `total` tiles: XCD b % 8 takes a contiguous range of
// them, so that tiles which share operands share an L2. -1: no tile.
__device__ __forceinline__ int64_t xcd_tile(int64_t total) {
    const int64_t per = (total + 7) / 8;
    const int64_t b = blockIdx.x;
    const int64_t id = (b & 7) * per + (b >> 3);
    return (b >> 3) < per && id < total ? id : -1;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
    return v < lo ? lo : v > hi ? hi : v;
}

struct Group {
    int expert, lo, hi, tile;  // rows [lo, hi), tile within them
};

// The experts' rows in tiles of bm rows, one after another, then the rows past
// the last expert (expert == experts). mt < 0: returns the number of tiles in
// .tile. Offsets are clamped into the matrix, so whatever they hold no access
// leaves it.
__device__ __forceinline__ Group find_group(const int *offsets, int experts, int rows, int bm,
                                            int mt) {
    const int lane = threadIdx.x & 63;
    Group r = {-1, 0, 0, 0};
    int before = 0;
    for (int e0 = 0; e0 <= experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e <= experts) {
            lo = clampi(offsets[e], 0, rows);
            hi = e < experts ? clampi(offsets[e + 1], lo, rows) : rows;
        }
        const int n = (hi - lo + bm - 1) / bm;
        const int incl = before + wave_incl_scan(n);
        if (mt >= 0) {
            const unsigned long long past = __ballot(incl > mt);
            if (past) {
                const int l = __builtin_ctzll(past);
                r.expert = e0 + l;
                r.lo = __builtin_amdgcn_readlane(lo, l);
                r.hi = __builtin_amdgcn_readlane(hi, l);
                r.tile = mt - __builtin_amdgcn_readlane(incl - n, l);
                return r;
            }
        }
        before = __builtin_amdgcn_readlane(incl, 63);
    }
    r.tile = before;
    return r;
}

// Four values of one row; `full`: all inside it and on a vector boundary.
template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p, int valid, bool full) {
    f32x4 r = {0, 0, 0, 0};
    if (full) {
        typedef T v4 __attribute__((ext_vector_type(4)));
        const v4 x = *reinterpret_cast<const v4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = (float)x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) r[i] = (float)p[i];
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store4(T *p, f32x4 v, int valid, bool full) {
    if (full) {
        typedef T v4 __attribute__((ext_vector_type(4)));
        v4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (T)v[i];
        *reinterpret_cast<v4 *>(p) = x;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) p[i] = (T)v[i];
    }
}

template <typename T>
struct RowsArgs {
    RowsProblem pr;
    bool vec;  // rows of out, pre, residual, in_pre and bias are whole 4-value vectors
    int gm;    // row tiles walked per column tile, so that a group's operands stay in L2
};

// Tile (mt, nt) of the walk's place id: groups of gm row tiles, row first.
__device__ __forceinline__ void walk(int64_t id, int tiles_m, int tiles_n, int gm, int &mt, int &nt) {
    const int64_t per = (int64_t)gm * tiles_n;
    const int64_t panel = id / per;
    const int first = (int)(panel * gm);
    const int height = tiles_m - first < gm ? tiles_m - first : gm;
    const int64_t in = id - panel * per;
    mt = first + (int)(in % height);
    nt = (int)(in / height);
}

template <class S>
__global__ __launch_bounds__(S::NW * 64, 1) void rows_kernel(RowsArgs<typename S::type> a) {
    typedef typename S::type T;
    __shared__ __align__(1024) char smem[2 * S::kStage];
    const RowsProblem &pr = a.pr;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)pr.rows, cols = (int)pr.cols;
    const int tiles_n = (cols + S::BN - 1) / S::BN;
    int tiles_m;
    if (pr.offsets)
        tiles_m = find_group(pr.offsets, pr.experts, rows, S::BM, -1).tile;
    else
        tiles_m = (rows + S::BM - 1) / S::BM;
    const int64_t id = xcd_tile((int64_t)tiles_m * tiles_n);
    if (id < 0) return;
    int mt, nt;
    walk(id, tiles_m, tiles_n, a.gm, mt, nt);
    Group gr = {0, 0, rows, mt};
    if (pr.offsets) gr = find_group(pr.offsets, pr.experts, rows, S::BM, mt);
    if (gr.expert < 0) return;
    const int m0 = gr.lo + gr.tile * S::BM, n0 = nt * S::BN;
    const bool tail = gr.expert == pr.experts;
    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    if (!tail) {
        const char *q = (const char *)pr.q + (int64_t)m0 * pr.ldq * sizeof(T);
        const char *p = (const char *)pr.p + (int64_t)gr.expert * pr.p_expert * sizeof(T);
        p += (S::p_mc ? (int64_t)n0 : (int64_t)n0 * pr.ldp) * sizeof(T);
        typename S::TileP tp;
        typename S::TileQ tq;
        tp.init(p, pr.ldp, S::p_mc ? pr.p_cols - n0 : (int64_t)cols - n0, pr.depth, wave, lane);
        tq.init(q, pr.ldq, gr.hi - m0, pr.depth, wave, lane);
        product<S>(smem, tp, tq, pr.depth, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM) + (lane & 15);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN) + (lane >> 4) * 4;
    T *out = (T *)pr.out, *pre = (T *)pr.pre;
    const T *bias = (const T *)pr.bias, *res = (const T *)pr.residual, *in = (const T *)pr.in_pre;
#pragma unroll
    for (int tn = 0; tn < S::TN; ++tn) {
        const int n = wn + tn * 16;
        const int valid = cols - n;
        if (valid <= 0) continue;
        const bool full = a.vec && valid >= 4;
        f32x4 b = {0, 0, 0, 0};
        if (bias && !tail) b = load4(bias + (int64_t)gr.expert * cols + n, valid, full);
#pragma unroll
        for (int tm = 0; tm < S::TM; ++tm) {
            const int64_t m = wm + tm * 16;
            if (m >= gr.hi) continue;
            f32x4 z = acc[tm][tn] + b;
            if (tail) z = f32x4{0, 0, 0, 0};
            if (pre) store4(pre + m * pr.ldpre + n, z, valid, full);
            if (pr.act != kActNone) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = act_value(z[i], pr.act);
            }
            if (!tail) {
                if (res) z += load4(res + m * pr.ldr + n, valid, full);
                if (in) {
                    const f32x4 y = load4(in + m * pr.ldin + n, valid, full);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] *= act_slope(y[i], pr.in_act);
                }
            }
            store4(out + m * pr.ldo + n, z, valid, full);
        }
    }
}

struct GradArgs {
    GradProblem pr;
    bool vec;
};

template <class S>
__global__ __launch_bounds__(S::NW * 64, 1) void grad_kernel(GradArgs a) {
    typedef typename S::type T;
    __shared__ __align__(1024) char smem[2 * S::kStage];
    const GradProblem &pr = a.pr;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mc = (int)pr.m_cols, nc = (int)pr.n_cols, rows = (int)pr.rows;
    const int tiles_m = (mc + S::BM - 1) / S::BM, tiles_n = (nc + S::BN - 1) / S::BN;
    const int64_t each = (int64_t)tiles_m * tiles_n;
    const int64_t id = xcd_tile(each * pr.experts);
    if (id < 0) return;
    const int e = (int)(id / each);
    int mt, nt;
    walk(id - e * each, tiles_m, tiles_n, 4, mt, nt);
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    int lo = 0, hi = rows;
    if (pr.offsets) {
        lo = clampi(pr.offsets[e], 0, rows);
        hi = clampi(pr.offsets[e + 1], lo, rows);
    }
    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    typename S::TileP tp;
    typename S::TileQ tq;
    tp.init((const char *)pr.x + ((int64_t)lo * pr.ldx + n0) * sizeof(T), pr.ldx, pr.x_cols - n0,
            hi - lo, wave, lane);
    tq.init((const char *)pr.dz + ((int64_t)lo * pr.lddz + m0) * sizeof(T), pr.lddz,
            pr.dz_cols - m0, hi - lo, wave, lane);
    product<S>(smem, tp, tq, hi - lo, wave, lane, acc);
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM) + (lane & 15);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN) + (lane >> 4) * 4;
    T *out = (T *)pr.out + (int64_t)e * mc * nc;
#pragma unroll
    for (int tn = 0; tn < S::TN; ++tn) {
        const int n = wn + tn * 16;
        const int valid = nc - n;
        if (valid <= 0) continue;
#pragma unroll
        for (int tm = 0; tm < S::TM; ++tm) {
            const int64_t m = wm + tm * 16;
            if (m < mc) store4(out + m * nc + n, acc[tm][tn], valid, a.vec && valid >= 4);
        }
    }
}

inline bool on_vector(const void *p, int64_t ld, int size) {
    return p == nullptr || ((uintptr_t)p % (4 * size) == 0 && ld % 4 == 0);
}
inline bool on_chunk(const void *p, int64_t ld, int64_t len, int size) {
    return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0 && len * size % 16 == 0;
}

// Row tiles of all experts at most: each may end in a partial tile.
inline int64_t most_row_tiles(int64_t rows, int bm, const void *offsets, int experts) {
    return offsets ? rows / bm + experts + 1 : cdiv(rows, bm);
}

template <class S>
hipError_t run_rows(const RowsProblem &pr, hipStream_t s) {
    constexpr int size = (int)sizeof(typename S::type);
    RowsArgs<typename S::type> a;
    a.pr = pr;
    a.vec = on_vector(pr.out, pr.ldo, size) && on_vector(pr.pre, pr.ldpre, size) &&
            on_vector(pr.residual, pr.ldr, size) && on_vector(pr.in_pre, pr.ldin, size) &&
            on_vector(pr.bias, pr.cols, size);
    a.gm = 8;
    const int64_t tiles = most_row_tiles(pr.rows, S::BM, pr.offsets, pr.experts) * cdiv(pr.cols, S::BN);
    rows_kernel<S><<<(unsigned)(cdiv(tiles, 8) * 8), S::NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

template <class S>
hipError_t run_grad(const GradProblem &pr, hipStream_t s) {
    constexpr int size = (int)sizeof(typename S::type);
    GradArgs a;
    a.pr = pr;
    a.vec = on_vector(pr.out, pr.n_cols, size);
    const int64_t tiles = cdiv(pr.m_cols, S::BM) * cdiv(pr.n_cols, S::BN) * pr.experts;
    grad_kernel<S><<<(unsigned)(cdiv(tiles, 8) * 8), S::NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

// Tiles that one launch computes with tiles of bm x bn.
inline int64_t rows_tiles(const RowsProblem &pr, int bm, int bn) {
    return (cdiv(pr.rows, bm) + (pr.offsets ? pr.experts / 2 : 0)) * cdiv(pr.cols, bn);
}

template <typename T, bool PMC, int DW>
hipError_t pick_rows(const RowsProblem &pr, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (rows_tiles(pr, 256, 256) >= 192)
            return run_rows<Shape<T, PMC, false, 256, 256, 2, 4, DW>>(pr, s);
    }
    if (rows_tiles(pr, 128, 128) >= 192)
        return run_rows<Shape<T, PMC, false, 128, 128, 2, 2, DW>>(pr, s);
    return run_rows<Shape<T, PMC, false, 64, 64, 2, 2, DW>>(pr, s);
}

template <typename T, int DW>
hipError_t pick_grad(const GradProblem &pr, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (cdiv(pr.m_cols, 256) * cdiv(pr.n_cols, 256) * pr.experts >= 192)
            return run_grad<Shape<T, true, true, 256, 256, 2, 4, DW>>(pr, s);
    }
    if (cdiv(pr.m_cols, 128) * cdiv(pr.n_cols, 128) * pr.experts >= 192)
        return run_grad<Shape<T, true, true, 128, 128, 2, 2, DW>>(pr, s);
    return run_grad<Shape<T, true, true, 64, 64, 2, 2, DW>>(pr, s);
}

}  // namespace

template <typename T>
hipError_t launch_rows_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_grad_t(const GradProblem &pr, hipStream_t s);

}  // namespace kx
