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
    int kc[2];        // KC: byte of k that this lane moves, by the parity of the issue
    uint64_t at;      // this stage's first row or column (the rest is wave-uniform too)
    int ld, left;     // bytes of a row; KC: bytes, MC: rows of k from this stage on
    int extent;       // KC: bytes before the last valid row (< 0: no row); MC: valid bytes of a row

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
    __device__ __forceinline__ void init(const char *p, int64_t ld_elems, int64_t valid, int depth,
                                         int wave, int lane) {
        const uint64_t a = (uint64_t)p;
        at = ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) << 32) |
             (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
        ld = __builtin_amdgcn_readfirstlane((int)(ld_elems * kSize));
        const int n = (int)(valid < 0 ? 0 : valid > R ? R : valid);
        // 16-bit rows are padded with zeros to whole 16 bytes; the range check
        // drops a 4-byte word that the records end inside of.
        left = __builtin_amdgcn_readfirstlane(
            MC ? depth : kSize == 2 ? (depth + 7) / 8 * 16 : depth * kSize);
        extent = __builtin_amdgcn_readfirstlane(MC ? n * kSize : n ? (n - 1) * ld : -(1 << 30));
#pragma unroll
        for (int i = 0; i < kIssues; ++i) {
            const int q = lds_byte(wave, lane, i);
            if (MC) {
                constexpr int kRowBytes = R * kSize;
                const int k = q / kRowBytes, c = q % kRowBytes;
                const int src = (((c >> 4) ^ swizzle(k)) << 4) | (c & 15);
                off[i] = src < extent ? (uint32_t)(k * ld + src) : kNowhere;
            } else {
                off[i] = (q >> 7) * ld + kc_byte(q);
            }
        }
        kc[0] = kc_byte(lds_byte(wave, lane, 0));
        kc[1] = kc_byte(lds_byte(wave, lane, kIssues > 1 ? 1 : 0));
    }

    // Moves this stage into LDS and steps to the next. Past the last stage
    // every lane is out of range, and zeros arrive.
    __device__ __forceinline__ void issue(lds_char *lds, int wave, int lane) {
        int records = 0;
        if (MC) {
            const int rows = left < kDepth ? left : kDepth;
            if (left > 0 && extent > 0) records = (rows - 1) * ld + extent;
        } else {
            if (left > 0) records = extent + left;
            if (records < 0) records = 0;
        }
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc((void *)at, 0, records, 0x00020000);
#pragma unroll
        for (int i = 0; i < kIssues; ++i) {
            uint32_t o = off[i];
            if (!MC) {
                // With 16 bytes a lane an issue covers 8 rows, so its bytes of k
                // depend on the parity of the issue alone; with 4, on i % 4.
                const int k = DW == 16 ? kc[i & 1] : kc_byte(lds_byte(wave, lane, i));
                o = k < left ? o : kNowhere;
            }
            lds_char *to = lds + (wave * kIssues + i) * 64 * DW;
            if constexpr (DW == 16)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)to, 16, (int)o, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)to, 4, (int)o, 0, 0, 0);
        }
        at += MC ? (uint64_t)ld * kDepth : (uint64_t)kRow;
        left -= MC ? kDepth : kRow;
    }
};

// Fragment reads of one operand: `first` = the wave's first output row/column.
template <typename T, bool MC, int R, int N>
struct Reader {
    typedef typename Frag<T>::type frag;
    typedef __attribute__((address_space(3))) const frag lds_frag;
    typedef __attribute__((address_space(3))) const float lds_float;
    int at[MC ? N : 2];  // MC: by block; KC: by half of the stage

    __device__ __forceinline__ void init(int first, int lane) {
        const int i = lane & 15, g = lane >> 4;
        if (!MC) {
#pragma unroll
            for (int s = 0; s < 2; ++s) at[s] = (first + i) * kRow + (((4 * s + g) ^ (i >> 1)) << 4);
        } else {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                if (sizeof(T) == 2) {
                    const int k = 8 * g + (i >> 2);
                    const int key = ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
                    at[t] = k * (R * 2) + (((first / 16 + t) ^ key) << 5) + (i & 3) * 8;
                } else {
                    at[t] = 4 * g * (R * 4) + (((first / 16 + t) ^ g) << 6) + i * 4;
                }
            }
        }
    }
    // Half `s` of the stage (64 of its 128 bytes of k), block t.
    __device__ __forceinline__ frag read(const lds_char *lds, int t, int s) const {
        if constexpr (!MC) {
            return *(lds_frag *)(lds + at[s] + t * 16 * kRow);
        } else if constexpr (sizeof(T) == 2) {
            const lds_char *p = lds + at[t] + s * 32 * (R * 2);
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
            for (int j = 0; j < 4; ++j) f[j] = *(lds_float *)(lds + at[t] + (s * 16 + j) * (R * 4));
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
    static constexpr bool p_mc = PMC, q_mc = QMC;
};

template <class S>
struct Frags {
    typename Frag<typename S::type>::type p[S::TN], q[S::TM];
};

template <class S>
__device__ __forceinline__ void read_half(const typename S::ReadP &rp, const typename S::ReadQ &rq,
                                          const lds_char *stage, int s, Frags<S> &f) {
#pragma unroll
    for (int t = 0; t < S::TN; ++t) f.p[t] = rp.read(stage, t, s);
#pragma unroll
    for (int t = 0; t < S::TM; ++t) f.q[t] = rq.read(stage + S::BN * kRow, t, s);
}
template <class S>
__device__ __forceinline__ void multiply(const Frags<S> &f, f32x4 (&acc)[S::TM][S::TN]) {
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n)
            acc[m][n] = Frag<typename S::type>::mma(f.p[n], f.q[m], acc[m][n]);
}

// The order of one half-stage: its LDS reads (for the half after it) and
// `moves` global-to-LDS loads spread evenly over its matrix instructions.
template <class S>
__device__ __forceinline__ void spread(bool moves) {
    constexpr int kMma = S::TM * S::TN * (sizeof(typename S::type) == 4 ? 4 : 1);
    constexpr int kReadsP = S::TN * (S::p_mc ? (sizeof(typename S::type) == 4 ? 4 : 2) : 1);
    constexpr int kReadsQ = S::TM * (S::q_mc ? (sizeof(typename S::type) == 4 ? 4 : 2) : 1);
    constexpr int kReads = kReadsP + kReadsQ;
    constexpr int kMoves = S::TileP::kIssues + S::TileQ::kIssues;
    constexpr int kSteps = kMma / 2;  // two matrix instructions a step
    int reads = 0, moved = 0;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        // The reads in the first three quarters, so that they have returned by the end.
        const int r = (j + 1) * kReads * 4 / (kSteps * 3) < kReads ? (j + 1) * kReads * 4 / (kSteps * 3) : kReads;
        for (; reads < r; ++reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (moves) {
            const int m = (j + 1) * kMoves / kSteps;
            for (; moved < m; ++moved) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    }
}

// acc[tm][tn] += the tile's product over the whole depth. Two stages in LDS and
// two half-stages of fragments in registers: while one half is multiplied, the
// next is read, and in the second half of a stage, whose buffer every wave has
// read by then, the stage after the next moves in.
template <class S>
__device__ __forceinline__ void product(lds_char *smem, typename S::TileP &tp,
                                        typename S::TileQ &tq, int depth, int wave, int lane,
                                        f32x4 (&acc)[S::TM][S::TN]) {
    typename S::ReadP rp;
    typename S::ReadQ rq;
    rp.init((wave % S::WN) * (S::BN / S::WN), lane);
    rq.init((wave / S::WN) * (S::BM / S::WM), lane);
    const int stages = __builtin_amdgcn_readfirstlane((depth + S::TileP::kDepth - 1) / S::TileP::kDepth);
    if (stages == 0) return;
    tp.issue(smem, wave, lane);
    tq.issue(smem + S::BN * kRow, wave, lane);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    tp.issue(smem + S::kStage, wave, lane);
    tq.issue(smem + S::kStage + S::BN * kRow, wave, lane);
    Frags<S> f[2];
    read_half<S>(rp, rq, smem, 0, f[0]);
    for (int it = 0; it < stages; ++it) {
        lds_char *cur = smem + (it & 1) * S::kStage;
        lds_char *nxt = smem + ((it & 1) ^ 1) * S::kStage;
        read_half<S>(rp, rq, cur, 1, f[1]);
        multiply<S>(f[0], acc);
        spread<S>(false);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();  // the next stage has landed, and this one is in registers
        read_half<S>(rp, rq, nxt, 0, f[0]);
        tp.issue(cur, wave, lane);
        tq.issue(cur + S::BN * kRow, wave, lane);
        multiply<S>(f[1], acc);
        spread<S>(true);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // the stages' memory is free
}

// Block b of a grid of `total` tiles: XCD b % 8 takes pieces of `piece`
// consecutive tiles, so that tiles which share operands share an L2; piece 0: one
// piece, an eighth of the tiles. -1: no tile. (total, piece < 2^31)
__device__ __forceinline__ int xcd_tile(int total, int piece) {
    const int b = blockIdx.x, x = b & 7, j = b >> 3;
    const int per = (total + 7) / 8;
    const int id = piece ? ((j / piece) * 8 + x) * piece + j % piece : j < per ? x * per + j : total;
    return id < total ? id : -1;
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

// Eight values of one row, `valid` of them inside it, at any alignment.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int valid, float (&r)[8]) {
    if (valid >= 8) {
        T x[8];
        load_vec(p, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (float)x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = i < valid ? (float)p[i] : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8], int valid) {
    T x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
    if (valid >= 8) {
        store_vec(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = x[i];
    }
}

// Hands the wave's tile to `use(row, col, values, aux)`, eight consecutive
// columns at a time: 16 rows at a time go through LDS (each wave's own part of the
// stages' memory), so that a wave's accesses to memory are whole rows of the tile,
// 16 bytes a lane, where the matrix instruction leaves a lane four columns of one
// row. `load(row, col)` gives the aux of a place; it is asked for two groups of rows
// ahead (the fragments' registers are free by then), or its latency would be paid
// again for every group.
template <class S, class Aux, class L, class F>
__device__ __forceinline__ void by_rows(lds_char *smem, int wave, int lane,
                                        const f32x4 (&acc)[S::TM][S::TN], L load, F use) {
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    constexpr int kCols = S::TN * 16, kLd = (kCols + 4) * 4;
    constexpr int kLanes = kCols / 8;   // lanes to a row
    constexpr int kRows = 64 / kLanes;  // rows at a time
    constexpr int kParts = 16 / kRows;
    constexpr int kAhead = 2;           // blocks of 16 rows in LDS at a time
    static_assert(kAhead * 16 * kLd * S::NW <= 2 * S::kStage, "the stages' memory");
    lds_char *own = smem + wave * kAhead * 16 * kLd;
    const int row = lane / kLanes, col = lane % kLanes * 8;
    Aux aux[S::TM][kParts];
#pragma unroll
    for (int tm = 0; tm < 2 * kAhead && tm < S::TM; ++tm)
#pragma unroll
        for (int r = 0; r < kParts; ++r) aux[tm][r] = load(tm * 16 + r * kRows + row, col);
#pragma unroll
    for (int t0 = 0; t0 < S::TM; t0 += kAhead) {
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int tn = 0; tn < S::TN; ++tn)
                *(lds_f32x4 *)(own + (h * 16 + (lane & 15)) * kLd + tn * 64 + (lane >> 4) * 16) =
                    acc[t0 + h][tn];
        // One wave's LDS accesses are done in order; only the compiler must keep it.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int r = 0; r < kParts; ++r) {
                const lds_char *p = own + (h * 16 + r * kRows + row) * kLd + col * 4;
                const f32x4 a = *(lds_f32x4 *)p, b = *(lds_f32x4 *)(p + 16);
                float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                use((t0 + h) * 16 + r * kRows + row, col, v, aux[t0 + h][r]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int tm = t0 + 2 * kAhead; tm < t0 + 3 * kAhead && tm < S::TM; ++tm)
#pragma unroll
            for (int r = 0; r < kParts; ++r) aux[tm][r] = load(tm * 16 + r * kRows + row, col);
    }
}

struct RowsArgs {
    RowsProblem pr;
    int gm;  // row tiles walked per column tile, so that a group's operands stay in L2
};

// Tile (mt, nt) of the walk's place id: groups of gm row tiles, row first.
__device__ __forceinline__ void walk(int id, int tiles_m, int tiles_n, int gm, int &mt, int &nt) {
    const int per = gm * tiles_n;
    const int panel = id / per;
    const int first = panel * gm;
    const int height = tiles_m - first < gm ? tiles_m - first : gm;
    const int in = id - panel * per;
    mt = __builtin_amdgcn_readfirstlane(first + in % height);
    nt = __builtin_amdgcn_readfirstlane(in / height);
}

template <class S>
__global__ __launch_bounds__(S::NW * 64, 1) void rows_kernel(RowsArgs a) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[2 * S::kStage];
    lds_char *smem = (lds_char *)memory;
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
    const int id = xcd_tile(tiles_m * tiles_n, 0);
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
        product<S>(smem, tp, tq, (int)pr.depth, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    T *out = (T *)pr.out, *pre = (T *)pr.pre;
    const T *bias = (const T *)pr.bias;
    // The residual of the forward product or the input's activation of dx.
    const T *extra = (const T *)(pr.residual ? pr.residual : pr.in_pre);
    const int64_t ldx = pr.residual ? pr.ldr : pr.ldin;
    const bool in = pr.in_pre != nullptr;
    float b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (bias && !tail) {
        const int n = wn + lane % (S::TN * 2) * 8;
        if (n < cols) load8(bias + (int64_t)gr.expert * cols + n, cols - n, b);
    }
    struct Aux {
        T v[8];
    };
    by_rows<S, Aux>(
        smem, wave, lane, acc,
        [&](int row, int col) {
            Aux x;
            const int64_t m = wm + row;
            const int n = wn + col, valid = cols - n;
            if (extra && !tail && m < gr.hi && valid >= 8) {
                load_vec(extra + m * ldx + n, x.v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x.v[i] = extra && !tail && m < gr.hi && i < valid ? extra[m * ldx + n + i] : (T)0.0f;
            }
            return x;
        },
        [&](int row, int col, float (&z)[8], const Aux &x) {
            const int64_t m = wm + row;
            const int n = wn + col, valid = cols - n;
            if (m >= gr.hi || valid <= 0) return;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = tail ? 0.0f : z[i] + b[i];
            if (pre) store8(pre + m * pr.ldpre + n, z, valid);
            if (pr.act != kActNone) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], pr.act);
            }
            if (in) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= act_slope((float)x.v[i], pr.in_act);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += (float)x.v[i];
            }
            store8(out + m * pr.ldo + n, z, valid);
        });
}

constexpr int kPiece = 16;  // tiles: 4 x 4 of the walk

template <class S>
__global__ __launch_bounds__(S::NW * 64, 1) void grad_kernel(GradProblem pr) {
    typedef typename S::type T;
    __shared__ __align__(1024) char memory[2 * S::kStage];
    lds_char *smem = (lds_char *)memory;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mc = (int)pr.m_cols, nc = (int)pr.n_cols, rows = (int)pr.rows;
    const int tiles_m = (mc + S::BM - 1) / S::BM, tiles_n = (nc + S::BN - 1) / S::BN;
    const int each = tiles_m * tiles_n;
    // Experts' tiles cost as many stages as the expert has rows: dealt out in
    // small pieces, every XCD gets tiles of every large expert.
    const int id = xcd_tile(each * pr.experts, pr.offsets ? kPiece : 0);
    if (id < 0) return;
    const int e = __builtin_amdgcn_readfirstlane(id / each);
    int mt, nt;
    walk(id - e * each, tiles_m, tiles_n, 4, mt, nt);
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    int lo = 0, hi = rows;
    if (pr.offsets) {
        lo = __builtin_amdgcn_readfirstlane(clampi(pr.offsets[e], 0, rows));
        hi = __builtin_amdgcn_readfirstlane(clampi(pr.offsets[e + 1], lo, rows));
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
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    T *out = (T *)pr.out + (int64_t)e * mc * nc;
    struct Aux {};
    by_rows<S, Aux>(
        smem, wave, lane, acc, [](int, int) { return Aux{}; },
        [&](int row, int col, float (&z)[8], const Aux &) {
            const int m = wm + row, n = wn + col;
            if (m < mc && n < nc) store8(out + (int64_t)m * nc + n, z, nc - n);
        });
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
    RowsArgs a;
    a.pr = pr;
    a.gm = 8;
    const int64_t tiles = most_row_tiles(pr.rows, S::BM, pr.offsets, pr.experts) * cdiv(pr.cols, S::BN);
    rows_kernel<S><<<(unsigned)(cdiv(tiles, 8) * 8), S::NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

template <class S>
hipError_t run_grad(const GradProblem &pr, hipStream_t s) {
    const int64_t tiles = cdiv(pr.m_cols, S::BM) * cdiv(pr.n_cols, S::BN) * pr.experts;
    const int64_t unit = pr.offsets ? 8 * kPiece : 8;
    grad_kernel<S><<<(unsigned)(cdiv(tiles, unit) * unit), S::NW * 64, 0, s>>>(pr);
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
