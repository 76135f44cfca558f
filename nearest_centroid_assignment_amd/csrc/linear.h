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
// output row or column (64 16-bit values, 32 floats; 64 bytes in product_in_turns),
// moved from global memory straight into LDS (buffer_load ... lds); whatever lies
// outside an operand is dropped by the buffer's range check and reads as zero.
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
//       (Rows of fewer granules use the low bits of the key.)
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

constexpr uint32_t kNowhere = 1u << 31;  // an offset past every buffer (records < 2^31)

template <typename T>
struct Frag;  // 16 bytes of k per lane
template <>
struct Frag<bf16> {
    typedef bf16x8 type;
    static constexpr int kSteps = 1;  // matrix instructions for a fragment
    static __device__ __forceinline__ f32x4 mma(bf16x8 p, bf16x8 q, f32x4 c, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
    }
};
template <>
struct Frag<f16> {
    typedef f16x8 type;
    static constexpr int kSteps = 1;
    static __device__ __forceinline__ f32x4 mma(f16x8 p, f16x8 q, f32x4 c, int) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, c, 0, 0, 0);
    }
};
template <>
struct Frag<float> {
    typedef f32x4 type;
    static constexpr int kSteps = 4;
    // Lane group g holds k = 4 g .. 4 g + 3 of both operands; instruction j
    // takes element j of each lane, so its four k are j, 4 + j, 8 + j, 12 + j.
    static __device__ __forceinline__ f32x4 mma(f32x4 p, f32x4 q, f32x4 c, int j) {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], q[j], c, 0, 0, 0);
    }
};

// Rows of 64 bytes: the key of row r. Four rows share a line of 64 banks, so rows r,
// r + 4, r + 8, r + 12 get different keys, in an order that also keeps apart the two
// chunks that a read's groups of 16 lanes mix (rows 0-3 and 12-15 of one, 4-11 of
// the next).
__device__ __forceinline__ int kc_key64(int r) {
    const int n = (r >> 2) & 3;
    return ((n & 1) << 1) ^ ((n >> 1) * 3);
}

// One operand's stage: R output rows (or columns) x 128 bytes of k, moved by
// NW waves with 16 bytes a lane and instruction. Rows may start on any 4 bytes:
// the buffer's range check works in 4-byte words, so a chunk that leaves the
// operand is cut there. A chunk that leaves its row reads the next row's start,
// which in an MC operand only reaches columns that are not stored; where a KC row ends
// inside a chunk (`ragged`), the last stage's fragments are cut in registers (cut).
template <typename T, bool MC, int R, int NW, int kRow>
struct Tile {
    static constexpr int kSize = (int)sizeof(T);
    static constexpr int kBytes = R * kRow;
    static constexpr int kDepth = kRow / kSize;  // k per stage
    static constexpr int kIssues = kBytes / (1024 * NW);
    static_assert(kIssues >= 1 && kIssues * 1024 * NW == kBytes, "tile and waves");

    uint32_t off[kIssues];
    int kc[2];        // KC: byte of k that this lane moves, by the parity of the issue (8 rows each)
    uint64_t at;      // this stage's first row or column (the rest is wave-uniform too)
    int ld, left;     // bytes of a row; KC: bytes, MC: rows of k from this stage on
    int extent;       // KC: bytes before the last valid row (< 0: no row); MC: valid bytes of a row

    static __device__ __forceinline__ int swizzle(int k) {  // MC, in 16-byte chunks
        if (kSize == 2) return (((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1)) << 1;
        return ((k >> 2) & 3 & (R / 16 - 1)) << 2;
    }
    // Byte q of the stage in LDS: its byte of the row in memory (KC).
    static __device__ __forceinline__ int kc_byte(int q) {
        const int key = kRow == 128 ? (q >> 8) & 7 : kc_key64(q / 64);
        return ((((q & (kRow - 1)) >> 4) ^ key) << 4) | (q & 15);
    }
    static __device__ __forceinline__ int lds_byte(int wave, int lane, int i) {
        return ((wave * kIssues + i) * 64 + lane) * 16;
    }

    // p: the tile's first row (KC) or column (MC) at k = 0; valid: rows or columns.
    __device__ __forceinline__ void init(const char *p, int64_t ld_elems, int64_t valid, int depth,
                                         int wave, int lane) {
        const uint64_t a = (uint64_t)p;
        at = ((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) << 32) |
             (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
        ld = __builtin_amdgcn_readfirstlane((int)(ld_elems * kSize));
        const int n = (int)(valid < 0 ? 0 : valid > R ? R : valid);
        // (A row of an odd number of 16-bit values comes padded with a zero.)
        left = __builtin_amdgcn_readfirstlane(MC ? depth : (depth * kSize + 3) & ~3);
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
                off[i] = q / kRow * ld + kc_byte(q);
            }
        }
        kc[0] = kc_byte(lds_byte(wave, lane, 0));
        kc[1] = kc_byte(lds_byte(wave, lane, kIssues > 1 ? 1 : 0));
    }

    // Whether the last stage's fragments have to be cut.
    __device__ __forceinline__ bool ragged() const { return !MC && (left & 15) != 0; }

    // Moves this stage into LDS and steps to the next. Past the last stage
    // every lane is out of range, and zeros arrive.
    __device__ __forceinline__ void issue(lds_char *lds, int wave) {
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
        lds_char *to = lds + wave * kIssues * 1024;
#pragma unroll
        for (int i = 0; i < kIssues; ++i) {
            uint32_t o = off[i];
            if (!MC) o = kc[i & 1] < left ? o : kNowhere;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(to + i * 1024), 16, (int)o, 0,
                                                     0, 0);
        }
        at += MC ? (uint64_t)ld * kDepth : (uint64_t)kRow;
        left -= MC ? kDepth : kRow;
    }
};

// Fragment reads of one operand: `first` = the wave's first output row/column.
template <typename T, bool MC, int R, int N, int kRow>
struct Reader {
    typedef typename Frag<T>::type frag;
    typedef __attribute__((address_space(3))) const frag lds_frag;
    typedef __attribute__((address_space(3))) const float lds_float;
    int at[MC ? N : 2];  // MC: by block; KC: by half of the stage

    __device__ __forceinline__ void init(int first, int lane) {
        const int i = lane & 15, g = lane >> 4;
        if (!MC) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                at[s] = (first + i) * kRow +
                        ((kRow == 128 ? (4 * s + g) ^ (i >> 1) : g ^ kc_key64(i)) << 4);
        } else {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                if (sizeof(T) == 2) {
                    const int k = 8 * g + (i >> 2);
                    const int key = ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
                    at[t] = k * (R * 2) + (((first / 16 + t) ^ key) << 5) + (i & 3) * 8;
                } else {
                    at[t] = 4 * g * (R * 4) + (((first / 16 + t) ^ (g & (R / 16 - 1))) << 6) + i * 4;
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

template <typename T, bool PMC, bool QMC, int BM_, int BN_, int WM_, int WN_, int NS_, int ROW = 128>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, kRow = ROW;
    static constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr int kStage = (BM + BN) * ROW;
    // The largest tiles belong to products whose outputs, residuals and input
    // activations pass through once and would push the operands out of L2:
    // 32768 x 4096 with depth 2048 and an input activation 597 -> 513 us,
    // 8192^3 dx 883 -> 793 us.
    static constexpr bool kOnce = BM * BN >= 1 << 16;
    typedef T type;
    typedef Tile<T, PMC, BN, NW, ROW> TileP;
    typedef Tile<T, QMC, BM, NW, ROW> TileQ;
    typedef Reader<T, PMC, BN, TN, ROW> ReadP;
    typedef Reader<T, QMC, BM, TM, ROW> ReadQ;
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
    for (int t = 0; t < S::TM; ++t) f.q[t] = rq.read(stage + S::BN * S::kRow, t, s);
}
// Zero for what the last stage's half s holds past its `valid` values of k, in
// the operands whose rows hold k.
template <class S>
__device__ __forceinline__ void cut(Frags<S> &f, int s, int valid, int lane) {
    constexpr int kLane = 16 / (int)sizeof(typename S::type);
    const int left = valid - (s * 4 + (lane >> 4)) * kLane;
#pragma unroll
    for (int j = 0; j < kLane; ++j) {
        if (!S::p_mc)
#pragma unroll
            for (int t = 0; t < S::TN; ++t) f.p[t][j] = j < left ? f.p[t][j] : 0;
        if (!S::q_mc)
#pragma unroll
            for (int t = 0; t < S::TM; ++t) f.q[t][j] = j < left ? f.q[t][j] : 0;
    }
}
template <class S>
__device__ __forceinline__ void multiply(const Frags<S> &f, f32x4 (&acc)[S::TM][S::TN]) {
    // One accumulator's instructions lie a whole block apart: back to back each
    // would wait for the one before it.
#pragma unroll
    for (int j = 0; j < Frag<typename S::type>::kSteps; ++j)
#pragma unroll
        for (int m = 0; m < S::TM; ++m)
#pragma unroll
            for (int n = 0; n < S::TN; ++n)
                acc[m][n] = Frag<typename S::type>::mma(f.p[n], f.q[m], acc[m][n], j);
}

// The order of one half-stage: its LDS reads (for the half after it) and
// `moves` global-to-LDS loads spread evenly over its matrix instructions.
template <class S>
__device__ __forceinline__ void spread(bool moves) {
    constexpr int kMma = S::TM * S::TN * Frag<typename S::type>::kSteps;
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

// Waits until at most `loads` loads of the wave are in flight, and for its LDS reads.
template <int loads>
__device__ __forceinline__ void wait_loads() {
    static_assert(loads < 64, "the counter's width");
    __builtin_amdgcn_s_waitcnt((loads & 15) | (7 << 4) | ((loads >> 4) << 14));
}

// The product of the largest tiles, whose compute unit holds one block of eight
// waves, two to a SIMD. Stages are 64 bytes of k, four in LDS. A wave alternates
// between reading a stage's fragments and multiplying them, and the second four waves
// run one phase behind the first four: on every SIMD one wave multiplies without a
// pause while the other reads, moves the stage three later in and waits for the next
// one. A barrier ends each phase.
// 8192^3 bf16, against `product` with two stages of 128 bytes: 9 % fewer cycles (the
// matrix units busy 72 % of them, before 66 %), but 2 to 3 % less time (872 us under the
// counters, before 901), since the clock falls to 1.66 GHz from 1.76: at this rate the
// chip's power sets the pace (a loop of nothing but these matrix instructions reaches 2.1
// PFLOP/s). Of 17 experts (32768 x 2048 with depth 4096, f16) the units are busy 51 % of
// the cycles: there each tile's first loads and its epilogue, in rounds of 256 tiles, count
// as much. dw, both of whose operands are read by column, has 8192^3 2 % and 8192 x 2048
// with depth 8192 6 % slower this way, 17 experts 2 % faster: it keeps `product`.
template <class S>
__device__ __forceinline__ void product_in_turns(lds_char *smem, typename S::TileP &tp,
                                                 typename S::TileQ &tq, int depth, int wave,
                                                 int lane, f32x4 (&acc)[S::TM][S::TN]) {
    static_assert(S::NS == 4 && S::kRow == 64 && S::NW == 8, "four short stages, eight waves");
    typename S::ReadP rp;
    typename S::ReadQ rq;
    rp.init((wave % S::WN) * (S::BN / S::WN), lane);
    rq.init((wave / S::WN) * (S::BM / S::WM), lane);
    const int stages = __builtin_amdgcn_readfirstlane((depth + S::TileP::kDepth - 1) / S::TileP::kDepth);
    if (stages == 0) return;
    constexpr int kMoves = S::TileP::kIssues + S::TileQ::kIssues;
    const bool ragged = tp.ragged() || tq.ragged();
    auto meet = [] {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        tp.issue(smem + i * S::kStage, wave);
        tq.issue(smem + i * S::kStage + S::BN * S::kRow, wave);
    }
    wait_loads<2 * kMoves>();
    meet();
    if (wave >= 4) meet();  // one phase behind
    Frags<S> f;
    int at = 0;
    const int valid = depth - (stages - 1) * S::TileP::kDepth;  // of the last stage
    auto stage = [&](bool last) {
        lds_char *cur = smem + at * S::kStage, *free = smem + ((at + 3) & 3) * S::kStage;
        read_half<S>(rp, rq, cur, 0, f);
        // Its last readers, the waves behind, were done a phase ago.
        tp.issue(free, wave);
        tq.issue(free + S::BN * S::kRow, wave);
        wait_loads<2 * kMoves>();  // the next stage has landed; the fragments are here
        meet();
        if (last) cut<S>(f, 0, valid, lane);
        __builtin_amdgcn_s_setprio(1);
        multiply<S>(f, acc);
        __builtin_amdgcn_s_setprio(0);
        meet();
        at = (at + 1) & 3;
    };
    const int plain = ragged ? stages - 1 : stages;
    for (int it = 0; it < plain; ++it) stage(false);
    if (ragged) stage(true);
    if (wave < 4) meet();
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // the stages' memory is free
}

// acc[tm][tn] += the tile's product over the whole depth. NS stages in LDS and two
// half-stages of fragments in registers: while one half is multiplied, the next
// is read, and in the second half of a stage, whose buffer every wave has read
// by then, the stage NS later moves in.
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
    constexpr int kMoves = S::TileP::kIssues + S::TileQ::kIssues;
    const bool ragged = tp.ragged() || tq.ragged();
#pragma unroll
    for (int i = 0; i < S::NS; ++i) {
        tp.issue(smem + i * S::kStage, wave);
        tq.issue(smem + i * S::kStage + S::BN * S::kRow, wave);
    }
    wait_loads<(S::NS - 1) * kMoves>();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    Frags<S> f[2];
    read_half<S>(rp, rq, smem, 0, f[0]);
    lds_char *cur = smem;
    const int valid = depth - (stages - 1) * S::TileP::kDepth;  // of the last stage
    auto stage = [&](bool last) {
        lds_char *nxt = cur + S::kStage == smem + S::NS * S::kStage ? smem : cur + S::kStage;
        read_half<S>(rp, rq, cur, 1, f[1]);
        if (last) cut<S>(f[0], 0, valid, lane);
        multiply<S>(f[0], acc);
        spread<S>(false);
        // Left alone, the compiler waits and meets after a quarter of these
        // multiplications and lets the rest cover the barrier. With one wave to a SIMD
        // (64 x 64) the loads then have too little time: 1000 x 777 with depth 1111 float32
        // 29 -> 26.5 us. Larger tiles are as fast either way, or faster left alone.
        if (S::BM * S::BN <= 64 * 64 && S::BM == S::BN) __builtin_amdgcn_sched_barrier(0);
        wait_loads<(S::NS - 2) * kMoves>();
        // The next stage has landed, and this one is in registers. (Loads of later
        // stages stay in flight across the barrier; __syncthreads would wait.)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        read_half<S>(rp, rq, nxt, 0, f[0]);
        tp.issue(cur, wave);
        tq.issue(cur + S::BN * S::kRow, wave);
        if (last) cut<S>(f[1], 1, valid, lane);
        multiply<S>(f[1], acc);
        spread<S>(true);
        cur = nxt;
    };
    const int plain = ragged ? stages - 1 : stages;
    for (int it = 0; it < plain; ++it) stage(false);
    if (ragged) stage(true);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // the stages' memory is free
}

template <class S>
__device__ __forceinline__ void run_product(lds_char *smem, typename S::TileP &tp,
                                            typename S::TileQ &tq, int depth, int wave, int lane,
                                            f32x4 (&acc)[S::TM][S::TN]) {
    if constexpr (S::kRow == 64)
        product_in_turns<S>(smem, tp, tq, depth, wave, lane, acc);
    else
        product<S>(smem, tp, tq, depth, wave, lane, acc);
}

// Block b of a grid of `total` tiles: XCD b % 8 takes pieces of `piece`
// consecutive tiles, so that tiles which share operands share an L2; piece 0: one
// piece, an eighth of the tiles. -1: no tile. (total, piece < 2^31)
__device__ __forceinline__ int xcd_tile(int b, int total, int piece) {
    const int x = b & 7, j = b >> 3;
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
// the last expert (expert == experts). Offsets are clamped into the matrix, so
// whatever they hold no access leaves it. The last 64 experts looked at stay in
// the lanes' registers: up to 63 experts are read once.
struct Groups {
    const int *offsets;
    int experts, rows, bm;
    int lo, hi, tiles, incl;  // of the lane's expert; incl: tiles up to and with it

    __device__ __forceinline__ void load(int e0, int before) {
        const int e = e0 + (threadIdx.x & 63);
        lo = hi = 0;
        if (e <= experts) {
            lo = clampi(offsets[e], 0, rows);
            hi = e < experts ? clampi(offsets[e + 1], lo, rows) : rows;
        }
        tiles = (hi - lo + bm - 1) / bm;
        incl = before + wave_incl_scan(tiles);
    }
    __device__ __forceinline__ int total() {
        int before = 0;
        for (int e0 = 0; e0 <= experts; e0 += 64) {
            load(e0, before);
            before = __builtin_amdgcn_readlane(incl, 63);
        }
        return before;
    }
    // The group that holds tile mt (expert -1: none). After total().
    __device__ __forceinline__ Group find(int mt) {
        Group r = {-1, 0, 0, 0};
        int before = 0;
        for (int e0 = 0; e0 <= experts; e0 += 64) {
            if (experts >= 64) load(e0, before);
            const unsigned long long past = __ballot(incl > mt);
            if (past) {
                const int l = __builtin_ctzll(past);
                r.expert = e0 + l;
                r.lo = __builtin_amdgcn_readlane(lo, l);
                r.hi = __builtin_amdgcn_readlane(hi, l);
                r.tile = mt - __builtin_amdgcn_readlane(incl - tiles, l);
                // (Offsets that no plan makes can give more tiles than an int counts.)
                if (r.tile < 0 || r.tile >= __builtin_amdgcn_readlane(tiles, l)) r.expert = -1;
                return r;
            }
            before = __builtin_amdgcn_readlane(incl, 63);
        }
        return r;
    }
};

template <bool ONCE, typename T>
__device__ __forceinline__ void store_whole(T *p, const float (&v)[8]) {
    T x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
    if (ONCE)
        store_once(p, x);
    else
        store_vec(p, x);
}

// Hands the wave's tile to `use(row, col, values, aux)`, eight consecutive
// columns at a time: 16 rows at a time go through LDS (each wave's own part of the
// stages' memory), so that a wave's accesses to memory are whole rows of the tile,
// 16 bytes a lane, where the matrix instruction leaves a lane four columns of one
// row. (Stored as it leaves them, 8 bytes a lane: 8192 x 8192 x 2048 with gelu 318 us
// against 287, both before the epilogue chose its activation once.) `load(row, col)`
// gives the aux of a place; it is asked for kAhead blocks of 16 rows ahead, or its latency
// would be paid again for every block.
template <class S, class Aux, class L, class F>
__device__ __forceinline__ void by_rows(lds_char *smem, int wave, int lane,
                                        const f32x4 (&acc)[S::TM][S::TN], L load, F use) {
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    constexpr int kCols = S::TN * 16, kLd = (kCols + 4) * 4;
    constexpr int kLanes = kCols / 8;   // lanes to a row
    constexpr int kRows = 64 / kLanes;  // rows at a time
    constexpr int kParts = 16 / kRows;
    constexpr int kAhead = S::TM < 2 ? S::TM : 2;
    static_assert(kParts >= 1, "two column blocks a wave at least");
    static_assert(16 * kLd * S::NW <= S::NS * S::kStage, "the stages' memory");
    lds_char *own = smem + wave * 16 * kLd;
    const int row = lane / kLanes, col = lane % kLanes * 8;
    Aux aux[S::TM][kParts];
#pragma unroll
    for (int tm = 0; tm < kAhead; ++tm)
#pragma unroll
        for (int r = 0; r < kParts; ++r) aux[tm][r] = load(tm * 16 + r * kRows + row, col);
#pragma unroll
    for (int tm = 0; tm < S::TM; ++tm) {
#pragma unroll
        for (int tn = 0; tn < S::TN; ++tn)
            *(lds_f32x4 *)(own + (lane & 15) * kLd + tn * 64 + (lane >> 4) * 16) = acc[tm][tn];
        // One wave's LDS accesses are done in order; only the compiler must keep it.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int r = 0; r < kParts; ++r) {
            const lds_char *p = own + (r * kRows + row) * kLd + col * 4;
            const f32x4 a = *(lds_f32x4 *)p, b = *(lds_f32x4 *)(p + 16);
            float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            use(tm * 16 + r * kRows + row, col, v, aux[tm][r]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (tm + kAhead < S::TM) {
#pragma unroll
            for (int r = 0; r < kParts; ++r)
                aux[tm + kAhead][r] = load((tm + kAhead) * 16 + r * kRows + row, col);
        }
    }
}

constexpr int kWalk = 8;

struct RowsArgs {
    RowsProblem pr;
    int gm;  // row tiles walked per column tile, so that a group's operands stay in L2
};

// Part `part` of `parts` of a depth of `stages` stages: whole stages.
__device__ __forceinline__ void part_of(int stages, int parts, int part, int &first, int &count) {
    const int per = (stages + parts - 1) / parts;
    first = part * per < stages ? part * per : stages;
    count = stages - first < per ? stages - first : per;
}

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
__device__ __forceinline__ void rows_block(const RowsArgs &a, int block, lds_char *smem) {
    typedef typename S::type T;
    const RowsProblem &pr = a.pr;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)pr.rows, cols = (int)pr.cols;
    const int tiles_n = (cols + S::BN - 1) / S::BN;
    Groups groups = {pr.offsets, pr.experts, rows, S::BM};
    const int tiles_m = pr.offsets ? groups.total() : (rows + S::BM - 1) / S::BM;
    const int tiles = tiles_m * tiles_n;
    int id = xcd_tile(block, tiles * pr.splits, 0);
    if (id < 0 || tiles_m < 1) return;  // (tiles_m < 1: an int did not hold them)
    const int part = __builtin_amdgcn_readfirstlane(id / tiles);
    id -= part * tiles;
    int mt, nt;
    walk(id, tiles_m, tiles_n, a.gm, mt, nt);
    Group gr = {0, 0, rows, mt};
    if (pr.offsets) gr = groups.find(mt);
    if (gr.expert < 0) return;
    const int m0 = gr.lo + gr.tile * S::BM, n0 = nt * S::BN;
    if (gr.expert == pr.experts) {  // rows past the last expert's: zero
        if (pr.splits > 1) return;    // (the join writes them)
        for (int i = threadIdx.x; i < S::BM * (S::BN / 8); i += S::NW * 64) {
            const int64_t m = m0 + i / (S::BN / 8);
            const int n = n0 + i % (S::BN / 8) * 8;
            if (m >= gr.hi || n >= cols) continue;
            const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            store_row((T *)pr.out + m * pr.ldo + n, zero, cols - n);
            if (pr.pre) store_row((T *)pr.pre + m * pr.ldpre + n, zero, cols - n);
        }
        return;
    }
    f32x4 acc[S::TM][S::TN];
#pragma unroll
    for (int m = 0; m < S::TM; ++m)
#pragma unroll
        for (int n = 0; n < S::TN; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    {
        constexpr int kDepth = S::TileP::kDepth;
        const int depth = (int)pr.depth;
        int first, count;
        part_of((depth + kDepth - 1) / kDepth, pr.splits, part, first, count);
        const int k0 = __builtin_amdgcn_readfirstlane(first * kDepth);
        const int len = depth - k0 < count * kDepth ? depth - k0 : count * kDepth;
        const char *q = (const char *)pr.q + ((int64_t)m0 * pr.ldq + k0) * sizeof(T);
        const char *p = (const char *)pr.p + (int64_t)gr.expert * pr.p_expert * sizeof(T);
        p += (S::p_mc ? k0 * pr.ldp + n0 : n0 * pr.ldp + k0) * sizeof(T);
        typename S::TileP tp;
        typename S::TileQ tq;
        tp.init(p, pr.ldp, S::p_mc ? pr.p_cols - n0 : (int64_t)cols - n0, len, wave, lane);
        tq.init(q, pr.ldq, gr.hi - m0, len, wave, lane);
        run_product<S>(smem, tp, tq, len, wave, lane, acc);
    }
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    struct None {};
    if (pr.splits > 1) {
        float *partial = pr.partial + (int64_t)part * pr.rows * cols;
        by_rows<S, None>(
            smem, wave, lane, acc, [](int, int) { return None{}; },
            [&](int row, int col, float (&z)[8], const None &) {
                const int64_t m = wm + row;
                const int n = wn + col;
                if (m < gr.hi && n < cols) store_row(partial + m * cols + n, z, cols - n);
            });
        return;
    }
    T *out = (T *)pr.out, *pre = (T *)pr.pre;
    const T *bias = (const T *)pr.bias;
    // The residual of the forward product (P by depth) or the input's activation of
    // dx (P by column).
    const T *extra = (const T *)(S::p_mc ? pr.in_pre : pr.residual);
    const int64_t ldx = S::p_mc ? pr.ldin : pr.ldr;
    struct Aux {
        T v[8];
    };
    float b[8];
    if (!S::p_mc) {
        T row[8];
        const int n = wn + lane % (S::TN * 2) * 8;
        load_row(bias + (int64_t)gr.expert * cols + n, bias ? cols - n : 0, row);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = (float)row[i];
    }
    if (m0 + S::BM <= gr.hi && n0 + S::BN <= cols) {
        // A whole tile: nothing to check.
        auto whole = [&](auto tag, auto has_extra) {
            constexpr int ACT = decltype(tag)::value;
            constexpr bool EXTRA = decltype(has_extra)::value != 0;
            by_rows<S, Aux>(
                smem, wave, lane, acc,
                [&](int row, int col) {
                    Aux x;
                    const T *at = extra + (int64_t)(wm + row) * ldx + wn + col;
                    if (EXTRA && S::kOnce)
                        load_once(at, x.v);
                    else if (EXTRA)
                        load_vec(at, x.v);
                    return x;
                },
                [&](int row, int col, float (&z)[8], const Aux &x) {
                    const int64_t m = wm + row;
                    const int n = wn + col;
                    if (S::p_mc) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (EXTRA) z[i] *= slope_of<ACT>((float)x.v[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] += b[i];
                        if (pre) store_whole<S::kOnce>(pre + m * pr.ldpre + n, z);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            z[i] = act_of<ACT>(z[i]);
                            if (EXTRA) z[i] += (float)x.v[i];
                        }
                    }
                    store_whole<S::kOnce>(out + m * pr.ldo + n, z);
                });
        };
        if (S::p_mc) {
            if (extra)
                with_act(pr.in_act, [&](auto tag) { whole(tag, ActTag<1>{}); });
            else
                whole(ActTag<kActNone>{}, ActTag<0>{});
        } else if (extra) {
            with_act(pr.act, [&](auto tag) { whole(tag, ActTag<1>{}); });
        } else {
            with_act(pr.act, [&](auto tag) { whole(tag, ActTag<0>{}); });
        }
        return;
    }
    by_rows<S, Aux>(
        smem, wave, lane, acc,
        [&](int row, int col) {
            Aux x;
            const int64_t m = wm + row;
            const int n = wn + col;
            load_row(extra + m * ldx + n, extra && m < gr.hi ? cols - n : 0, x.v);
            return x;
        },
        [&](int row, int col, float (&z)[8], const Aux &x) {
            const int64_t m = wm + row;
            const int n = wn + col, valid = cols - n;
            if (m >= gr.hi || valid <= 0) return;
            if (S::p_mc) {
                if (extra) apply_slope(z, x.v, pr.in_act);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += b[i];
                if (pre) store_row(pre + m * pr.ldpre + n, z, valid);
                apply_act(z, pr.act);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] += (float)x.v[i];
            }
            store_row(out + m * pr.ldo + n, z, valid);
        });
}

constexpr int kPiece = 16;  // tiles: 4 x 4 of the walk

template <class S>
__device__ __forceinline__ void grad_block(const GradProblem &pr, int block, lds_char *smem) {
    typedef typename S::type T;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mc = (int)pr.m_cols, nc = (int)pr.n_cols, rows = (int)pr.rows;
    const int tiles_m = (mc + S::BM - 1) / S::BM, tiles_n = (nc + S::BN - 1) / S::BN;
    const int each = tiles_m * tiles_n;
    // Experts' tiles cost as many stages as the expert has rows: dealt out in
    // small pieces, every XCD gets tiles of every large expert.
    const int tiles = each * pr.experts;
    int id = xcd_tile(block, tiles * pr.splits, pr.offsets ? kPiece : 0);
    if (id < 0) return;
    const int part = __builtin_amdgcn_readfirstlane(id / tiles);
    id -= part * tiles;
    const int e = __builtin_amdgcn_readfirstlane(id / each);
    int mt, nt;
    walk(id - e * each, tiles_m, tiles_n, 4, mt, nt);
    const int m0 = mt * S::BM, n0 = nt * S::BN;
    int lo = 0, hi = rows;
    if (pr.offsets) {
        lo = __builtin_amdgcn_readfirstlane(clampi(pr.offsets[e], 0, rows));
        hi = __builtin_amdgcn_readfirstlane(clampi(pr.offsets[e + 1], lo, rows));
    }
    {
        constexpr int kDepth = S::TileP::kDepth;
        int first, count;
        part_of((hi - lo + kDepth - 1) / kDepth, pr.splits, part, first, count);
        lo = __builtin_amdgcn_readfirstlane(lo + first * kDepth);
        hi = __builtin_amdgcn_readfirstlane(hi - lo < count * kDepth ? hi : lo + count * kDepth);
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
    run_product<S>(smem, tp, tq, hi - lo, wave, lane, acc);
    const int wm = m0 + (wave / S::WN) * (S::BM / S::WM);
    const int wn = n0 + (wave % S::WN) * (S::BN / S::WN);
    T *out = (T *)pr.out + (int64_t)e * mc * nc;
    float *partial = pr.partial + ((int64_t)part * pr.experts + e) * mc * nc;
    struct None {};
    auto write = [&](auto *to, bool whole) {
        by_rows<S, None>(
            smem, wave, lane, acc, [](int, int) { return None{}; },
            [&](int row, int col, float (&z)[8], const None &) {
                const int m = wm + row, n = wn + col;
                if (whole)
                    store_whole<S::kOnce>(to + (int64_t)m * nc + n, z);
                else if (m < mc && n < nc)
                    store_row(to + (int64_t)m * nc + n, z, nc - n);
            });
    };
    if (pr.splits > 1)
        write(partial, false);
    else if (m0 + S::BM <= mc && n0 + S::BN <= nc)
        write(out, true);
    else
        write(out, false);
}

template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void rows_kernel(RowsArgs a) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    rows_block<S>(a, blockIdx.x, (lds_char *)memory);
}
template <class S>
__global__ __launch_bounds__(S::NW * 64, 2) void grad_kernel(GradProblem pr) {
    __shared__ __align__(1024) char memory[S::NS * S::kStage];
    grad_block<S>(pr, blockIdx.x, (lds_char *)memory);
}

// dx and dw of one call (where both_plan finds it better): the blocks of the one follow
// those of the other, the deeper (longer) ones first. The last blocks add the parts of
// dbias.
template <class SR, class SG>
__global__ __launch_bounds__(SR::NW * 64, 2) void both_kernel(RowsArgs a, GradProblem g, int first,
                                                              bool rows_first, int products,
                                                              SlopeSum sum) {
    static_assert(SR::NW == SG::NW, "one block size");
    constexpr int kBytes = SR::NS * SR::kStage > SG::NS * SG::kStage ? SR::NS * SR::kStage
                                                                     : SG::NS * SG::kStage;
    __shared__ __align__(1024) char memory[kBytes];
    const int b = blockIdx.x;
    if (b >= products) {
        slope_sum<typename SR::type>(sum, b - products, (float *)memory);
        return;
    }
    const int in = b < first ? b : b - first;
    if ((b < first) == rows_first)
        rows_block<SR>(a, in, (lds_char *)memory);
    else
        grad_block<SG>(g, in, (lds_char *)memory);
}

template <class S>
int64_t rows_blocks(const RowsProblem &pr) {
    const int64_t tiles = most_row_tiles(pr.rows, S::BM, pr.offsets != nullptr, pr.experts) *
                          cdiv(pr.cols, S::BN) * pr.splits;
    return cdiv(tiles, 8) * 8;
}
template <class S>
int64_t grad_blocks(const GradProblem &pr) {
    const int64_t tiles = cdiv(pr.m_cols, S::BM) * cdiv(pr.n_cols, S::BN) * pr.experts * pr.splits;
    const int64_t unit = pr.offsets ? 8 * kPiece : 8;
    return cdiv(tiles, unit) * unit;
}

template <class S>
hipError_t run_rows(const RowsProblem &pr, hipStream_t s) {
    return launch(rows_kernel<S>, rows_blocks<S>(pr), S::NW * 64, 0, s, RowsArgs{pr, kWalk});
}
template <class S>
hipError_t run_grad(const GradProblem &pr, hipStream_t s) {
    return launch(grad_kernel<S>, grad_blocks<S>(pr), S::NW * 64, 0, s, pr);
}
template <class SR, class SG>
hipError_t run_both(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum, hipStream_t s) {
    const int64_t nr = rows_blocks<SR>(r), ng = grad_blocks<SG>(g);
    const bool rows_first = r.depth * g.experts >= g.rows;
    const int64_t ns = sum.splits ? cdiv(sum.n, 64) : 0;
    return launch(both_kernel<SR, SG>, nr + ng + ns, SR::NW * 64, 0, s, RowsArgs{r, kWalk}, g,
                  (int)(rows_first ? nr : ng), rows_first, (int)(nr + ng), sum);
}

// The tiles of a type: forward product (PMC false), dx (PMC true), dw.
template <typename T, bool PMC>
using Rows256 = Shape<T, PMC, false, 256, 256, 2, 4, 4, 64>;
template <typename T, bool PMC>
using Rows129 = Shape<T, PMC, false, 128, 128, 2, 4, 3>;
template <typename T, bool PMC>
using Rows128 = Shape<T, PMC, false, 128, 128, 2, 4, 2>;
template <typename T, bool PMC>
using Rows64 = Shape<T, PMC, false, 64, 64, 2, 2, 2>;
template <typename T, bool PMC>
using Rows32 = Shape<T, PMC, false, 32, 64, 2, 2, 2>;
template <typename T>
using Grad256 = Shape<T, true, true, 256, 256, 2, 4, 2>;
template <typename T>
using Grad129 = Shape<T, true, true, 128, 128, 2, 4, 3>;
template <typename T>
using Grad128 = Shape<T, true, true, 128, 128, 2, 4, 2>;
template <typename T>
using Grad64 = Shape<T, true, true, 64, 64, 2, 2, 2>;
template <typename T>
using Grad32 = Shape<T, true, true, 32, 64, 2, 2, 2>;

template <typename T, bool PMC>
hipError_t pick_rows(const RowsProblem &pr, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (pr.tile == 256) return run_rows<Rows256<T, PMC>>(pr, s);
        if (pr.tile == 129) return run_rows<Rows129<T, PMC>>(pr, s);
    } else {
        if (pr.tile == 32) return run_rows<Rows32<T, PMC>>(pr, s);
    }
    if (pr.tile == 128) return run_rows<Rows128<T, PMC>>(pr, s);
    return run_rows<Rows64<T, PMC>>(pr, s);
}

template <typename T>
hipError_t pick_grad(const GradProblem &pr, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (pr.tile == 256) return run_grad<Grad256<T>>(pr, s);
        if (pr.tile == 129) return run_grad<Grad129<T>>(pr, s);
    } else {
        if (pr.tile == 32) return run_grad<Grad32<T>>(pr, s);
    }
    if (pr.tile == 128) return run_grad<Grad128<T>>(pr, s);
    return run_grad<Grad64<T>>(pr, s);
}

template <typename T>
hipError_t pick_both(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                     hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (r.tile == 256) return run_both<Rows256<T, true>, Grad256<T>>(r, g, sum, s);
    }
    if (r.tile == 128) return run_both<Rows128<T, true>, Grad128<T>>(r, g, sum, s);
    return run_both<Rows64<T, true>, Grad64<T>>(r, g, sum, s);
}

// Products with few rows an expert (BM = 16 MT of them to a block): bound by
// reading w once, so nothing is shared through LDS. A block has 16 columns; its
// eight waves take an eighth of the depth each, every lane loading its fragments
// straight from memory, 16 bytes at any alignment, a batch of them in flight, and
// the eight partial tiles meet in LDS. Rows and columns past the end are read at
// the last valid one and not stored.
template <typename T, int MT>
__global__ __launch_bounds__(512) void thin_kernel(RowsProblem pr) {
    typedef typename Frag<T>::type frag;
    constexpr int kWaves = 8, kLane = 16 / (int)sizeof(T), kStep = 4 * kLane;
    constexpr int kBatch = MT == 1 ? 8 : 6;
    __shared__ float part[kWaves][MT][64][4];
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = (int)pr.rows, cols = (int)pr.cols, depth = (int)pr.depth;
    const int tiles_n = (cols + 15) / 16;
    const int mt = __builtin_amdgcn_readfirstlane(blockIdx.x / tiles_n);
    const int n0 = (blockIdx.x - mt * tiles_n) * 16;
    Group gr = {0, 0, rows, mt};
    if (pr.offsets) {
        Groups groups = {pr.offsets, pr.experts, rows, 16 * MT};
        groups.total();
        gr = groups.find(mt);
    }
    if (gr.expert < 0) return;
    const int m0 = gr.lo + gr.tile * 16 * MT;
    const bool tail = gr.expert == pr.experts;
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    if (!tail) {
        const int steps = (depth + kStep - 1) / kStep;
        int first, count;
        part_of(steps, kWaves, wave, first, count);
        const int n = n0 + i < cols ? n0 + i : cols - 1;
        const T *p = (const T *)pr.p + gr.expert * pr.p_expert + n * pr.ldp + g * kLane;
        const T *q[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + 16 * t + i < gr.hi ? m0 + 16 * t + i : gr.hi - 1;
            q[t] = (const T *)pr.q + (int64_t)m * pr.ldq + g * kLane;
        }
        int s = first;
        const int whole = depth / kStep < first + count ? depth / kStep : first + count;
        union Chunk {
            T v[kLane];
            frag f;
        };
        for (; s + kBatch <= whole; s += kBatch) {
            Chunk a[kBatch], b[kBatch][MT];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                load_vec(p + (s + u) * kStep, a[u].v);
#pragma unroll
                for (int t = 0; t < MT; ++t) load_vec(q[t] + (s + u) * kStep, b[u][t].v);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < Frag<T>::kSteps; ++j)
                        acc[t] = Frag<T>::mma(a[u].f, b[u][t].f, acc[t], j);
        }
        for (; s < first + count; ++s) {
            // One step at a time, the last of them possibly past the depth's end.
            const int left = depth - s * kStep - g * kLane;
            Chunk a, b;
            auto some = [&](const T *x, Chunk &c) {
                if (left >= kLane) {
                    load_vec(x + s * kStep, c.v);
                } else {
#pragma unroll
                    for (int j = 0; j < kLane; ++j) c.v[j] = j < left ? x[s * kStep + j] : (T)0.0f;
                }
            };
            some(p, a);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                some(q[t], b);
#pragma unroll
                for (int j = 0; j < Frag<T>::kSteps; ++j) acc[t] = Frag<T>::mma(a.f, b.f, acc[t], j);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][t][lane][r] = acc[t][r];
    __syncthreads();
    // Lane l of the tile holds columns 4 (l / 16) .. + 3 of row l % 16.
    for (int j = threadIdx.x; j < MT * 256; j += 512) {
        const int t = j >> 8, row = (j >> 4) & 15, col = j & 15;
        const int64_t m = m0 + 16 * t + row;
        const int n = n0 + col;
        if (m >= gr.hi || n >= cols) continue;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) z += part[w][t][(col >> 2) * 16 + row][col & 3];
        if (tail) z = 0.0f;
        if (pr.bias && !tail) z += (float)((const T *)pr.bias)[(int64_t)gr.expert * cols + n];
        if (pr.pre) ((T *)pr.pre)[m * pr.ldpre + n] = (T)z;
        float act[1] = {z};
        apply_act(act, pr.act);
        z = act[0];
        if (pr.residual && !tail) z += (float)((const T *)pr.residual)[m * pr.ldr + n];
        ((T *)pr.out)[m * pr.ldo + n] = (T)z;
    }
}

template <typename T, int MT>
hipError_t run_thin(const RowsProblem &pr, hipStream_t s) {
    const int64_t tiles = most_row_tiles(pr.rows, 16 * MT, pr.offsets != nullptr, pr.experts);
    return launch(thin_kernel<T, MT>, tiles * cdiv(pr.cols, 16), 512, 0, s, pr);
}
template <typename T>
hipError_t pick_thin(const RowsProblem &pr, hipStream_t s) {
    return pr.tile == 16 ? run_thin<T, 1>(pr, s) : run_thin<T, 2>(pr, s);
}

}  // namespace

template <typename T>
hipError_t launch_rows_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_thin_t(const RowsProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_grad_t(const GradProblem &pr, hipStream_t s);
template <typename T>
hipError_t launch_both_t(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                         hipStream_t s);

}  // namespace kx
