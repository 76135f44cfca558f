// adamw.hip - one AdamW step over many tensors in one launch, moments in
// float32 or in 8 bits.
//
// A wave takes 256 consecutive elements of one tensor, four a lane: the block of
// elements that shares the scales of 8-bit moments is then one wave's registers,
// and its largest magnitude one reduction over the wave. A workgroup takes
// kChunk elements of one tensor; the tensors' pointers travel in the kernel's
// arguments (kTensors to a launch), so nothing is copied to the device and a
// step can be captured in a graph.
//
// Bound by memory: everything is read and written once, past the caches (12 tensors, 189
// million elements, float32 moments: 1000 us through them, 909 to 935 past them, 5.7 to 5.8
// TB/s).
//
// The arithmetic is float32 without contraction, in the order of the formulas:
// a moment that lies between two codes gets the same one wherever these
// formulas are evaluated in IEEE float32.
#include "experts.h"

namespace kx {
namespace {

constexpr int kTensors = 64;        // per launch: 2.9 KB of kernel arguments
constexpr int kBlock = 256;         // elements that share a scale
constexpr int kPerWave = 4;         // blocks per wave
constexpr int kChunk = 4 * kPerWave * kBlock;
constexpr int64_t kMaxBlocks = 4294967295LL / 256;

struct Tensor {
    void *p;
    const void *g;
    bf16 *copy;
    int64_t n, at;  // length, first element of its moments
};
struct Batch {
    Tensor t[kTensors];
    int first[kTensors + 1];  // first workgroup of each
    int count;
};

template <typename T>
__device__ __forceinline__ void load_some(const T *p, int64_t left, float (&v)[4]) {
    if (left >= 4) {
        T x[4];
        load_once(p, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? (float)p[i] : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store_some(T *p, int64_t left, const float (&v)[4]) {
    T x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (T)v[i];
    if (left >= 4) {
        store_once(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = x[i];
    }
}

// Largest |x| of the wave, as bits: unsigned order puts infinity above every
// number and NaN above infinity, so neither is lost. DPP moves, as in a scan: lane
// 63 ends with the maximum of all.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto step = [](uint32_t a, int b) { return (uint32_t)b > a ? (uint32_t)b : a; };
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, true));   // row_shr:1
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, true));   // row_shr:2
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, true));   // row_shr:4
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, true));   // row_shr:8
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float block_scale(const float (&x)[4]) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
        big = b > big ? b : big;
    }
    big = wave_max(big);
    return big >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(big);
}

__device__ __forceinline__ float decode_m(int q, float scale) {
#pragma clang fp contract(off)
    const float t = (float)q * (float)(1.0 / 127.0);
    return (t * fabsf(t)) * scale;
}
__device__ __forceinline__ float decode_v(int q, float scale) {
#pragma clang fp contract(off)
    float t = (float)q * (float)(1.0 / 255.0);
    t = t * t;
    return (t * t) * scale;
}
// Codes of a value whose block has this scale (not a number above 0: code 0),
// rounded as IEEE divisions and square roots would have it.
__device__ __forceinline__ int encode_m(float m, float scale) {
#pragma clang fp contract(off)
    if (!(scale > 0.0f)) return 0;
    const float r = m / scale;
    const float q = rintf(sqrtf(fabsf(r)) * 127.0f);
    return (int)(r < 0.0f ? -q : q);
}
__device__ __forceinline__ int encode_v(float v, float scale) {
#pragma clang fp contract(off)
    if (!(scale > 0.0f)) return 0;
    const float q = rintf(sqrtf(sqrtf(v / scale)) * 255.0f);
    return v > 0.0f && q < 1.0f ? 1 : (int)q;
}
// Four codes from the hardware's reciprocal and square root, good to 1 ulp each.
// Before rounding they are then within 6e-5 (m: 127 times 2.7e-7, and as IEEE's own
// roundings 2e-5) or 1.2e-4 (v: 255 times 2.9e-7, and 4e-5) of what encode_m and
// encode_v round, so a code can differ only within 2e-4 of a half: there, in one
// block of ten, the wave takes the exact form. Blocks whose quotients or reciprocal of
// the scale may leave the normal range (the hardware's reciprocal is 0 there) take it
// always: scales below 1e-30 or above 8e37, just under 2^126, and NaN.
// (189 million elements: all exact 740 us, VALU bound; so 540.)
constexpr float kNearHalf = 0.4998f;
__device__ __forceinline__ bool plain_scale(float scale) { return scale >= 1e-30f && scale <= 8e37f; }
__device__ __forceinline__ void encode_m4(const float (&m)[4], float scale, int8_t (&q)[4]) {
    bool exact = !plain_scale(scale);
    const float inv = __builtin_amdgcn_rcpf(scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float t = __builtin_amdgcn_sqrtf(fabsf(m[k]) * inv) * 127.0f;
        const float n = rintf(t);
        exact |= fabsf(t - n) > kNearHalf;
        q[k] = (int8_t)(int)(m[k] < 0.0f ? -n : n);
    }
    if (__any(exact)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = (int8_t)encode_m(m[k], scale);
    }
}
__device__ __forceinline__ void encode_v4(const float (&v)[4], float scale, uint8_t (&q)[4]) {
    bool exact = !plain_scale(scale);
    const float inv = __builtin_amdgcn_rcpf(scale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float t = __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v[k] * inv)) * 255.0f;
        const float n = rintf(t);
        exact |= fabsf(t - n) > kNearHalf;
        q[k] = (uint8_t)(v[k] > 0.0f && n < 1.0f ? 1 : (int)n);
    }
    if (__any(exact)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = (uint8_t)encode_v(v[k], scale);
    }
}

template <typename P, typename G, bool CODES>
__global__ __launch_bounds__(256) void adamw_kernel(Batch b, AdamwStep st) {
#pragma clang fp contract(off)
    const int blk = blockIdx.x;
    int lo = 0, hi = b.count;  // the tensor whose workgroups hold blk
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.first[mid] <= blk)
            lo = mid;
        else
            hi = mid;
    }
    const Tensor t = b.t[lo];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t start = (int64_t)(blk - b.first[lo]) * kChunk + wave * kPerWave * kBlock;
    const float gs = st.grad_scale ? *st.grad_scale : 1.0f;
#pragma unroll
    for (int u = 0; u < kPerWave; ++u) {
        const int64_t base = start + u * kBlock;
        if (base >= t.n) break;
        const int64_t i = base + lane * 4;
        const int64_t left = t.n - i;
        const int64_t j = t.at + i;
        float p[4], g[4], m[4], v[4];
        load_some((const P *)t.p + i, left, p);
        load_some((const G *)t.g + i, left, g);
        if (CODES) {
            int8_t mq[4];
            uint8_t vq[4];
            load_once((const int8_t *)st.m + j, mq);
            load_once((const uint8_t *)st.v + j, vq);
            const float ms = st.m_scale[(t.at + base) / kBlock], vs = st.v_scale[(t.at + base) / kBlock];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = decode_m(mq[k], ms);
                v[k] = decode_v(vq[k], vs);
            }
        } else {
            load_once((const float *)st.m + j, m);
            load_once((const float *)st.v + j, v);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gk = g[k] * gs;
            m[k] = m[k] * st.beta1 + gk * st.one_minus_beta1;
            v[k] = v[k] * st.beta2 + (gk * gk) * st.one_minus_beta2;
            p[k] = p[k] * st.keep - (m[k] * st.rate) / (sqrtf(v[k]) * st.root + st.eps);
        }
        store_some((P *)t.p + i, left, p);
        if (t.copy) store_some(t.copy + i, left, p);
        if (CODES) {
            const float ms = block_scale(m), vs = block_scale(v);
            int8_t mq[4];
            uint8_t vq[4];
            encode_m4(m, ms, mq);
            encode_v4(v, vs, vq);
            store_once((int8_t *)st.m + j, mq);
            store_once((uint8_t *)st.v + j, vq);
            if (lane == 0) {
                st.m_scale[(t.at + base) / kBlock] = ms;
                st.v_scale[(t.at + base) / kBlock] = vs;
            }
        } else {
            store_once((float *)st.m + j, m);
            store_once((float *)st.v + j, v);
        }
    }
}

__global__ __launch_bounds__(256) void moments_kernel(const int8_t *__restrict__ m,
                                                      const uint8_t *__restrict__ v,
                                                      const float *__restrict__ m_scale,
                                                      const float *__restrict__ v_scale,
                                                      int64_t elements, float *__restrict__ m_out,
                                                      float *__restrict__ v_out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= elements) return;
    if (m_out) {
        int8_t q[4];
        load_vec(m + i, q);
        const float s = m_scale[i / kBlock];
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = decode_m(q[k], s);
        store_once(m_out + i, x);
    }
    if (v_out) {
        uint8_t q[4];
        load_vec(v + i, q);
        const float s = v_scale[i / kBlock];
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = decode_v(q[k], s);
        store_once(v_out + i, x);
    }
}

template <typename P, typename G>
hipError_t run(const Batch &b, const AdamwStep &st, hipStream_t s) {
    return launch(st.bits == 8 ? adamw_kernel<P, G, true> : adamw_kernel<P, G, false>,
                  b.first[b.count], 256, 0, s, b, st);
}
template <typename P>
hipError_t run_grads(const Batch &b, const AdamwStep &st, hipStream_t s) {
    if (st.grad_dtype == 0) return run<P, float>(b, st, s);
    return st.grad_dtype == 1 ? run<P, bf16>(b, st, s) : run<P, f16>(b, st, s);
}
hipError_t run_batch(const Batch &b, const AdamwStep &st, hipStream_t s) {
    if (b.count == 0) return hipSuccess;
    if (st.param_dtype == 0) return run_grads<float>(b, st, s);
    return st.param_dtype == 1 ? run_grads<bf16>(b, st, s) : run_grads<f16>(b, st, s);
}

}  // namespace

hipError_t launch_adamw(void *const *params, const void *const *grads, void *const *copies,
                        const int64_t *numels, int64_t count, const AdamwStep &st, hipStream_t s) {
    Batch b;
    b.count = 0;
    b.first[0] = 0;
    int64_t at = 0;
    const int psize = st.param_dtype == 0 ? 4 : 2, gsize = st.grad_dtype == 0 ? 4 : 2;
    for (int64_t i = 0; i < count; ++i) {
        // A tensor longer than one launch's workgroups is taken in pieces.
        for (int64_t done = 0; done < numels[i];) {
            const int64_t room = (kMaxBlocks - b.first[b.count]) * kChunk;
            if (b.count == kTensors || room == 0) {
                const hipError_t e = run_batch(b, st, s);
                if (e != hipSuccess) return e;
                b.count = 0;
                continue;
            }
            const int64_t n = numels[i] - done < room ? numels[i] - done : room;
            Tensor &t = b.t[b.count];
            t.p = (char *)params[i] + done * psize;
            t.g = (const char *)grads[i] + done * gsize;
            t.copy = copies && copies[i] != params[i] ? (bf16 *)copies[i] + done : nullptr;
            t.n = n;
            t.at = at + done;
            b.first[b.count + 1] = b.first[b.count] + (int)cdiv(n, kChunk);
            ++b.count;
            done += n;
        }
        at += cdiv(numels[i], kBlock) * kBlock;
    }
    return run_batch(b, st, s);
}

hipError_t launch_moments(const int8_t *m, const uint8_t *v, const float *m_scale,
                          const float *v_scale, int64_t elements, float *m_out, float *v_out,
                          hipStream_t s) {
    if (elements == 0) return hipSuccess;
    return launch(moments_kernel, cdiv(elements, 1024), 256, 0, s, m, v, m_scale, v_scale, elements,
                  m_out, v_out);
}

}  // namespace kx
