// route.hip - from the scores of the experts to the experts of each token and their
// weights, and the scores' gradient.
//
//   s = softmax(z) or 1 / (1 + e^-z),  c = s + bias  (c = z where nothing is added: the
//   order is the same), a group's rank = its largest c, or the sum of its two largest;
//   of the best groups the `top` largest c, ties to the lower number;
//   weights = scale s / (sum of the chosen s), or scale s.
//
// Bound by memory at best (z read once, dz written once), in fact by the vector units: the
// choice is a partial sort. L lanes (16 or 64) hold a token's choices, V each, as doubles
// whose bits are 1.mantissa = (the float's bits in an order that integers have, then the
// complement of the expert's number): every key is different, a tie goes to the lower
// number, and one v_max_f64 and one v_min_f64 exchange two. Each lane sorts its V keys
// with a network; then, `top` times, the largest head of the lanes is taken out.
//
// A choice between sums of float32 roundings can differ from the formula's where two
// choices lie within those roundings. Where any two that follow each other, or two groups
// at the border, come that near, the token's wave chooses again in float64.
#include "layers.h"
#include "rows.h"

namespace kx {
namespace {

constexpr float kLog2e = 1.44269504088896f;
constexpr int kNumber = 20;  // bits of a key for the expert's number

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Larger for larger floats; -0 as 0. 0 is no float's that is not a NaN.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ double key_of(float choice, int expert) {
    const uint64_t m = ((uint64_t)ordered(choice) << kNumber) | (((1u << kNumber) - 1) - (uint32_t)expert);
    return __longlong_as_double((long long)(m | 0x3ff0000000000000ull));
}
__device__ __forceinline__ int number_of(double key) {
    return (int)(((1u << kNumber) - 1) - ((uint32_t)__double_as_longlong(key) & ((1u << kNumber) - 1)));
}
__device__ __forceinline__ float choice_of(double key) {
    const uint32_t o = (uint32_t)((uint64_t)__double_as_longlong(key) >> kNumber);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Batcher's odd-even merge sort of V keys, largest first.
template <int V>
__device__ __forceinline__ void sort_keys(double (&k)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    const int a = i + j, b = a + q;
                    if (b < V && a / (2 * p) == b / (2 * p)) {
                        const double hi = fmax(k[a], k[b]), lo = fmin(k[a], k[b]);
                        k[a] = hi;
                        k[b] = lo;
                    }
                }
}

template <int CTRL>
__device__ __forceinline__ double rotated(double x) {  // within 16 lanes
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xf, 0xf, false);
    return __longlong_as_double((long long)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo));
}
template <int L>
__device__ __forceinline__ double lanes_max(double x) {
    x = fmax(x, rotated<0x128>(x));  // row_ror:8, 4, 2, 1
    x = fmax(x, rotated<0x124>(x));
    x = fmax(x, rotated<0x122>(x));
    x = fmax(x, rotated<0x121>(x));
    if (L == 64) {
        x = fmax(x, __shfl_xor(x, 16));
        x = fmax(x, __shfl_xor(x, 32));
    }
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) x += __shfl_xor(x, d);
    return x;
}
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// Of the lane's group: the sum of its one or two largest choices, and whether it is
// among the `kept` best (ties to the lower group). `first` and `second`: the lane's two
// largest (-inf: none). `least`: the least distance of a rank to one on the other side.
template <int L, typename F>
__device__ __forceinline__ bool group_kept(F first, F second, int groups, int kept, int best,
                                           int lanes, int group, F &least) {
    const int base = threadIdx.x & 63 & ~(L - 1), own = threadIdx.x & (L - 1);
    const int start = group * lanes;
    F a = first, b = second;
    for (int i = 1; i < lanes; ++i) {
        int from = own + i;
        from -= from >= start + lanes ? lanes : 0;
        const int at = base + (from & (L - 1));
        const F c = __shfl(first, at), d = __shfl(second, at);
        if (c > a) {
            b = a > d ? a : d;
            a = c;
        } else {
            b = b > c ? b : c;
        }
    }
    const F none = -(F)INFINITY;
    const F rank = best == 2 && b > none ? a + b : a;
    int before = 0;
    for (int g = 0; g < groups; ++g) {
        const F other = __shfl(rank, base + g * lanes);
        before += other > rank || (other == rank && g < group);
    }
    const bool keep = group < groups && before < kept;
    least = (F)INFINITY;
    for (int g = 0; g < groups; ++g) {
        const F other = __shfl(rank, base + g * lanes);
        const bool there = __shfl((int)keep, base + g * lanes);
        const F d = other > rank ? other - rank : rank - other;
        if (group < groups && there != keep && d < least) least = d;
    }
    return keep;
}

// The order of the wave's lanes over the experts: L / groups lanes to a group, V experts
// to a lane, one after another.
struct Layout {
    int lanes, group, first, n;  // n: the lane's experts, from `first` on
};
template <int L, int V>
__device__ __forceinline__ Layout layout_of(int experts, int groups) {
    Layout l;
    const int own = threadIdx.x & (L - 1), size = experts / groups;
    l.lanes = L / groups;
    l.group = own / l.lanes;
    const int in = (own - l.group * l.lanes) * V;
    l.first = l.group * size + in;
    l.n = l.group < groups ? (size - in < 0 ? 0 : size - in < V ? size - in : V) : 0;
    return l;
}

template <typename T, int V>
__device__ __forceinline__ void load_scores(const T *p, const Layout &l, float (&z)[V]) {
    T v[V];
    if (l.n == V) {
        load_vec(p + l.first, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < l.n ? p[l.first + j] : (T)(-INFINITY);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = (float)v[j];
}

// The same choice in float64 (see the top): the t-th expert in lane t.
template <int L, int V>
__device__ __forceinline__ int choose_exactly(const float (&z)[V], const RouteProblem &pr, const Layout &l) {
    double c[V];
    double m = -INFINITY, sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) m = z[j] > m ? (double)z[j] : m;
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d));
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool live = z[j] > -INFINITY;
        c[j] = !live ? 0.0 : pr.sigmoid ? 1.0 / (1.0 + exp(-(double)z[j])) : exp((double)z[j] - m);
        sum += c[j];
    }
    sum = lanes_sum<L>(sum);
    double first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (!pr.sigmoid) c[j] /= sum;
        if (pr.bias && j < l.n) c[j] += (double)pr.bias[l.first + j];
        if (!(z[j] > -INFINITY) || !(c[j] > -INFINITY)) c[j] = -INFINITY;
        if (c[j] > first) {
            second = first;
            first = c[j];
        } else if (c[j] > second) {
            second = c[j];
        }
    }
    bool keep = true;
    if (pr.groups > 1) {
        double least;
        keep = group_kept<L, double>(first, second, pr.groups, pr.kept, pr.best, l.lanes, l.group, least);
    }
    int mine = -1;
    for (int t = 0; t < pr.top; ++t) {
        double best = -INFINITY;
        int at = 1 << kNumber;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (keep && c[j] > best) {
                best = c[j];
                at = l.first + j;
            }
#pragma unroll
        for (int d = L / 2; d >= 1; d >>= 1) {
            const double other = __shfl_xor(best, d);
            const int where = __shfl_xor(at, d);
            if (other > best || (other == best && where < at)) {
                best = other;
                at = where;
            }
        }
        if ((int)(threadIdx.x & (L - 1)) == t) mine = best > -INFINITY ? at : -1;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (l.first + j == at) c[j] = -INFINITY;
    }
    return mine;
}

template <typename T, int L, int V>
__global__ __launch_bounds__(256) void route_kernel(RouteProblem pr) {
    const int own = threadIdx.x & (L - 1);
    int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool there = t < pr.tokens;
    if (!there) t = pr.tokens - 1;  // its lanes go along, and store nothing
    const Layout l = layout_of<L, V>(pr.experts, pr.groups);
    const T *row = (const T *)pr.logits + t * pr.ld;
    float z[V], c[V];
    load_scores<T, V>(row, l, z);
    const bool scored = pr.bias || (pr.groups > 1 && pr.best == 2);
    // The largest and the sum of e^(z - largest) where they are needed.
    float top = -INFINITY, total = 1.0f;
    if (scored || (!pr.sigmoid && !pr.renormalize)) {
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, z[j]);
        top = lanes_max<L>(top);
        if (!pr.sigmoid) {
            const float from = top > -INFINITY ? top : 0.0f;
            total = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                c[j] = exp_of(z[j] - from);
                total += c[j];
            }
            total = lanes_sum<L>(total);
        }
    }
    float far = 0.0f;   // what two choices may be off by together
    float most = 0.0f;  // the largest |c|
    if (scored) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            c[j] = pr.sigmoid ? sigmoid(z[j]) : c[j] / total;
            if (pr.bias && j < l.n) c[j] += pr.bias[l.first + j];
            if (!(z[j] > -INFINITY) || !(c[j] > -INFINITY)) c[j] = -INFINITY;
            if (c[j] > -INFINITY) most = fmaxf(most, fabsf(c[j]));
        }
        most = lanes_max<L>(most);
        // The scores' own errors (the argument's rounding times s'(z) |z|, the hardware's
        // 2^x and reciprocal; the softmax's sum), and that of adding the bias.
        const float s = pr.sigmoid ? sigmoid(top) : 1.0f / total;
        const float slope = pr.sigmoid ? (top > -1.0f ? 0.25f : s * -top) : 0.0f;
        far = 2.0f * ((pr.sigmoid ? 0x1p-21f : 0x1p-18f) * s + 0x1p-23f * slope + 0x1p-24f * most);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = z[j];
    }
    bool again = false;
    bool keep = true;
    if (pr.groups > 1) {
        float first = -INFINITY, second = -INFINITY, least;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (c[j] > first) {
                second = first;
                first = c[j];
            } else if (c[j] > second) {
                second = c[j];
            }
        }
        keep = group_kept<L, float>(first, second, pr.groups, pr.kept, pr.best, l.lanes, l.group, least);
        again = scored && least <= 2.0f * far + 0x1p-22f * most;
    }
    double key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = keep && c[j] > -INFINITY ? key_of(c[j], l.first + j) : 0.0;
    sort_keys<V>(key);
    int mine = -1;  // the t-th chosen, in lane t
    double before = 0.0;
    for (int i = 0; i < pr.top + (scored ? 1 : 0); ++i) {
        const double best = lanes_max<L>(key[0]);
        if (key[0] == best) {
#pragma unroll
            for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
            key[V - 1] = 0.0;
        }
        if (own == i && i < pr.top && best != 0.0) mine = number_of(best);
        if (scored) {
            if (i > 0 && best != 0.0) again |= choice_of(before) - choice_of(best) <= far;
            before = best;
        }
    }
    if (scored && __any(again)) mine = choose_exactly<L, V>(z, pr, l);

    const bool chosen = mine >= 0;
    const float score = chosen ? (float)row[mine] : -INFINITY;
    float w = 0.0f;
    if (pr.renormalize) {
        // The denominators cancel: softmax over the chosen, or their sigmoids, which
        // far below zero are e^z (the shift keeps them from all being zero).
        const float highest = lanes_max<L>(score);
        if (pr.sigmoid && highest > -60.0f)
            w = chosen ? sigmoid(score) : 0.0f;
        else
            w = chosen ? exp_of(score - highest) : 0.0f;
        const float sum = lanes_sum<L>(w);
        w = chosen ? pr.scale * (w / sum) : 0.0f;
    } else if (chosen) {
        w = pr.scale * (pr.sigmoid ? sigmoid(score) : exp_of(score - top) / total);
    }
    if (there && own < pr.top) {
        pr.ids[t * pr.top + own] = mine;
        pr.weights[t * pr.top + own] = w;
    }
}

// With r the chosen's shares (their sum 1) and d = scale dweights:
//   renormalised  dz = r (d - sum r d), for sigmoids times 1 - s
//   sigmoid       dz = s (1 - s) d
//   softmax       dz = p (d - sum p d), of the others -p sum p d
// One row for L lanes: lane i has the i-th chosen, then every lane looks through the
// chosen for its V of the row's places.
template <typename T, int L>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteProblem pr) {
    constexpr int V = vec<T>();
    const int own = threadIdx.x & (L - 1), base = threadIdx.x & 63 & ~(L - 1);
    int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool there = t < pr.tokens;
    if (!there) t = pr.tokens - 1;
    const T *row = (const T *)pr.logits + t * pr.ld;
    int64_t id = own < pr.top ? pr.chosen[t * pr.top + own] : -1;
    const bool live = id >= 0 && id < pr.experts;
    const int at = live ? (int)id : -1;
    const float score = live ? (float)row[at] : -INFINITY;
    const float d = live ? pr.scale * pr.dweights[t * pr.top + own] : 0.0f;
    const bool dense = !pr.sigmoid && !pr.renormalize;
    float top = 0.0f, total = 1.0f, inner = 0.0f, dz;
    if (pr.renormalize) {
        const float most = lanes_max<L>(score);
        float r = 0.0f;
        if (live) r = pr.sigmoid && most > -60.0f ? sigmoid(score) : exp_of(score - most);
        const float sum = lanes_sum<L>(r);
        r = live ? r / sum : 0.0f;
        dz = r * (d - lanes_sum<L>(live ? r * d : 0.0f));
        if (pr.sigmoid) dz *= sigmoid(-score);
    } else if (pr.sigmoid) {
        dz = d * sigmoid(score) * sigmoid(-score);
    } else {
        top = -INFINITY;
        for (int c = own; c < pr.experts; c += L) top = fmaxf(top, (float)row[c]);
        top = lanes_max<L>(top);
        if (!(top > -INFINITY)) top = 0.0f;
        total = 0.0f;
        for (int c = own; c < pr.experts; c += L) total += exp_of((float)row[c] - top);
        total = lanes_sum<L>(total);
        const float p = live ? exp_of(score - top) / total : 0.0f;
        dz = p * d;
        inner = lanes_sum<L>(dz);
    }
    if (!live) dz = 0.0f;
    T *out = (T *)pr.dlogits + t * pr.lddl;
    for (int c0 = 0; c0 < pr.experts; c0 += L * V) {
        const int c = c0 + own * V;
        float g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = 0.0f;
        if (dense) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (c + j >= pr.experts) continue;
                const float z = (float)row[c + j];
                if (z > -INFINITY) g[j] = -inner * (exp_of(z - top) / total);
            }
        }
        for (int i = 0; i < pr.top; ++i) {
            const int e = __shfl(at, base + i) - c;
            const float v = __shfl(dz, base + i);
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] += e == j ? v : 0.0f;
        }
        if (there && c < pr.experts) store_row(out + c, g, pr.experts - c);
    }
}

struct Form {
    int lanes, each;
};
// 16 lanes to a token where they hold its experts with 16 each, else a wave with up to 32.
Form form_of(int64_t experts, int64_t groups, int64_t top) {
    const int64_t size = experts / groups;
    if (top <= 16 && groups <= 16) {
        const int64_t each = cdiv(size, 16 / groups);
        if (each <= 16) return {16, each <= 4 ? 4 : each <= 8 ? 8 : 16};
    }
    if (groups > 64) return {64, 0};
    const int64_t each = cdiv(size, 64 / groups);
    return {64, each <= 8 ? 8 : each <= 16 ? 16 : each <= 32 ? 32 : 0};
}

template <typename T>
hipError_t route_t(const RouteProblem &pr, hipStream_t s) {
    const Form f = form_of(pr.experts, pr.groups, pr.top);
    const int64_t blocks = cdiv(pr.tokens, 256 / f.lanes);
    if (f.lanes == 16) {
        if (f.each == 4) return launch(route_kernel<T, 16, 4>, blocks, 256, 0, s, pr);
        if (f.each == 8) return launch(route_kernel<T, 16, 8>, blocks, 256, 0, s, pr);
        return launch(route_kernel<T, 16, 16>, blocks, 256, 0, s, pr);
    }
    if (f.each == 8) return launch(route_kernel<T, 64, 8>, blocks, 256, 0, s, pr);
    if (f.each == 16) return launch(route_kernel<T, 64, 16>, blocks, 256, 0, s, pr);
    return launch(route_kernel<T, 64, 32>, blocks, 256, 0, s, pr);
}
template <typename T>
hipError_t backward_t(const RouteProblem &pr, hipStream_t s) {
    if (pr.top <= 16 && pr.experts <= 16 * 2 * vec<T>())
        return launch(route_backward_kernel<T, 16>, cdiv(pr.tokens, 16), 256, 0, s, pr);
    return launch(route_backward_kernel<T, 64>, cdiv(pr.tokens, 4), 256, 0, s, pr);
}

}  // namespace

bool route_fits(int64_t experts, int64_t groups, int64_t top) {
    return form_of(experts, groups, top).each > 0;
}

hipError_t launch_route(int dtype, const RouteProblem &pr, hipStream_t s) {
    if (pr.tokens == 0) return hipSuccess;
    if (dtype == 0) return route_t<float>(pr, s);
    return dtype == 1 ? route_t<bf16>(pr, s) : route_t<f16>(pr, s);
}
hipError_t launch_route_backward(int dtype, const RouteProblem &pr, hipStream_t s) {
    if (pr.tokens == 0) return hipSuccess;
    if (dtype == 0) return backward_t<float>(pr, s);
    return dtype == 1 ? backward_t<bf16>(pr, s) : backward_t<f16>(pr, s);
}

}  // namespace kx
