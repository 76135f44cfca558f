// route.hip - from the scores of the experts to the experts of each token and their
// weights, and the scores' gradient.
//
//   s = softmax(z) or 1 / (1 + e^-z),  c = s + bias  (c = z where nothing is added: the
//   order is the same), a group's rank = its largest c, or the sum of its two largest;
//   of the best groups the `top` largest c, ties to the lower number;
//   weights = scale s / (sum of the chosen s), or scale s.
//
// Bound by memory at best (z read once, dz written once), in fact by the vector units: the
// choice is a partial sort. L lanes (16 or 64) hold a token's choices, V each, as keys in
// which a tie goes to the lower number. Each lane sorts its V keys with a network of
// maxima and minima; then, `top` times, the largest head of the lanes is taken out. Keys:
//   kWide    float32 logits: a double 1.mantissa of the float's 32 bits, put in an order that
//            integers have, and the complement of the expert's number.
//   kNarrow  16-bit logits leave 13 bits of a float32 empty, which hold that complement.
//   kScored  c is a float32 sum of roundings: 23 bits of it as an integer, of the largest |c|,
//            and 8 for the lane and the place in it (with 64 lanes 20 or 21, and 10 or 11), so
//            that no two are the same. Where two choices that follow each other, or two groups
//            at the border, lie within the roundings of each other, float64 tells: for choices
//            each lane computes its own again and the lanes sort them (at the size below in
//            0.3 to 1.2 % of the waves, by the logits' spread), for groups the token's wave
//            chooses again.
// 65536 tokens, 8 of 256 from 4 of 8 groups, sigmoids and a bias, bf16: with wide keys for
// everything 58 us and 1550 vector instructions a wave of four tokens, so 36 to 38 and 950.
#include "layers.h"
#include "rows.h"

namespace kx {
namespace {

constexpr float kLog2e = 1.44269504088896f;
constexpr int kNumber = 20;  // bits of a key for the expert's number

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

enum { kWide, kNarrow, kScored };

// float's bits in the order that integers have.
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
constexpr int kNone = (int)0x807fffff;  // ordered(-inf) with any low bits is at most this

// (Without the canonicalising of fmax: a key is never a NaN.)
__device__ __forceinline__ double key_max(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double key_min(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ int key_max(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int key_min(int a, int b) { return a < b ? a : b; }

template <int K, int L, int V>
struct Key {  // kNarrow
    typedef int type;
    static constexpr int kMask = (1 << 13) - 1;
    static constexpr int kEmpty = INT32_MIN;
    static __device__ __forceinline__ int of(float c, int expert, int) {
        return (ordered(c) & ~kMask) | (kMask - expert);
    }
    static __device__ __forceinline__ bool live(int k) { return k > kNone; }
    static __device__ __forceinline__ int number(int k) { return kMask - (k & kMask); }
};
template <int L, int V>
struct Key<kScored, L, V> {
    typedef int type;
    static constexpr int kPlace = V <= 16 ? 4 : 5, kBits = kPlace + (L == 16 ? 4 : 6);
    static constexpr int kEmpty = INT32_MIN;
    // c times the power of two that leaves it below 2^(30 - kBits) in magnitude, or an
    // infinity. `at`: the lane, and the place in it.
    static __device__ __forceinline__ int of(float c, int, int at) {
        const float held = __builtin_amdgcn_fmed3f(c, -(float)(1 << (31 - kBits)), (float)(1 << (30 - kBits)));
        return (int)((uint32_t)(int)held << kBits) | at;
    }
    static __device__ __forceinline__ bool live(int k) { return k >= -(1 << 30); }
    static __device__ __forceinline__ int place(int k) { return k & ((1 << kPlace) - 1); }
    static __device__ __forceinline__ int lane(int k) { return (k >> kPlace) & (L - 1); }
    static __device__ __forceinline__ int choice(int k) { return k >> kBits; }
};
template <int L, int V>
struct Key<kWide, L, V> {
    typedef double type;
    static constexpr double kEmpty = 0.0;
    static __device__ __forceinline__ double of(float c, int expert, int) {
        const uint32_t o = (uint32_t)ordered(c) ^ 0x80000000u;
        const uint32_t hi = __builtin_amdgcn_alignbit(0x3ffu, o, 12);  // 0x3ff00000 | o >> 12
        const uint32_t lo = o << kNumber | (((1u << kNumber) - 1) - (uint32_t)expert);
        return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
    }
    static __device__ __forceinline__ bool live(double k) {
        const uint64_t m = (uint64_t)(((uint32_t)kNone ^ 0x80000000u) + 1) << kNumber;
        return k >= __longlong_as_double((long long)(m | 0x3ff0000000000000ull));
    }
    static __device__ __forceinline__ int number(double k) {
        return (int)(((1u << kNumber) - 1) - ((uint32_t)__double_as_longlong(k) & ((1u << kNumber) - 1)));
    }
};

// Batcher's odd-even merge sort of V keys, largest first.
template <int V, typename K>
__device__ __forceinline__ void sort_keys(K (&k)[V]) {
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
                        const K hi = key_max(k[a], k[b]), lo = key_min(k[a], k[b]);
                        k[a] = hi;
                        k[b] = lo;
                    }
                }
}

template <int CTRL>
__device__ __forceinline__ double rotated(double x) {  // within 16 lanes
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const int lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
    const int hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __longlong_as_double((long long)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo));
}
template <int CTRL>
__device__ __forceinline__ int rotated(int x) {
    return __builtin_amdgcn_mov_dpp(x, CTRL, 0xf, 0xf, true);
}
template <int L, typename K>
__device__ __forceinline__ K lanes_most(K x) {  // of keys
    x = key_max(x, rotated<0x128>(x));  // row_ror:8, 4, 2, 1
    x = key_max(x, rotated<0x124>(x));
    x = key_max(x, rotated<0x122>(x));
    x = key_max(x, rotated<0x121>(x));
    if (L == 64) {
        x = key_max(x, __shfl_xor(x, 16));
        x = key_max(x, __shfl_xor(x, 32));
    }
    return x;
}
template <int L>
__device__ __forceinline__ double lanes_max(double x) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) x = fmax(x, __shfl_xor(x, d));
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
    x = fmaxf(x, rotated<0x128>(x));
    x = fmaxf(x, rotated<0x124>(x));
    x = fmaxf(x, rotated<0x122>(x));
    x = fmaxf(x, rotated<0x121>(x));
    if (L == 64) {
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
    }
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {  // to all lanes, of one order
    x += rotated<0x128>(x);
    x += rotated<0x124>(x);
    x += rotated<0x122>(x);
    x += rotated<0x121>(x);
    if (L == 64) {
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
    }
    return x;
}
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
    for (int d = L / 2; d >= 1; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// (v_max and v_min: a NaN gives way to the other operand.)
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

// first >= second, with one more value.
template <typename F>
__device__ __forceinline__ void two_largest(F c, F &first, F &second) {
    second = larger(second, smaller(first, c));
    first = larger(first, c);
}

// x of the lane i places before, within the L lanes.
template <int L, typename F>
__device__ __forceinline__ F turned(F x, int i) {
    const int lane = threadIdx.x & 63;
    return __shfl(x, (lane & ~(L - 1)) | ((lane - i) & (L - 1)));
}

// Of every STEP-th of the 16 lanes, those before this one in the order of the keys.
template <int STEP, int I = STEP>
__device__ __forceinline__ int count_before(double key) {
    if constexpr (I < 16)
        return (int)(rotated<0x120 + I>(key) > key) + count_before<STEP, I + STEP>(key);
    else
        return 0;
}

// Of the lane's group: the sum of its one or two largest choices, and whether it is
// among the `kept` best (ties to the lower group). `first` and `second`: the lane's two
// largest (-inf: none). `least`: how far the groups that stay lie from the others.
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
        two_largest(c, a, b);
        b = larger(b, d);
    }
    const F none = -(F)INFINITY;
    // (Half of the sum, which no finite biases overflow. Infinite ranks are those of the formulas.)
    const F rank = best == 2 ? (F)0.5 * a + (b > none ? (F)0.5 * b : (F)0) : a;
    int before = 0;
    if constexpr (L == 16 && sizeof(F) == 4) {
        // (A group's lanes hold the same key.)
        const double key = Key<kWide, 16, 1>::of(rank + 0.0f, group, 0);
        if (lanes == 2)
            before = 2 * count_before<2>(key);
        else if (lanes == 4)
            before = 4 * count_before<4>(key);
        else
            before = count_before<1>(key);
    } else {
        for (int i = 1; i < L; ++i) {
            const F other = turned<L>(rank, i);
            before += (int)(other > rank) | ((int)(other == rank) & (int)(((own - i) & (L - 1)) < start));
        }
    }
    const bool keep = group < groups && before < kept * lanes;
    const F worst = lanes_max<L>(keep ? -rank : none), other = lanes_max<L>(keep || group >= groups ? none : rank);
    least = (best == 2 ? (F)2 : (F)1) * (-worst - other);
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
__device__ __forceinline__ void load_own(const T *p, const Layout &l, T none, T (&v)[V]) {
    if (l.n == V) {
        load_vec(p + l.first, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < l.n ? p[l.first + j] : none;
    }
}
// The same choice in float64 (see the top): the t-th expert in lane t. (As a function of
// its own, or with rolled loops, it took 101 to 130 registers, which are every wave's, in
// place of 90, and the size above 49 to 55 us in place of 46, before the lanes sorted.)
template <int L, int V>
__device__ __forceinline__ int choose_exactly(const float (&z)[V], const RouteProblem &pr, const Layout &l) {
    double c[V];
    double m = -INFINITY, sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) m = z[j] > m ? (double)z[j] : m;
    m = lanes_max<L>(m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        // (A NaN, or a softmax's +inf, makes the sum a NaN: nothing to choose by, as in route_token.)
        const bool out = z[j] == -INFINITY;
        c[j] = out ? 0.0 : pr.sigmoid ? 1.0 / (1.0 + exp(-(double)z[j])) : exp((double)z[j] - m);
        sum += c[j];
    }
    sum = lanes_sum<L>(sum);
    double first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (!pr.sigmoid) c[j] /= sum;
        if (pr.bias && j < l.n) c[j] += (double)pr.bias[l.first + j];
        if (!(z[j] > -INFINITY) || !(c[j] > -INFINITY)) c[j] = -INFINITY;
        two_largest(c[j], first, second);
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

// The lane's candidate (`mine`, the t-th in lane t, -1: none) by its choice in float64: the
// lanes up to `last` in order, ties to the lower number.
template <int L, int V>
__device__ __forceinline__ int resolve(const float (&z)[V], const RouteProblem &pr, float score, int mine,
                                       int last) {
    const int own = threadIdx.x & (L - 1);
    double c = -INFINITY;
    if (pr.sigmoid) {
        c = 1.0 / (1.0 + exp(-(double)score));
    } else {
        double m = -INFINITY, sum = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) m = z[j] > m ? (double)z[j] : m;
        m = lanes_max<L>(m);
#pragma unroll
        for (int j = 0; j < V; ++j) sum += z[j] > -INFINITY ? exp((double)z[j] - m) : 0.0;
        c = exp((double)score - m) / lanes_sum<L>(sum);
    }
    if (pr.bias && mine >= 0) c += (double)pr.bias[mine];
    if (mine < 0) c = -INFINITY;
    for (int pass = 0; pass <= last; ++pass) {  // odd-even transposition
        const int with = ((own ^ pass) & 1) ? own - 1 : own + 1;
        const int at = (threadIdx.x & 63 & ~(L - 1)) + (with & (L - 1));
        const double other = __shfl(c, at);
        const int number = __shfl(mine, at);
        const bool before = other > c || (other == c && (uint32_t)number < (uint32_t)mine);
        if (with >= 0 && with <= last && own <= last && (with > own) == before) {
            c = other;
            mine = number;
        }
    }
    return mine;
}

// The `top` largest keys of the lanes that `keep` theirs, one after another: the t-th in lane
// t. D keys of a lane can come up.
template <int L, int D, typename Keys>
__device__ __forceinline__ void take(Keys &key, bool keep, int top, typename Keys::type &won) {
    const int own = threadIdx.x & (L - 1);
    sort_keys(key.k);
    key.k[0] = keep ? key.k[0] : Keys::kEmpty;
    for (int i = 0; i < top; ++i) {
        const auto best = lanes_most<L>(key.k[0]);
        const bool had = keep & (key.k[0] == best);
#pragma unroll
        for (int j = 0; j + 1 < D; ++j) key.k[j] = had ? key.k[j + 1] : key.k[j];
        if (D == Keys::kCount) key.k[D - 1] = had ? Keys::kEmpty : key.k[D - 1];
        won = own == i ? best : won;
    }
}
template <int K, int L, int V>
struct Keys : Key<K, L, V> {
    static constexpr int kCount = V;
    typename Key<K, L, V>::type k[V];
};

// The choice for the token of the L lanes, and its weights.
template <typename T, int L, int V, int K, int B>
__device__ __forceinline__ void route_token(const RouteProblem &pr, const Layout &l, const float (&bias)[B],
                                            const float (&z)[V], bool there, const T *row, int64_t t) {
    const int own = threadIdx.x & (L - 1);
    float c[V];
    // The largest and the sum of e^(z - largest) where they are needed.
    float top = -INFINITY, total = 1.0f;
    if (K == kScored || (!pr.sigmoid && !pr.renormalize)) {
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
    if (K == kScored) {
        const float each = 1.0f / total;
        const bool sound = total == total;
        if (pr.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = sigmoid(z[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] *= each;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] += bias[j];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            most = fmaxf(most, fabsf(c[j]));
            // A NaN, or -inf. (The bias holds no NaN, and the sum none but for a NaN or an
            // infinite logit, which leave a softmax nothing to choose by.)
            const bool out = __builtin_amdgcn_classf(z[j], 0x007);
            c[j] = (out | !sound) ? -INFINITY : c[j];
        }
        most = lanes_max<L>(most);
        if (most == INFINITY) {  // a bias that takes experts out: of the others
            most = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) most = fmaxf(most, fabsf(c[j]) < INFINITY ? fabsf(c[j]) : 0.0f);
            most = lanes_max<L>(most);
        }
        // The scores' own errors (the argument's rounding times s'(z) |z|, the hardware's
        // 2^x and reciprocal; the softmax's sum), and that of adding the bias.
        const float s = pr.sigmoid ? sigmoid(top) : each;
        const float slope = pr.sigmoid ? (top > -1.0f ? 0.25f : s * -top) : 0.0f;
        far = 2.0f * ((pr.sigmoid ? 0x1p-21f : 0x1p-18f) * s + 0x1p-23f * slope + 0x1p-24f * most);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = z[j] == z[j] ? z[j] + 0.0f : -INFINITY;  // not a NaN, nor -0
    }
    bool again = false;
    bool keep = true;
    if (pr.groups > 1) {
        float first = -INFINITY, second = -INFINITY, least;
#pragma unroll
        for (int j = 0; j < V; ++j) two_largest(c[j], first, second);
        keep = group_kept<L, float>(first, second, pr.groups, pr.kept, pr.best, l.lanes, l.group, least);
        again = K == kScored && least <= 2.0f * far + 0x1p-22f * most;
    }
    float unit = 1.0f;  // the power of two that makes integers of c
    if constexpr (K == kScored) {
        const int e = __builtin_amdgcn_frexp_expf(most);
        const int up = 30 - Key<K, L, V>::kBits - e;
        unit = ldexpf(1.0f, up < 120 ? up : 120);
    }
    Keys<K, L, V> key;
#pragma unroll
    for (int j = 0; j < V; ++j)
        key.k[j] = key.of(K == kScored ? c[j] * unit : c[j], l.first + j, own * (V <= 16 ? 16 : 32) + j);
    typename Key<K, L, V>::type best = Keys<K, L, V>::kEmpty;
    // One more than is returned, where choices may have to be told apart. Of a lane's keys
    // only as many can come up as are asked for, and the one after them.
    const int asked = K == kScored && pr.top < L ? pr.top + 1 : pr.top;
    if (V > 10 && asked <= 9)
        take<L, V < 10 ? V : 10>(key, keep, asked, best);
    else
        take<L, V>(key, keep, asked, best);
    int mine = -1;
    if constexpr (K == kScored) {
        const int first = __shfl(l.first, (threadIdx.x & 63 & ~(L - 1)) + key.lane(best));
        if (own < asked && key.live(best)) mine = first + key.place(best);
        // Does any of them come near the one after it? (In units of the keys' choices, to
        // which each is cut off.)
        const int next = lanes_most<L>(keep ? key.k[0] : key.kEmpty);
        int after = __shfl_down((int)best, 1, L);
        after = own == asked - 1 ? next : after;
        const bool near = mine >= 0 && key.live(after) &&
                          (float)(key.choice(best) - key.choice(after)) <= far * unit + 2.0f;
        const int last = asked - 1;
        // The last asked for is not returned, unless there was no lane for one more.
        const bool past = near && own == last;
        const bool border = asked == pr.top ? past : __shfl((int)near, (threadIdx.x & 63 & ~(L - 1)) + last - 1) && past;
        if (__any(again || border))
            mine = choose_exactly<L, V>(z, pr, l);
        else if (__any(near && own < last))
            mine = resolve<L, V>(z, pr, mine >= 0 ? (float)row[mine] : -INFINITY, mine, last);
        if (own >= pr.top) mine = -1;
    } else if (own < pr.top && key.live(best)) {
        mine = key.number(best);
    }

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

template <typename T, int L, int V, int K>
__global__ __launch_bounds__(256) void route_kernel(RouteProblem pr) {
    const Layout l = layout_of<L, V>(pr.experts, pr.groups);
    float bias[K == kScored ? V : 1];
    if constexpr (K == kScored) {
#pragma unroll
        for (int j = 0; j < V; ++j) bias[j] = 0.0f;
        if (pr.bias) load_own<float, V>(pr.bias, l, 0.0f, bias);
#pragma unroll
        for (int j = 0; j < V; ++j) bias[j] = bias[j] == bias[j] ? bias[j] : -INFINITY;
    }
    int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool there = t < pr.tokens;
    if (!there) t = pr.tokens - 1;  // its lanes go along, and store nothing
    const T *row = (const T *)pr.logits + t * pr.ld;
    T raw[V];
    load_own<T, V>(row, l, (T)(-INFINITY), raw);
    float z[V];
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = (float)raw[j];
    route_token<T, L, V, K>(pr, l, bias, z, there, row, t);
}

// With r the chosen's shares (their sum 1) and d = scale dweights:
//   renormalised  dz = r (d - sum r d), for sigmoids times 1 - s
//   sigmoid       dz = s (1 - s) d
//   softmax       dz = p (d - sum p d), of the others -p sum p d
// One row for L lanes: lane i has the i-th chosen and puts its dz into the row in LDS, which the
// lanes then store, V places each. (65536 tokens, 8 of 256, bf16: 15.9 us, 4.6 TB/s with every logit's
// line read; every lane looking through the chosen for its places 18.2, 630 vector
// instructions a wave.)
template <typename T, int L>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteProblem pr) {
    constexpr int V = vec<T>();
    extern __shared__ __align__(16) float rows[];  // 256 / L, each a whole number of V
    float *sums = rows + threadIdx.x / L * ((pr.experts + V - 1) / V * V);
    const int own = threadIdx.x & (L - 1), base = threadIdx.x & 63 & ~(L - 1);
    int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool there = t < pr.tokens;
    if (!there) t = pr.tokens - 1;
    for (int c = own * V; c < pr.experts; c += L * V)
#pragma unroll
        for (int j = 0; j < V; ++j) sums[c + j] = 0.0f;
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
    // Is one chosen twice? (Not by route.) Then its first lane adds them.
    bool first = live;
    in_order();
    if (live) ((int *)sums)[at] = own;
    in_order();
    if (__any(live && ((int *)sums)[at] != own)) {
        for (int i = 0; i < pr.top; ++i) {
            const int e = __shfl(at, base + i);
            const float v = __shfl(dz, base + i);
            if (live && e == at && i < own) first = false;
            if (live && e == at && i > own) dz += v;
        }
    }
    in_order();
    if (first) sums[at] = dz;
    in_order();
    T *out = (T *)pr.dlogits + t * pr.lddl;
    for (int c0 = 0; c0 < pr.experts; c0 += L * V) {
        const int c = c0 + own * V;
        float g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = c < pr.experts ? sums[c + j] : 0.0f;
        if (dense) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (c + j >= pr.experts) continue;
                const float z = (float)row[c + j];
                if (z > -INFINITY) g[j] -= inner * (exp_of(z - top) / total);
            }
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

template <typename T, int K>
hipError_t route_k(const RouteProblem &pr, hipStream_t s) {
    const Form f = form_of(pr.experts, pr.groups, pr.top);
    const int64_t blocks = cdiv(pr.tokens, 256 / f.lanes);
    if (f.lanes == 16) {
        if (f.each == 4) return launch(route_kernel<T, 16, 4, K>, blocks, 256, 0, s, pr);
        if (f.each == 8) return launch(route_kernel<T, 16, 8, K>, blocks, 256, 0, s, pr);
        return launch(route_kernel<T, 16, 16, K>, blocks, 256, 0, s, pr);
    }
    if (f.each == 8) return launch(route_kernel<T, 64, 8, K>, blocks, 256, 0, s, pr);
    if (f.each == 16) return launch(route_kernel<T, 64, 16, K>, blocks, 256, 0, s, pr);
    return launch(route_kernel<T, 64, 32, K>, blocks, 256, 0, s, pr);
}
template <typename T>
hipError_t route_t(const RouteProblem &pr, hipStream_t s) {
    if (pr.bias || (pr.groups > 1 && pr.best == 2)) return route_k<T, kScored>(pr, s);
    return route_k<T, sizeof(T) == 4 ? kWide : kNarrow>(pr, s);
}
template <typename T>
hipError_t backward_t(const RouteProblem &pr, hipStream_t s) {
    const size_t row = (size_t)cdiv(pr.experts, vec<T>()) * vec<T>() * sizeof(float);  // at most 8 KB
    if (pr.top <= 16 && pr.experts <= 16 * 2 * vec<T>())
        return launch(route_backward_kernel<T, 16>, cdiv(pr.tokens, 16), 256, 16 * row, s, pr);
    return launch(route_backward_kernel<T, 64>, cdiv(pr.tokens, 4), 256, 4 * row, s, pr);
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
