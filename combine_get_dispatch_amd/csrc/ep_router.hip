// ep_router.hip -- the router: experts and weights of every token from the
// gate's logits, and the weights' gradient in them.
//
// A token is L lanes of a wave (16, four tokens to a wave, or 64), each with P
// neighbouring experts; a group of experts is a power of two of neighbouring
// lanes. What is chosen is ordered by one 64-bit number per expert: its c_e (a
// logit, or with a bias the sum in 64 bits, since neighbouring 32-bit sums tie or
// change places by a rounding) with the expert's index in the ten low bits of
// the mantissa, so that the lower index wins a tie and one maximum over the
// lanes finds value and index. Every lane sorts its own numbers once; each of
// the k choices is then the maximum of the lanes' first ones, and the lane that
// had it moves up.
//
// What bounds it, on MI355X: few tokens a launch and the chain of k maxima (128
// tokens x 256 experts, k = 8: 3.7 us, an empty kernel 2.3); many tokens chains of
// lane exchanges and vector instructions (issued in 60% of the SIMDs' cycles, waves
// waiting in 49% of theirs), which for 64-bit numbers of every expert took twice the
// time of the candidates' form (k_route_many). Memory would allow 2.5 us for the 18
// MB of 16384 tokens x 256 experts in fp32. What the candidates' form does not take
// (more than 256 experts or 8 choices, softmax with a bias), 16384 tokens in fp32: 256
// experts, softmax with a bias, k = 8, 21.4 us, sigmoid with one, k = 10, 26.4; 384
// experts with a bias, k = 8, 34.4, in groups 37.8; 512 experts, k = 10, 26.7 (2.5,
// 2.6, 3.7 and 5.0 by memory).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ep.h"
#include "ep_groups.h"

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxTokens = 1 << 24;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *w;
    int T, E, k, G, kept, top;
    int gs, lg, lg_log;  // experts and lanes per group, and the lanes' logarithm
    int exact;       // c_e is a score in 64 bits, else the logit
    int sigmoid, renorm;
    int vector, quads;  // logits come in vectors; a lane's experts start at a multiple of four
    float scale;
};

// ---------------------------------------------------------------------------
// over a token's lanes
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// `op` of a value with that of the lane 1, 2, 4, 8, 16, 32 away (STEP 0 to 5;
// a mirror image from step 2 on, where the lanes nearer already hold the same)
template <int STEP, class F>
__device__ __forceinline__ double step(double v, F op) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    u32x2 a;
    if constexpr (STEP < 4) {
        constexpr int CTRL = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
        a = u32x2{from_lane<CTRL>(w.x), from_lane<CTRL>(w.y)};
        return op(v, __builtin_bit_cast(double, a));
    } else {
        u32x2 lo, hi;
        if constexpr (STEP == 4) {
            lo = __builtin_amdgcn_permlane16_swap(w.x, w.x, false, false);
            hi = __builtin_amdgcn_permlane16_swap(w.y, w.y, false, false);
        } else {
            lo = __builtin_amdgcn_permlane32_swap(w.x, w.x, false, false);
            hi = __builtin_amdgcn_permlane32_swap(w.y, w.y, false, false);
        }
        return op(__builtin_bit_cast(double, (u32x2{lo.x, hi.x})), __builtin_bit_cast(double, (u32x2{lo.y, hi.y})));
    }
}
template <int STEP, class F>
__device__ __forceinline__ float step(float v, F op) {
    const uint32_t w = __float_as_uint(v);
    if constexpr (STEP < 4) {
        constexpr int CTRL = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
        return op(v, __uint_as_float(from_lane<CTRL>(w)));
    } else {
        const u32x2 s = STEP == 4 ? u32x2(__builtin_amdgcn_permlane16_swap(w, w, false, false))
                                  : u32x2(__builtin_amdgcn_permlane32_swap(w, w, false, false));
        return op(__uint_as_float(s.x), __uint_as_float(s.y));
    }
}

// over all L lanes of a token, in every lane
template <int L, class T, class F>
__device__ __forceinline__ T all(T v, F op) {
    v = step<0>(v, op);
    v = step<1>(v, op);
    v = step<2>(v, op);
    v = step<3>(v, op);
    if constexpr (L == 64) {
        v = step<4>(v, op);
        v = step<5>(v, op);
    }
    return v;
}

struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ __forceinline__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
};
struct Sum {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
    __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};

// ---------------------------------------------------------------------------
// arithmetic
// ---------------------------------------------------------------------------

// exp(x) for x <= 0 (below -745: 0) in 64 bits, to some 2^-47: x = n ln 2 + r by
// ln 2 in two parts, Taylor's series of exp(r) to the eleventh power (|r| <= 0.35).
__device__ __forceinline__ double exp64(double x) {
    x = __builtin_fmax(x, -800.0);
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0x1.62e42fefa0000p-1, x);
    r = __builtin_fma(n, -0x1.cf79abc9e3b39p-40, r);
    double p = 1.0 / 39916800;
    p = __builtin_fma(p, r, 1.0 / 3628800);
    p = __builtin_fma(p, r, 1.0 / 362880);
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// 1 / d, d a normal number well inside the range: the hardware's estimate and two of Newton's steps
__device__ __forceinline__ double recip64(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

__device__ __forceinline__ double sigmoid64(double l) {
    const double e = exp64(-__builtin_fabs(l)), r = recip64(1.0 + e);
    return l >= 0 ? r : e * r;
}

// exp(x) for x <= 0 in 32 bits: 2^t with t = x log2 e rounded, and what the
// rounding left out; below 2^-126 it may be 0
__device__ __forceinline__ float exp32(float x) {
    constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596299112661746887e-8f;
    const float t = x * kLog2e, y = __builtin_amdgcn_exp2f(t);
    const float r = fmaf(x, kLog2e, -t) + x * kRest;
    return t > -128.0f ? fmaf(y, r * 0.693147180559945309f, y) : y;
}

// sigmoid(l) = exp(min(l, 0)) over this
__device__ __forceinline__ float sigmoid_den(float l) { return 1.0f + exp32(-fabsf(l)); }

// ---------------------------------------------------------------------------
// what orders experts
// ---------------------------------------------------------------------------

constexpr uint64_t kIndexBits = 1023;

__device__ __forceinline__ double minus_inf() { return -__builtin_inf(); }

// c with the index e in its low bits: of two that agree but there the one of the
// lower index is larger. -infinity (not to be chosen) stays.
__device__ __forceinline__ double with_index(double c, int e) {
    const double v = __builtin_fmin(c, 1.7976931348623157e308) + 0.0;  // -0 is 0
    const uint64_t low = v < 0 ? (uint64_t)e : kIndexBits - (uint64_t)e;
    const uint64_t b = (__builtin_bit_cast(uint64_t, v) & ~kIndexBits) | low;
    return c > minus_inf() ? __builtin_bit_cast(double, b) : minus_inf();
}
__device__ __forceinline__ int index_of(double v) {
    const int low = (int)(__builtin_bit_cast(uint64_t, v) & kIndexBits);
    return v < 0 ? low : (int)kIndexBits - low;
}
__device__ __forceinline__ double value_of(double v) {
    return v > minus_inf() ? __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, v) & ~kIndexBits) : minus_inf();
}

template <int P>
__device__ __forceinline__ void sort_down(double (&v)[P]) {  // Batcher's odd-even merge sort
#pragma unroll
    for (int p = 1; p < P; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < P; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < P && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const double a = v[i + j], b = v[i + j + q];
                        v[i + j] = __builtin_fmax(a, b);
                        v[i + j + q] = __builtin_fmin(a, b);
                    }
}

// the k largest of the lanes' sorted numbers, the j-th in lane j of the token
template <int L, int Q, int P>
__device__ __forceinline__ double choose(double (&v)[P], int k, int sub) {
    double mine = minus_inf();
    for (int j = 0; j < k; ++j) {
        const double m = all<L>(v[0], Max());
        const bool won = v[0] == m;
#pragma unroll
        for (int p = 0; p < Q; ++p) v[p] = won ? (p + 1 < Q ? v[p + 1] : minus_inf()) : v[p];
        mine = sub == j ? m : mine;
    }
    return mine;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t at) {
    if (BF16) return __uint_as_float((uint32_t)((const uint16_t *)p)[at] << 16);
    return ((const float *)p)[at];
}

// P neighbouring logits; their place is a multiple of P (and the row's start too)
template <bool BF16, int P>
__device__ __forceinline__ void load_logits(const void *p, int64_t at, float (&l)[P]) {
    if constexpr (BF16) {
        uint32_t w[P / 2 > 0 ? P / 2 : 1];
        const uint16_t *s = (const uint16_t *)p + at;
        if constexpr (P >= 8) {
#pragma unroll
            for (int i = 0; i < P / 8; ++i) {
                const u32x4 v = *(const u32x4 *)(s + 8 * i);
#pragma unroll
                for (int c = 0; c < 4; ++c) w[4 * i + c] = v[c];
            }
        } else if constexpr (P == 4) {
            const u32x2 v = *(const u32x2 *)s;
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (P == 2) {
            w[0] = *(const uint32_t *)s;
        } else {
            w[0] = *s;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) l[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
        const float *s = (const float *)p + at;
        if constexpr (P >= 4) {
#pragma unroll
            for (int i = 0; i < P / 4; ++i) {
                const f32x4 v = *(const f32x4 *)(s + 4 * i);
#pragma unroll
                for (int c = 0; c < 4; ++c) l[4 * i + c] = v[c];
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) l[i] = s[i];
        }
    }
}

// ---------------------------------------------------------------------------
// route
// ---------------------------------------------------------------------------

// Whether a lane's group stays, one and two its two largest numbers (with indices), in all its lanes.
template <int L>
__device__ __forceinline__ bool group_kept(const RouteArgs &a, double one, double two, float top, int group) {
    double value = value_of(one);
    if (a.top == 2) {
        const double second = value_of(two);
        if (a.exact) {
            value += two > minus_inf() ? second : 0.0;
        } else {  // the scores of the two logits (softmax's without its sum)
            auto score = [&](double l) __attribute__((always_inline)) {
                const float x = (float)l;  // (the largest numbers stand for infinity)
                return a.sigmoid ? sigmoid64(x) : x == top ? 1.0 : exp64((double)x - (double)top);
            };
            value = one > minus_inf() ? score(value) + (two > minus_inf() ? score(second) : 0.0) : minus_inf();
        }
    }
    int ahead = 0;
    for (int g = 0; g < a.G; ++g) {
        const double other = __shfl(value, g * a.lg, L);
        ahead += other > value || (other == value && g < group);
    }
    return ahead < a.kept;
}

// Weights of the chosen experts (open: this lane has one, of logit x): divided by their sum, or of all scores' (total, over
// top's exponential, for softmax).
template <int L>
__device__ __forceinline__ float weight_of(const RouteArgs &a, bool open, float x, float top, float total) {
    float w;
    if (a.renorm) {  // over the largest of the chosen logits, so that none underflows all
        const float y = a.sigmoid ? fminf(x, 0.0f) : x;
        const float m = all<L>(open ? y : -INFINITY, Max());
        w = open ? exp32(y == m ? 0.0f : y - m) : 0.0f;
        if (a.sigmoid && open) w /= sigmoid_den(x);
        const float sum = all<L>(w, Sum());
        w = w / sum * a.scale;
    } else if (a.sigmoid) {
        w = exp32(fminf(x, 0.0f)) / sigmoid_den(x) * a.scale;
    } else {
        w = exp32(x == top ? 0.0f : x - top) / total * a.scale;
    }
    return open ? w : 0.0f;
}

// softmax's sum over a token's experts, over the exponential of their largest logit
template <int L, int P>
__device__ __forceinline__ float sum_of(const float (&l)[P], int mine, float top) {
    float total = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) total += p < mine ? exp32(l[p] == top ? 0.0f : l[p] - top) : 0.0f;
    return all<L>(total, Sum());
}

template <int L, int P, bool BF16>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
    const int lane = threadIdx.x & 63, sub = lane % L;
    const int group = sub / a.lg, first = (sub % a.lg) * P, e0 = group * a.gs + first;
    const int mine = group < a.G ? min(max(a.gs - first, 0), P) : 0;  // experts of this lane
    const bool whole = a.vector && mine == P;
    float bias[P];
#pragma unroll
    for (int p = 0; p < P; ++p) bias[p] = a.bias && p < mine ? a.bias[e0 + p] : 0.0f;
    const int per = 64 / L;
    const int64_t waves = (int64_t)gridDim.x * (blockDim.x / 64);
    for (int64_t at = (int64_t)blockIdx.x * (blockDim.x / 64) + threadIdx.x / 64; at * per < a.T; at += waves) {
        const int64_t token = at * per + lane / L;
        const bool on = token < a.T;
        const int64_t row = (on ? token : (int64_t)a.T - 1) * a.E;  // (a wave's last tokens may be none: the last again)
        float l[P];
        if (whole) {
            load_logits<BF16, P>(a.logits, row + e0, l);
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) l[p] = p < mine ? load_logit<BF16>(a.logits, row + e0 + p) : -INFINITY;
        }
        bool bad = false;
        float top = -INFINITY;  // (fmaxf leaves NaN out)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            bad |= l[p] != l[p];
            top = fmaxf(top, l[p]);
        }
        // any NaN logit of the token?
        const uint64_t nans = __ballot(bad);
        const bool poisoned = (L == 64 ? nans : nans >> (lane & 48) & 0xFFFF) != 0;
        double v[P];
        float total = 1.0f;  // softmax's sum, where the weights or the scores need it
        const bool sums = !a.sigmoid && !a.renorm;
        if (!a.sigmoid && (a.exact || a.G > 1 || sums)) top = all<L>(top, Max());
        if (!a.exact) {
#pragma unroll
            for (int p = 0; p < P; ++p) v[p] = l[p];
            if (sums) total = sum_of<L>(l, mine, top);
        } else if (a.sigmoid) {
#pragma unroll
            for (int p = 0; p < P; ++p) v[p] = sigmoid64(l[p]) + (double)bias[p];
        } else {
            double sum = 0.0;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                v[p] = l[p] == top ? 1.0 : exp64((double)l[p] - (double)top);
                sum += p < mine ? v[p] : 0.0;
            }
            sum = all<L>(sum, Sum());
            total = (float)sum;
            const double r = recip64(sum);
#pragma unroll
            for (int p = 0; p < P; ++p) v[p] = fma(v[p], r, (double)bias[p]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p)  // (comparisons that NaN fails)
            v[p] = p < mine && l[p] > -INFINITY && v[p] > minus_inf() ? with_index(v[p], e0 + p) : minus_inf();
        if (a.G > 1) {
            double one = v[0], two = minus_inf();
#pragma unroll
            for (int p = 1; p < P; ++p) {
                two = __builtin_fmax(two, __builtin_fmin(one, v[p]));
                one = __builtin_fmax(one, v[p]);
            }
            // the two largest of both sides: the larger first, and the smaller of the firsts or either second
            auto merge = [&](auto s) __attribute__((always_inline)) {
                constexpr int S = decltype(s)::value;
                const double low = step<S>(one, [](double x, double y) { return __builtin_fmin(x, y); });
                two = __builtin_fmax(low, step<S>(two, Max()));
                one = step<S>(one, Max());
            };
            if (a.lg > 1) merge(std::integral_constant<int, 0>());
            if (a.lg > 2) merge(std::integral_constant<int, 1>());
            if (a.lg > 4) merge(std::integral_constant<int, 2>());
            if (a.lg > 8) merge(std::integral_constant<int, 3>());
            if constexpr (L == 64) {
                if (a.lg > 16) merge(std::integral_constant<int, 4>());
                if (a.lg > 32) merge(std::integral_constant<int, 5>());
            }
            if (!group_kept<L>(a, one, two, top, group)) {
#pragma unroll
                for (int p = 0; p < P; ++p) v[p] = minus_inf();
            }
        }
        sort_down(v);
        const double won = a.k <= 8 ? choose<L, (P < 8 ? P : 8)>(v, a.k, sub) : choose<L, P>(v, a.k, sub);
        const bool open = sub < a.k && won > minus_inf();
        const int e = open ? index_of(won) : 0;
        const float x = open ? load_logit<BF16>(a.logits, row + e) : -INFINITY;
        float w = weight_of<L>(a, open, x, top, total);
        if (poisoned) w = __builtin_nanf("");
        if (on && sub < a.k) {
            a.idx[token * a.k + sub] = open ? e : -1;
            a.w[token * a.k + sub] = w;
        }
    }
}

// Numbers that are compared as integers as floats are: the largest of a token's
// lanes is then one instruction a step.
__device__ __forceinline__ int ordered(float f) {
    const int b = __float_as_int(f);
    return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_ordered(int b) { return __int_as_float(b ^ (b >> 31 & 0x7FFFFFFF)); }
template <int CTRL>
__device__ __forceinline__ int lane_max(int v) {
    return max(v, (int)from_lane<CTRL>((uint32_t)v));
}
__device__ __forceinline__ int max16(int v) {
    return lane_max<0x140>(lane_max<0x141>(lane_max<0x4E>(lane_max<0xB1>(v))));
}

// 16 lanes' numbers in falling order: of sorted runs of 1, 2, 4 and 8 lanes the
// larger halves against the other run's mirror image, then within the halves.
template <int CTRL>
__device__ __forceinline__ double other(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, (u32x2{from_lane<CTRL>(w.x), from_lane<CTRL>(w.y)}));
}
__device__ __forceinline__ double pick(double a, double b, bool larger) {
    const double most = __builtin_fmax(a, b), least = __builtin_fmin(a, b);
    return larger ? most : least;
}
__device__ __forceinline__ double sort16(double v, int sub) {
    constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror4 = 0x1B, kMirror8 = 0x141, kMirror16 = 0x140;
    const bool b0 = !(sub & 1), b1 = !(sub & 2), b2 = !(sub & 4), b3 = !(sub & 8);
    v = pick(v, other<kXor1>(v), b0);
    v = pick(v, other<kMirror4>(v), b1);
    v = pick(v, other<kXor1>(v), b0);
    v = pick(v, other<kMirror8>(v), b2);
    v = pick(v, other<kXor2>(v), b1);
    v = pick(v, other<kXor1>(v), b0);
    v = pick(v, other<kMirror16>(v), b3);
    v = pick(v, other<kMirror8>(other<kMirror4>(v)), b2);  // four lanes away
    v = pick(v, other<kXor2>(v), b1);
    return pick(v, other<kXor1>(v), b0);
}

// The same for many tokens: 16 lanes a token, k <= 8 of at most 256 experts, no
// bias with softmax. 64-bit numbers only for candidates: by c_e in 32 bits, off
// by little, every lane finds its two largest, the k-th largest of all lanes' two
// bounds the k-th largest of all from below, and what may reach it, some 8 to 12
// experts (more where many logits are equal), goes to a lane each, 16 at a time,
// to be ordered by the exact numbers. Groups are ordered by 32 bits where those
// decide, else exactly. 16384 tokens x 256 experts in fp32, k = 8: softmax 8.9 us
// (12.7 by k_route), in groups 9.8; sigmoid in groups with a bias 9.0 where 32 bits
// decide every token's groups, 10.5 to 13.3 with one to three tokens where they do not
// (one in some 15000 of normal logits; their waves end last), 22.4 by k_route. With
// biases of 1000 and -1000 by turns, one token in 200 undecided, 18.1.
__host__ __device__ constexpr int place(int e) { return e + e / 16 * 4; }

template <int P, bool BF16>
__global__ __launch_bounds__(256) void k_route_many(RouteArgs a) {
    constexpr int L = 16, kTokens = 256 / L, kRow = L * P, kVec = BF16 ? 8 : 4;
    constexpr float kMost = 3.402823466e38f;
    // logits and biases, four words left out after 16: lanes that read 16 neighbours each then fall on different banks
    __shared__ alignas(16) float rows[kTokens][place(kRow)], biases[place(kRow)];
    __shared__ uint8_t found[kTokens][kRow];  // candidates
    const int lane = threadIdx.x & 63, sub = lane % L, slot = threadIdx.x / L;
    const int group = sub >> a.lg_log, first = (sub & (a.lg - 1)) * P, e0 = group * a.gs + first;
    const int mine = group < a.G ? min(max(a.gs - first, 0), P) : 0;
    const int64_t token = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
    const bool on = token < a.T;
    const int64_t row = (on ? token : (int64_t)a.T - 1) * a.E;
    // neighbouring lanes read neighbouring logits; by way of LDS every lane gets its own
    if (a.vector) {
        float v[P / kVec > 0 ? P / kVec : 1][kVec];
#pragma unroll
        for (int i = 0; i * kVec < P; ++i) {
            const int e = (i * L + sub) * kVec;
            if (e < a.E) load_logits<BF16, kVec>(a.logits, row + e, v[i]);
        }
#pragma unroll
        for (int i = 0; i * kVec < P; ++i) {
            const int e = (i * L + sub) * kVec;
            if (e < a.E)
#pragma unroll
                for (int q = 0; q < kVec; q += 4) *(f32x4 *)&rows[slot][place(e + q)] = f32x4{v[i][q], v[i][q + 1], v[i][q + 2], v[i][q + 3]};
        }
    } else {
        for (int e = sub; e < a.E; e += L) rows[slot][place(e)] = load_logit<BF16>(a.logits, row + e);
    }
    if (a.bias && (int)threadIdx.x < a.E) biases[place(threadIdx.x)] = a.bias[threadIdx.x];
    __syncthreads();
    float l[P], c[P];
    if (P >= 4 && a.quads && mine == P) {
#pragma unroll
        for (int p = 0; p < P; p += 4) {
            const f32x4 v = *(const f32x4 *)&rows[slot][place(e0 + p)];
            const f32x4 b = a.bias ? *(const f32x4 *)&biases[place(e0 + p)] : f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (p + q < P) l[p + q] = v[q], c[p + q] = b[q];
        }
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            l[p] = p < mine ? rows[slot][place(e0 + p)] : -INFINITY;
            c[p] = a.bias && p < mine ? biases[place(e0 + p)] : 0.0f;
        }
    }
    bool bad = false;
    float top = -INFINITY;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        bad |= l[p] != l[p];
        top = fmaxf(top, l[p]);
    }
    const bool poisoned = (__ballot(bad) >> (lane & 48) & 0xFFFF) != 0;
    top = of_ordered(max16(ordered(top)));
    const float total = !a.sigmoid && !a.renorm ? sum_of<L>(l, mine, top) : 1.0f;
    float one = -INFINITY, two = -INFINITY;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        // within 2^-22 of the score, and the sum's rounding (NaN: not open)
        float v = l[p];
        if (a.exact) v = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[p] * -1.44269504f)) + c[p];
        c[p] = l[p] > -INFINITY && v > -INFINITY ? v : -INFINITY;
        two = __builtin_amdgcn_fmed3f(one, two, c[p]);
        one = __builtin_amdgcn_fmed3f(one, c[p], INFINITY);
    }
    // exact number of expert e, -infinity if it is not open
    auto number = [&](int e, bool in) __attribute__((always_inline)) {
        const float x = in ? rows[slot][place(e)] : -INFINITY;
        double v = x;
        if (a.exact) v = sigmoid64(x) + (double)biases[place(e)];
        return x > -INFINITY && v > minus_inf() ? with_index(v, e) : minus_inf();
    };
    if (a.G > 1) {
        float g1 = one, g2 = two;
        auto merge = [&](auto s) __attribute__((always_inline)) {
            constexpr int S = decltype(s)::value;
            const float low = step<S>(g1, [](float x, float y) { return fminf(x, y); });
            g2 = fmaxf(low, step<S>(g2, Max()));
            g1 = step<S>(g1, Max());
        };
        if (a.lg > 1) merge(std::integral_constant<int, 0>());
        if (a.lg > 2) merge(std::integral_constant<int, 1>());
        if (a.lg > 4) merge(std::integral_constant<int, 2>());
        // The group's value and what 32 bits may be off of it. With a bias, each score: 2^-22; both numbers, their sum and the
        // bounds below: a rounding each, 2^-24 of what was added, by its size, since biases of opposite signs leave a small sum.
        // Without a bias a largest logit is exact; the sum of two scores is off by 9 roundings at most (exponential 3, quotient
        // and denominator 4, sum, bounds), softmax's by its logits' differences' too, 2^-24 of a difference, by which the
        // exponential grows. Scores that underflow are never told apart.
        float value = g1, off = 0.0f;
        if (a.exact) {
            const float more = a.top == 2 && g2 > -INFINITY ? g2 : 0.0f;
            value = g1 > -INFINITY ? fminf(fmaxf(g1 + more, -kMost), kMost) : -INFINITY;  // (beyond the range: all the same)
            off = 0x1p-21f + 0x1.9p-23f * fabsf(g1) + 0x1.9p-23f * fabsf(more);
        } else if (a.top == 2) {
            auto score = [&](float x) __attribute__((always_inline)) {
                if (a.sigmoid) return exp32(fminf(x, 0.0f)) / sigmoid_den(x);
                const float far = x == top ? 0.0f : x - top, y = exp32(far);
                off = fmaf(y, fminf(-far, 128.0f), off);
                return y;
            };
            value = g1 > -INFINITY ? score(g1) + (g2 > -INFINITY ? score(g2) : 0.0f) : -INFINITY;
            off = 0x1p-24f * off + 0x1.4p-21f * value + 0x1p-100f;
        }
        const int mark = ordered(value);
        int left = mark, last = 0;
        for (int j = 0; j < a.kept; ++j) {
            last = max16(left);
            left = left == last ? ordered(-INFINITY) : left;
        }
        bool closed = mark < last;
        // sure if those that stay are not too many (equal ones were counted once) and the least that each can be is more than the
        // most that any other can be
        const bool open = value > -INFINITY, in = open && !closed;
        const int stay = __popcll(__ballot(in && (sub & (a.lg - 1)) == 0) >> (lane & 48) & 0xFFFF);
        const float least_in = -of_ordered(max16(ordered(in ? off - value : -INFINITY)));
        const float most_out = of_ordered(max16(ordered(open && closed ? value + off : -INFINITY)));
        const bool unsure = in && (stay > a.kept || !(least_in > most_out));
        if (__builtin_expect(__ballot(unsure) != 0, 0)) {  // some group of the wave's tokens: all its groups exactly
            double d1 = minus_inf(), d2 = minus_inf();
#pragma unroll 1
            for (int p = 0; p < P; ++p) {
                const double v = number(p < mine ? e0 + p : 0, p < mine);
                d2 = __builtin_fmax(d2, __builtin_fmin(d1, v));
                d1 = __builtin_fmax(d1, v);
            }
            auto merge64 = [&](auto s) __attribute__((always_inline)) {
                constexpr int S = decltype(s)::value;
                const double low = step<S>(d1, [](double x, double y) { return __builtin_fmin(x, y); });
                d2 = __builtin_fmax(low, step<S>(d2, Max()));
                d1 = step<S>(d1, Max());
            };
            if (a.lg > 1) merge64(std::integral_constant<int, 0>());
            if (a.lg > 2) merge64(std::integral_constant<int, 1>());
            if (a.lg > 4) merge64(std::integral_constant<int, 2>());
            closed = !group_kept<L>(a, d1, d2, top, group);
        }
        if (closed) {
            one = two = -INFINITY;
#pragma unroll
            for (int p = 0; p < P; ++p) c[p] = -INFINITY;
        }
    }
    // the k-th largest of the lanes' two (equal ones counted once: lower still), and what it may be off
    int mark = 0;
    for (int j = 0, x = ordered(one), y = ordered(two); j < a.k; ++j) {
        mark = max16(x);
        const bool won = x == mark;
        x = won ? y : x;
        y = won ? ordered(-INFINITY) : y;
    }
    float least = fminf(fmaxf(of_ordered(mark), -kMost), kMost);
    if (a.exact) least = fmaxf(least - (0x1p-20f + 0x1p-21f * fabsf(least)), -kMost);
    uint32_t those = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) those |= c[p] >= least ? 1u << p : 0u;
    const int n = __popc(those);
    int before = n;  // candidates of the lanes up to this one
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        const int u = __shfl_up(before, d, L);
        before += sub >= d ? u : 0;
    }
    const int many = __shfl(before, L - 1, L);
    for (int i = before - n; those; ++i) {
        found[slot][i] = (uint8_t)(e0 + __builtin_ctz(those));
        those &= those - 1;
    }
    __builtin_amdgcn_wave_barrier();  // (a token's candidates are its wave's own)
    double won = minus_inf();
#pragma unroll 1
    for (int from = 0; __ballot(from < many); from += L) {  // the 16 largest so far, the j-th in lane j, and 16 more
        const bool in = from + sub < many;
        const double v = sort16(number(in ? found[slot][from + sub] : 0, in), sub);
        won = from == 0 ? v : sort16(__builtin_fmax(won, other<0x140>(v)), sub);
    }
    const bool open = sub < a.k && won > minus_inf();
    const int e = open ? index_of(won) : 0;
    const float x = open ? rows[slot][place(e)] : -INFINITY;
    float w = weight_of<L>(a, open, x, top, total);
    if (poisoned) w = __builtin_nanf("");
    if (on && sub < a.k) {
        a.idx[token * a.k + sub] = open ? e : -1;
        a.w[token * a.k + sub] = w;
    }
}

// ---------------------------------------------------------------------------
// its gradient
// ---------------------------------------------------------------------------

struct GradArgs {
    const void *logits;
    const int32_t *idx;
    const float *d;
    void *out;
    int T, E, k, sigmoid, renorm;
    float scale;
};

constexpr int kGradThreads = 256;

// A token's row is put together in LDS: zeros, the chosen experts' numbers at
// their places, and then written as a row (softmax that is not renormalized:
// with every expert's share added). Lanes take V neighbours in turn, at most 16
// in all. What bounds it is writing the row, and a launch's latency: 16384
// tokens x 256 experts in fp32 6.6 us one by one, 6.3 in fours (2.8 TB/s; softmax
// not renormalized 13.3 and 7.9, its logits read once: 4.4 TB/s). 173 tokens x 48
// experts 3.5 us: a launch, and two loads that depend on each other.
template <int L, bool BF16, int V>
__global__ __launch_bounds__(kGradThreads) void k_route_grad(GradArgs a) {
    constexpr int kRow = L * 16, kTurns = 16 / V;
    __shared__ alignas(16) float rows[kGradThreads / L][kRow];
    const int lane = threadIdx.x & 63, sub = lane % L, slot = threadIdx.x / L;
    const int64_t token = ((int64_t)blockIdx.x * kGradThreads + threadIdx.x) / L;
    const bool on = token < a.T;
    const int64_t at = (on ? token : 0) * a.E;
    const bool dense = !a.sigmoid && !a.renorm;
    float l[kTurns][V];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int from = (i * L + sub) * V;
        if (dense && from < a.E) load_logits<BF16, V>(a.logits, at + from, l[i]);
#pragma unroll
        for (int q = 0; q < V; ++q) rows[slot][from + q] = 0.0f;
    }
    int e = on && sub < a.k ? a.idx[token * a.k + sub] : -1;
    bool ok = e >= 0 && e < a.E;
    for (int j = 0; j < a.k; ++j) {
        const int other = __shfl(e, j, L);
        ok &= j >= sub || other != e;
    }
    e = ok ? e : 0;
    const float d = ok ? a.d[token * a.k + sub] * a.scale : 0.0f;
    const float x = ok ? load_logit<BF16>(a.logits, at + e) : -INFINITY;
    float value, top = 0.0f, total = 1.0f, share = 0.0f;
    if (a.renorm) {
        const float y = a.sigmoid ? fminf(x, 0.0f) : x;
        const float m = all<L>(y, Max());
        const float den = sigmoid_den(x);
        float p = ok ? exp32(y == m ? 0.0f : y - m) : 0.0f;
        if (a.sigmoid && ok) p /= den;
        p = p / all<L>(p, Sum());
        p = ok ? p : 0.0f;
        value = p * (d - all<L>(p * d, Sum()));
        if (a.sigmoid) value *= exp32(fminf(-x, 0.0f)) / den;  // 1 - s
    } else if (a.sigmoid) {
        const float den = sigmoid_den(x);
        value = d * (exp32(-fabsf(x)) / (den * den));
    } else {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) top = fmaxf(top, (i * L + sub) * V < a.E ? l[i][q] : -INFINITY);
        top = all<L>(top, Max());
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q)
                if ((i * L + sub) * V < a.E) {
                    l[i][q] = exp32(l[i][q] == top ? 0.0f : l[i][q] - top);
                    total += l[i][q];
                }
        total = all<L>(total, Sum());
        const float p = ok ? exp32(x == top ? 0.0f : x - top) / total : 0.0f;
        share = all<L>(p * d, Sum());
        value = d;
    }
    const float scale = 1.0f / total;
    __syncthreads();
    if (ok) rows[slot][e] = value;
    __syncthreads();
    if (!on) return;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int from = (i * L + sub) * V;
        if (from >= a.E) continue;
        float v[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            v[q] = rows[slot][from + q];
            if (dense) v[q] = l[i][q] * scale * (v[q] - share);
        }
        if constexpr (V == 1) {
            if (BF16)
                ((__bf16 *)a.out)[at + from] = (__bf16)v[0];
            else
                ((float *)a.out)[at + from] = v[0];
        } else if constexpr (BF16) {
            u32x4 w;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bf16x2 b = {(__bf16)v[2 * q], (__bf16)v[2 * q + 1]};
                w[q] = __builtin_bit_cast(uint32_t, b);
            }
            *(u32x4 *)((uint16_t *)a.out + at + from) = w;
        } else {
            *(f32x4 *)((float *)a.out + at + from) = f32x4{v[0], v[1], v[2], v[3]};
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int power_of_two(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

int bad_router(const ep_router *r) {
    if (!r) return EP_ERR_ARG;
    if (r->num_experts < 1 || r->num_experts > 1024 || r->num_topk < 1 || r->num_topk > 32) return EP_ERR_ARG;
    if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_ERR_ARG;
    if (r->renormalize != 0 && r->renormalize != 1) return EP_ERR_ARG;
    if (r->num_groups < 1 || r->num_groups > 64 || r->num_experts % r->num_groups) return EP_ERR_ARG;
    if (r->topk_groups < 1 || r->topk_groups > r->num_groups) return EP_ERR_ARG;
    if (r->num_topk > r->topk_groups * (r->num_experts / r->num_groups)) return EP_ERR_ARG;
    if (r->group_top != 1 && r->group_top != 2) return EP_ERR_ARG;
    if (!isfinite(r->scale)) return EP_ERR_ARG;
    return EP_OK;
}

template <int L>
hipError_t launch_route_grad(const GradArgs &a, bool bf16, bool vector, hipStream_t s) {
    const int per = kGradThreads / L, grid = (a.T + per - 1) / per;
    if (bf16 && vector)
        k_route_grad<L, true, 8><<<grid, kGradThreads, 0, s>>>(a);
    else if (bf16)
        k_route_grad<L, true, 1><<<grid, kGradThreads, 0, s>>>(a);
    else if (vector)
        k_route_grad<L, false, 4><<<grid, kGradThreads, 0, s>>>(a);
    else
        k_route_grad<L, false, 1><<<grid, kGradThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int P>
hipError_t launch_route_many(const RouteArgs &a, bool bf16, hipStream_t s) {
    const int grid = (a.T + 15) / 16;
    if (bf16)
        k_route_many<P, true><<<grid, 256, 0, s>>>(a);
    else
        k_route_many<P, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int L, int P>
hipError_t launch_route(const RouteArgs &a, bool bf16, int cus, hipStream_t s) {
    const int64_t waves = ((int64_t)a.T * L + 63) / 64;
    const int threads = waves < 4 * (int64_t)cus ? 64 : 256;
    const int64_t blocks = (waves + threads / 64 - 1) / (threads / 64), most = (int64_t)cus * 8;
    const int grid = (int)(blocks < most ? blocks : most);
    if (bf16)
        k_route<L, P, true><<<grid, threads, 0, s>>>(a);
    else
        k_route<L, P, false><<<grid, threads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

extern "C" {

int ep_route(const ep_router *router, const void *logits, int logits_f32, const float *bias, int num_tokens,
             int32_t *topk_idx, float *topk_weights, ep_stream_t stream) {
    if (int r = bad_router(router)) return r;
    if (num_tokens < 0 || num_tokens > kMaxTokens || (logits_f32 != 0 && logits_f32 != 1)) return EP_ERR_ARG;
    if (num_tokens == 0) return EP_OK;
    if (!logits || !topk_idx || !topk_weights) return EP_ERR_ARG;
    if (misaligned(logits, logits_f32 ? 4 : 2) || misaligned(bias, 4) || misaligned(topk_idx, 4) || misaligned(topk_weights, 4))
        return EP_ERR_ALIGN;
    const int64_t T = num_tokens, E = router->num_experts, in = T * E * (logits_f32 ? 4 : 2), out = T * router->num_topk * 4;
    if (ep::overlap(topk_idx, out, topk_weights, out) || ep::overlap(topk_idx, out, logits, in) ||
        ep::overlap(topk_weights, out, logits, in) || ep::overlap(topk_idx, out, bias, E * 4) ||
        ep::overlap(topk_weights, out, bias, E * 4))
        return EP_ERR_ARG;
    int cus;
    if (int r = ep::device_cus(&cus)) return r;
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.idx = topk_idx;
    a.w = topk_weights;
    a.T = num_tokens;
    a.E = router->num_experts;
    a.k = router->num_topk;
    const bool grouped = router->topk_groups < router->num_groups;  // all groups stay: none
    a.G = grouped ? router->num_groups : 1;
    a.kept = router->topk_groups;
    a.top = router->group_top;
    a.gs = a.E / a.G;
    a.exact = bias != nullptr;
    a.sigmoid = router->score == EP_SCORE_SIGMOID;
    a.renorm = router->renormalize;
    a.scale = router->scale;
    const int all = power_of_two(a.G);
    // 16 lanes a token where its experts, choices and groups fit them and there are tokens enough for that to be faster: by
    // candidates from 8 a compute unit on (2048 tokens, 256 experts: 4.5 to 6.0 us against 4.6 to 6.2; 512 tokens 4.5 to 5.3
    // against 4.0 to 5.3), else from 16 on
    const bool few = a.k <= 8 && (a.sigmoid || !a.exact);
    const bool narrow = all <= 16 && a.k <= 16 && (int64_t)(a.gs + 16 / all - 1) / (16 / all) <= 16 &&
                        T >= (few ? 8 : 16) * (int64_t)cus;
    const int L = narrow ? 16 : 64;
    a.lg = L / all;
    a.lg_log = __builtin_ctz(a.lg);
    const int P = power_of_two((a.gs + a.lg - 1) / a.lg);
    a.quads = 0;
    a.vector = a.gs % P == 0 && !misaligned(logits, 16);  // P experts at a multiple of their size
    const hipStream_t s = (hipStream_t)stream;
    const bool bf16 = !logits_f32;
    hipError_t e;
    const bool many = narrow && few;
    if (many) {
        a.vector = a.E % (bf16 ? 8 : 4) == 0 && P >= (bf16 ? 8 : 4) && !misaligned(logits, 16);
        a.quads = P >= 4 && a.gs % 4 == 0;
    }
    if (many)
        e = P == 1   ? launch_route_many<1>(a, bf16, s)
            : P == 2 ? launch_route_many<2>(a, bf16, s)
            : P == 4 ? launch_route_many<4>(a, bf16, s)
            : P == 8 ? launch_route_many<8>(a, bf16, s)
                     : launch_route_many<16>(a, bf16, s);
    else if (narrow)
        e = P == 1   ? launch_route<16, 1>(a, bf16, cus, s)
            : P == 2 ? launch_route<16, 2>(a, bf16, cus, s)
            : P == 4 ? launch_route<16, 4>(a, bf16, cus, s)
            : P == 8 ? launch_route<16, 8>(a, bf16, cus, s)
                     : launch_route<16, 16>(a, bf16, cus, s);
    else
        e = P == 1    ? launch_route<64, 1>(a, bf16, cus, s)
            : P == 2  ? launch_route<64, 2>(a, bf16, cus, s)
            : P == 4  ? launch_route<64, 4>(a, bf16, cus, s)
            : P == 8  ? launch_route<64, 8>(a, bf16, cus, s)
            : P == 16 ? launch_route<64, 16>(a, bf16, cus, s)
                      : launch_route<64, 32>(a, bf16, cus, s);
    return ep::hip_status(e, "ep_route");
}

int ep_route_backward(const ep_router *router, const void *logits, int logits_f32, const int32_t *topk_idx,
                      const float *grad_weights, int num_tokens, void *grad_logits, ep_stream_t stream) {
    if (int r = bad_router(router)) return r;
    if (num_tokens < 0 || num_tokens > kMaxTokens || (logits_f32 != 0 && logits_f32 != 1)) return EP_ERR_ARG;
    if (num_tokens == 0) return EP_OK;
    if (!logits || !topk_idx || !grad_weights || !grad_logits) return EP_ERR_ARG;
    const size_t each = logits_f32 ? 4 : 2;
    if (misaligned(logits, each) || misaligned(grad_logits, each) || misaligned(topk_idx, 4) || misaligned(grad_weights, 4))
        return EP_ERR_ALIGN;
    const int64_t T = num_tokens, n = T * router->num_experts * (logits_f32 ? 4 : 2), picks = T * router->num_topk * 4;
    if (ep::overlap(grad_logits, n, logits, n) || ep::overlap(grad_logits, n, topk_idx, picks) ||
        ep::overlap(grad_logits, n, grad_weights, picks))
        return EP_ERR_ARG;
    GradArgs a;
    a.logits = logits;
    a.idx = topk_idx;
    a.d = grad_weights;
    a.out = grad_logits;
    a.T = num_tokens;
    a.E = router->num_experts;
    a.k = router->num_topk;
    a.sigmoid = router->score == EP_SCORE_SIGMOID;
    a.renorm = router->renormalize;
    a.scale = router->scale;
    const bool vector = a.E % (logits_f32 ? 4 : 8) == 0 && !misaligned(logits, 16) && !misaligned(grad_logits, 16);
    const hipStream_t s = (hipStream_t)stream;
    // 16 lanes a token where its experts and slots fit them
    const hipError_t e = a.E <= 256 && a.k <= 16 ? launch_route_grad<16>(a, !logits_f32, vector, s)
                                                 : launch_route_grad<64>(a, !logits_f32, vector, s);
    return ep::hip_status(e, "ep_route_backward");
}

}  // extern "C"
