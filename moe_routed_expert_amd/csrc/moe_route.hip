// Choice of each token's experts, the chosen experts' weights, and their gradient (gfx950).
//
// A token takes 16 lanes (32 and 64 above 256 and 512 experts) with up to 16
// experts in a row each. A lane sorts its own, and lists are joined lane by
// lane, which keeps the 8 largest of two sorted lists by comparing one with the
// other reversed; more than 8 are taken one after the other from sorted lanes.
// Keys are float64, with the expert's number below a float32 value. The order of
// logits is exact; a token with biased scores too near to tell, or groups' sums,
// is chosen again in float64, by its whole wavefront: with equal biases and bfloat16
// logits, of which many are equal, that is a third of the tokens (65536 x 256 in
// groups 140 us instead of 48). An expert that a bias of -1e4 or -1e9 switches off
// changes nothing (47 us).
//
// Bound by vector instructions: 65536 tokens, 8 of 256 experts by logits 22 us
// (15 at a copy's rate), in groups by biased sigmoids 48 us; 131072 tokens, 8
// of 64 25 us. A kernel takes each token once, without a loop around it: with
// one the compiler keeps the constants of exponentials and divisions in
// registers, 204 instead of 84 for 256 experts, and the times are 31, 75 and 28.
//
// The gradient is bound by memory where every score counts (131072 x 64 19.2
// us, 4.0 TB/s): a token's slots go through LDS, and each lane adds up those of
// its experts, in their order.
#include <type_traits>

#include "epi_common.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMostTokens = 1 << 20;  // of a launch
constexpr int kMostExperts = 1024, kMostGroups = 64, kMostChosen = 64;
constexpr float kInf = __builtin_inff();

struct Choice {
    int experts, top_k, groups, top_groups;
    bool sigmoid, top2, renormalise;
    float scale;
};

// ---- over the L lanes of a token -------------------------------------------------

// The lane's partner in step `kXor` (1, 2, 4, 8, 16, 32) of an exchange that
// leaves every lane of an aligned group of 2 kXor with the group's result: the
// steps up to 8 mirror quads, halves and rows of 16 lanes, the others swap rows
// and halves of the wavefront; none goes through LDS.
template <int kXor>
__device__ __forceinline__ int partner(int v) {
    if constexpr (kXor == 1)
        return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
    else if constexpr (kXor == 2)
        return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
    else if constexpr (kXor == 4)
        return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
    else if constexpr (kXor == 8)
        return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
    else {
        // the rows (halves) of the pair: their own in one of the two, the partner's in the other
        const auto r = kXor == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                  : __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (threadIdx.x & kXor) != 0 ? r[0] : r[1];
    }
}
template <int kXor>
__device__ __forceinline__ float partner(float v) {
    return __int_as_float(partner<kXor>(__float_as_int(v)));
}
template <int kXor>
__device__ __forceinline__ double partner(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = static_cast<uint32_t>(partner<kXor>(static_cast<int>(u)));
    const uint32_t hi = static_cast<uint32_t>(partner<kXor>(static_cast<int>(u >> 32)));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
template <int L, int kXor = 1, class V, class F>
__device__ __forceinline__ V over_lanes(V v, F f) {
    if constexpr (kXor < L)
        return over_lanes<L, 2 * kXor>(f(v, partner<kXor>(v)), f);
    else
        return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    return over_lanes<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, class V>
__device__ __forceinline__ V lanes_sum(V v) {
    return over_lanes<L>(v, [](V a, V b) { return a + b; });
}
template <int L>
__device__ __forceinline__ bool lanes_any(bool v) {
    if constexpr (L == 64)
        return __any(v);
    else
        return (__ballot(v) >> (threadIdx.x & 63 & ~(L - 1)) & ((1ull << L) - 1)) != 0;
}

// ---- keys ----------------------------------------------------------------------------
//
// A key is a float32 value as a float64, whose last 10 bits (of the 29 that the
// value leaves free) are the expert's number, turned so that of equal values the
// lowest expert has the largest key. -inf: not to be chosen.

constexpr uint64_t kNumber = kMostExperts - 1;

__device__ __forceinline__ double key_of(float value, int expert) {
    if (!(value > -kInf)) return -kInf;  // NaN too
    const double v = fmin(static_cast<double>(value) + 0.0, 0x1p1000);  // +0 for -0; a number for infinity
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, u | static_cast<uint64_t>(v >= 0 ? kNumber - expert : expert));
}
__device__ __forceinline__ int expert_of(double key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int n = static_cast<int>(u & kNumber);
    return key == -kInf ? -1 : (u >> 63 ? n : static_cast<int>(kNumber) - n);
}
__device__ __forceinline__ double value_of(double key) {
    return key == -kInf ? key : __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~kNumber);
}
// One instruction each: keys are never NaN, so they need not be made quiet first.
__device__ __forceinline__ double larger(double a, double b) {
    double d;
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double smaller(double a, double b) {
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
// Descending, by Batcher's odd-even merge.
template <int N>
__device__ __forceinline__ void sort_keys(double (&key)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const double a = key[i + j], b = key[i + j + k];
                        key[i + j] = larger(a, b);
                        key[i + j + k] = smaller(a, b);
                    }
}

// A sequence that rises and falls, descending.
template <int N, int M>
__device__ __forceinline__ void settle(double (&key)[M]) {
#pragma unroll
    for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!(i & d)) {
                const double a = key[i], b = key[i + d];
                key[i] = larger(a, b);
                key[i + d] = smaller(a, b);
            }
}
// The K largest of two descending lists of K, in `a`; `left` grows to the largest that is left out.
template <int K>
__device__ __forceinline__ void join(double (&a)[K], const double (&b)[K], double& left) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
        left = larger(left, smaller(a[i], b[K - 1 - i]));
        a[i] = larger(a[i], b[K - 1 - i]);
    }
    settle<K>(a);
}
// The K largest keys of L lanes that have n each, descending, in every lane.
template <int L, int K, int n, int kXor = 1>
__device__ __forceinline__ void join_lanes(double (&key)[K], double& left) {
    if constexpr (kXor < L) {
        if constexpr (2 * n <= K) {
#pragma unroll
            for (int i = 0; i < n; ++i) key[2 * n - 1 - i] = partner<kXor>(key[i]);
            settle<2 * n>(key);
            join_lanes<L, K, 2 * n, 2 * kXor>(key, left);
        } else {
            double other[K];
#pragma unroll
            for (int i = 0; i < K; ++i) other[i] = partner<kXor>(key[i]);
            join<K>(key, other, left);
            left = larger(left, partner<kXor>(left));
            join_lanes<L, K, n, 2 * kXor>(key, left);
        }
    }
}

// The K largest keys of L lanes that have N each, descending, in every lane.
template <int L, int K, int N>
__device__ __forceinline__ void best_keys(const double (&key)[N], double (&list)[K], double& left) {
    constexpr int n = N < K ? N : K;
    static_assert(n * L >= K, "");
#pragma unroll
    for (int c = 0; c < N; c += n) {
        double part[n];
#pragma unroll
        for (int i = 0; i < n; ++i) part[i] = key[c + i];
        sort_keys<n>(part);
        if constexpr (n == K) {
            if (c > 0) {
                join<K>(list, part, left);
                continue;
            }
        }
#pragma unroll
        for (int i = 0; i < n; ++i) list[i] = part[i];
    }
    if constexpr (N > K) left = over_lanes<L>(left, [](double a, double c) { return larger(a, c); });
    join_lanes<L, K, n>(list, left);
}

// ---- scores ----------------------------------------------------------------------------

__device__ __forceinline__ float sigmoid32(float l) {
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}
// As sigmoid32 with the hardware's exponential and reciprocal, for the choice.
__device__ __forceinline__ float rough_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float rough_sigmoid(float l) {
    const float e = rough_exp(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
}
// sigmoid(l) over e^min(most, 0), which does not underflow for the largest of some logits.
__device__ __forceinline__ float over_most(float l, float most) {
    return expf(fminf(l, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(l)));
}
// What a float32 score may be off, in steps of 2^-24. A sigmoid: 0.3 for the
// exponential's argument and 0.5 for its last place (passed on by e / (1 + e)^2),
// 1 for the sum, 1 for the reciprocal's last place and 0.25 for the product,
// below 2^-22. A softmax: |l - m| of itself (m - l is at most log(experts) on
// average over the scores, which the sum is off by, and at most 0.4 of the
// largest score for the score itself), up to 22 additions and 8 for exponentials
// and quotient, below 2^-18 of the largest score, 1 / sum.
__device__ __forceinline__ float score_error(bool sigmoid, float sum) { return sigmoid ? 0x1p-22f : 0x1p-18f / sum; }

template <int T>
__device__ __forceinline__ float load_logit(const char* row, int e) {
    return Elem<T>::load1(row, e);
}
// Experts e0 .. e0 + N - 1 of a row, -inf past the last.
template <int T, int N>
__device__ __forceinline__ void load_logits(const char* row, int e0, int experts, float (&l)[N]) {
    constexpr int V = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += V) {
        if (V == 4 && e0 + i + 4 <= experts) {
            if constexpr (T == MOE_EPI_F32) {
                typedef u32x4 loose __attribute__((aligned(4)));
                const u32x4 w = *reinterpret_cast<const loose*>(row + 4 * (e0 + i));
#pragma unroll
                for (int j = 0; j < V; ++j) l[i + j] = __uint_as_float(w[j]);
            } else {
                typedef u32x2 loose __attribute__((aligned(2)));
                const u32x2 w = *reinterpret_cast<const loose*>(row + 2 * (e0 + i));
                float f[8];
                Elem<T>::unpack(u32x4{w[0], w[1], 0, 0}, f);
#pragma unroll
                for (int j = 0; j < V; ++j) l[i + j] = f[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) l[i + j] = e0 + i + j < experts ? load_logit<T>(row, e0 + i + j) : -kInf;
        }
    }
}

// The groups (a bit each) that fewer than top_groups others come before.
template <int L>
__device__ __forceinline__ uint64_t best_groups(const double* value, const Choice& p, int lane) {
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    uint64_t kept = 0;
#pragma unroll 1
    for (int g0 = 0; g0 < p.groups; g0 += L) {
        const int g = g0 + lane;
        const double v = g < p.groups ? value[g] : -kInf;
        int before = g < p.groups ? 0 : kMostGroups;

#pragma unroll 1
        for (int o = 0; o < p.groups; ++o) {
            const double w = value[o];
            before += w > v || (w == v && o < g);
        }
        const uint64_t best = __ballot(before < p.top_groups);
        if constexpr (L == 64)
            kept |= best;
        else
            kept |= (best >> (threadIdx.x & 63 & ~(L - 1)) & ((1ull << L) - 1)) << g0;
    }
    __builtin_amdgcn_wave_barrier();
    return kept;
}

// e^x to an ulp or so: x = n ln 2 + r, the Taylor series to r^13 (|r| <= 0.35: what is left out is 2^-57), times
// 2^n. The coefficients are read in a loop: as constants they would be kept in registers from every token.
__device__ const double kOverFactorial[14] = {1.0 / 6227020800.0, 1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0,
                                              1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0,
                                              1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
template <int N>
__device__ __forceinline__ void exp64(double (&x)[N]) {
    double n[N], r[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        x[j] = fmin(fmax(x[j], -800.0), 800.0);  // 0 and infinity from there on
        n[j] = rint(x[j] * 0x1.71547652b82fep+0);
        r[j] = fma(-n[j], 0x1.62e42fefa39efp-1, x[j]);
        r[j] = fma(-n[j], 0x1.abc9e3b39803fp-56, r[j]);
        x[j] = kOverFactorial[0];
    }
#pragma unroll 1
    for (int i = 1; i < 14; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = fma(x[j], r[j], kOverFactorial[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = ldexp(x[j], static_cast<int>(n[j]));
}

// Token t by float64 values, by the whole wavefront, an expert that is chosen in each lane. Few tokens come here, so
// its code is kept short: what is not in the instruction cache takes longer to read than to run.
template <int T>
__device__ __forceinline__ void route64(const char* logits, const float* bias, int32_t* ids, float* weights, int64_t t,
                                        const Choice& p, double* value, double* of_group) {
    const int lane = threadIdx.x & 63, size = p.experts / p.groups;
    const char* row = logits + t * p.experts * Elem<T>::kBytes;
    float m = -kInf;
    double all = 0.0;
    bool bad = false;
    // four experts at a time, so that their loads and exponentials go side by side
    auto each4 = [&](auto f) {
#pragma unroll 1
        for (int e = lane; e < p.experts; e += 256) {
            float l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) l[j] = e + 64 * j < p.experts ? load_logit<T>(row, e + 64 * j) : -kInf;
            f(e, l);
        }
    };
    if (!p.sigmoid) {
        each4([&](int, const float (&l)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, l[j]);
        });
        m = lanes_max<64>(m);
        each4([&](int, const float (&l)[4]) {
            double x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = static_cast<double>(l[j]) - m;
            exp64(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) all += l[j] > -kInf ? x[j] : 0.0;
        });
        all = lanes_sum<64>(all);
    }
    // an expert's value, its score where groups count sums of those and there is no bias
    const bool sums = p.top2 && p.groups > 1;
    auto fill = [&](bool by_score) {
        each4([&](int e, const float (&l)[4]) {
            double x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= l[j] != l[j] || (!p.sigmoid && l[j] == kInf);
                x[j] = p.sigmoid ? -static_cast<double>(l[j]) : static_cast<double>(l[j]) - m;
            }
            exp64(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e + 64 * j >= p.experts) continue;
                double v = l[j];
                if (by_score) v = p.sigmoid ? 1.0 / (1.0 + x[j]) : x[j] / all;
                if (bias) v += static_cast<double>(bias[e + 64 * j]);
                value[e + 64 * j] = l[j] > -kInf && v > -kInf ? v : -kInf;  // not where either is NaN
            }
        });
        __threadfence_block();
        __builtin_amdgcn_wave_barrier();
    };
    fill(bias || sums);
    bad = lanes_any<64>(bad);
    uint64_t kept = ~0ull;
    if (p.groups > 1) {
        if (lane < p.groups) {
            double first = -kInf, second = -kInf;

#pragma unroll 4
            for (int i = 0; i < size; ++i) {
                const double v = value[lane * size + i];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
            of_group[lane] = sums ? first + second : first;
        }
        kept = best_groups<64>(of_group, p, lane);
        if (sums && !bias) {
#pragma unroll 1
            for (int e = lane; e < p.experts; e += 64) value[e] = value[e] > -kInf ? load_logit<T>(row, e) : -kInf;
            __threadfence_block();
            __builtin_amdgcn_wave_barrier();
        }
    }
    // a lane holds experts in a row, so that of equal ones the lowest lane has the lowest
    const int n = (p.experts + 63) / 64;
    int id = -1;
#pragma unroll 1
    for (int r = 0; r < p.top_k; ++r) {
        double best = -kInf;
        int expert = -1;

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int e = lane * n + i;
            const double v = e < p.experts && (kept >> (e / size & 63) & 1) ? value[e] : -kInf;
            if (v > best) {
                best = v;
                expert = e;
            }
        }
        const double most = over_lanes<64>(best, [](double a, double c) { return larger(a, c); });
        const int at = __builtin_ctzll(__ballot(best == most));  // -inf: the first lane, which has no expert then
        const int e = __shfl(expert, at, 64);
        if (lane == r) id = e;
        if (lane == at && expert >= 0) value[expert] = -kInf;
        __threadfence_block();
        __builtin_amdgcn_wave_barrier();
    }
    const float l = id >= 0 ? load_logit<T>(row, id) : -kInf, most = lanes_max<64>(l);
    float w;
    if (!p.renormalise)
        w = p.sigmoid ? sigmoid32(l) : expf(l - m) / static_cast<float>(all);
    else if (!p.sigmoid)
        w = expf(l - most);
    else
        w = over_most(l, most);
    if (id < 0) w = 0.0f;
    if (p.renormalise) {
        const float sum = lanes_sum<64>(w);
        if (id >= 0) w /= sum;
    }
    if (lane < p.top_k) {
        ids[t * p.top_k + lane] = id;
        weights[t * p.top_k + lane] = bad ? __builtin_nanf("") : w * p.scale;
    }
}

// L lanes per token, N experts in a lane, S chosen experts in a lane. K: the
// lanes' lists are joined, of which the K >= top_k largest are kept; 0: one
// expert at a time. kScored: the order is that of scores, with a bias or as sums
// of two for a group's value, and not that of the logits.
template <int T, int L, int N, int S, int K, bool kScored>
__global__ __launch_bounds__(kBlock) void route_kernel(const char* __restrict__ logits, const float* __restrict__ bias,
                                                       int32_t* __restrict__ ids, float* __restrict__ weights,
                                                       int64_t tokens, Choice p) {
    constexpr int kTokens = kBlock / L;
    __shared__ double of_group[kTokens][kMostGroups];  // only of groups that do not lie in whole lanes
    __shared__ f32x2_t range_group[kScored ? kTokens : 1][kScored ? kMostGroups : 1];
    __shared__ double value64[kScored ? kBlock / 64 : 1][kScored ? (L * N < 64 ? 64 : L * N) : 1];
    __shared__ double group64[kScored ? kBlock / 64 : 1][kScored ? kMostGroups : 1];
    const int lane = threadIdx.x % L, e0 = lane * N, size = p.experts / p.groups;
    const bool grouped = p.groups > 1, biased = kScored && bias;
    // lanes of a group, where its experts are those of 2^n lanes
    const int wide = size % N == 0 ? size / N : 0;
    const bool whole = grouped && wide >= 1 && wide <= L && (wide & (wide - 1)) == 0;

    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
    const int64_t mine = t0 + threadIdx.x / L, t = mine < tokens ? mine : tokens - 1;
    const char* row = logits + t * p.experts * Elem<T>::kBytes;
    float l[N], b[N], m = -kInf;
    load_logits<T, N>(row, e0, p.experts, l);
    if (biased) load_logits<MOE_EPI_F32, N>(reinterpret_cast<const char*>(bias), e0, p.experts, b);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        bad |= l[i] != l[i] || (!p.sigmoid && l[i] == kInf);
        m = fmaxf(m, l[i]);
    }
    bad = lanes_any<L>(bad);
    float sum = 0.0f;
    if (!p.sigmoid) {
        m = lanes_max<L>(m);
        if (kScored || !p.renormalise) {
#pragma unroll
            for (int i = 0; i < N; ++i) sum += expf(l[i] - m);
            sum = lanes_sum<L>(sum);
        }
    }

    int id[S];
    // The choice by logits, which is exact.
    auto choose = [&]() {
        double key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = key_of(l[i], e0 + i);
        const auto larger2 = [](double a, double c) { return larger(a, c); };
        if (grouped && !whole) {
            double* value = of_group[threadIdx.x / L];
            for (int g = 0; g < p.groups; ++g) {
                double first = -kInf;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (e0 + i >= g * size && e0 + i < (g + 1) * size) first = larger(first, key[i]);
                first = over_lanes<L>(first, larger2);
                if (lane == 0) value[g] = value_of(first);
            }
            const uint64_t kept = best_groups<L>(value, p, lane);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!(kept >> ((e0 + i) / size & 63) & 1)) key[i] = -kInf;
        }
        if (whole) {
            double first = -kInf;
#pragma unroll
            for (int i = 0; i < N; ++i) first = larger(first, key[i]);
            for (int x = 1; x < wide; x *= 2) first = larger(first, __shfl_xor(first, x, 64));
            const double v = value_of(first);
            const int group = lane / wide;
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const double w = __shfl(v, g * wide, L);
                before += w > v || (w == v && g < group);
            }
            if (before >= p.top_groups || group >= p.groups)
#pragma unroll
                for (int i = 0; i < N; ++i) key[i] = -kInf;
        }
        if constexpr (K > 0) {
            double list[K], left = -kInf, mine = -kInf;
            best_keys<L, K>(key, list, left);
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (lane == j) mine = list[j];
            id[0] = lane < p.top_k ? expert_of(mine) : -1;
        } else {
            sort_keys<N>(key);
            for (int r = 0; r < p.top_k; ++r) {
                const double best = over_lanes<L>(key[0], larger2);
                const bool pop = key[0] == best;
#pragma unroll
                for (int i = 0; i + 1 < N; ++i) key[i] = pop ? key[i + 1] : key[i];
                key[N - 1] = pop ? static_cast<double>(-kInf) : key[N - 1];
                const int e = expert_of(best);
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (r == lane + s * L) id[s] = e;
            }
        }
    };
    // The choice by float32 scores; returns whether some were too near to tell.
    auto choose_scored = [&]() {
        const float over = p.sigmoid ? 0.0f : 1.0f / sum;
        const float score_off = score_error(p.sigmoid, sum);
        bool near = false;
        float c[N];
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = l[i] > -kInf ? l[i] : -kInf;  // for NaN too
        if (biased) {
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < N; ++i) c[i] = rough_sigmoid(l[i]) + b[i];
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) c[i] = rough_exp(l[i] - m) * over + b[i];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = l[i] > -kInf && c[i] > -kInf ? c[i] : -kInf;
        }
        auto group_value = [&](float first, float second) {
            if (!p.top2 || second == -kInf) return p.top2 ? second : first;
            return biased ? first + second
                          : (p.sigmoid ? rough_sigmoid(first) + rough_sigmoid(second)
                                       : (rough_exp(first - m) + rough_exp(second - m)) * over);
        };
        // Where a group's value is: it is off by two scores, each rounded with its bias, which may be far larger than
        // the sum of both, and by that sum's rounding: 2^-24 of the biased scores' sizes each time, and once more for
        // the border. A sum beyond float32 may be anywhere; -inf for a lack of experts is what it is.
        struct Within {
            float least, most;
        };
        auto range_of_group = [&](float v, float first, float second) {
            if ((p.top2 ? second : first) == -kInf) return Within{-kInf, -kInf};
            if (!(fabsf(v) < kInf)) return Within{-kInf, kInf};
            const float sizes = biased ? fabsf(first) + (p.top2 ? fabsf(second) : 0.0f) : fabsf(v);
            const float off_by = 2.0f * score_off + sizes * 0x1p-22f;
            return Within{v - off_by, v + off_by};
        };
        // in: the least of the groups that stay, out: the most of the others
        auto tell_groups = [&](float in, float out) { near |= out > -kInf && !(in > out); };
        if (grouped && !whole) {
            double* value = of_group[threadIdx.x / L];
            f32x2_t* range = range_group[kScored ? threadIdx.x / L : 0];
            for (int g = 0; g < p.groups; ++g) {
                float first = -kInf, second = -kInf;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float v = e0 + i >= g * size && e0 + i < (g + 1) * size ? c[i] : -kInf;
                    second = fmaxf(second, fminf(first, v));
                    first = fmaxf(first, v);
                }
#pragma unroll
                for (int x = 1; x < L; x *= 2) {
                    const float a = __shfl_xor(first, x, 64), o = __shfl_xor(second, x, 64);
                    second = fmaxf(fminf(first, a), fmaxf(second, o));
                    first = fmaxf(first, a);
                }
                const float v = group_value(first, second);
                if (lane == 0) {
                    const Within r = range_of_group(v, first, second);
                    value[g] = v;
                    range[g] = f32x2_t{r.least, r.most};
                }
            }
            const uint64_t kept = best_groups<L>(value, p, lane);
            float in = kInf, out = -kInf;
            for (int g = 0; g < p.groups; ++g) {
                const bool stays = kept >> g & 1;
                in = fminf(in, stays ? range[g][0] : kInf);
                out = fmaxf(out, stays ? -kInf : range[g][1]);
            }
            tell_groups(in, out);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!(kept >> ((e0 + i) / size & 63) & 1)) c[i] = -kInf;
        }
        if (whole) {
            float first = -kInf, second = -kInf;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                second = fmaxf(second, fminf(first, c[i]));
                first = fmaxf(first, c[i]);
            }
            for (int x = 1; x < wide; x *= 2) {
                const float a = __shfl_xor(first, x, 64), o = __shfl_xor(second, x, 64);
                second = fmaxf(fminf(first, a), fmaxf(second, o));
                first = fmaxf(first, a);
            }
            const float v = group_value(first, second);
            const int group = lane / wide;
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const float w = __shfl(v, g * wide, L);
                before += w > v || (w == v && g < group);
            }
            const bool stays = before < p.top_groups && group < p.groups;
            const Within r = range_of_group(v, first, second);
            tell_groups(-lanes_max<L>(stays ? -r.least : -kInf), lanes_max<L>(stays || group >= p.groups ? -kInf : r.most));
            if (!stays)
#pragma unroll
                for (int i = 0; i < N; ++i) c[i] = -kInf;
        }
        double key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = key_of(c[i], e0 + i);
        // Two biased scores of which a is not the smaller: each off, and rounded with its bias to half an ulp, 2^-24 of
        // itself. Logits are exact.
        auto tell = [&](double a, double o) {
            const double more = value_of(a), less = value_of(o);
            near |= biased && o > -kInf && more - less <= 2.0 * score_off + (fabs(more) + fabs(less)) * 0x1p-24;
        };
        const auto larger2 = [](double a, double o) { return larger(a, o); };
        if constexpr (K > 0) {
            double list[K], left = -kInf, mine = -kInf;
            best_keys<L, K>(key, list, left);
            double next = left;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (lane == j) mine = list[j];
                if (lane + 1 == j) next = list[j];
            }
            if (lane < p.top_k) tell(mine, next);
            id[0] = lane < p.top_k ? expert_of(mine) : -1;
        } else {
            sort_keys<N>(key);
            double last = -kInf;
            for (int r = 0; r <= p.top_k; ++r) {  // also the best that is left
                const double best = over_lanes<L>(key[0], larger2);
                if (r > 0) tell(last, best);
                last = best;
                const bool pop = key[0] == best;
#pragma unroll
                for (int i = 0; i + 1 < N; ++i) key[i] = pop ? key[i + 1] : key[i];
                key[N - 1] = pop ? static_cast<double>(-kInf) : key[N - 1];
                const int e = expert_of(best);
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (r < p.top_k && r == lane + s * L) id[s] = e;
            }
        }
        return lanes_any<L>(near);
    };
#pragma unroll
    for (int s = 0; s < S; ++s) id[s] = -1;
    bool near = false;
    if constexpr (kScored)
        near = choose_scored();
    else
        choose();
    float w[S], lw[S], most = -kInf, all = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        lw[s] = id[s] >= 0 ? load_logit<T>(row, id[s]) : -kInf;
        most = fmaxf(most, lw[s]);
    }
    most = lanes_max<L>(most);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (!p.renormalise)
            w[s] = p.sigmoid ? sigmoid32(lw[s]) : expf(lw[s] - m) / sum;
        else if (!p.sigmoid)
            w[s] = expf(lw[s] - most);
        else
            w[s] = over_most(lw[s], most);
        if (id[s] < 0) w[s] = 0.0f;
        all += w[s];
    }
    if (p.renormalise) all = lanes_sum<L>(all);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int j = lane + s * L;
        if (p.renormalise && id[s] >= 0) w[s] /= all;
        if (j < p.top_k && mine < tokens && !(kScored && near)) {
            ids[t * p.top_k + j] = id[s];
            weights[t * p.top_k + j] = bad ? __builtin_nanf("") : w[s] * p.scale;
        }
    }
    if constexpr (kScored) {
        // float32 values tell nearly all tokens; the others are chosen again, one after the other
        for (uint64_t left = __ballot(near && mine < tokens); left != 0;) {
            const int at = __builtin_amdgcn_readfirstlane(__builtin_ctzll(left) / L);  // of the wavefront's tokens
            left &= L == 64 ? 0 : ~(((1ull << (L & 63)) - 1) << (at * L));
            const int64_t again = t0 + (threadIdx.x & ~63) / L + at;
            route64<T>(logits, bias, ids, weights, again, p, value64[threadIdx.x / 64], group64[threadIdx.x / 64]);
        }
    }
}

// L lanes per token, N experts and S slots in a lane.
template <int T, int L, int N, int S>
__global__ __launch_bounds__(kBlock) void route_grad_kernel(const float* __restrict__ grad_weights,
                                                            const char* __restrict__ logits,
                                                            const int32_t* __restrict__ ids,
                                                            char* __restrict__ grad_logits, int64_t tokens, Choice p) {
    constexpr int kTokens = kBlock / L;
    struct Slot {
        int id;
        float d;
    };
    __shared__ Slot slots[kTokens][S * L];
    const int lane = threadIdx.x % L, e0 = lane * N;
    Slot* mine_slots = slots[threadIdx.x / L];
    const bool dense = !p.sigmoid && !p.renormalise;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
    const int64_t mine = t0 + threadIdx.x / L, t = mine < tokens ? mine : tokens - 1;
    const char* row = logits + t * p.experts * Elem<T>::kBytes;
    float l[N], m = -kInf, sum = 0.0f;
    if (dense) {
        load_logits<T, N>(row, e0, p.experts, l);
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
        m = lanes_max<L>(m);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            l[i] = m > -kInf ? expf(l[i] - m) : 0.0f;
            sum += l[i];
        }
        sum = lanes_sum<L>(sum);
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = m > -kInf ? l[i] / sum : 0.0f;
    }
    int id[S];
    float u[S], lw[S], v[S], most = -kInf;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int j = lane + s * L;
        id[s] = j < p.top_k ? ids[t * p.top_k + j] : -1;
        if (id[s] < 0 || id[s] >= p.experts) id[s] = -1;
        u[s] = id[s] >= 0 ? grad_weights[t * p.top_k + j] * p.scale : 0.0f;
        lw[s] = id[s] >= 0 ? load_logit<T>(row, id[s]) : -kInf;
        most = fmaxf(most, lw[s]);
    }
    float dot = 0.0f, all = 0.0f;
    if (p.renormalise) {
        most = lanes_max<L>(most);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            v[s] = 0.0f;
            if (id[s] >= 0 && !(most == -kInf))
                v[s] = p.sigmoid ? over_most(lw[s], most) : expf(lw[s] - most);
            all += v[s];
        }
        all = lanes_sum<L>(all);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            v[s] = all == 0.0f ? 0.0f : v[s] / all;
            dot += u[s] * v[s];
        }
        dot = lanes_sum<L>(dot);
    } else if (!p.sigmoid) {
#pragma unroll
        for (int s = 0; s < S; ++s) dot += id[s] >= 0 && m > -kInf ? u[s] * (expf(lw[s] - m) / sum) : 0.0f;
        dot = lanes_sum<L>(dot);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float d = u[s];
        if (p.renormalise) d = v[s] * (u[s] - dot);
        if (p.sigmoid) d *= p.renormalise ? sigmoid32(-lw[s]) : sigmoid32(lw[s]) * sigmoid32(-lw[s]);
        mine_slots[lane + s * L] = Slot{id[s], id[s] >= 0 ? d : 0.0f};
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const Slot s = mine_slots[j];
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] += s.id == e0 + i ? s.d : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    if (dense)
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = l[i] * (g[i] - dot);
    if (mine >= tokens) return;
    char* to = grad_logits + t * p.experts * Elem<T>::kBytes;
    constexpr int V = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += V) {
        if (V == 4 && e0 + i + 4 <= p.experts) {
            if constexpr (T == MOE_EPI_F32) {
                typedef u32x4 loose __attribute__((aligned(4)));
                u32x4 w;
#pragma unroll
                for (int j = 0; j < V; ++j) w[j] = __float_as_uint(g[i + j]);
                *reinterpret_cast<loose*>(to + 4 * (e0 + i)) = w;
            } else {
                typedef u32x2 loose __attribute__((aligned(2)));
                const float f[8] = {g[i], g[i + 1 < N ? i + 1 : i], g[i + 2 < N ? i + 2 : i],
                                    g[i + 3 < N ? i + 3 : i], 0, 0, 0, 0};
                const u32x4 w = Elem<T>::pack(f);
                *reinterpret_cast<loose*>(to + 2 * (e0 + i)) = u32x2{w[0], w[1]};
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e0 + i + j < p.experts) Elem<T>::store1(to, e0 + i + j, g[i + j]);
        }
    }
}

// f(lanes of a token, experts of a lane, chosen of a lane, length of a list)
template <class F>
void by_size(int experts, int top_k, F f) {
    auto go = [&](auto l, auto n) {
        constexpr int L = decltype(l)::value;
        const std::integral_constant<int, 1> one;
        if (top_k <= 8) return f(l, n, one, std::integral_constant<int, 8>());
        f(l, n, std::integral_constant<int, kMostChosen / L>(), std::integral_constant<int, 0>());
    };
    const std::integral_constant<int, 16> l16, n16;
    if (experts <= 16) return go(l16, std::integral_constant<int, 1>());
    if (experts <= 32) return go(l16, std::integral_constant<int, 2>());
    if (experts <= 64) return go(l16, std::integral_constant<int, 4>());
    if (experts <= 128) return go(l16, std::integral_constant<int, 8>());
    if (experts <= 256) return go(l16, n16);
    if (experts <= 512) return go(std::integral_constant<int, 32>(), n16);
    go(std::integral_constant<int, 64>(), n16);
}

template <class F>
void by_type(int dtype, F f) {
    if (dtype == MOE_EPI_BF16) return f(std::integral_constant<int, MOE_EPI_BF16>());
    if (dtype == MOE_EPI_F16) return f(std::integral_constant<int, MOE_EPI_F16>());
    f(std::integral_constant<int, MOE_EPI_F32>());
}

bool sizes_ok(int64_t tokens, int64_t experts, int64_t top_k) {
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= kMostExperts && top_k >= 1 &&
           top_k <= kMostChosen && top_k <= experts;
}
bool score_ok(int score) { return score == MOE_EPI_SOFTMAX || score == MOE_EPI_SIGMOID; }

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int moe_route_fwd(const void* logits, int dtype, const float* bias, int32_t* ids, float* weights,
                             int64_t tokens, int64_t experts, int64_t top_k, int64_t groups, int64_t top_groups,
                             int score, int group_score, int renormalise, float scale, void* stream) {
    if (!dtype_ok(dtype) || !score_ok(score) ||
        !(group_score == MOE_EPI_GROUP_MAX || group_score == MOE_EPI_GROUP_TOP2))
        return MOE_EPI_ERR_BAD_DTYPE;
    if (!sizes_ok(tokens, experts, top_k) || groups < 1 || groups > kMostGroups || experts % groups != 0 ||
        top_groups < 1 || top_groups > groups || top_k > top_groups * (experts / groups) ||
        (group_score == MOE_EPI_GROUP_TOP2 && groups > 1 && experts / groups < 2))
        return MOE_EPI_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return MOE_EPI_ERR_BAD_LIMIT;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if (!logits || !ids || !weights) return MOE_EPI_ERR_NULL_POINTER;
    const int e = elem_bytes(dtype);
    if (!aligned(logits, e) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range rl = range_of(logits, tokens * experts * e), rb = range_of(bias, bias ? 4 * experts : 0);
    const Range ri = range_of(ids, 4 * tokens * top_k), rw = range_of(weights, 4 * tokens * top_k);
    if (overlaps(ri, rl) || overlaps(ri, rb) || overlaps(rw, rl) || overlaps(rw, rb) || overlaps(ri, rw))
        return MOE_EPI_ERR_ALIAS;
    const Choice p = {static_cast<int>(experts), static_cast<int>(top_k), static_cast<int>(groups),
                      static_cast<int>(top_groups), score == MOE_EPI_SIGMOID, group_score == MOE_EPI_GROUP_TOP2,
                      renormalise != 0, scale};
    (void)hipGetLastError();
    by_type(dtype, [&](auto t) {
        by_size(p.experts, p.top_k, [&](auto l, auto n, auto s, auto k) {
            constexpr int L = decltype(l)::value;
            auto go = [&](auto kernel) {
                for (int64_t t = 0; t < tokens; t += kMostTokens) {
                    const int64_t here = tokens - t < kMostTokens ? tokens - t : kMostTokens;
                    hipLaunchKernelGGL(kernel, dim3(grid_for_rows(here, kBlock / L)), dim3(kBlock), 0,
                                       as_stream(stream), static_cast<const char*>(logits) + t * experts * e, bias,
                                       ids + t * top_k, weights + t * top_k, here, p);
                }
            };
            constexpr int T = decltype(t)::value, N = decltype(n)::value, S = decltype(s)::value, K = decltype(k)::value;
            bias || (p.top2 && p.groups > 1) ? go(route_kernel<T, L, N, S, K, true>)
                                             : go(route_kernel<T, L, N, S, K, false>);
        });
    });
    return launch_status();
}

extern "C" int moe_route_bwd(const float* grad_weights, const void* logits, int dtype, const int32_t* ids,
                             void* grad_logits, int64_t tokens, int64_t experts, int64_t top_k, int score,
                             int renormalise, float scale, void* stream) {
    if (!dtype_ok(dtype) || !score_ok(score)) return MOE_EPI_ERR_BAD_DTYPE;
    if (!sizes_ok(tokens, experts, top_k)) return MOE_EPI_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return MOE_EPI_ERR_BAD_LIMIT;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if (!grad_weights || !logits || !ids || !grad_logits) return MOE_EPI_ERR_NULL_POINTER;
    const int e = elem_bytes(dtype);
    if (!aligned(grad_weights, 4) || !aligned(logits, e) || !aligned(ids, 4) || !aligned(grad_logits, e))
        return MOE_EPI_ERR_MISALIGNED;
    const Range rg = range_of(grad_logits, tokens * experts * e);
    if (overlaps(rg, range_of(logits, tokens * experts * e)) || overlaps(rg, range_of(ids, 4 * tokens * top_k)) ||
        overlaps(rg, range_of(grad_weights, 4 * tokens * top_k)))
        return MOE_EPI_ERR_ALIAS;
    const Choice p = {static_cast<int>(experts), static_cast<int>(top_k), 1, 1, score == MOE_EPI_SIGMOID, false,
                      renormalise != 0, scale};
    (void)hipGetLastError();
    by_type(dtype, [&](auto t_) {
        by_size(p.experts, p.top_k, [&](auto l, auto n, auto s, auto k) {
            constexpr int L = decltype(l)::value;
            for (int64_t t = 0; t < tokens; t += kMostTokens) {
                const int64_t here = tokens - t < kMostTokens ? tokens - t : kMostTokens;
                hipLaunchKernelGGL((route_grad_kernel<decltype(t_)::value, L, decltype(n)::value, decltype(s)::value>),
                                   dim3(grid_for_rows(here, kBlock / L)), dim3(kBlock), 0, as_stream(stream),
                                   grad_weights + t * top_k, static_cast<const char*>(logits) + t * experts * e,
                                   ids + t * top_k, static_cast<char*>(grad_logits) + t * experts * e, here, p);
            }
        });
    });
    return launch_status();
}
