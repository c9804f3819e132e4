// Choice of each token's experts, the chosen experts' weights, and their gradient (gfx950).
#include <type_traits>

#include "epi_common.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kMostExperts = 1024, kMostGroups = 64, kMostChosen = 64;
constexpr float kInf = __builtin_inff();

struct Choice {
    int experts, top_k, groups, top_groups;
    bool sigmoid, top2, renormalise;
    float scale;
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// One wavefront per token. An expert's place is the number of experts that come before it.
template <int T>
__global__ __launch_bounds__(64) void route_kernel(const void* logits, const float* bias, int32_t* ids, float* weights,
                                                   int64_t tokens, Choice p) {
    __shared__ double c[kMostExperts], of_group[kMostGroups];
    __shared__ int chosen[kMostChosen];
    const int lane = threadIdx.x, size = p.experts / p.groups;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        auto logit = [&](int e) { return Elem<T>::load1(logits, t * p.experts + e); };
        float m = -kInf;
        bool bad = false;
        for (int e = lane; e < p.experts; e += 64) {
            const float l = logit(e);
            bad |= l != l || (!p.sigmoid && l == kInf);
            m = fmaxf(m, l);
        }
        m = wave_max(m);
        bad = __any(bad);
        double sum = 0.0;
        if (!p.sigmoid) {
            for (int e = lane; e < p.experts; e += 64) sum += exp(static_cast<double>(logit(e)) - m);
            sum = wave_sum(sum);
        }
        auto score = [&](float l) {
            return p.sigmoid ? sigmoid64(l) : exp(static_cast<double>(l) - m) / sum;
        };
        for (int e = lane; e < p.experts; e += 64) {
            const float l = logit(e);
            double v = bias ? score(l) + static_cast<double>(bias[e]) : static_cast<double>(l);
            if (!(v > -kInf) || !(l > -kInf)) v = -kInf;  // NaN too
            c[e] = v;
        }
        if (lane < kMostChosen) chosen[lane] = -1;
        __syncthreads();
        if (lane < p.groups) {
            double a = -kInf, b = -kInf;
            for (int i = 0; i < size; ++i) {
                double v = c[lane * size + i];
                if (p.top2 && !bias && v > -kInf) v = score(static_cast<float>(v));
                if (v > a) {
                    b = a;
                    a = v;
                } else if (v > b) {
                    b = v;
                }
            }
            of_group[lane] = p.top2 && p.groups > 1 ? a + b : a;
        }
        __syncthreads();
        bool keep = false;
        if (lane < p.groups) {
            int before = 0;
            for (int g = 0; g < p.groups; ++g)
                before += of_group[g] > of_group[lane] || (of_group[g] == of_group[lane] && g < lane);
            keep = before < p.top_groups;
        }
        const uint64_t mask = __ballot(keep);
        for (int e = lane; e < p.experts; e += 64) {
            if (!(mask >> (e / size) & 1) || !(c[e] > -kInf)) continue;
            int before = 0;
            for (int i = 0; i < p.experts; ++i)
                before += (mask >> (i / size) & 1) && (c[i] > c[e] || (c[i] == c[e] && i < e));
            if (before < p.top_k) chosen[before] = e;
        }
        __syncthreads();
        const int id = lane < p.top_k ? chosen[lane] : -1;
        const float l = id >= 0 ? logit(id) : -kInf;
        const float most = wave_max(l);
        double w = 0.0;
        if (id >= 0) {
            if (!p.renormalise)
                w = score(l);
            else if (!p.sigmoid)
                w = exp(static_cast<double>(l) - most);
            else  // sigmoid(l) over e^min(most, 0), which does not underflow
                w = exp(fmin(static_cast<double>(l), 0.0) - fmin(static_cast<double>(most), 0.0)) /
                    (1.0 + exp(-fabs(static_cast<double>(l))));
        }
        if (p.renormalise) {
            const double all = wave_sum(w);
            w = id >= 0 ? w / all : 0.0;
        }
        if (lane < p.top_k) {
            ids[t * p.top_k + lane] = id;
            weights[t * p.top_k + lane] = bad ? __builtin_nanf("") : static_cast<float>(w * p.scale);
        }
        __syncthreads();
    }
}

template <int T>
__global__ __launch_bounds__(64) void route_grad_kernel(const float* grad_weights, const void* logits,
                                                        const int32_t* ids, void* grad_logits, int64_t tokens,
                                                        Choice p) {
    __shared__ double part[kMostChosen];
    __shared__ int chosen[kMostChosen];
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        auto logit = [&](int64_t e) { return static_cast<double>(Elem<T>::load1(logits, t * p.experts + e)); };
        int id = lane < p.top_k ? ids[t * p.top_k + lane] : -1;
        if (id < 0 || id >= p.experts) id = -1;
        const double u = id >= 0 ? static_cast<double>(grad_weights[t * p.top_k + lane]) * p.scale : 0.0;
        const double l = id >= 0 ? logit(id) : -kInf;
        double m = -kInf, sum = 0.0;
        if (!p.sigmoid && !p.renormalise) {
            for (int e = lane; e < p.experts; e += 64) m = fmax(m, logit(e));
            m = static_cast<double>(wave_max(static_cast<float>(m)));
            for (int e = lane; e < p.experts; e += 64) sum += m > -kInf ? exp(logit(e) - m) : 0.0;
            sum = wave_sum(sum);
        }
        auto softmax = [&](double v) { return m > -kInf ? exp(v - m) / sum : 0.0; };
        double d = 0.0, dot = 0.0;
        if (p.renormalise) {
            const double most = wave_max(static_cast<float>(l));
            double v = 0.0;
            if (id >= 0 && most > -kInf)
                v = p.sigmoid ? exp(fmin(l, 0.0) - fmin(most, 0.0)) / (1.0 + exp(-fabs(l))) : exp(l - most);
            const double all = wave_sum(v);
            v = all > 0.0 || all != all ? v / all : 0.0;
            dot = wave_sum(u * v);
            d = id >= 0 ? v * (u - dot) : 0.0;
            if (p.sigmoid && id >= 0) d *= 1.0 / (1.0 + exp(l));
        } else if (p.sigmoid) {
            const double s = 1.0 / (1.0 + exp(-l));
            d = id >= 0 ? u * s / (1.0 + exp(l)) : 0.0;
        } else {
            dot = wave_sum(id >= 0 ? u * softmax(l) : 0.0);
            d = u;
        }
        part[lane] = d;
        chosen[lane] = id;
        __syncthreads();
        for (int e = lane; e < p.experts; e += 64) {
            double g = 0.0;
            for (int j = 0; j < p.top_k; ++j) g += chosen[j] == e ? part[j] : 0.0;
            if (!p.sigmoid && !p.renormalise) g = softmax(logit(e)) * (g - dot);
            Elem<T>::store1(grad_logits, t * p.experts + e, static_cast<float>(g));
        }
        __syncthreads();
    }
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
    const dim3 grid(grid_for_rows(tokens, 1)), block(64);
    const hipStream_t st = as_stream(stream);
    switch (dtype) {
        case MOE_EPI_BF16: hipLaunchKernelGGL((route_kernel<MOE_EPI_BF16>), grid, block, 0, st, logits, bias, ids, weights, tokens, p); break;
        case MOE_EPI_F16: hipLaunchKernelGGL((route_kernel<MOE_EPI_F16>), grid, block, 0, st, logits, bias, ids, weights, tokens, p); break;
        default: hipLaunchKernelGGL((route_kernel<MOE_EPI_F32>), grid, block, 0, st, logits, bias, ids, weights, tokens, p); break;
    }
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
    const dim3 grid(grid_for_rows(tokens, 1)), block(64);
    const hipStream_t st = as_stream(stream);
    switch (dtype) {
        case MOE_EPI_BF16: hipLaunchKernelGGL((route_grad_kernel<MOE_EPI_BF16>), grid, block, 0, st, grad_weights, logits, ids, grad_logits, tokens, p); break;
        case MOE_EPI_F16: hipLaunchKernelGGL((route_grad_kernel<MOE_EPI_F16>), grid, block, 0, st, grad_weights, logits, ids, grad_logits, tokens, p); break;
        default: hipLaunchKernelGGL((route_grad_kernel<MOE_EPI_F32>), grid, block, 0, st, grad_weights, logits, ids, grad_logits, tokens, p); break;
    }
    return launch_status();
}
