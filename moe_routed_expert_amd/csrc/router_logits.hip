// The router's product and its gradients (gfx950).
#include <type_traits>

#include "epi_common.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMostExperts = 1024;

template <int T, int W>
__global__ __launch_bounds__(kBlock) void logits_kernel(const void* x, const void* weight, float* logits,
                                                        int64_t tokens, int64_t hidden, int64_t experts) {
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
        for (int64_t e = threadIdx.x / 64; e < experts; e += kBlock / 64) {
            float sum = 0.0f;
            for (int64_t h = threadIdx.x & 63; h < hidden; h += 64)
                sum = __fmaf_rn(Elem<T>::load1(x, t * hidden + h), Elem<W>::load1(weight, e * hidden + h), sum);
            sum = group_sum<64>(sum);
            if ((threadIdx.x & 63) == 0) logits[t * experts + e] = sum;
        }
}

template <int T, int W>
__global__ __launch_bounds__(kBlock) void grad_x_kernel(const float* grad, const void* weight, void* grad_x,
                                                        int64_t tokens, int64_t hidden, int64_t experts) {
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
        for (int64_t h = threadIdx.x; h < hidden; h += kBlock) {
            float sum = 0.0f;
            for (int64_t e = 0; e < experts; ++e)
                sum = __fmaf_rn(grad[t * experts + e], Elem<W>::load1(weight, e * hidden + h), sum);
            Elem<T>::store1(grad_x, t * hidden + h, sum);
        }
}

template <int T, int W>
__global__ __launch_bounds__(kBlock) void grad_weight_kernel(const float* grad, const void* x, void* grad_weight,
                                                             int64_t tokens, int64_t hidden, int64_t experts) {
    const int64_t e = blockIdx.y, h = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
    if (h >= hidden) return;
    float sum = 0.0f;
    for (int64_t t = 0; t < tokens; ++t)
        sum = __fmaf_rn(grad[t * experts + e], Elem<T>::load1(x, t * hidden + h), sum);
    Elem<W>::store1(grad_weight, e * hidden + h, sum);
}

bool sizes_ok(int64_t tokens, int64_t hidden, int64_t experts) {
    int64_t a;
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= kMostExperts &&
           bytes_ok(tokens, hidden, 4, &a) && bytes_ok(experts, hidden, 4, &a) && bytes_ok(tokens, experts, 4, &a) &&
           row_fits_u32_offsets(hidden, 4);
}

template <class F>
void by_types(int t, int w, F f) {
    const std::integral_constant<int, MOE_EPI_BF16> bf16;
    const std::integral_constant<int, MOE_EPI_F16> f16;
    const std::integral_constant<int, MOE_EPI_F32> f32;
    if (t == MOE_EPI_BF16) return w == MOE_EPI_F32 ? f(bf16, f32) : f(bf16, bf16);
    if (t == MOE_EPI_F16) return w == MOE_EPI_F32 ? f(f16, f32) : f(f16, f16);
    f(f32, f32);
}

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int64_t moe_router_logits_workspace_bytes(int64_t tokens, int64_t hidden, int64_t experts) {
    return sizes_ok(tokens, hidden, experts) ? 0 : -1;
}

extern "C" int moe_router_logits_fwd(const void* x, int dtype, const void* weight, int w_dtype, float* logits,
                                     void* workspace, int64_t workspace_bytes, int64_t tokens, int64_t hidden,
                                     int64_t experts, void* stream) {
    if (!dtype_ok(dtype) || !(w_dtype == dtype || w_dtype == MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    if (!sizes_ok(tokens, hidden, experts)) return MOE_EPI_ERR_BAD_SHAPE;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if (!x || !weight || !logits) return MOE_EPI_ERR_NULL_POINTER;
    const int64_t need = moe_router_logits_workspace_bytes(tokens, hidden, experts);
    if (need && !workspace) return MOE_EPI_ERR_NULL_POINTER;
    if (workspace_bytes < need) return MOE_EPI_ERR_BAD_SHAPE;
    const int e = elem_bytes(dtype), ew = elem_bytes(w_dtype);
    if (!aligned(x, e) || !aligned(weight, ew) || !aligned(logits, 4) || (need && !aligned(workspace, 16)))
        return MOE_EPI_ERR_MISALIGNED;
    const Range rx = range_of(x, tokens * hidden * e), rw = range_of(weight, experts * hidden * ew);
    const Range rl = range_of(logits, tokens * experts * 4), rs = range_of(workspace, need);
    if (overlaps(rl, rx) || overlaps(rl, rw) || overlaps(rs, rx) || overlaps(rs, rw) || overlaps(rs, rl))
        return MOE_EPI_ERR_ALIAS;
    (void)hipGetLastError();
    by_types(dtype, w_dtype, [&](auto t, auto w) {
        hipLaunchKernelGGL((logits_kernel<decltype(t)::value, decltype(w)::value>), dim3(grid_for_rows(tokens, 1)),
                           dim3(kBlock), 0, as_stream(stream), x, weight, logits, tokens, hidden, experts);
    });
    return launch_status();
}

extern "C" int64_t moe_router_logits_bwd_workspace_bytes(int64_t tokens, int64_t hidden, int64_t experts) {
    return sizes_ok(tokens, hidden, experts) ? 0 : -1;
}

extern "C" int moe_router_logits_bwd(const float* grad_logits, const void* x, int dtype, const void* weight,
                                     int w_dtype, void* grad_x, void* grad_weight, void* workspace,
                                     int64_t workspace_bytes, int64_t tokens, int64_t hidden, int64_t experts,
                                     void* stream) {
    if (!dtype_ok(dtype) || !(w_dtype == dtype || w_dtype == MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    if (!sizes_ok(tokens, hidden, experts)) return MOE_EPI_ERR_BAD_SHAPE;
    const int64_t need = grad_weight ? moe_router_logits_bwd_workspace_bytes(tokens, hidden, experts) : 0;
    if (tokens == 0 && !grad_weight) return MOE_EPI_SUCCESS;
    if (!grad_x && !grad_weight) return MOE_EPI_ERR_NULL_POINTER;
    if (tokens && (!grad_logits || (grad_x && !weight) || (grad_weight && !x))) return MOE_EPI_ERR_NULL_POINTER;
    if (need && !workspace) return MOE_EPI_ERR_NULL_POINTER;
    if (workspace_bytes < need) return MOE_EPI_ERR_BAD_SHAPE;
    const int e = elem_bytes(dtype), ew = elem_bytes(w_dtype);
    if (!aligned(grad_logits, 4) || !aligned(x, e) || !aligned(weight, ew) || !aligned(grad_x, e) ||
        !aligned(grad_weight, ew) || (need && !aligned(workspace, 16)))
        return MOE_EPI_ERR_MISALIGNED;
    const int64_t nx = tokens * hidden * e, nw = experts * hidden * ew;
    const Range in[] = {range_of(grad_logits, tokens * experts * 4), range_of(x, grad_weight ? nx : 0),
                        range_of(weight, grad_x ? nw : 0)};
    const Range to[] = {range_of(grad_x, grad_x ? nx : 0), range_of(grad_weight, grad_weight ? nw : 0),
                        range_of(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlaps(to[i], r)) return MOE_EPI_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(to[i], to[j])) return MOE_EPI_ERR_ALIAS;
    }
    (void)hipGetLastError();
    const hipStream_t st = as_stream(stream);
    by_types(dtype, w_dtype, [&](auto t, auto w) {
        constexpr int T = decltype(t)::value, W = decltype(w)::value;
        if (grad_x && tokens)
            hipLaunchKernelGGL((grad_x_kernel<T, W>), dim3(grid_for_rows(tokens, 1)), dim3(kBlock), 0, st, grad_logits,
                               weight, grad_x, tokens, hidden, experts);
        if (grad_weight)
            hipLaunchKernelGGL((grad_weight_kernel<T, W>),
                               dim3(static_cast<unsigned>((hidden + kBlock - 1) / kBlock),
                                    static_cast<unsigned>(experts)),
                               dim3(kBlock), 0, st, grad_logits, x, grad_weight, tokens, hidden, experts);
    });
    return launch_status();
}
