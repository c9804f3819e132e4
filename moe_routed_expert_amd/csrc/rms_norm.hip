// Root-mean-square norm with the residual's addition, and its gradients (gfx950).
#include "epi_common.h"
#include "int8_rows.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kRowsPerPart = 64;
constexpr int64_t kMostParts = 512;

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off, 64));
        v = o > v ? o : v;
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int w = 0; w < kBlock / 64; ++w) v = part[w] > v ? part[w] : v;
    __syncthreads();
    return v;
}

template <int T>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (T == MOE_EPI_BF16) {
        return __uint_as_float(static_cast<uint32_t>(to_bf16(v)) << 16);
    } else if constexpr (T == MOE_EPI_F16) {
        asm volatile("" : "+v"(v));
        return static_cast<float>(static_cast<_Float16>(v));
    } else {
        return v;
    }
}

template <int T, int W>
__global__ __launch_bounds__(kBlock) void rms_norm_kernel(const void* x, const void* residual, const void* weight,
                                                          float eps, void* out, void* residual_out, int8_t* q,
                                                          float* scale, float* rstd, int64_t rows, int64_t cols) {
    __shared__ float part[kBlock / 64];
    __shared__ uint32_t most_part[kBlock / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t at = r * cols;
        auto stream = [&](int64_t c) {
            float v = Elem<T>::load1(x, at + c);
            if (residual) v = rounded<T>(v + Elem<T>::load1(residual, at + c));
            return v;
        };
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kBlock) {
            const float h = stream(c);
            sum = __fmaf_rn(h, h, sum);
        }
        sum = row_sum<kBlock>(sum, part);
        const float n = 1.0f / sqrtf(sum / static_cast<float>(cols) + eps);
        uint32_t most = 0;
        if (q) {
            for (int64_t c = threadIdx.x; c < cols; c += kBlock) {
                const uint32_t m = magnitude(stream(c) * n * Elem<W>::load1(weight, c));
                most = m > most ? m : most;
            }
            most = block_max(most, most_part);
        }
        const RowScale s(most);
        for (int64_t c = threadIdx.x; c < cols; c += kBlock) {
            const float h = stream(c), y = h * n * Elem<W>::load1(weight, c);
            if (residual_out) Elem<T>::store1(residual_out, at + c, h);
            if (out) Elem<T>::store1(out, at + c, y);
            if (q) q[at + c] = static_cast<int8_t>(s.finite ? static_cast<int>(rintf(y * s.mul / s.den)) : 0);
        }
        if (threadIdx.x == 0) {
            if (scale) scale[r] = s.scale;
            if (rstd) rstd[r] = n;
        }
    }
}

template <int T, int W>
__global__ __launch_bounds__(kBlock) void grad_x_kernel(const void* grad_out, const void* h, const void* weight,
                                                        const float* rstd, const void* grad_residual, void* grad_x,
                                                        int64_t rows, int64_t cols) {
    __shared__ float part[kBlock / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t at = r * cols;
        const float n = rstd[r];
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += kBlock) {
            const float a = Elem<T>::load1(h, at + c) * n;
            sum = __fmaf_rn(Elem<T>::load1(grad_out, at + c) * Elem<W>::load1(weight, c), a, sum);
        }
        const float mean = row_sum<kBlock>(sum, part) / static_cast<float>(cols);
        for (int64_t c = threadIdx.x; c < cols; c += kBlock) {
            const float a = Elem<T>::load1(h, at + c) * n;
            const float g = Elem<T>::load1(grad_out, at + c) * Elem<W>::load1(weight, c);
            float d = n * __fmaf_rn(-a, mean, g);
            if (grad_residual) d += Elem<T>::load1(grad_residual, at + c);
            Elem<T>::store1(grad_x, at + c, d);
        }
    }
}

// parts[p][c]: the sum of grad_out * h * rstd over the rows of part p
template <int T>
__global__ __launch_bounds__(kBlock) void grad_weight_parts_kernel(const void* grad_out, const void* h,
                                                                   const float* rstd, float* parts, int64_t rows,
                                                                   int64_t cols) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x, p = blockIdx.y, n = gridDim.y;
    if (c >= cols) return;
    float sum = 0.0f;
    for (int64_t r = rows * p / n; r < rows * (p + 1) / n; ++r)
        sum = __fmaf_rn(Elem<T>::load1(grad_out, r * cols + c), Elem<T>::load1(h, r * cols + c) * rstd[r], sum);
    parts[p * cols + c] = sum;
}

template <int W>
__global__ __launch_bounds__(kBlock) void grad_weight_kernel(const float* parts, void* grad_weight, int64_t n,
                                                             int64_t cols) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
    if (c >= cols) return;
    float sum = 0.0f;
    for (int64_t p = 0; p < n; ++p) sum += parts[p * cols + c];
    Elem<W>::store1(grad_weight, c, sum);
}

int64_t parts_of(int64_t rows) {
    const int64_t n = (rows + kRowsPerPart - 1) / kRowsPerPart;
    return n < 1 ? 1 : (n > kMostParts ? kMostParts : n);
}

bool sizes_ok(int64_t rows, int64_t cols, int64_t* bytes4) {
    return bytes_ok(rows, cols, 4, bytes4) && row_fits_u32_offsets(cols, 4);
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

extern "C" int rms_norm_fwd(const void* x, const void* residual, int dtype, const void* weight, int w_dtype, float eps,
                            void* out, void* residual_out, int8_t* q, float* scale, float* rstd, int64_t rows,
                            int64_t cols, void* stream) {
    if (!dtype_ok(dtype) || !(w_dtype == dtype || w_dtype == MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    int64_t all;
    if (!sizes_ok(rows, cols, &all)) return MOE_EPI_ERR_BAD_SHAPE;
    if (!(eps >= 0.0f) || !isfinite(eps)) return MOE_EPI_ERR_BAD_LIMIT;
    if (rows == 0) return MOE_EPI_SUCCESS;
    if (!x || !weight || (!out && !q) || (q != nullptr) != (scale != nullptr) || (residual_out && !residual))
        return MOE_EPI_ERR_NULL_POINTER;
    const int e = elem_bytes(dtype);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(weight, elem_bytes(w_dtype)) || !aligned(out, e) ||
        !aligned(residual_out, e) || !aligned(scale, 4) || !aligned(rstd, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const int64_t n = rows * cols;
    const Range in[] = {range_of(x, n * e), range_of(residual, residual ? n * e : 0),
                        range_of(weight, cols * elem_bytes(w_dtype))};
    const Range to[] = {range_of(out, out ? n * e : 0), range_of(residual_out, residual_out ? n * e : 0),
                        range_of(q, q ? n : 0), range_of(scale, scale ? 4 * rows : 0),
                        range_of(rstd, rstd ? 4 * rows : 0)};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlaps(to[i], in[j]) && !(i == 1 && j == 1 && residual_out == residual)) return MOE_EPI_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(to[i], to[j])) return MOE_EPI_ERR_ALIAS;
    }
    (void)hipGetLastError();
    by_types(dtype, w_dtype, [&](auto t, auto w) {
        hipLaunchKernelGGL((rms_norm_kernel<decltype(t)::value, decltype(w)::value>), dim3(grid_for_rows(rows, 1)),
                           dim3(kBlock), 0, as_stream(stream), x, residual, weight, eps, out, residual_out, q, scale,
                           rstd, rows, cols);
    });
    return launch_status();
}

extern "C" int64_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
    int64_t all;
    if (!sizes_ok(rows, cols, &all)) return -1;
    return parts_of(rows) * cols * 4;
}

extern "C" int rms_norm_bwd(const void* grad_out, const void* h, int dtype, const void* weight, int w_dtype,
                            const float* rstd, const void* grad_residual, void* grad_x, void* grad_weight,
                            void* workspace, int64_t workspace_bytes, int64_t rows, int64_t cols, void* stream) {
    if (!dtype_ok(dtype) || !(w_dtype == dtype || w_dtype == MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    int64_t all;
    if (!sizes_ok(rows, cols, &all)) return MOE_EPI_ERR_BAD_SHAPE;
    const int64_t need = grad_weight ? parts_of(rows) * cols * 4 : 0;
    if (rows == 0 && !grad_weight) return MOE_EPI_SUCCESS;
    if (rows != 0 && (!grad_out || !h || !weight || !rstd || !grad_x)) return MOE_EPI_ERR_NULL_POINTER;
    if (grad_weight && !workspace) return MOE_EPI_ERR_NULL_POINTER;
    if (workspace_bytes < need) return MOE_EPI_ERR_BAD_SHAPE;
    const int e = elem_bytes(dtype), ew = elem_bytes(w_dtype);
    if (!aligned(grad_out, e) || !aligned(h, e) || !aligned(weight, ew) || !aligned(rstd, 4) ||
        !aligned(grad_residual, e) || !aligned(grad_x, e) || !aligned(grad_weight, ew) ||
        (grad_weight && !aligned(workspace, 16)))
        return MOE_EPI_ERR_MISALIGNED;
    const int64_t n = rows * cols * e;
    const Range in[] = {range_of(grad_out, n), range_of(h, n), range_of(weight, rows ? cols * ew : 0),
                        range_of(rstd, 4 * rows), range_of(grad_residual, grad_residual ? n : 0)};
    const Range to[] = {range_of(grad_x, n), range_of(grad_weight, grad_weight ? cols * ew : 0),
                        range_of(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlaps(to[i], r)) return MOE_EPI_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(to[i], to[j])) return MOE_EPI_ERR_ALIAS;
    }
    (void)hipGetLastError();
    const hipStream_t st = as_stream(stream);
    float* parts = static_cast<float*>(workspace);
    by_types(dtype, w_dtype, [&](auto t, auto w) {
        constexpr int T = decltype(t)::value, W = decltype(w)::value;
        if (rows)
            hipLaunchKernelGGL((grad_x_kernel<T, W>), dim3(grid_for_rows(rows, 1)), dim3(kBlock), 0, st, grad_out, h,
                               weight, rstd, grad_residual, grad_x, rows, cols);
        if (grad_weight) {
            const unsigned blocks = static_cast<unsigned>((cols + kBlock - 1) / kBlock);
            const unsigned n_parts = static_cast<unsigned>(parts_of(rows));
            hipLaunchKernelGGL((grad_weight_parts_kernel<T>), dim3(blocks, n_parts), dim3(kBlock), 0, st, grad_out, h,
                               rstd, parts, rows, cols);
            hipLaunchKernelGGL((grad_weight_kernel<W>), dim3(blocks), dim3(kBlock), 0, st, parts, grad_weight,
                               static_cast<int64_t>(n_parts), cols);
        }
    });
    return launch_status();
}
