// Root-mean-square norm with the residual's addition, and its gradients (gfx950).
//
//   h = round(x + residual),  n = 1 / sqrt(mean(h^2) + eps),  y = h n weight
//   grad_x = n (g - a mean(g a)) + grad_residual,  grad_weight = sum_r grad_out a
//   with a = h n, g = grad_out weight
//
// Bound by memory: a row is read once and kept in registers, as it is stored,
// between its sum and its results; 65536 x 7168 bf16 with the residual 639 us
// (5.9 TB/s), 16384 x 7168 with rows also in 8 bits 175 us (6.0 TB/s).
//
// Lanes of a row are chosen as in quantize_rows.hip, which has both sides of
// each: the fewest that hold it with four vectors each, and up to 512 rows more
// lanes with one or two. The order of a row's sum is that of its vectors and
// not of its lanes, so the choice does not show in the results.
//
// Gradients: a lane also keeps the sums of its columns of the weight's gradient
// over the rows of its block, of which there are up to four per CU; the blocks'
// sums are added by a second launch. 32768 x 7168 bf16 365 + 9 us (5.2 TB/s);
// with four vectors a lane instead of two the registers held one block a CU. Rows
// wider than 8192 columns are read by elements, twice for grad_x and once more for
// the weight: 8192 x 12288 351 us, where the bytes take 125.
#include <type_traits>

#include "bf16_pieces.h"
#include "epi_common.h"
#include "int8_rows.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;              // threads, or the lanes of a row if they are more
constexpr int64_t kFewRows = 512;
constexpr int64_t kMostRows = 1 << 20;   // of a launch
constexpr int64_t kRowsPerPart = 64;
constexpr int64_t kMostParts = 512;

// ---- vectors of 8 elements --------------------------------------------------------

// Vector v of a row of cols elements, of which the last may have fewer than 8.
// kAligned: whole vectors at 16-byte addresses, read and written once.
template <int T, bool kAligned>
struct Vec {
    typedef Piece8<T> P;
    typedef typename P::Raw Raw;
    __device__ __forceinline__ static Raw load(const char* row, uint32_t v, uint32_t cols) {
        const uint32_t e = v * 8;
        if (e >= cols) return Raw{};
        const char* p = row + e * P::kBytes;
        if constexpr (kAligned) {
            Raw r;
#pragma unroll
            for (int i = 0; i < P::kWords; ++i) r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 16 * i));
            return r;
        } else {
            return P::load_first(p, cols - e);
        }
    }
    __device__ __forceinline__ static void store(char* row, uint32_t v, uint32_t cols, const Raw& r) {
        const uint32_t e = v * 8;
        if (e >= cols) return;
        char* p = row + e * P::kBytes;
        if constexpr (kAligned) {
#pragma unroll
            for (int i = 0; i < P::kWords; ++i) __builtin_nontemporal_store(r.w[i], reinterpret_cast<u32x4*>(p + 16 * i));
        } else if (e + 8 <= cols) {
#pragma unroll
            for (int i = 0; i < P::kWords; ++i) *reinterpret_cast<typename P::loose*>(p + 16 * i) = r.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e + i < cols) {
                    if constexpr (T == MOE_EPI_F32)
                        reinterpret_cast<uint32_t*>(p)[i] = r.w[i / 4][i % 4];
                    else
                        reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r.w[0][i / 2] >> (16 * (i % 2)));
                }
        }
    }
    __device__ __forceinline__ static Raw round(float (&f)[8]) {
        if constexpr (T == MOE_EPI_F32) {
            const typename Elem<T>::Raw r = Elem<T>::pack(f);
            return Raw{{r.a, r.b}};
        } else {
            if constexpr (T == MOE_EPI_F16) {
                // finished float32 values: not a product that is rounded straight to half
#pragma unroll
                for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(f[i]));
            }
            return Raw{{Elem<T>::pack(f)}};
        }
    }
};

// Vector v of the weight, which is of the rows' type T or float32.
template <int T, bool kAligned>
struct Weight {
    u32x4 w[2];
    __device__ __forceinline__ void load(const char* weight, bool f32, uint32_t v, uint32_t cols) {
        const uint32_t e = v * 8;
        if (e >= cols) {
            w[0] = w[1] = u32x4{0, 0, 0, 0};
        } else if (T == MOE_EPI_F32 || f32) {
            typedef Piece8<MOE_EPI_F32> P;
            const P::Raw r = kAligned ? P::load(weight + e * 4) : P::load_first(weight + e * 4, cols - e);
            w[0] = r.w[0];
            w[1] = r.w[1];
        } else {
            typedef Piece8<T> P;
            w[0] = (kAligned ? P::load(weight + e * 2) : P::load_first(weight + e * 2, cols - e)).w[0];
        }
    }
    __device__ __forceinline__ void widen(bool f32, float (&f)[8]) const {
        if (T == MOE_EPI_F32 || f32)
            Piece8<MOE_EPI_F32>::widen(Piece8<MOE_EPI_F32>::Raw{{w[0], w[1]}}, f);
        else if constexpr (T != MOE_EPI_F32)
            Elem<T>::unpack(w[0], f);
    }
};

// ---- over the L lanes of a row ------------------------------------------------------

// As group_sum, lowest bit first.
template <int G>
__device__ __forceinline__ float group_sum_up(float v) {
#pragma unroll
    for (int off = 1; off < G; off *= 2) v += __shfl_xor(v, off, 64);
    return v;
}

// The sum of a row's vectors' values, of which lane l has s[k] of vector
// l + k L. The order depends on the vectors alone, so that a row's result is
// the same whatever lanes it is given: 64 vectors by halves, lowest bit first,
// then those sums one after the other. part: kVecs L / 64 words, at least 1.
template <int L, int V>
__device__ __forceinline__ float vectors_sum(float (&s)[V], float* part) {
    constexpr int kLanes = L < 64 ? L : 64;
#pragma unroll
    for (int k = 0; k < V; ++k) s[k] = group_sum_up<kLanes>(s[k]);
    if constexpr (L < 64) {
        static_assert(V * L <= 64 || 64 % L == 0, "");
        // vectors of one lane that belong to the same 64: 64 / L of them
        constexpr int kSame = 64 / L < V ? 64 / L : V;
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < V; c += kSame) {
            float t[kSame];
#pragma unroll
            for (int i = 0; i < kSame; ++i) t[i] = s[c + i];
#pragma unroll
            for (int d = 1; d < kSame; d *= 2)
#pragma unroll
                for (int i = 0; i + d < kSame; i += 2 * d) t[i] += t[i + d];
            sum += t[0];
        }
        return sum;
    } else if constexpr (L == 64) {
        float sum = s[0];
#pragma unroll
        for (int k = 1; k < V; ++k) sum += s[k];
        return sum;
    } else {
        constexpr int kWaves = L / 64;
        const int wave = threadIdx.x / 64, first = wave / kWaves * kWaves * V;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < V; ++k) part[first + k * kWaves + wave % kWaves] = s[k];
        __syncthreads();
        float sum = part[first];
#pragma unroll
        for (int i = 1; i < kWaves * V; ++i) sum += part[first + i];
        return sum;
    }
}

template <int L>
__device__ __forceinline__ uint32_t lanes_most(uint32_t v, uint32_t* part) {
#pragma unroll
    for (int off = (L < 64 ? L : 64) / 2; off > 0; off >>= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off, 64));
        v = o > v ? o : v;
    }
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        const int first = threadIdx.x / L * (L / 64);
#pragma unroll
        for (int w = 0; w < L / 64; ++w) v = part[first + w] > v ? part[first + w] : v;
    }
    return v;
}

// ---- norm -----------------------------------------------------------------------------

// L lanes per row, V vectors in a lane. kInt8: also (or only) 8-bit rows.
// kWide: rows of more vectors, of which those that the lanes do not hold are
// read again; the stream from residual_out if it is written.
template <int T, int L, int V, bool kAligned, bool kInt8, bool kWide>
__global__ __launch_bounds__(L > kBlock ? L : kBlock) void rms_norm_kernel(
    const char* x, const char* residual, const char* __restrict__ weight, bool w32, float eps, char* __restrict__ out,
    char* residual_out, int8_t* __restrict__ q, float* __restrict__ scale, float* __restrict__ rstd, uint32_t rows,
    uint32_t cols) {
    typedef Vec<T, kAligned> X;
    constexpr int kThreads = L > kBlock ? L : kBlock, kRows = kThreads / L;
    __shared__ float part[kThreads / 64 * V];
    __shared__ uint32_t most_part[kThreads / 64];
    const uint32_t lane = threadIdx.x % L, r0 = blockIdx.x * kRows + group_in_block<L>();
    const bool live = r0 < rows;
    const int64_t r = live ? r0 : rows - 1, at = r * cols;  // spare lanes of the last block repeat its last row
    const char* xr = x + at * Elem<T>::kBytes;
    const char* rr = residual ? residual + at * Elem<T>::kBytes : nullptr;
    char* hr = residual_out ? residual_out + at * Elem<T>::kBytes : nullptr;
    typename X::Raw h[V];
    Weight<T, kAligned> w[V];
    float s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = X::load(xr, lane + k * L, cols);
    auto add = [&](typename X::Raw& a, const typename X::Raw& b) {
        float f[8], g[8];
        X::P::widen(a, f);
        X::P::widen(b, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        a = X::round(f);
    };
    auto squares = [&](const typename X::Raw& a) {
        float f[8], sum = 0.0f;
        X::P::widen(a, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __fmaf_rn(f[i], f[i], sum);
        return sum;
    };
    if (residual) {
        typename X::Raw b[V];
#pragma unroll
        for (int k = 0; k < V; ++k) b[k] = X::load(rr, lane + k * L, cols);
#pragma unroll
        for (int k = 0; k < V; ++k) w[k].load(weight, w32, lane + k * L, cols);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            add(h[k], b[k]);
            if (residual_out && live) X::store(hr, lane + k * L, cols, h[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k].load(weight, w32, lane + k * L, cols);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) s[k] = squares(h[k]);
    if constexpr (kWide) {
        for (uint32_t v = lane + V * L; v * 8 < cols; v += L) {
            typename X::Raw a = X::load(xr, v, cols);
            if (residual) {
                add(a, X::load(rr, v, cols));
                if (residual_out && live) X::store(hr, v, cols, a);
            }
            s[0] += squares(a);
        }
    }
    const float n = 1.0f / sqrtf(vectors_sum<L, V>(s, part) / static_cast<float>(cols) + eps);
    auto normed = [&](const typename X::Raw& a, const Weight<T, kAligned>& b, float (&y)[8]) {
        float g[8];
        X::P::widen(a, y);
        b.widen(w32, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * n * g[i];
    };
    auto again = [&](uint32_t v, Weight<T, kAligned>& b) {  // a vector that the lanes do not hold
        b.load(weight, w32, v, cols);
        if (residual_out && live) return X::load(hr, v, cols);
        typename X::Raw a = X::load(xr, v, cols);
        if (residual) add(a, X::load(rr, v, cols));
        return a;
    };
    uint32_t most = 0;
    if constexpr (kInt8) {
        auto grow = [&](const typename X::Raw& a, const Weight<T, kAligned>& b) {
            float y[8];
            normed(a, b, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = magnitude(y[i]);
                most = m > most ? m : most;
            }
        };
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (kAligned || (lane + k * L) * 8 < cols) grow(h[k], w[k]);
        if constexpr (kWide)
            for (uint32_t v = lane + V * L; v * 8 < cols; v += L) {
                Weight<T, kAligned> b;
                const typename X::Raw a = again(v, b);
                grow(a, b);
            }
        most = lanes_most<L>(most, most_part);
    }
    const RowScale rs(most);
    if (!live) return;
    auto put = [&](uint32_t v, const typename X::Raw& a, const Weight<T, kAligned>& b) {
        if (v * 8 >= cols) return;
        float y[8];
        normed(a, b, y);
        if constexpr (kInt8) {
            const u32x2 bytes = rs.finite ? quantize8(rs, y) : u32x2{0u, 0u};
            int8_t* to = q + at + v * 8;
            if constexpr (kAligned) {
                __builtin_nontemporal_store(bytes, reinterpret_cast<u32x2*>(to));
            } else if (v * 8 + 8 <= cols) {
                typedef u32x2 loose __attribute__((aligned(1)));
                *reinterpret_cast<loose*>(to) = bytes;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (v * 8 + i < cols) to[i] = static_cast<int8_t>(bytes[i / 4] >> (8 * (i % 4)));
            }
        }
        if (!kInt8 || out) X::store(out + at * Elem<T>::kBytes, v, cols, X::round(y));
    };
#pragma unroll
    for (int k = 0; k < V; ++k) put(lane + k * L, h[k], w[k]);
    if constexpr (kWide)
        for (uint32_t v = lane + V * L; v * 8 < cols; v += L) {
            Weight<T, kAligned> b;
            const typename X::Raw a = again(v, b);
            put(v, a, b);
        }
    if (lane == 0) {
        if (kInt8) scale[r] = rs.scale;
        if (rstd) rstd[r] = n;
    }
}

struct NormCall {
    const char *x, *residual, *weight;
    bool w32;
    float eps;
    char *out, *residual_out;
    int8_t* q;
    float *scale, *rstd;
    int64_t rows, cols;
};

template <int T>
void launch_norm(const NormCall& c, hipStream_t st) {
    const int e = Elem<T>::kBytes;
    const bool fit = c.cols % 8 == 0 && aligned(c.x, 16) && aligned(c.residual, 16) && aligned(c.weight, 16) &&
                     aligned(c.out, 16) && aligned(c.residual_out, 16) && aligned(c.q, 8);
    auto go = [&](auto lanes, auto vecs, auto is_fit, auto wide) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value, kThreads = L > kBlock ? L : kBlock;
        constexpr bool kFit = decltype(is_fit)::value, kWide = decltype(wide)::value;
        for (int64_t r = 0; r < c.rows; r += kMostRows) {
            const int64_t here = c.rows - r < kMostRows ? c.rows - r : kMostRows, at = r * c.cols;
            auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, dim3(grid_for_rows(here, kThreads / L)), dim3(kThreads), 0, st, c.x + at * e,
                                   c.residual ? c.residual + at * e : nullptr, c.weight, c.w32, c.eps,
                                   c.out ? c.out + at * e : nullptr, c.residual_out ? c.residual_out + at * e : nullptr,
                                   c.q ? c.q + at : nullptr, c.scale ? c.scale + r : nullptr,
                                   c.rstd ? c.rstd + r : nullptr, static_cast<uint32_t>(here),
                                   static_cast<uint32_t>(c.cols));
            };
            c.q ? launch(rms_norm_kernel<T, L, V, kFit, true, kWide>) : launch(rms_norm_kernel<T, L, V, kFit, false, kWide>);
        }
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 16> l16;
    const std::integral_constant<int, 64> l64;
    const std::integral_constant<int, 256> l256;
    const std::integral_constant<int, 512> l512;
    const std::integral_constant<int, 1024> l1024;
    const std::true_type yes;
    const std::false_type no;
    const int64_t vecs = (c.cols + 7) / 8;
    if (vecs > 2048) return fit ? go(l1024, two, yes, yes) : go(l1024, two, no, yes);
    if (!fit) {
        if (vecs <= 64) return go(l16, four, no, no);
        if (vecs <= 256) return go(l64, four, no, no);
        if (vecs <= 1024) return go(l256, four, no, no);
        return go(l1024, two, no, no);
    }
    if (vecs <= 64) return go(l16, four, yes, no);
    if (c.rows <= kFewRows) {
        if (vecs <= 128) return go(std::integral_constant<int, 128>(), one, yes, no);
        if (vecs <= 256) return go(l256, one, yes, no);
        if (vecs <= 512) return go(l512, one, yes, no);
        if (vecs <= 1024) return go(l512, two, yes, no);
        return go(l1024, two, yes, no);
    }
    if (vecs <= 128) return go(std::integral_constant<int, 32>(), four, yes, no);
    if (vecs <= 256) return go(l64, four, yes, no);
    if (vecs <= 512) return go(std::integral_constant<int, 128>(), four, yes, no);
    if (vecs <= 1024) return go(l256, four, yes, no);
    return go(l1024, two, yes, no);
}

// ---- gradients ------------------------------------------------------------------------

// L lanes per row, V vectors in a lane, which keeps the sums of its columns of
// the weight's gradient over the rows that it has: rows group, group + groups,
// ... of the call. With kWeight the row groups of a block then add theirs.
template <int T, int L, int V, bool kAligned, bool kWeight>
__global__ __launch_bounds__(L > kBlock ? L : kBlock) void rms_norm_grad_kernel(
    const char* __restrict__ grad_out, const char* __restrict__ h, const char* __restrict__ weight, bool w32,
    const float* __restrict__ rstd, const char* __restrict__ grad_residual, char* __restrict__ grad_x,
    float* __restrict__ parts, int64_t rows, uint32_t cols) {
    typedef Vec<T, kAligned> X;
    constexpr int kThreads = L > kBlock ? L : kBlock, kRows = kThreads / L;
    __shared__ float part[kThreads / 64 * V];
    const uint32_t lane = threadIdx.x % L;
    const int group = group_in_block<L>();
    Weight<T, kAligned> w[V];
    float dw[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        w[k].load(weight, w32, lane + k * L, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
    }
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
        const bool live = r0 + group < rows;
        const int64_t r = live ? r0 + group : rows - 1, at = r * cols * Elem<T>::kBytes;
        typename X::Raw dy[V], a[V], more[V];
        float s[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dy[k] = X::load(grad_out + at, lane + k * L, cols);
            a[k] = X::load(h + at, lane + k * L, cols);
        }
        if (grad_residual)
#pragma unroll
            for (int k = 0; k < V; ++k) more[k] = X::load(grad_residual + at, lane + k * L, cols);
        const float n = rstd[r];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float g[8], f[8], b[8];
            X::P::widen(dy[k], g);
            X::P::widen(a[k], f);
            w[k].widen(w32, b);
            s[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = f[i] * n;
                if (kWeight && live) dw[k][i] = __fmaf_rn(g[i], x, dw[k][i]);
                s[k] = __fmaf_rn(g[i] * b[i], x, s[k]);
            }
        }
        const float mean = vectors_sum<L, V>(s, part) / static_cast<float>(cols);
        if (L > 64) __syncthreads();  // part is used again
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float g[8], f[8], b[8], d[8];
            X::P::widen(dy[k], g);
            X::P::widen(a[k], f);
            w[k].widen(w32, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = n * __fmaf_rn(-(f[i] * n), mean, g[i] * b[i]);
            if (grad_residual) {
                X::P::widen(more[k], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += f[i];
            }
            if (live) X::store(grad_x + at, lane + k * L, cols, X::round(d));
        }
    }
    if constexpr (kWeight) {
        constexpr int kLater = kRows > 1 ? (kRows - 1) * L * V * 8 : 1;
        __shared__ float sums[kLater];
        if constexpr (kRows > 1) {
            if (group > 0)
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sums[(((group - 1) * V + k) * 8 + i) * L + lane] = dw[k][i];
            __syncthreads();
            if (group > 0) return;
            for (int o = 0; o < kRows - 1; ++o)
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[k][i] += sums[((o * V + k) * 8 + i) * L + lane];
        }
        char* to = reinterpret_cast<char*>(parts + static_cast<int64_t>(blockIdx.x) * cols);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            typedef Vec<MOE_EPI_F32, kAligned> F;
            F::store(to, lane + k * L, cols, F::round(dw[k]));
        }
    }
}

// Rows of any width: one block per row, and the weight's gradient apart.
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

// 64 columns a block, and a multiple of the grid's beyond; its 16 wavefronts share the parts, and their sums are added in
// order.
template <int W>
__global__ __launch_bounds__(1024) void grad_weight_kernel(const float* __restrict__ parts, void* __restrict__ grad_weight,
                                                           int64_t n, int64_t cols) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * 64; c0 < cols; c0 += static_cast<int64_t>(gridDim.x) * 64) {
        const int64_t c = c0 + lane;
        float sum = 0.0f;
        if (c < cols) {
#pragma unroll 8
            for (int64_t p = n * wave / 16; p < n * (wave + 1) / 16; ++p) sum += parts[p * cols + c];
        }
        sums[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && c < cols) {
#pragma unroll
            for (int i = 1; i < 16; ++i) sum += sums[i][lane];
            Elem<W>::store1(grad_weight, c, sum);
        }
        __syncthreads();  // sums is used again
    }
}

constexpr int64_t kMostHeld = 8192;  // columns that the lanes of a block hold: with 1024 lanes the registers do not do

// Lanes of a row that the gradient's lanes hold.
int grad_lanes(int64_t cols) {
    const int64_t vecs = (cols + 7) / 8;
    int l = 16;
    while (l * 2 < vecs) l *= 2;
    return l;
}
// Parts of the weight's gradient, each the sum of some rows: a block's, of up to
// four blocks per CU, or 64 rows of rows that are wider than a block holds.
int64_t parts_of(int64_t rows, int64_t cols) {
    int64_t n;
    if (cols > kMostHeld) {
        n = (rows + kRowsPerPart - 1) / kRowsPerPart;
        n = n > kMostParts ? kMostParts : n;
    } else {
        const int l = grad_lanes(cols), at_once = l > kBlock ? 1 : kBlock / l;
        n = (rows + at_once - 1) / at_once;
        n = n > 1024 ? 1024 : n;
    }
    return n < 1 ? 1 : n;
}

template <int T>
void launch_norm_grad(const char* grad_out, const char* h, const char* weight, bool w32, const float* rstd,
                      const char* grad_residual, char* grad_x, float* parts, int64_t blocks, int64_t rows, int64_t cols,
                      hipStream_t st) {
    const bool fit = cols % 8 == 0 && aligned(grad_out, 16) && aligned(h, 16) && aligned(weight, 16) &&
                     aligned(grad_residual, 16) && aligned(grad_x, 16);
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value, kThreads = L > kBlock ? L : kBlock;
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st, grad_out, h, weight, w32,
                               rstd, grad_residual, grad_x, parts, rows, static_cast<uint32_t>(cols));
        };
        if (fit)
            parts ? launch(rms_norm_grad_kernel<T, L, 2, true, true>) : launch(rms_norm_grad_kernel<T, L, 2, true, false>);
        else
            parts ? launch(rms_norm_grad_kernel<T, L, 2, false, true>) : launch(rms_norm_grad_kernel<T, L, 2, false, false>);
    };
    switch (grad_lanes(cols)) {
        case 16: return go(std::integral_constant<int, 16>());
        case 32: return go(std::integral_constant<int, 32>());
        case 64: return go(std::integral_constant<int, 64>());
        case 128: return go(std::integral_constant<int, 128>());
        case 256: return go(std::integral_constant<int, 256>());
        default: return go(std::integral_constant<int, 512>());
    }
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
    const NormCall c = {static_cast<const char*>(x), static_cast<const char*>(residual), static_cast<const char*>(weight),
                        w_dtype == MOE_EPI_F32, eps, static_cast<char*>(out), static_cast<char*>(residual_out), q, scale,
                        rstd, rows, cols};
    switch (dtype) {
        case MOE_EPI_BF16: launch_norm<MOE_EPI_BF16>(c, as_stream(stream)); break;
        case MOE_EPI_F16: launch_norm<MOE_EPI_F16>(c, as_stream(stream)); break;
        default: launch_norm<MOE_EPI_F32>(c, as_stream(stream)); break;
    }
    return launch_status();
}

extern "C" int64_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
    int64_t all;
    if (!sizes_ok(rows, cols, &all)) return -1;
    return parts_of(rows, cols) * cols * 4;
}

extern "C" int rms_norm_bwd(const void* grad_out, const void* h, int dtype, const void* weight, int w_dtype,
                            const float* rstd, const void* grad_residual, void* grad_x, void* grad_weight,
                            void* workspace, int64_t workspace_bytes, int64_t rows, int64_t cols, void* stream) {
    if (!dtype_ok(dtype) || !(w_dtype == dtype || w_dtype == MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    int64_t all;
    if (!sizes_ok(rows, cols, &all)) return MOE_EPI_ERR_BAD_SHAPE;
    const int64_t need = grad_weight ? parts_of(rows, cols) * cols * 4 : 0;
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
        const int64_t n_parts = parts_of(rows, cols);
        if (cols > kMostHeld || rows == 0) {
            const unsigned blocks = static_cast<unsigned>((cols + kBlock - 1) / kBlock);
            if (rows)
                hipLaunchKernelGGL((grad_x_kernel<T, W>), dim3(grid_for_rows(rows, 1)), dim3(kBlock), 0, st, grad_out, h,
                                   weight, rstd, grad_residual, grad_x, rows, cols);
            if (grad_weight)
                hipLaunchKernelGGL((grad_weight_parts_kernel<T>), dim3(blocks, static_cast<unsigned>(n_parts)),
                                   dim3(kBlock), 0, st, grad_out, h, rstd, parts, rows, cols);
        } else {
            launch_norm_grad<T>(static_cast<const char*>(grad_out), static_cast<const char*>(h),
                                static_cast<const char*>(weight), W == MOE_EPI_F32, rstd,
                                static_cast<const char*>(grad_residual), static_cast<char*>(grad_x),
                                grad_weight ? parts : nullptr, n_parts, rows, cols, st);
        }
        if (grad_weight)
            hipLaunchKernelGGL((grad_weight_kernel<W>), dim3(grid_for_rows(cols, 64)), dim3(1024), 0, st,
                               parts, grad_weight, n_parts, cols);
    });
    return launch_status();
}
