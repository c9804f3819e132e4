// Rows to 8-bit integers with one scale each (gfx950).
//
//   scale = max|x| / 127,  q = rint(127 x / max|x|), ties to even.
//
// Bound by memory: a row is read once and kept in registers, as it came,
// between its maximum and its rounding (rows wider than the registers hold are
// read again, from L2). The maximum is taken over the bit patterns without
// sign: their order is that of the magnitudes, with infinity above every
// number and NaN above that, so one integer maximum also finds rows that are
// not finite. x and max|x| are first scaled by the power of two that brings
// the maximum near 1 (exact), so that 127 x cannot overflow and the quotient
// of a tiny maximum stays in range.
//
// An IEEE division per element is 22 instructions and set the pace (32768 x
// 7168 bf16 149 us, 65536 x 2048 81 us). quantize8 rounds the product with a
// reciprocal instead, and takes the remainder: where it shows that the nearest
// integer is within 0.4999, that is what the rounded quotient gives too;
// vectors with an element nearer to a tie are divided. The bits are the same
// and the times 109 us (6.4 TB/s) and 63 us (6.3 TB/s).
//
// A row takes the fewest lanes that hold it, four vectors each: 65536 rows of
// 256 13 us with 16 lanes, 19 with 32, 30 with 64; of 512 20, 25, 35; of 1024
// 35 with 32, 45 with 64; 32768 of 7168 109 with 256 lanes, 139 with 512. Up to
// 512 rows, two per CU, do not fill the chip, and a row is done sooner by more
// lanes with one or two vectors each: 32 rows of 2048 3.4 -> 2.6 us, of 4096 3.6
// -> 2.9, of 7168 3.6 -> 3.4, of 16384 6.0 -> 4.5; 512 rows 3.9 -> 3.3, 4.4 -> 3.9,
// 5.3 -> 5.1, 11.2 -> 8.0; but 1024 rows of 640 3.56 and 3.58, of 7168 6.5 and 6.7.
#include <type_traits>

#include "epi_common.h"
#include "int8_rows.h"
#include "moe_routed.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;         // threads, or the lanes of a row if they are more
constexpr int64_t kFewRows = 512;

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
#pragma unroll
    for (int off = (L < 64 ? L : 64) / 2; off > 0; off >>= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off, 64));
        v = o > v ? o : v;
    }
    if constexpr (L > kBlock) {
        if ((threadIdx.x & 63) == 0) atomicMax(part, v);  // any order, one maximum; cleared before the row's loads
        __syncthreads();
        v = *part;
        __syncthreads();
    } else if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        const int first = threadIdx.x / L * (L / 64);
#pragma unroll
        for (int w = 0; w < L / 64; ++w) v = part[first + w] > v ? part[first + w] : v;
        __syncthreads();
    }
    return v;
}

// L lanes per row, from part of a wavefront to the block; kVecs vectors of 8
// elements that a lane keeps.
template <int T, int L, int kVecs, bool kAligned>
__global__ __launch_bounds__(L > kBlock ? L : kBlock) void quantize_rows_kernel(
    const char* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale, int64_t rows, int64_t cols) {
    typedef Eight<T, kAligned> X;
    constexpr int kThreads = L > kBlock ? L : kBlock, kRowsPerBlock = kThreads / L;
    __shared__ uint32_t part[kBlock / 64];  // a word per wavefront, or one for a row of more
    const uint32_t lane = threadIdx.x % L;
    const uint32_t nvec = static_cast<uint32_t>(cols / 8), left = static_cast<uint32_t>(cols) - nvec * 8;
    const int64_t groups = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t r0 = g * kRowsPerBlock + group_in_block<L>();
        const bool live = r0 < rows;
        const int64_t r = live ? r0 : rows - 1;  // spare wavefronts of the last block repeat its last row
        const char* row = x + r * cols * X::kBytes;
        int8_t* qrow = q + r * cols;
        typename X::Raw raw[kVecs];
        uint32_t most = 0;
        if constexpr (L > kBlock) {
            if (threadIdx.x == 0) *part = 0;
            __syncthreads();
        }
        auto grow = [&](const typename X::Raw& v) {
            float f[8];
            X::widen(v, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = magnitude(f[i]);
                most = m > most ? m : most;
            }
        };
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            raw[k] = lane + k * L < nvec ? X::load(row, (lane + k * L) * 8) : typename X::Raw{};
#pragma unroll
        for (int k = 0; k < kVecs; ++k) grow(raw[k]);
        for (uint32_t c = lane + kVecs * L; c < nvec; c += L) grow(X::load(row, c * 8));
        float last = 0.0f;
        if (lane < left) {
            last = Elem<T>::load1(row, nvec * 8 + lane);
            const uint32_t m = magnitude(last);
            most = m > most ? m : most;
        }
        const RowScale s(row_max<L>(most, part));
        auto put = [&](uint32_t c, const typename X::Raw& v) {
            typedef u32x2 loose __attribute__((aligned(1)));
            float f[8];
            X::widen(v, f);
            const u32x2 w = s.finite ? quantize8(s, f) : u32x2{0u, 0u};
            if constexpr (kAligned)
                __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(qrow + c * 8));
            else
                *reinterpret_cast<loose*>(qrow + c * 8) = w;
        };
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            if (lane + k * L < nvec) put(lane + k * L, raw[k]);
        for (uint32_t c = lane + kVecs * L; c < nvec; c += L) put(c, X::load(row, c * 8));
        if (lane < left)
            qrow[nvec * 8 + lane] = static_cast<int8_t>(s.finite ? static_cast<int>(rintf(last * s.mul / s.den)) : 0);
        if (lane == 0) scale[r] = s.scale;
    }
}

template <int T>
void launch_quantize(const void* x, int8_t* q, float* scale, int64_t rows, int64_t cols, hipStream_t st) {
    const bool fit = cols % 8 == 0 && aligned(x, 16) && aligned(q, 8);
    auto go = [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value, kThreads = L > kBlock ? L : kBlock;
        const dim3 block(kThreads), grid(grid_for_rows(rows, kThreads / L));
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, st, static_cast<const char*>(x), q, scale, rows, cols);
        };
        fit ? launch(quantize_rows_kernel<T, L, V, true>) : launch(quantize_rows_kernel<T, L, V, false>);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 128> l128;
    const std::integral_constant<int, 256> l256;
    const std::integral_constant<int, 512> l512;
    // the fewest lanes that hold a row; of the widest rows what they do not hold is read again
    const int64_t vecs = (cols + 7) / 8;
    if (vecs <= 16 * 4) return go(std::integral_constant<int, 16>(), four);
    if (rows <= kFewRows) {
        if (vecs <= 128) return go(l128, one);
        if (vecs <= 256) return go(l256, one);
        if (vecs <= 512) return go(l512, one);
        if (vecs <= 512 * 2) return go(l512, two);
        return go(std::integral_constant<int, 1024>(), two);
    }
    if (vecs <= 32 * 4) return go(std::integral_constant<int, 32>(), four);
    if (vecs <= 64 * 4) return go(std::integral_constant<int, 64>(), four);
    if (vecs <= 128 * 4) return go(l128, four);
    return go(l256, four);
}

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int quantize_rows_int8_fwd(const void* x, int dtype, int8_t* q, float* scale, int64_t rows, int64_t cols,
                                      void* stream) {
    if (!dtype_ok(dtype)) return MOE_EPI_ERR_BAD_DTYPE;
    const int e = elem_bytes(dtype);
    int64_t xb, qb, sb;
    if (!bytes_ok(rows, cols, e, &xb) || !bytes_ok(rows, cols, 1, &qb) || !bytes_ok(rows, 1, 4, &sb) ||
        !row_fits_u32_offsets(cols, 4))
        return MOE_EPI_ERR_BAD_SHAPE;
    if (rows == 0) return MOE_EPI_SUCCESS;
    if (!x || !q || !scale) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(x, e) || !aligned(scale, 4)) return MOE_EPI_ERR_MISALIGNED;
    const Range rx = range_of(x, xb), rq = range_of(q, qb), rs = range_of(scale, sb);
    if (overlaps(rq, rx) || overlaps(rs, rx) || overlaps(rq, rs)) return MOE_EPI_ERR_ALIAS;
    (void)hipGetLastError();
    const hipStream_t st = as_stream(stream);
    switch (dtype) {
        case MOE_EPI_BF16: launch_quantize<MOE_EPI_BF16>(x, q, scale, rows, cols, st); break;
        case MOE_EPI_F16: launch_quantize<MOE_EPI_F16>(x, q, scale, rows, cols, st); break;
        default: launch_quantize<MOE_EPI_F32>(x, q, scale, rows, cols, st); break;
    }
    return launch_status();
}
