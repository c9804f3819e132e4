// Rows to 8-bit integers with one scale each (gfx950).
//
//   scale = max|x| / 127,  q = rint(127 x / max|x|), ties to even.
//
// Bound by memory: a row is read once and kept in registers between its
// maximum and its rounding (rows wider than the registers hold are read
// again, from L2). The maximum is taken over the bit patterns without sign:
// their order is that of the magnitudes, with infinity above every number and
// NaN above that, so one integer maximum also finds rows that are not finite.
// x and max|x| are first scaled by the power of two that brings the maximum
// near 1 (exact), so that 127 x cannot overflow and the quotient of a tiny
// maximum stays in range.
#include "epi_common.h"
#include "moe_routed.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int kVecs = 4;  // vectors of 8 elements that a lane keeps

// Eight elements at element e of a row, widened. kAligned: 16-byte aligned rows.
template <int T, bool kAligned>
__device__ __forceinline__ void load8(const char* row, uint32_t e, float (&f)[8]) {
    typedef u32x4 loose __attribute__((aligned(2)));
    auto word = [](const char* p) {
        if constexpr (kAligned)
            return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
        else
            return static_cast<u32x4>(__builtin_nontemporal_load(reinterpret_cast<const loose*>(p)));
    };
    if constexpr (T == MOE_EPI_F32) {
        const typename Elem<T>::Raw r{word(row + e * 4u), word(row + e * 4u + 16)};
        Elem<T>::unpack(r, f);
    } else {
        Elem<T>::unpack(word(row + e * 2u), f);
    }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What a row's maximum gives: q = rint(x * mul / den).
struct RowScale {
    float mul, den, scale;
    bool finite;
    __device__ __forceinline__ explicit RowScale(uint32_t most) {
        finite = most < 0x7F800000u;
        int e = static_cast<int>(most >> 23) - 127;  // exponent of the maximum
        e = e < -120 ? -120 : (e > 126 ? 126 : e);   // 2^-e and 127 * 2^-e stay normal
        const float m = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
        mul = 127.0f * m;
        den = most == 0 ? 1.0f : __uint_as_float(most) * m;
        scale = finite ? __uint_as_float(most) / 127.0f : __uint_as_float(0x7FC00000u);
    }
    __device__ __forceinline__ int q(float x) const {
        return finite ? static_cast<int>(rintf(x * mul / den)) : 0;
    }
};

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), off, 64));
        v = o > v ? o : v;
    }
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < L / 64; ++w) v = part[w] > v ? part[w] : v;
        __syncthreads();
    }
    return v;
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (static_cast<uint32_t>(a) & 0xFFu) | (static_cast<uint32_t>(b) & 0xFFu) << 8 |
           (static_cast<uint32_t>(c) & 0xFFu) << 16 | static_cast<uint32_t>(d) << 24;
}

// L lanes per row (64: a wavefront; 256: the block).
template <int T, int L, bool kAligned>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(const char* __restrict__ x, int8_t* __restrict__ q,
                                                               float* __restrict__ scale, int64_t rows,
                                                               int64_t cols) {
    constexpr int E = T == MOE_EPI_F32 ? 4 : 2, kRowsPerBlock = kBlock / L;
    __shared__ uint32_t part[kBlock / 64];
    const uint32_t lane = threadIdx.x % L;
    const uint32_t nvec = static_cast<uint32_t>(cols / 8), left = static_cast<uint32_t>(cols) - nvec * 8;
    const int64_t groups = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t r0 = g * kRowsPerBlock + group_in_block<L>();
        const bool live = r0 < rows;
        const int64_t r = live ? r0 : rows - 1;  // spare wavefronts of the last block repeat its last row
        const char* row = x + r * cols * E;
        int8_t* qrow = q + r * cols;
        float f[kVecs][8];
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const uint32_t c = lane + k * L;
            if (c < nvec) {
                load8<T, kAligned>(row, c * 8, f[k]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[k][i] = 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = magnitude(f[k][i]);
                most = m > most ? m : most;
            }
        for (uint32_t c = lane + kVecs * L; c < nvec; c += L) {
            float h[8];
            load8<T, kAligned>(row, c * 8, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = magnitude(h[i]);
                most = m > most ? m : most;
            }
        }
        float last = 0.0f;
        if (lane < left) {
            last = Elem<T>::load1(row, nvec * 8 + lane);
            const uint32_t m = magnitude(last);
            most = m > most ? m : most;
        }
        const RowScale s(row_max<L>(most, part));
        auto put = [&](uint32_t c, const float (&v)[8]) {
            typedef u32x2 loose __attribute__((aligned(1)));
            const u32x2 w = {pack4(s.q(v[0]), s.q(v[1]), s.q(v[2]), s.q(v[3])),
                             pack4(s.q(v[4]), s.q(v[5]), s.q(v[6]), s.q(v[7]))};
            if constexpr (kAligned)
                *reinterpret_cast<u32x2*>(qrow + c * 8) = w;
            else
                *reinterpret_cast<loose*>(qrow + c * 8) = w;
        };
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
            if (lane + k * L < nvec) put(lane + k * L, f[k]);
        for (uint32_t c = lane + kVecs * L; c < nvec; c += L) {
            float h[8];
            load8<T, kAligned>(row, c * 8, h);
            put(c, h);
        }
        if (lane < left) qrow[nvec * 8 + lane] = static_cast<int8_t>(s.q(last));
        if (lane == 0) scale[r] = s.scale;
    }
}

template <int T>
void launch_quantize(const void* x, int8_t* q, float* scale, int64_t rows, int64_t cols, hipStream_t st) {
    const bool fit = cols % 8 == 0 && aligned(x, 16) && aligned(q, 8);
    // a wavefront holds 2048 elements; wider rows take the block
    const bool wave = cols <= 64 * 8 * kVecs;
    const dim3 block(kBlock), grid(grid_for_rows(rows, wave ? kBlock / 64 : 1));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, st, static_cast<const char*>(x), q, scale, rows, cols);
    };
    if (wave)
        fit ? go(quantize_rows_kernel<T, 64, true>) : go(quantize_rows_kernel<T, 64, false>);
    else
        fit ? go(quantize_rows_kernel<T, kBlock, true>) : go(quantize_rows_kernel<T, kBlock, false>);
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
