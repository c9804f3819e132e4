// Rows of 8 elements a lane, and their rounding to 8-bit integers (gfx950):
// shared by quantize_rows.hip, which says what it is made of, and rms_norm.hip.
#pragma once

#include "epi_common.h"

namespace moe_epi {

// Eight elements at element e of a row, as stored. kAligned: 16-byte aligned
// rows, read once; others share cache lines between lanes and rows, so they
// are read with the caches' default policy.
template <int T, bool kAligned>
struct Eight {
    typedef u32x4 loose __attribute__((aligned(2)));
    static constexpr int kWords = T == MOE_EPI_F32 ? 2 : 1, kBytes = T == MOE_EPI_F32 ? 4 : 2;
    struct Raw {
        u32x4 w[kWords];
    };
    __device__ __forceinline__ static Raw load(const char* row, uint32_t e) {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const char* p = row + e * kBytes + 16 * i;
            if constexpr (kAligned)
                r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
            else
                r.w[i] = *reinterpret_cast<const loose*>(p);
        }
        return r;
    }
    __device__ __forceinline__ static void widen(const Raw& r, float (&f)[8]) {
        if constexpr (T == MOE_EPI_F32)
            Elem<T>::unpack(typename Elem<T>::Raw{r.w[0], r.w[1]}, f);
        else
            Elem<T>::unpack(r.w[0], f);
    }
};

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What a row's maximum gives: q = rint(x * mul / den), about x * near.
struct RowScale {
    float mul, den, scale, near;
    bool finite;
    __device__ __forceinline__ explicit RowScale(uint32_t most) {
        finite = most < 0x7F800000u;
        int e = static_cast<int>(most >> 23) - 127;  // exponent of the maximum
        e = e < -120 ? -120 : (e > 126 ? 126 : e);   // 2^-e and 127 * 2^-e stay normal
        const float m = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
        mul = 127.0f * m;
        den = most == 0 ? 1.0f : __uint_as_float(most) * m;
        near = mul / den;
        if (!(near < __uint_as_float(0x7F800000u))) near = 0.0f;  // max|x| below 2^-121: every element is divided
        scale = finite ? __uint_as_float(most) / 127.0f : __uint_as_float(0x7FC00000u);
    }
};
// 1.5 * 2^23: added to a float32 of small magnitude it leaves the nearest
// integer (ties to even) in the low bits, in two's complement.
constexpr float kMagic = 12582912.0f;

// rint(x * mul / den) of eight elements, as bytes. |x * mul / den| <= 127 (1 + 2^-23).
__device__ __forceinline__ u32x2 quantize8(const RowScale& s, const float (&x)[8]) {
    float t[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = __fmaf_rn(x[i], s.near, kMagic);
        const float q = t[i] - kMagic, c = x[i] * s.mul;
        far = fmaxf(far, fabsf(__fmaf_rn(-q, s.den, c)));
    }
    if (__any(far > 0.4999f * s.den)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = x[i] * s.mul / s.den + kMagic;
    }
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // the low byte of each, two at a time
        auto bits = [&](int i) { return __float_as_uint(t[4 * h + i]); };
        w[h] = __builtin_amdgcn_perm(bits(1), bits(0), 0x0c0c0400u) |
               __builtin_amdgcn_perm(bits(3), bits(2), 0x04000c0cu);
    }
    return w;
}

}  // namespace moe_epi
