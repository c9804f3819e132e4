// Eight elements of a row as operands of the bfloat16 matrix instructions (gfx950).
//
// The matrix cores multiply float32 at an eighth of their 16-bit rate, so a
// float32 is cut into up to three bfloat16 pieces, each the nearest bfloat16 to
// what the ones before leave: x = x0 + x1 + x2 exactly (8 significant bits and a
// sign each) from 2^-110 on, below to 2^-134, half the least bfloat16; |x1| <=
// 2^-8 |x|, |x2| <= 2^-16 |x|. Products of pieces are exact in float32. Of the pairs of pieces those with i + j <= 2 are summed; what is left
// out is at most 2^-23 of a product. A float16 (11 bits) is two pieces.
#pragma once

#include "epi_common.h"

namespace moe_epi {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// D += A B for 16 x 32 and 32 x 16 operands: lane l holds row (of A) or column
// (of B) l % 16 and k = 8 (l / 16) .. + 7; D has column l % 16 and rows
// 4 (l / 16) .. + 3 in it.
template <bool kF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 d) {
    if constexpr (kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), d,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       d, 0, 0, 0);
}

// Eight elements of storage type T as they lie in memory, at any alignment of
// the element (the hardware takes loads at any address).
template <int T>
struct Piece8 {
    typedef u32x4 loose __attribute__((aligned(2)));
    static constexpr int kWords = T == MOE_EPI_F32 ? 2 : 1, kBytes = Elem<T>::kBytes;
    struct Raw {
        u32x4 w[kWords];
    };
    __device__ __forceinline__ static Raw load(const char* p) {
        Raw r;
#pragma unroll
        for (int i = 0; i < kWords; ++i) r.w[i] = *reinterpret_cast<const loose*>(p + 16 * i);
        return r;
    }
    // the first n of eight elements, zeros after them
    __device__ __forceinline__ static Raw load_first(const char* p, int64_t n) {
        if (n >= 8) return load(p);
        Raw r = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) continue;
            if constexpr (T == MOE_EPI_F32)
                r.w[i / 4][i % 4] = reinterpret_cast<const uint32_t*>(p)[i];
            else
                r.w[0][i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
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

// Two values' piece, which leaves f what the next pieces are of. Values beyond
// the largest bfloat16 have that as theirs, and not an infinity: what is left of
// a finite one is its next pieces, and of an infinity or a NaN its last piece,
// which is not held back (kLast). Float32 logits of 16384 x 7168 x 64 take 137
// us so, 133 without.
template <bool kLast>
__device__ __forceinline__ uint32_t cut2(float& a, float& b) {
    constexpr float kMost = 0x1.fep127f;
    const uint32_t w = kLast ? pack_bf16x2(a, b)
                             : pack_bf16x2(__builtin_amdgcn_fmed3f(a, -kMost, kMost), __builtin_amdgcn_fmed3f(b, -kMost, kMost));
    a -= bf16_lo(w);
    b -= bf16_hi(w);
    return w;
}
// f as P pieces.
template <int P>
__device__ __forceinline__ void cut(float (&f)[8], u32x4 (&piece)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            piece[p][i] = p + 1 < P ? cut2<false>(f[2 * i], f[2 * i + 1]) : cut2<true>(f[2 * i], f[2 * i + 1]);
}
// Four values as P pieces.
template <int P>
__device__ __forceinline__ void cut4(float (&f)[4], u32x2 (&piece)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            piece[p][i] = p + 1 < P ? cut2<false>(f[2 * i], f[2 * i + 1]) : cut2<true>(f[2 * i], f[2 * i + 1]);
}
// r as P pieces; the type itself where it has one piece.
template <int T, int P>
__device__ __forceinline__ void cut_raw(const typename Piece8<T>::Raw& r, u32x4 (&piece)[P]) {
    if constexpr (P == 1 && T != MOE_EPI_F32) {
        piece[0] = r.w[0];
    } else {
        float f[8];
        Piece8<T>::widen(r, f);
        cut<P>(f, piece);
    }
}

// r: eight 16-bit elements of each of eight rows; out[j]: the rows' elements j.
__device__ __forceinline__ void turn8(const u32x4 (&r)[8], u32x4 (&out)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[j][i] = __builtin_amdgcn_perm(r[2 * i + 1][j / 2], r[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
}

// The sum over the pairs of pieces that count: i + j <= 2.
template <bool kF16, int PA, int PB>
__device__ __forceinline__ f32x4 mfma_pieces(const u32x4 (&a)[PA], const u32x4 (&b)[PB], f32x4 d) {
#pragma unroll
    for (int i = PA - 1; i >= 0; --i)
#pragma unroll
        for (int j = PB - 1; j >= 0; --j)
            if (i + j <= 2) d = mfma16<kF16>(a[i], b[j], d);
    return d;
}

}  // namespace moe_epi
