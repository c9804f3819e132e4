// Moves of the tokens into expert order and back, and their gradients (gfx950).
//
//   dispatch        out[r] = x[slot_of[r] / k]                               (bits copied)
//   its gradient    grad_x[t] = sum_j grad_out[row_of[t, j]]
//   combine         out[t] = sum_j w[t, j] * rows[row_of[t, j]]
//   its gradients   grad_rows[row_of[t, j]] = w[t, j] * grad_out[t]
//                   grad_w[t, j] = sum_h grad_out[t, h] * rows[row_of[t, j], h]
//
// All of them are bound by the bytes they move: each row is read or written
// once and each token once, with a multiply-add per element at most. Sums are
// float32 in a fixed order (slots ascending; lanes, then wavefronts for the
// weights' gradient), rounded once when stored, so that a run repeats bit for
// bit: the alternative, one row per block with atomic additions into the
// token, would read and write the token once per row and in any order.
//
// A lane moves vectors of N elements: 16 bytes of 16-bit storage, or 4
// elements where float32 takes part (16 bytes of float32), so that the
// accesses of a wavefront are one contiguous run on both sides. Rows of odd
// width or address are moved by the same vectors at the element's alignment
// (the hardware takes any), with the last few elements one per lane.
#include <type_traits>

#include "epi_common.h"
#include "moe_routed.h"

namespace moe_epi {
namespace {

constexpr int64_t kMaxTopK = 1024;
constexpr int kSlotChunk = 8;  // slots taken together: their indices are read at once, a lane each

// ---- N elements of storage type T at element `e` of a row --------------------------

template <int T>
constexpr int kBytesOf = T == MOE_EPI_F32 ? 4 : 2;

// Unsigned vectors of 1 to 16 bytes, at their own or at the element's alignment.
template <int kBytes, int kAlign> struct Word;
#define MOE_WORD(BYTES, TYPE, ALIGN)                                   \
    template <> struct Word<BYTES, ALIGN> {                            \
        typedef TYPE plain;                                            \
        typedef TYPE type __attribute__((aligned(ALIGN)));             \
    };
MOE_WORD(16, u32x4, 16)
MOE_WORD(16, u32x4, 4)
MOE_WORD(16, u32x4, 2)
MOE_WORD(8, u32x2, 8)
MOE_WORD(8, u32x2, 4)
MOE_WORD(8, u32x2, 2)
#undef MOE_WORD

// Aligned words are streamed (nontemporal); words at the element's alignment
// share cache lines with their neighbours, whose loads should find them: a
// weighted sum of 30021 rows of 1001 float16 22.2 -> 19.8 us (18.1 now).
template <int kBytes, int kAlign>
__device__ __forceinline__ typename Word<kBytes, kAlign>::plain load_word(const void* p) {
    const typename Word<kBytes, kAlign>::type* w = static_cast<const typename Word<kBytes, kAlign>::type*>(p);
    if constexpr (kAlign == kBytes)
        return __builtin_nontemporal_load(w);
    else
        return *w;
}
template <int kBytes, int kAlign>
__device__ __forceinline__ void store_word(void* p, typename Word<kBytes, kAlign>::plain v) {
    __builtin_nontemporal_store(v, static_cast<typename Word<kBytes, kAlign>::type*>(p));
}

__device__ __forceinline__ float half_at(uint32_t w, int hi) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hi ? w >> 16 : w & 0xFFFFu)));
}

// N consecutive elements widened to float32, and rounded back to T.
template <int T, int N, bool kAligned>
struct Vec {
    static constexpr int kBytes = N * kBytesOf<T>, kAlign = kAligned ? kBytes : kBytesOf<T>;
    static_assert(kBytes == 16 || kBytes == 8, "one access");
    typedef typename Word<kBytes, kAlign>::plain Raw;

    __device__ __forceinline__ static Raw load(const void* row, uint32_t e) {
        return load_word<kBytes, kAlign>(static_cast<const char*>(row) + e * kBytesOf<T>);
    }
    __device__ __forceinline__ static void widen(Raw r, float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
            const uint32_t w = r[i];
            if constexpr (T == MOE_EPI_F32) {
                f[i] = __uint_as_float(w);
            } else if constexpr (T == MOE_EPI_BF16) {
                f[2 * i] = bf16_lo(w);
                f[2 * i + 1] = bf16_hi(w);
            } else {
                f[2 * i] = half_at(w, 0);
                f[2 * i + 1] = half_at(w, 1);
            }
        }
    }
    __device__ __forceinline__ static void store(void* row, uint32_t e, const float (&f)[N]) {
        Raw r;
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
            if constexpr (T == MOE_EPI_F32) {
                r[i] = __float_as_uint(f[i]);
            } else if constexpr (T == MOE_EPI_BF16) {
                r[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
            } else {
                // finished binary32 values first: see Elem<MOE_EPI_F16>::store1
                float a = f[2 * i], b = f[2 * i + 1];
                asm volatile("" : "+v"(a), "+v"(b));
                r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, f16x2_t));
            }
        }
        store_word<kBytes, kAlign>(static_cast<char*>(row) + e * kBytesOf<T>, r);
    }
};

// ---- dispatch ------------------------------------------------------------------------

constexpr int kCopyLanes = 64;

// One wavefront per (row, segment of kCopyLanes * V 16-byte pieces): bytes are
// copied, whatever they stand for. kAlign: of every row on both sides. Tokens
// are read with the caches' default policy, since a token with several rows
// here is read again. One piece a lane streams best (131072 rows of 7168 bf16,
// about one a token: 592 us, 6.3 TB/s moved; 2 pieces 634, 4 with 128 lanes
// 687; a residency limit on the latter 652 to 675); where tokens have many
// rows, which come from the Infinity Cache, two pieces do (262144 rows of 2048,
// 8 a token: 299 us against 330).
template <int kAlign, int V>
__global__ __launch_bounds__(kCopyLanes) void moe_dispatch_kernel(const char* __restrict__ x,
                                                                  const int32_t* __restrict__ slot_of,
                                                                  char* __restrict__ out, int64_t rows, int64_t slots,
                                                                  uint32_t top_k, int64_t row_bytes, uint32_t nseg) {
    const uint32_t pieces = static_cast<uint32_t>(row_bytes / 16);
    const int64_t pairs = rows * static_cast<int64_t>(nseg);
    for (int64_t b = blockIdx.x; b < pairs; b += gridDim.x) {
        const int64_t r = b / nseg;
        const uint32_t seg = static_cast<uint32_t>(b - r * nseg);
        const int32_t slot = __builtin_amdgcn_readfirstlane(slot_of[r]);
        const bool has = slot >= 0 && slot < slots;  // a row without a slot is zeros
        const char* src = x + (has ? static_cast<int64_t>(static_cast<uint32_t>(slot) / top_k) * row_bytes : 0);
        char* dst = out + r * row_bytes;
        const uint32_t c0 = seg * (kCopyLanes * V) + threadIdx.x;
        u32x4 v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            v[k] = u32x4{0u, 0u, 0u, 0u};
            if (has && c0 + k * kCopyLanes < pieces)
                v[k] = *reinterpret_cast<const typename Word<16, kAlign>::type*>(src + (c0 + k * kCopyLanes) * 16u);
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (c0 + k * kCopyLanes < pieces) store_word<16, kAlign>(dst + (c0 + k * kCopyLanes) * 16u, v[k]);
        if constexpr (kAlign < 16) {  // the row's last bytes, two at a time
            const uint32_t done = pieces * 16, left = static_cast<uint32_t>(row_bytes) - done;
            if (seg + 1 == nseg && threadIdx.x < left / 2)
                *reinterpret_cast<uint16_t*>(dst + done + 2 * threadIdx.x) =
                    has ? *reinterpret_cast<const uint16_t*>(src + done + 2 * threadIdx.x) : uint16_t{0};
        }
    }
}

// ---- sums over a token's rows ------------------------------------------------------

constexpr int kSumLanes = 64;

// One wavefront per (token, segment of kSumLanes * kVecs vectors), with 8 / kVecs
// rows' loads in flight together. Its slots' rows and weights are read by a lane
// each, so that a call of few tokens waits once for them and not once a slot
// (sums of 8 rows for 32 tokens of 7168 bf16 4.9 -> 4.1 us on the GPU), those
// with a row are kept as a bit mask and taken in ascending order.
//
// Two vectors a lane and four rows stream best. Measured (us): 8 rows a token,
// 32768 tokens of 2048 bf16 204, 5.9 TB/s (128 lanes 214; one vector and 8 rows
// 203); about one row a token, 131072 of 7168 bf16 602, 6.2 TB/s (637; 964);
// float32 rows, 65536 of 7168, 600 (606; 953). Where tokens have several rows
// and the call has fewer wavefronts than the chip holds at once, the waits set
// the time, and one vector a lane with eight rows in flight is faster: 1, 32,
// 64 and 128 tokens of 7168 2.9, 3.5, 3.9, 4.8 us against 3.3, 4.1, 4.5, 5.6;
// 256 tokens 7.2 against 7.0; 512 of 2048 5.1 against 5.9, 1024 8.0 against 7.6;
// with about one row a token 128 of 7168 3.6 against 3.2.
template <int TI, int TO, int N, int kVecs, bool kWeighted, bool kAligned>
__global__ __launch_bounds__(kSumLanes) void moe_row_sum_kernel(const char* __restrict__ in,
                                                                const int32_t* __restrict__ row_of,
                                                                const float* __restrict__ weights,
                                                                char* __restrict__ out, int64_t rows, int64_t tokens,
                                                                int64_t top_k, int64_t hidden, uint32_t nseg) {
    constexpr int kRows = 8 / kVecs;
    typedef Vec<TI, N, kAligned> In;
    typedef Vec<TO, N, kAligned> Out;
    const uint32_t nvec = static_cast<uint32_t>(hidden / N), done = nvec * N;
    const uint32_t left = static_cast<uint32_t>(hidden) - done;
    const int64_t pairs = tokens * static_cast<int64_t>(nseg);
    for (int64_t b = blockIdx.x; b < pairs; b += gridDim.x) {
        const int64_t t = b / nseg;
        const uint32_t seg = static_cast<uint32_t>(b - t * nseg);
        const uint32_t c0 = seg * (kSumLanes * kVecs) + threadIdx.x;
        const bool tail = !kAligned && seg + 1 == nseg && threadIdx.x < left;
        float acc[kVecs][N] = {};
        float acc1 = 0.0f;
        for (int64_t j0 = 0; j0 < top_k; j0 += kSlotChunk) {
            // a lane per slot: their indices and weights are one read each
            const int64_t j = j0 + threadIdx.x % kSlotChunk;
            const int32_t slot_row = j < top_k ? row_of[t * top_k + j] : -1;
            const float slot_weight = kWeighted && j < top_k ? weights[t * top_k + j] : 1.0f;
            uint32_t mask =
                static_cast<uint32_t>(__ballot(slot_row >= 0 && slot_row < rows)) & ((1u << kSlotChunk) - 1u);
            while (mask) {
                int64_t at[kRows];
                float ww[kRows];
                int n = 0;
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    at[q] = 0;
                    ww[q] = 0.0f;
                    if (mask) {  // the lowest flagged slot
                        const int slot = __builtin_ctz(mask);
                        mask &= mask - 1;
                        at[q] = __builtin_amdgcn_readlane(slot_row, slot);
                        ww[q] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(slot_weight), slot));
                        n = q + 1;
                    }
                }
                typename In::Raw v[kRows][kVecs];
                float v1[kRows];
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    v1[q] = 0.0f;
                    if (q >= n) continue;
                    const void* row = in + at[q] * hidden * kBytesOf<TI>;
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) {
                        const uint32_t c = c0 + k * kSumLanes;
                        v[q][k] = c < nvec ? In::load(row, c * N) : typename In::Raw{};
                    }
                    if (tail) v1[q] = Elem<TI>::load1(row, done + threadIdx.x);
                }
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    if (q >= n) continue;
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) {
                        float f[N];
                        In::widen(v[q][k], f);
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            acc[k][i] = kWeighted ? __fmaf_rn(ww[q], f[i], acc[k][i]) : acc[k][i] + f[i];
                    }
                    acc1 = kWeighted ? __fmaf_rn(ww[q], v1[q], acc1) : acc1 + v1[q];
                }
            }
        }
        char* orow = out + t * hidden * kBytesOf<TO>;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const uint32_t c = c0 + k * kSumLanes;
            if (c < nvec) Out::store(orow, c * N, acc[k]);
        }
        if (tail) Elem<TO>::store1(orow, done + threadIdx.x, acc1);
    }
}

// ---- gradients of the weighted combine -----------------------------------------------

constexpr int kGradVecs = 4;  // vectors per lane and pass over the row
constexpr int kGradRows = 2;  // rows whose loads are in flight together

// L lanes per token: its gradient is read once for up to kSlotChunk slots,
// each of their rows is read and its gradient written in the same pass, and
// the products' partial sums stay in one register per slot. Lanes by the row's
// vectors, four each, up to 256 lanes. 65536 tokens of 7168 bf16, about one row
// each: 432 us, 5.8 TB/s (128 lanes 456, 64 476; one vector at a time 450; 2
// vectors a lane 445; 448 lanes of 2, an exact fit, 483; default-policy stores
// 448; 4 instead of 5 blocks per CU 459, registers for 6 wavefronts a SIMD 470);
// of 4096: 262 us (256 lanes 281, 64 271).
//
// Few tokens leave most CUs without a block, each going through its token's
// slots: then a token's slots are spread over `parts` blocks, `span` each, and
// its gradient is read once more by each of them (from L2). 8 rows a token, us
// with spans of 1, 2, 4 and with all slots in one block: 32 tokens of 7168 5.9,
// 6.2, 7.7, 11.0, 128 12.2, 9.0, 10.0, 14.3, 256 20.5, 15.5, 15.3, 16.9, 512
// 35.3, 29.4, 26.8, 26.7; of 2048, 128 tokens 6.1, 6.2, 7.1, 10.4, 512 12.7,
// 11.0, 10.9, 13.7, 2048 38.9, 33.6, 30.7, 30.3. About one row a token: 32
// tokens of 7168 3.8, 4.3, 4.7, 5.7, 128 5.9, 5.8, 6.1, 7.1.
template <int TG, int TE, int N, int L, bool kDot, bool kAligned>
__global__ __launch_bounds__(L) void moe_combine_grad_kernel(
    const char* __restrict__ grad, const char* __restrict__ in, const int32_t* __restrict__ row_of,
    const float* __restrict__ weights, char* __restrict__ grad_in, float* __restrict__ grad_w, int64_t rows,
    int64_t tokens, int64_t top_k, int64_t hidden, uint32_t parts, uint32_t span) {
    typedef Vec<TG, N, kAligned> G;
    typedef Vec<TE, N, kAligned> E;
    constexpr int kWaves = L / 64;
    __shared__ float part[kWaves][kSlotChunk];
    const uint32_t nvec = static_cast<uint32_t>(hidden / N), done = nvec * N;
    const uint32_t left = static_cast<uint32_t>(hidden) - done;
    for (int64_t b = blockIdx.x; b < tokens * parts; b += gridDim.x) {
        const int64_t t = parts == 1 ? b : static_cast<uint32_t>(b) / parts;
        const int64_t first = (b - t * parts) * span, end = first + span < top_k ? first + span : top_k;
        const char* grow = grad + t * hidden * kBytesOf<TG>;
        for (int64_t j0 = first; j0 < end; j0 += kSlotChunk) {
            int64_t at[kSlotChunk];
            float w[kSlotChunk], dot[kSlotChunk];
            // a lane per slot: their indices and weights are one read each
            const int64_t mine = j0 + threadIdx.x % kSlotChunk;
            const int32_t slot_row = mine < end ? row_of[t * top_k + mine] : -1;
            const float slot_weight = mine < end ? weights[t * top_k + mine] : 0.0f;
            const uint32_t mask =
                static_cast<uint32_t>(__ballot(slot_row >= 0 && slot_row < rows)) & ((1u << kSlotChunk) - 1u);
#pragma unroll
            for (int j = 0; j < kSlotChunk; ++j) {
                dot[j] = 0.0f;
                w[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(slot_weight), j));
                at[j] = static_cast<int64_t>(__builtin_amdgcn_readlane(slot_row, j)) * hidden * kBytesOf<TE>;
            }
            if (mask) {
                for (uint32_t c0 = threadIdx.x; c0 < nvec; c0 += L * kGradVecs) {
                    typename G::Raw gr[kGradVecs];
#pragma unroll
                    for (int u = 0; u < kGradVecs; ++u)
                        gr[u] = c0 + u * L < nvec ? G::load(grow, (c0 + u * L) * N) : typename G::Raw{};
#pragma unroll
                    for (int jj = 0; jj < kSlotChunk; jj += kGradRows) {
                        typename E::Raw er[kGradRows][kGradVecs];
                        if constexpr (kDot) {
#pragma unroll
                            for (int q = 0; q < kGradRows; ++q) {
                                if (!(mask >> (jj + q) & 1u)) continue;
#pragma unroll
                                for (int u = 0; u < kGradVecs; ++u)
                                    er[q][u] = c0 + u * L < nvec ? E::load(in + at[jj + q], (c0 + u * L) * N)
                                                                 : typename E::Raw{};
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kGradRows; ++q) {
                            if (!(mask >> (jj + q) & 1u)) continue;
#pragma unroll
                            for (int u = 0; u < kGradVecs; ++u) {
                                float g[N], o[N];
                                G::widen(gr[u], g);
                                if constexpr (kDot) {
                                    float f[N];
                                    E::widen(er[q][u], f);
#pragma unroll
                                    for (int i = 0; i < N; ++i) dot[jj + q] = __fmaf_rn(g[i], f[i], dot[jj + q]);
                                }
#pragma unroll
                                for (int i = 0; i < N; ++i) o[i] = w[jj + q] * g[i];
                                if (c0 + u * L < nvec) E::store(grad_in + at[jj + q], (c0 + u * L) * N, o);
                            }
                        }
                    }
                }
                if (!kAligned && threadIdx.x < left) {
                    const float g = Elem<TG>::load1(grow, done + threadIdx.x);
#pragma unroll
                    for (int j = 0; j < kSlotChunk; ++j) {
                        if (!(mask >> j & 1u)) continue;
                        if constexpr (kDot)
                            dot[j] = __fmaf_rn(g, Elem<TE>::load1(in + at[j], done + threadIdx.x), dot[j]);
                        Elem<TE>::store1(grad_in + at[j], done + threadIdx.x, w[j] * g);
                    }
                }
            }
            if constexpr (kDot) {
                const int lane = static_cast<int>(threadIdx.x & 63u), wave = static_cast<int>(threadIdx.x >> 6);
#pragma unroll
                for (int j = 0; j < kSlotChunk; ++j) {
                    const float s = mask >> j & 1u ? group_sum<64>(dot[j]) : 0.0f;
                    if (lane == 0) part[wave][j] = s;
                }
                __syncthreads();
                if (threadIdx.x < kSlotChunk && j0 + threadIdx.x < end) {
                    float s = 0.0f;
#pragma unroll
                    for (int v = 0; v < kWaves; ++v) s += part[v][threadIdx.x];
                    grad_w[t * top_k + j0 + threadIdx.x] = s;
                }
                __syncthreads();
            }
        }
    }
}

// ---- narrow rows --------------------------------------------------------------------------
//
// A row of up to 32 vectors leaves most lanes of a wavefront idle, and the
// kernels above are then bound by the wavefronts they start. Here 2^gs lanes
// (8, 16 or 32) take a row or token, so that a wavefront takes 8, 4 or 2. The
// slots' indices differ between the lanes' groups and are read by the lanes.
// bf16 rows of 64 / 128 / 256, us with these and with the kernels above:
// dispatch of 262144 rows 10.6 / 20.3 / 39.3 against 57 / 58 / 58; sums of 4
// rows for 131072 tokens 16.6 / 30.5 / 56 against 92 / 93 / 94; their gradients
// 31 / 60 / 116 against 177 / 184 / 201.

constexpr int kNarrowLanes = 256;
constexpr int64_t kNarrowVecs = 32;
constexpr int kNarrowRows = 4;  // rows whose loads are in flight together

inline int group_shift(int64_t nvec) { return nvec > 16 ? 5 : (nvec > 8 ? 4 : 3); }

template <int kAlign>
__global__ __launch_bounds__(kNarrowLanes) void moe_dispatch_narrow_kernel(const char* __restrict__ x,
                                                                           const int32_t* __restrict__ slot_of,
                                                                           char* __restrict__ out, int64_t rows,
                                                                           int64_t slots, uint32_t top_k,
                                                                           int row_bytes, int gs) {
    typedef typename Word<16, kAlign>::type Piece;
    const int group = static_cast<int>(threadIdx.x) >> gs, lane = static_cast<int>(threadIdx.x) & ((1 << gs) - 1);
    const int64_t per = kNarrowLanes >> gs;
    const int pieces = row_bytes / 16, done = pieces * 16, left = (row_bytes - done) / 2;
    for (int64_t b = blockIdx.x; b * per * kNarrowRows < rows; b += gridDim.x) {
        int32_t slot[kNarrowRows];
        u32x4 v[kNarrowRows];
        uint16_t v1[kNarrowRows];
#pragma unroll
        for (int k = 0; k < kNarrowRows; ++k) {
            const int64_t r = (b * kNarrowRows + k) * per + group;
            slot[k] = r < rows ? slot_of[r] : -1;
        }
#pragma unroll
        for (int k = 0; k < kNarrowRows; ++k) {
            v[k] = u32x4{0u, 0u, 0u, 0u};
            v1[k] = 0;
            if (slot[k] < 0 || slot[k] >= slots) continue;
            const char* src = x + static_cast<int64_t>(static_cast<uint32_t>(slot[k]) / top_k) * row_bytes;
            if (lane < pieces) v[k] = *reinterpret_cast<const Piece*>(src + lane * 16);
            if (kAlign < 16 && lane < left) v1[k] = *reinterpret_cast<const uint16_t*>(src + done + 2 * lane);
        }
#pragma unroll
        for (int k = 0; k < kNarrowRows; ++k) {
            const int64_t r = (b * kNarrowRows + k) * per + group;
            if (r >= rows) continue;
            char* dst = out + r * row_bytes;
            if (lane < pieces) store_word<16, kAlign>(dst + lane * 16, v[k]);
            if (kAlign < 16 && lane < left) *reinterpret_cast<uint16_t*>(dst + done + 2 * lane) = v1[k];
        }
    }
}

template <int TI, int TO, int N, bool kWeighted, bool kAligned>
__global__ __launch_bounds__(kNarrowLanes) void moe_row_sum_narrow_kernel(
    const char* __restrict__ in, const int32_t* __restrict__ row_of, const float* __restrict__ weights,
    char* __restrict__ out, int64_t rows, int64_t tokens, int64_t top_k, int hidden, int gs) {
    typedef Vec<TI, N, kAligned> In;
    typedef Vec<TO, N, kAligned> Out;
    const int group = static_cast<int>(threadIdx.x) >> gs, lane = static_cast<int>(threadIdx.x) & ((1 << gs) - 1);
    const int64_t per = kNarrowLanes >> gs;
    const int nvec = hidden / N, done = nvec * N;
    const bool full = lane < nvec, tail = !kAligned && lane < hidden - done;
    for (int64_t t0 = blockIdx.x * per; t0 < tokens; t0 += gridDim.x * per) {
        const int64_t t = t0 + group;
        if (t >= tokens) continue;
        float acc[N] = {};
        float acc1 = 0.0f;
        for (int64_t j0 = 0; j0 < top_k; j0 += kNarrowRows) {
            int32_t r[kNarrowRows];
            float w[kNarrowRows], v1[kNarrowRows];
            typename In::Raw v[kNarrowRows];
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                r[q] = j0 + q < top_k ? row_of[t * top_k + j0 + q] : -1;
                w[q] = kWeighted && j0 + q < top_k ? weights[t * top_k + j0 + q] : 1.0f;
            }
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                v[q] = typename In::Raw{};
                v1[q] = 0.0f;
                if (r[q] < 0 || r[q] >= rows) continue;
                const char* row = in + static_cast<int64_t>(r[q]) * hidden * kBytesOf<TI>;
                if (full) v[q] = In::load(row, lane * N);
                if (tail) v1[q] = Elem<TI>::load1(row, done + lane);
            }
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                if (r[q] < 0 || r[q] >= rows) continue;
                float f[N];
                In::widen(v[q], f);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = kWeighted ? __fmaf_rn(w[q], f[i], acc[i]) : acc[i] + f[i];
                acc1 = kWeighted ? __fmaf_rn(w[q], v1[q], acc1) : acc1 + v1[q];
            }
        }
        char* orow = out + t * hidden * kBytesOf<TO>;
        if (full) Out::store(orow, lane * N, acc);
        if (tail) Elem<TO>::store1(orow, done + lane, acc1);
    }
}

template <int TG, int TE, int N, bool kDot, bool kAligned>
__global__ __launch_bounds__(kNarrowLanes) void moe_combine_grad_narrow_kernel(
    const char* __restrict__ grad, const char* __restrict__ in, const int32_t* __restrict__ row_of,
    const float* __restrict__ weights, char* __restrict__ grad_in, float* __restrict__ grad_w, int64_t rows,
    int64_t tokens, int64_t top_k, int hidden, int gs) {
    typedef Vec<TG, N, kAligned> G;
    typedef Vec<TE, N, kAligned> E;
    const int group = static_cast<int>(threadIdx.x) >> gs, lane = static_cast<int>(threadIdx.x) & ((1 << gs) - 1);
    const int64_t per = kNarrowLanes >> gs;
    const int nvec = hidden / N, done = nvec * N;
    const bool full = lane < nvec, tail = !kAligned && lane < hidden - done;
    for (int64_t t0 = blockIdx.x * per; t0 < tokens; t0 += gridDim.x * per) {
        const int64_t t = t0 + group;
        if (t >= tokens) continue;
        const char* grow = grad + t * hidden * kBytesOf<TG>;
        float g[N], g1 = 0.0f;
        typename G::Raw raw{};
        if (full) raw = G::load(grow, lane * N);
        if (tail) g1 = Elem<TG>::load1(grow, done + lane);
        G::widen(raw, g);
        for (int64_t j0 = 0; j0 < top_k; j0 += kNarrowRows) {
            int32_t r[kNarrowRows];
            float w[kNarrowRows], v1[kNarrowRows];
            typename E::Raw v[kNarrowRows];
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                r[q] = j0 + q < top_k ? row_of[t * top_k + j0 + q] : -1;
                w[q] = j0 + q < top_k ? weights[t * top_k + j0 + q] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                v[q] = typename E::Raw{};
                v1[q] = 0.0f;
                if (!kDot || r[q] < 0 || r[q] >= rows) continue;
                const char* row = in + static_cast<int64_t>(r[q]) * hidden * kBytesOf<TE>;
                if (full) v[q] = E::load(row, lane * N);
                if (tail) v1[q] = Elem<TE>::load1(row, done + lane);
            }
#pragma unroll
            for (int q = 0; q < kNarrowRows; ++q) {
                const bool has = r[q] >= 0 && r[q] < rows;
                if (has) {
                    char* row = grad_in + static_cast<int64_t>(r[q]) * hidden * kBytesOf<TE>;
                    float o[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = w[q] * g[i];
                    if (full) E::store(row, lane * N, o);
                    if (tail) Elem<TE>::store1(row, done + lane, w[q] * g1);
                }
                if constexpr (kDot) {
                    if (j0 + q >= top_k) continue;
                    float dot = 0.0f;
                    if (has) {
                        float f[N];
                        E::widen(v[q], f);
                        dot = g1 * v1[q];
#pragma unroll
                        for (int i = 0; i < N; ++i) dot = __fmaf_rn(g[i], f[i], dot);
                    }
                    for (int off = (1 << gs) / 2; off > 0; off >>= 1) dot += __shfl_xor(dot, off, 64);
                    if (lane == 0) grad_w[t * top_k + j0 + q] = has ? dot : 0.0f;
                }
            }
        }
    }
}

// ---- launches ------------------------------------------------------------------------

template <int TI, int TO, bool kWeighted>
int launch_sum(const void* in, const int32_t* row_of, const float* weights, void* out, int64_t rows, int64_t tokens,
               int64_t top_k, int64_t hidden, hipStream_t st) {
    constexpr int N = TI == MOE_EPI_F32 || TO == MOE_EPI_F32 ? 4 : 8;
    const bool fit = hidden % N == 0 && aligned(in, N * kBytesOf<TI>) && aligned(out, N * kBytesOf<TO>);
    const int64_t nvec = hidden / N;
    // few wavefronts, tokens with several rows (at the kernel)
    const bool few = rows > 2 * tokens && tokens * ((nvec + 2 * kSumLanes - 1) / (2 * kSumLanes)) <= 1024;
    const int64_t per = kSumLanes * (few ? 1 : 2);
    const int64_t nseg = nvec <= per ? 1 : (nvec + per - 1) / per;
    const dim3 grid(grid_for_rows(tokens * nseg, 1)), block(kSumLanes);
    const char* i = static_cast<const char*>(in);
    char* o = static_cast<char*>(out);
    (void)hipGetLastError();
    if (nvec <= kNarrowVecs) {
        const int gs = group_shift(nvec);
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(grid_for_rows(tokens, kNarrowLanes >> gs)), dim3(kNarrowLanes), 0, st, i,
                               row_of, weights, o, rows, tokens, top_k, static_cast<int>(hidden), gs);
        };
        fit ? go(moe_row_sum_narrow_kernel<TI, TO, N, kWeighted, true>)
            : go(moe_row_sum_narrow_kernel<TI, TO, N, kWeighted, false>);
    } else {
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, st, i, row_of, weights, o, rows, tokens, top_k, hidden,
                               static_cast<uint32_t>(nseg));
        };
        if (few)
            fit ? go(moe_row_sum_kernel<TI, TO, N, 1, kWeighted, true>)
                : go(moe_row_sum_kernel<TI, TO, N, 1, kWeighted, false>);
        else
            fit ? go(moe_row_sum_kernel<TI, TO, N, 2, kWeighted, true>)
                : go(moe_row_sum_kernel<TI, TO, N, 2, kWeighted, false>);
    }
    return launch_status();
}

template <int TG, int TE>
int launch_grad(const void* grad, const void* in, const int32_t* row_of, const float* weights, void* grad_in,
                float* grad_w, int64_t rows, int64_t tokens, int64_t top_k, int64_t hidden, hipStream_t st) {
    constexpr int N = TG == MOE_EPI_F32 || TE == MOE_EPI_F32 ? 4 : 8;
    const bool fit = hidden % N == 0 && aligned(grad, N * kBytesOf<TG>) && aligned(in, N * kBytesOf<TE>) &&
                     aligned(grad_in, N * kBytesOf<TE>);
    auto go = [&](int lanes, auto kernel) {
        const int64_t waves = tokens * top_k * (lanes / 64);  // with a block for every slot
        const int64_t span = waves <= 1024 ? 1 : (waves <= 4096 ? 2 : (waves <= 8192 ? 4 : top_k));
        const int64_t parts = (top_k + span - 1) / span;
        const dim3 grid(grid_for_rows(tokens * parts, 1));
        hipLaunchKernelGGL(kernel, grid, dim3(lanes), 0, st, static_cast<const char*>(grad),
                           static_cast<const char*>(in), row_of, weights, static_cast<char*>(grad_in), grad_w, rows,
                           tokens, top_k, hidden, static_cast<uint32_t>(parts), static_cast<uint32_t>(span));
    };
    auto pick = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        if (fit && grad_w)
            go(L, moe_combine_grad_kernel<TG, TE, N, L, true, true>);
        else if (fit)
            go(L, moe_combine_grad_kernel<TG, TE, N, L, false, true>);
        else if (grad_w)
            go(L, moe_combine_grad_kernel<TG, TE, N, L, true, false>);
        else
            go(L, moe_combine_grad_kernel<TG, TE, N, L, false, false>);
    };
    (void)hipGetLastError();
    const int64_t nvec = hidden / N;
    if (nvec <= kNarrowVecs) {
        const int gs = group_shift(nvec);
        auto narrow = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(grid_for_rows(tokens, kNarrowLanes >> gs)), dim3(kNarrowLanes), 0, st,
                               static_cast<const char*>(grad), static_cast<const char*>(in), row_of, weights,
                               static_cast<char*>(grad_in), grad_w, rows, tokens, top_k, static_cast<int>(hidden), gs);
        };
        if (grad_w)
            fit ? narrow(moe_combine_grad_narrow_kernel<TG, TE, N, true, true>)
                : narrow(moe_combine_grad_narrow_kernel<TG, TE, N, true, false>);
        else
            fit ? narrow(moe_combine_grad_narrow_kernel<TG, TE, N, false, true>)
                : narrow(moe_combine_grad_narrow_kernel<TG, TE, N, false, false>);
    } else if (nvec <= 64 * kGradVecs)
        pick(std::integral_constant<int, 64>());
    else if (nvec <= 128 * kGradVecs)
        pick(std::integral_constant<int, 128>());
    else
        pick(std::integral_constant<int, 256>());
    return launch_status();
}

// Sizes and byte counts shared by the calls below.
struct Sizes {
    int64_t row_bytes = 0, token_bytes = 0, slot_bytes = 0;
    bool ok = false;
    Sizes(int64_t rows, int64_t tokens, int64_t top_k, int64_t hidden, int row_elem, int token_elem) {
        ok = rows >= 0 && tokens >= 0 && rows <= INT32_MAX && top_k >= 1 && top_k <= kMaxTopK && hidden >= 1 &&
             row_fits_u32_offsets(hidden, 4) && tokens <= INT32_MAX / top_k &&
             bytes_ok(rows, hidden, row_elem, &row_bytes) && bytes_ok(tokens, hidden, token_elem, &token_bytes);
        slot_bytes = ok ? tokens * top_k * 4 : 0;
    }
};

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int moe_dispatch_fwd(const void* x, int dtype, const int32_t* slot_of, void* out, int64_t rows,
                                int64_t tokens, int64_t top_k, int64_t hidden, void* stream) {
    if (!dtype_ok(dtype)) return MOE_EPI_ERR_BAD_DTYPE;
    const int e = elem_bytes(dtype);
    const Sizes n(rows, tokens, top_k, hidden, e, e);
    if (!n.ok) return MOE_EPI_ERR_BAD_SHAPE;
    if (rows == 0) return MOE_EPI_SUCCESS;
    if ((tokens > 0 && !x) || !slot_of || !out) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(x, e) || !aligned(out, e) || !aligned(slot_of, 4)) return MOE_EPI_ERR_MISALIGNED;
    const Range ro = range_of(out, n.row_bytes);
    if (overlaps(ro, range_of(x, n.token_bytes)) || overlaps(ro, range_of(slot_of, rows * 4))) return MOE_EPI_ERR_ALIAS;
    const bool again = rows > 2 * tokens;  // tokens have several rows each
    const int64_t bytes = hidden * e, per = kCopyLanes * (again ? 2 : 1);
    const int64_t nseg = bytes / 16 <= per ? 1 : (bytes / 16 + per - 1) / per;
    const dim3 grid(grid_for_rows(rows * nseg, 1)), block(kCopyLanes);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, as_stream(stream), static_cast<const char*>(x), slot_of,
                           static_cast<char*>(out), rows, tokens * top_k, static_cast<uint32_t>(top_k), bytes,
                           static_cast<uint32_t>(nseg));
    };
    auto narrow = [&](auto kernel) {
        const int gs = group_shift(bytes / 16);
        hipLaunchKernelGGL(kernel, dim3(grid_for_rows(rows, (kNarrowLanes >> gs) * kNarrowRows)), dim3(kNarrowLanes), 0,
                           as_stream(stream), static_cast<const char*>(x), slot_of, static_cast<char*>(out), rows,
                           tokens * top_k, static_cast<uint32_t>(top_k), static_cast<int>(bytes), gs);
    };
    const bool sixteen = bytes % 16 == 0 && aligned(x, 16) && aligned(out, 16),
               four = bytes % 4 == 0 && aligned(x, 4) && aligned(out, 4);
    (void)hipGetLastError();
    if (bytes / 16 <= kNarrowVecs) {
        if (sixteen)
            narrow(moe_dispatch_narrow_kernel<16>);
        else
            four ? narrow(moe_dispatch_narrow_kernel<4>) : narrow(moe_dispatch_narrow_kernel<2>);
    } else if (sixteen)
        again ? go(moe_dispatch_kernel<16, 2>) : go(moe_dispatch_kernel<16, 1>);
    else if (four)
        again ? go(moe_dispatch_kernel<4, 2>) : go(moe_dispatch_kernel<4, 1>);
    else
        again ? go(moe_dispatch_kernel<2, 2>) : go(moe_dispatch_kernel<2, 1>);
    return launch_status();
}

extern "C" int moe_dispatch_bwd(const void* grad_out, int dtype, const int32_t* row_of, void* grad_x, int64_t rows,
                                int64_t tokens, int64_t top_k, int64_t hidden, void* stream) {
    if (!dtype_ok(dtype)) return MOE_EPI_ERR_BAD_DTYPE;
    const int e = elem_bytes(dtype);
    const Sizes n(rows, tokens, top_k, hidden, e, e);
    if (!n.ok) return MOE_EPI_ERR_BAD_SHAPE;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if ((rows > 0 && !grad_out) || !row_of || !grad_x) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(grad_out, e) || !aligned(grad_x, e) || !aligned(row_of, 4)) return MOE_EPI_ERR_MISALIGNED;
    const Range ro = range_of(grad_x, n.token_bytes);
    if (overlaps(ro, range_of(grad_out, n.row_bytes)) || overlaps(ro, range_of(row_of, n.slot_bytes)))
        return MOE_EPI_ERR_ALIAS;
    const hipStream_t st = as_stream(stream);
    switch (dtype) {
        case MOE_EPI_BF16:
            return launch_sum<MOE_EPI_BF16, MOE_EPI_BF16, false>(grad_out, row_of, nullptr, grad_x, rows, tokens,
                                                                 top_k, hidden, st);
        case MOE_EPI_F16:
            return launch_sum<MOE_EPI_F16, MOE_EPI_F16, false>(grad_out, row_of, nullptr, grad_x, rows, tokens, top_k,
                                                               hidden, st);
        default:
            return launch_sum<MOE_EPI_F32, MOE_EPI_F32, false>(grad_out, row_of, nullptr, grad_x, rows, tokens, top_k,
                                                               hidden, st);
    }
}

extern "C" int moe_combine_weighted_fwd(const void* expert_out, int eo_dtype, const int32_t* row_of,
                                        const float* weights, void* out, int out_dtype, int64_t rows, int64_t tokens,
                                        int64_t top_k, int64_t hidden, void* stream) {
    if (!dtype_ok(eo_dtype) || (out_dtype != eo_dtype && out_dtype != MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    const int e = elem_bytes(eo_dtype), eo = elem_bytes(out_dtype);
    const Sizes n(rows, tokens, top_k, hidden, e, eo);
    if (!n.ok) return MOE_EPI_ERR_BAD_SHAPE;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if ((rows > 0 && !expert_out) || !row_of || !weights || !out) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(expert_out, e) || !aligned(out, eo) || !aligned(row_of, 4) || !aligned(weights, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range ro = range_of(out, n.token_bytes);
    if (overlaps(ro, range_of(expert_out, n.row_bytes)) || overlaps(ro, range_of(row_of, n.slot_bytes)) ||
        overlaps(ro, range_of(weights, n.slot_bytes)))
        return MOE_EPI_ERR_ALIAS;
    const hipStream_t st = as_stream(stream);
    auto go = [&](auto launch) { return launch(expert_out, row_of, weights, out, rows, tokens, top_k, hidden, st); };
    if (eo_dtype == MOE_EPI_F32) return go(launch_sum<MOE_EPI_F32, MOE_EPI_F32, true>);
    if (eo_dtype == MOE_EPI_BF16)
        return out_dtype == MOE_EPI_F32 ? go(launch_sum<MOE_EPI_BF16, MOE_EPI_F32, true>)
                                        : go(launch_sum<MOE_EPI_BF16, MOE_EPI_BF16, true>);
    return out_dtype == MOE_EPI_F32 ? go(launch_sum<MOE_EPI_F16, MOE_EPI_F32, true>)
                                    : go(launch_sum<MOE_EPI_F16, MOE_EPI_F16, true>);
}

extern "C" int moe_combine_weighted_bwd(const void* grad_out, int go_dtype, const void* expert_out, int eo_dtype,
                                        const int32_t* row_of, const float* weights, void* grad_expert_out,
                                        float* grad_weights, int64_t rows, int64_t tokens, int64_t top_k,
                                        int64_t hidden, void* stream) {
    if (!dtype_ok(eo_dtype) || (go_dtype != eo_dtype && go_dtype != MOE_EPI_F32)) return MOE_EPI_ERR_BAD_DTYPE;
    const int e = elem_bytes(eo_dtype), g = elem_bytes(go_dtype);
    const Sizes n(rows, tokens, top_k, hidden, e, g);
    if (!n.ok) return MOE_EPI_ERR_BAD_SHAPE;
    if (tokens == 0) return MOE_EPI_SUCCESS;
    if (!grad_out || !row_of || !weights || (rows > 0 && !grad_expert_out) ||
        (rows > 0 && grad_weights && !expert_out))
        return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(grad_out, g) || !aligned(expert_out, e) || !aligned(grad_expert_out, e) || !aligned(row_of, 4) ||
        !aligned(weights, 4) || !aligned(grad_weights, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range in[4] = {range_of(grad_out, n.token_bytes), range_of(expert_out, expert_out ? n.row_bytes : 0),
                         range_of(row_of, n.slot_bytes), range_of(weights, n.slot_bytes)},
                gi = range_of(grad_expert_out, n.row_bytes),
                gw = range_of(grad_weights, grad_weights ? n.slot_bytes : 0);
    for (const Range& r : in)
        if (overlaps(gi, r) || overlaps(gw, r)) return MOE_EPI_ERR_ALIAS;
    if (overlaps(gi, gw)) return MOE_EPI_ERR_ALIAS;
    const hipStream_t st = as_stream(stream);
    auto go = [&](auto launch) {
        return launch(grad_out, expert_out, row_of, weights, grad_expert_out, grad_weights, rows, tokens, top_k,
                      hidden, st);
    };
    if (eo_dtype == MOE_EPI_F32) return go(launch_grad<MOE_EPI_F32, MOE_EPI_F32>);
    if (eo_dtype == MOE_EPI_BF16)
        return go_dtype == MOE_EPI_F32 ? go(launch_grad<MOE_EPI_F32, MOE_EPI_BF16>)
                                       : go(launch_grad<MOE_EPI_BF16, MOE_EPI_BF16>);
    return go_dtype == MOE_EPI_F32 ? go(launch_grad<MOE_EPI_F32, MOE_EPI_F16>)
                                   : go(launch_grad<MOE_EPI_F16, MOE_EPI_F16>);
}
