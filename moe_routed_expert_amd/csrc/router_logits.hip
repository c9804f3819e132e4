// The router's product and its gradients (gfx950).
#include <type_traits>

#include "bf16_pieces.h"
#include "epi_common.h"
#include "moe_prologue.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMostExperts = 1024;

// ---- logits ---------------------------------------------------------------------

constexpr int kStep = 64;       // of hidden, in one pass of the loop
constexpr int kTileRows = 128;  // tokens of a block: 32 for each of 4 wavefronts
constexpr int64_t kMostRows = 1 << 24;  // tokens of a launch
constexpr int kFewRows = 64;
constexpr int kFewWaves = 8;

// Pieces that x and the weight are cut into.
template <int T, int W>
struct Pieces {
    static constexpr bool kF16 = T == MOE_EPI_F16 && W == MOE_EPI_F16;
    static constexpr int kX = T == MOE_EPI_F32 ? 3 : (T == MOE_EPI_F16 && !kF16 ? 2 : 1);
    static constexpr int kW = W == MOE_EPI_F32 ? 3 : 1;
};

// The 16-byte store of four experts' logits of one token, or what of it there is.
__device__ __forceinline__ void put4(float* row, int64_t e, int64_t experts, f32x4 v) {
    typedef f32x4 loose __attribute__((aligned(4)));
    if (experts % 4 == 0) {
        if (e < experts) *reinterpret_cast<loose*>(row + e) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < experts) row[e + i] = v[i];
    }
}

// 128 tokens x 16 NT experts, over the steps [steps z / n, steps (z + 1) / n) of hidden.
template <int T, int W, int NT>
__global__ __launch_bounds__(kBlock) void logits_tile_kernel(const char* __restrict__ x, const char* __restrict__ weight,
                                                             float* __restrict__ out, int64_t tokens, int64_t hidden,
                                                             int64_t experts) {
    typedef Pieces<T, W> P;
    typedef Piece8<T> X;
    typedef Piece8<W> Y;
    constexpr int kFrags = 2 * NT, kMine = (kFrags + 3) / 4;
    __shared__ u32x4 lds[2][P::kW][kFrags][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTileRows + 32 * wave, e0 = blockIdx.y * 16 * NT;
    const int64_t steps = (hidden + kStep - 1) / kStep;
    const int64_t first = steps * blockIdx.z / gridDim.z, last = steps * (blockIdx.z + 1) / gridDim.z;
    const char* px[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int64_t t = row0 + 16 * m + of16;
        px[m] = x + ((t < tokens ? t : tokens - 1) * hidden + k8) * X::kBytes;
    }
    const char* pw[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int f = wave + 4 * i;
        const int64_t e = e0 + 16 * (f / 2) + of16;
        pw[i] = weight + ((e < experts ? e : experts - 1) * hidden + 32 * (f % 2) + k8) * Y::kBytes;
    }
    f32x4 d[2][NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) d[m][n] = f32x4{0, 0, 0, 0};

    struct Ahead {
        typename X::Raw x[2][2];
        typename Y::Raw w[kMine];
    };
    auto load = [&](int64_t step, Ahead& a) {
        const int64_t k = step * kStep, left = hidden - k - k8;
        if (k + kStep <= hidden) {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                if (kFrags >= 4 || wave < kFrags) a.w[i] = Y::load(pw[i] + k * Y::kBytes);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) a.x[m][h] = X::load_nt(px[m] + (k + 32 * h) * X::kBytes);
        } else {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                if (kFrags >= 4 || wave < kFrags)
                    a.w[i] = Y::load_first(pw[i] + k * Y::kBytes, left - 32 * ((wave + 4 * i) % 2));
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) a.x[m][h] = X::load_first(px[m] + (k + 32 * h) * X::kBytes, left - 32 * h);
        }
    };
    auto stage = [&](const Ahead& a, int buf) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (kFrags < 4 && wave >= kFrags) continue;
            u32x4 piece[P::kW];
            cut_raw<W, P::kW>(a.w[i], piece);
#pragma unroll
            for (int p = 0; p < P::kW; ++p) lds[buf][p][wave + 4 * i][lane] = piece[p];
        }
    };
    auto multiply = [&](const Ahead& a, int buf) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 xp[2][P::kX];
#pragma unroll
            for (int m = 0; m < 2; ++m) cut_raw<T, P::kX>(a.x[m][h], xp[m]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                u32x4 wp[P::kW];
#pragma unroll
                for (int p = 0; p < P::kW; ++p) wp[p] = lds[buf][p][2 * n + h][lane];
#pragma unroll
                for (int m = 0; m < 2; ++m) d[m][n] = mfma_pieces<P::kF16>(wp, xp[m], d[m][n]);
            }
        }
    };
    auto pass = [&](int64_t s, const Ahead& now, Ahead& next, int buf) {
        if (s + 1 < last) load(s + 1, next);
        multiply(now, buf);
        if (s + 1 < last) stage(next, buf ^ 1);
        __syncthreads();
    };
    Ahead a, b;
    if (first < last) {
        load(first, a);
        stage(a, 0);
    }
    __syncthreads();
    for (int64_t s = first; s < last; s += 2) {
        pass(s, a, b, 0);
        if (s + 1 < last) pass(s + 1, b, a, 1);
    }
    float* to = out + blockIdx.z * tokens * experts;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int64_t t = row0 + 16 * m + of16;
        if (t >= tokens) continue;
#pragma unroll
        for (int n = 0; n < NT; ++n) put4(to + t * experts, e0 + 16 * n + lane / 16 * 4, experts, d[m][n]);
    }
}

// Up to 16 MT tokens x 16 experts: 8 wavefronts share the steps of hidden that
// the block has, and their sums are added in their order.
template <int T, int W, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void logits_few_kernel(const char* __restrict__ x,
                                                                    const char* __restrict__ weight,
                                                                    float* __restrict__ out, int64_t tokens,
                                                                    int64_t hidden, int64_t experts) {
    typedef Pieces<T, W> P;
    typedef Piece8<T> X;
    typedef Piece8<W> Y;
    __shared__ f32x4 part[kFewWaves][MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t e = blockIdx.x * 16 + of16, row0 = static_cast<int64_t>(blockIdx.y) * 16 * MT;
    const char* pw = weight + ((e < experts ? e : experts - 1) * hidden + k8) * Y::kBytes;
    const char* px[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t t = row0 + 16 * m + of16;
        px[m] = x + ((t < tokens ? t : tokens - 1) * hidden + k8) * X::kBytes;
    }
    f32x4 d[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) d[m] = f32x4{0, 0, 0, 0};
    const int64_t steps = (hidden + 31) / 32, full = hidden / 32, all = static_cast<int64_t>(gridDim.z) * kFewWaves;
    const int64_t me = blockIdx.z * kFewWaves + wave;
    const int64_t first = steps * me / all, last = steps * (me + 1) / all;
    auto multiply = [&](const typename Y::Raw& w, const typename X::Raw (&v)[MT]) {
        u32x4 wp[P::kW];
        cut_raw<W, P::kW>(w, wp);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            u32x4 xp[P::kX];
            cut_raw<T, P::kX>(v[m], xp);
            d[m] = mfma_pieces<P::kF16>(wp, xp, d[m]);
        }
    };
    int64_t s = first;
    constexpr int kAhead = 4;
    for (; s + kAhead <= (last < full ? last : full); s += kAhead) {
        typename Y::Raw w[kAhead];
        typename X::Raw v[kAhead][MT];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            w[i] = Y::load(pw + (s + i) * 32 * Y::kBytes);
#pragma unroll
            for (int m = 0; m < MT; ++m) v[i][m] = X::load(px[m] + (s + i) * 32 * X::kBytes);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) multiply(w[i], v[i]);
    }
    for (; s < last; ++s) {
        const int64_t left = hidden - s * 32 - k8;
        typename X::Raw v[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) v[m] = X::load_first(px[m] + s * 32 * X::kBytes, left);
        multiply(Y::load_first(pw + s * 32 * Y::kBytes, left), v);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][m][lane] = d[m];
    __syncthreads();
    if (wave >= MT) return;
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) sum += part[i][wave][lane];
    const int64_t t = row0 + 16 * wave + of16;
    if (t < tokens)
        put4(out + (blockIdx.z * tokens + t) * experts, blockIdx.x * 16 + lane / 16 * 4, experts, sum);
}

// out[i] = the sum of parts[s][i], in their order
__global__ __launch_bounds__(kBlock) void add_parts_kernel(const float* __restrict__ parts, float* __restrict__ out,
                                                           int n_parts, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kBlock) {
        float sum = parts[i];
        for (int s = 1; s < n_parts; ++s) sum += parts[s * n + i];
        out[i] = sum;
    }
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts that hidden is shared by: enough blocks for the chip, and a few steps each.
int64_t logits_parts(int64_t tokens, int64_t hidden, int64_t experts) {
    const bool few = tokens <= kFewRows;
    const int64_t blocks = few ? up(experts, 16) : up(tokens, kTileRows) * up(experts, 64);
    const int64_t wanted = up(few ? 16 : 256, blocks), most = up(hidden, few ? 32 * kFewWaves : 4 * kStep);
    const int64_t n = wanted < most ? wanted : most;
    return n < 1 ? 1 : n;
}

// ---- gradients ----------------------------------------------------------------------

// Pieces of the factors. A result of 16 bits is rounded to 2^-9 of itself or
// 2^-12: two pieces of the float32 factors (2^-17 of each term) are beyond that
// even where terms cancel to a hundredth; a float32 result takes all three.
template <int T, int Out>
struct GradPieces {
    static constexpr int kMost = Out == MOE_EPI_F32 ? 2 : 1;   // largest i + j of a pair that counts
    static constexpr int kGrad = kMost + 1;
    static constexpr int kOther = T == MOE_EPI_BF16 ? 1 : (T == MOE_EPI_F16 ? 2 : kMost + 1);
};

// The elements j of eight rows of 16 bytes each, as pieces.
template <int T, int P>
__device__ __forceinline__ void turn_rows(const u32x4 (&r)[8], u32x4 (&piece)[16 / Elem<T>::kBytes][P]) {
    if constexpr (T == MOE_EPI_BF16) {
        u32x4 t[8];
        turn8(r, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) piece[j][0] = t[j];
    } else if constexpr (T == MOE_EPI_F16) {
        u32x4 t[8];
        turn8(r, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) cut_raw<T, P>(typename Piece8<T>::Raw{{t[j]}}, piece[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i][j]);
            cut<P>(f, piece[j]);
        }
    }
}

// 16 bytes of a row, of which `left` elements exist.
template <int T>
__device__ __forceinline__ u32x4 load16(const char* p, int64_t left) {
    typedef u32x4 loose __attribute__((aligned(2)));
    constexpr int n = 16 / Elem<T>::kBytes;
    if (left >= n) return *reinterpret_cast<const loose*>(p);
    u32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < n; ++i) {
        if (i >= left) continue;
        if constexpr (T == MOE_EPI_F32)
            r[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else
            r[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    }
    return r;
}

// 16 HT hidden x the tokens of a block, the experts being the inner dimension.
// The weight's columns lie in LDS as operands, and each wavefront takes 16 MT
// tokens at a time through all of them.
template <int T, int W, int KS, int HT, int MT>
__global__ __launch_bounds__(kBlock) void grad_x_kernel(const float* __restrict__ grad, const char* __restrict__ weight,
                                                        char* __restrict__ grad_x, int64_t tokens, int64_t hidden,
                                                        int64_t experts, int64_t tokens_a_block) {
    typedef GradPieces<W, T> P;
    typedef Piece8<MOE_EPI_F32> G;
    constexpr int V = 16 / Elem<W>::kBytes;  // weights of a 16-byte load
    __shared__ u32x4 lds[HT * KS * P::kOther][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t h0 = static_cast<int64_t>(blockIdx.x) * 16 * HT;
    // Operand row m of tile j is the hidden element that makes a lane's results
    // neighbours in memory: with 16-bit results two tiles give 8 of them.
    constexpr bool kPairs = T != MOE_EPI_F32 && HT % 2 == 0;
    auto place = [&](int h, int& tile, int& m) {  // of hidden element h0 + h
        if constexpr (kPairs) {
            const int in32 = h % 32;
            tile = h / 32 * 2 + in32 % 8 / 4;
            m = in32 / 8 * 4 + in32 % 4;
        } else {
            tile = h / 16;
            m = h % 16;
        }
    };
    for (int i = threadIdx.x; i < 16 * HT / V * KS * 4; i += kBlock) {
        const int hv = i % (16 * HT / V) * V, e8 = i / (16 * HT / V) * 8;
        u32x4 r[8], piece[V][P::kOther];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = e8 + j < experts ? load16<W>(weight + ((e8 + j) * hidden + h0 + hv) * Elem<W>::kBytes, hidden - h0 - hv)
                                    : u32x4{0, 0, 0, 0};
        turn_rows<W, P::kOther>(r, piece);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            int tile, m;
            place(hv + j, tile, m);
#pragma unroll
            for (int p = 0; p < P::kOther; ++p)
                lds[(tile * KS + e8 / 32) * P::kOther + p][m + 16 * (e8 % 32 / 8)] = piece[j][p];
        }
    }
    __syncthreads();
    const int64_t begin = blockIdx.y * tokens_a_block;
    const int64_t end = begin + tokens_a_block < tokens ? begin + tokens_a_block : tokens;
    for (int64_t t0 = begin + wave * 16 * MT; t0 < end; t0 += 4 * 16 * MT) {
        u32x4 g[MT][KS][P::kGrad];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int64_t t = t0 + 16 * m + of16;
            const char* row = reinterpret_cast<const char*>(grad + (t < tokens ? t : tokens - 1) * experts);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int64_t e = 32 * k + k8;
                const typename G::Raw raw = e < experts ? G::load_first(row + 4 * e, experts - e) : typename G::Raw{};
                cut_raw<MOE_EPI_F32, P::kGrad>(raw, g[m][k]);
            }
        }
        constexpr int kAtOnce = kPairs ? 2 : 1;
#pragma unroll 2
        for (int j = 0; j < HT; j += kAtOnce) {
            f32x4 d[kAtOnce][MT];
#pragma unroll
            for (int a = 0; a < kAtOnce; ++a) {
#pragma unroll
                for (int m = 0; m < MT; ++m) d[a][m] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    u32x4 w[P::kOther];
#pragma unroll
                    for (int p = 0; p < P::kOther; ++p) w[p] = lds[((j + a) * KS + k) * P::kOther + p][lane];
#pragma unroll
                    for (int m = 0; m < MT; ++m) d[a][m] = mfma_pieces<false, P::kMost>(w, g[m][k], d[a][m]);
                }
            }
            const int64_t h = h0 + 16 * j + (kPairs ? 8 : 4) * (lane / 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int64_t t = t0 + 16 * m + of16;
                if (t >= end) continue;
                char* to = grad_x + (t * hidden + h) * Elem<T>::kBytes;
                if constexpr (kPairs) {
                    typedef u32x4 loose __attribute__((aligned(2)));
                    const float f[8] = {d[0][m][0], d[0][m][1], d[0][m][2], d[0][m][3],
                                        d[1][m][0], d[1][m][1], d[1][m][2], d[1][m][3]};
                    if (h + 8 <= hidden) {
                        __builtin_nontemporal_store(Elem<T>::pack(f), reinterpret_cast<loose*>(to));
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (h + i < hidden) Elem<T>::store1(to, i, f[i]);
                    }
                } else if constexpr (T == MOE_EPI_F32) {
                    typedef f32x4 loose __attribute__((aligned(4)));
                    if (h + 4 <= hidden) {
                        __builtin_nontemporal_store(d[0][m], reinterpret_cast<loose*>(to));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (h + i < hidden) Elem<T>::store1(to, i, d[0][m][i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (h + i < hidden) Elem<T>::store1(to, i, d[0][m][i]);
                }
            }
        }
    }
}

// As above for more than 256 experts, 256 at a time: 16 hidden a block.
template <int T, int W>
__global__ __launch_bounds__(kBlock) void grad_x_many_kernel(const float* __restrict__ grad,
                                                             const char* __restrict__ weight,
                                                             char* __restrict__ grad_x, int64_t tokens, int64_t hidden,
                                                             int64_t experts, int64_t tokens_a_block) {
    typedef GradPieces<W, T> P;
    typedef Piece8<MOE_EPI_F32> G;
    constexpr int V = 16 / Elem<W>::kBytes, KS = kMostExperts / 32;
    __shared__ u32x4 lds[KS * P::kOther][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t h0 = static_cast<int64_t>(blockIdx.x) * 16;
    for (int i = threadIdx.x; i < 16 / V * KS * 4; i += kBlock) {
        const int hv = i % (16 / V) * V, e8 = i / (16 / V) * 8;
        u32x4 r[8], piece[V][P::kOther];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = e8 + j < experts ? load16<W>(weight + ((e8 + j) * hidden + h0 + hv) * Elem<W>::kBytes, hidden - h0 - hv)
                                    : u32x4{0, 0, 0, 0};
        turn_rows<W, P::kOther>(r, piece);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int p = 0; p < P::kOther; ++p)
                lds[e8 / 32 * P::kOther + p][hv + j + 16 * (e8 % 32 / 8)] = piece[j][p];
    }
    __syncthreads();
    const int64_t begin = blockIdx.y * tokens_a_block;
    const int64_t end = begin + tokens_a_block < tokens ? begin + tokens_a_block : tokens;
    for (int64_t t0 = begin + wave * 16; t0 < end; t0 += 4 * 16) {
        const int64_t t = t0 + of16;
        const char* row = reinterpret_cast<const char*>(grad + (t < tokens ? t : tokens - 1) * experts);
        f32x4 d = {0, 0, 0, 0};
        for (int k = 0; k < (experts + 31) / 32; ++k) {
            const int64_t e = 32 * k + k8;
            const typename G::Raw raw = e < experts ? G::load_first(row + 4 * e, experts - e) : typename G::Raw{};
            u32x4 g[P::kGrad], w[P::kOther];
            cut_raw<MOE_EPI_F32, P::kGrad>(raw, g);
#pragma unroll
            for (int p = 0; p < P::kOther; ++p) w[p] = lds[k * P::kOther + p][lane];
            d = mfma_pieces<false, P::kMost>(w, g, d);
        }
        if (t >= end) continue;
        const int64_t h = h0 + lane / 16 * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (h + i < hidden) Elem<T>::store1(grad_x, t * hidden + h + i, d[i]);
    }
}

// 16 ET experts x 64 HT hidden, over the tokens of part z: the tokens are the
// inner dimension. A wavefront reads 8 tokens' elements of its hidden and turns
// them into operands in registers; the operands of grad are made once a block.
template <int T, int W, int ET>
__global__ __launch_bounds__(kBlock) void grad_weight_kernel(const float* __restrict__ grad, const char* __restrict__ x,
                                                             float* __restrict__ parts, int64_t tokens, int64_t hidden,
                                                             int64_t experts) {
    typedef GradPieces<T, W> P;
    constexpr int HT = 16 / Elem<T>::kBytes;  // hidden of a lane: 16 bytes
    __shared__ u32x4 lds[2][ET][P::kGrad][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t h = static_cast<int64_t>(blockIdx.x) * 64 * HT + wave * 16 * HT + of16 * HT;
    const int64_t e0 = blockIdx.y * 16 * ET, mine = e0 + 16 * wave + of16;
    const int64_t steps = (tokens + 31) / 32;
    const int64_t first = steps * blockIdx.z / gridDim.z, last = steps * (blockIdx.z + 1) / gridDim.z;
    const int64_t left = hidden - h;
    f32x4 d[ET][HT];
#pragma unroll
    for (int e = 0; e < ET; ++e)
#pragma unroll
        for (int j = 0; j < HT; ++j) d[e][j] = f32x4{0, 0, 0, 0};
    struct Ahead {
        u32x4 x[8];
        float g[8];
    };
    auto load = [&](int64_t s, Ahead& a) {
        const int64_t t = s * 32 + k8;
        const char* px = x + (t * hidden + h) * Elem<T>::kBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            a.x[i] = t + i < tokens && left > 0 ? load16<T>(px + i * hidden * Elem<T>::kBytes, left) : u32x4{0, 0, 0, 0};
        if (wave < ET) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a.g[i] = t + i < tokens && mine < experts ? grad[(t + i) * experts + mine] : 0.0f;
        }
    };
    auto stage = [&](Ahead& a, int buf) {
        if (wave >= ET) return;
        u32x4 piece[P::kGrad];
        cut<P::kGrad>(a.g, piece);
#pragma unroll
        for (int p = 0; p < P::kGrad; ++p) lds[buf][wave][p][lane] = piece[p];
    };
    auto pass = [&](int64_t s, Ahead& now, Ahead& next, int buf) {
        if (s + 1 < last) load(s + 1, next);
        u32x4 v[HT][P::kOther];
        turn_rows<T, P::kOther>(now.x, v);
#pragma unroll
        for (int e = 0; e < ET; ++e) {
            u32x4 g[P::kGrad];
#pragma unroll
            for (int p = 0; p < P::kGrad; ++p) g[p] = lds[buf][e][p][lane];
#pragma unroll
            for (int j = 0; j < HT; ++j) d[e][j] = mfma_pieces<false, P::kMost>(g, v[j], d[e][j]);
        }
        if (s + 1 < last) stage(next, buf ^ 1);
        __syncthreads();
    };
    Ahead a, b;
    if (first < last) {
        load(first, a);
        stage(a, 0);
    }
    __syncthreads();
    for (int64_t s = first; s < last; s += 2) {
        pass(s, a, b, 0);
        if (s + 1 < last) pass(s + 1, b, a, 1);
    }
    float* to = parts + blockIdx.z * experts * hidden;
#pragma unroll
    for (int e = 0; e < ET; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t expert = e0 + 16 * e + lane / 16 * 4 + i;
            if (expert >= experts) continue;
#pragma unroll
            for (int j = 0; j < HT; ++j)
                if (j < left) to[expert * hidden + h + j] = d[e][j][i];
        }
}

template <int W>
__global__ __launch_bounds__(kBlock) void add_weight_parts_kernel(const float* __restrict__ parts,
                                                                  void* __restrict__ grad_weight, int n_parts,
                                                                  int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kBlock) {
        float sum = parts[i];
        for (int s = 1; s < n_parts; ++s) sum += parts[s * n + i];
        Elem<W>::store1(grad_weight, i, sum);
    }
}

// Parts that the tokens are shared by for the weight's gradient.
int64_t grad_parts(int64_t tokens, int64_t hidden, int64_t experts) {
    const int64_t blocks = up(hidden, 512) * up(experts, 64), wanted = up(512, blocks), most = up(tokens, 4 * 32);
    const int64_t n = wanted < most ? wanted : most;
    return n < 1 ? 1 : n;
}

bool sizes_ok(int64_t tokens, int64_t hidden, int64_t experts) {
    int64_t a;
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= kMostExperts &&
           bytes_ok(tokens, hidden, 4, &a) && bytes_ok(experts, hidden, 4, &a) && bytes_ok(tokens, experts, 4, &a) &&
           row_fits_u32_offsets(hidden, 4);
}

template <int T, int W>
void launch_logits(const void* x, const void* weight, float* logits, float* workspace, int64_t tokens, int64_t hidden,
                   int64_t experts, hipStream_t st) {
    const int64_t n = logits_parts(tokens, hidden, experts);
    float* to = n > 1 ? workspace : logits;
    const char *px = static_cast<const char*>(x), *pw = static_cast<const char*>(weight);
    if (tokens <= kFewRows) {
        const dim3 grid(static_cast<unsigned>(up(experts, 16)), 1, static_cast<unsigned>(n)), block(64 * kFewWaves);
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, px, pw, to, tokens, hidden, experts); };
        if (tokens <= 16)
            go(logits_few_kernel<T, W, 1>);
        else if (tokens <= 32)
            go(logits_few_kernel<T, W, 2>);
        else
            go(logits_few_kernel<T, W, 4>);
    } else {
        auto go = [&](auto kernel, int nt) {
            // a grid has fewer than 2^32 work-items; calls of so many tokens have one part
            for (int64_t t = 0; t < tokens; t += kMostRows) {
                const int64_t here = tokens - t < kMostRows ? tokens - t : kMostRows;
                const dim3 grid(static_cast<unsigned>(up(here, kTileRows)), static_cast<unsigned>(up(experts, 16 * nt)),
                                static_cast<unsigned>(n));
                hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, st, px + t * hidden * Elem<T>::kBytes, pw,
                                   to + t * experts, here, hidden, experts);
            }
        };
        if (experts <= 16)
            go(logits_tile_kernel<T, W, 1>, 1);
        else if (experts <= 32)
            go(logits_tile_kernel<T, W, 2>, 2);
        else
            go(logits_tile_kernel<T, W, 4>, 4);
    }
    if (n > 1) {
        const int64_t all = tokens * experts, blocks = up(all, kBlock);
        hipLaunchKernelGGL(add_parts_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(kBlock), 0,
                           st, workspace, logits, static_cast<int>(n), all);
    }
}

template <int T, int W>
void launch_grad_x(const float* grad, const void* weight, void* grad_x, int64_t tokens, int64_t hidden, int64_t experts,
                   hipStream_t st) {
    auto go = [&](auto kernel, int width, int wave_tokens) {
        const int64_t columns = up(hidden, width), wanted = up(1024, columns);
        int64_t each = up(up(tokens, wanted), 4 * wave_tokens) * 4 * wave_tokens;
        if (up(tokens, each) > 65535) each = up(up(tokens, 65535), 4 * wave_tokens) * 4 * wave_tokens;
        const dim3 grid(static_cast<unsigned>(columns), static_cast<unsigned>(up(tokens, each)));
        hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, st, grad, static_cast<const char*>(weight),
                           static_cast<char*>(grad_x), tokens, hidden, experts, each);
    };
    // hidden of a block: as many as 64 KB of LDS hold, up to 512
    constexpr int kW = GradPieces<W, T>::kOther;
    auto by_steps = [&](auto ks) {
        constexpr int KS = decltype(ks)::value, kFit = 64 * 1024 / (KS * kW * 1024), MT = KS > 4 ? 1 : 2;
        constexpr int HT = kFit >= 32 ? 32 : (kFit >= 16 ? 16 : (kFit >= 8 ? 8 : (kFit >= 4 ? 4 : 2)));
        go(grad_x_kernel<T, W, KS, HT, MT>, 16 * HT, 16 * MT);
    };
    if (experts <= 32)
        by_steps(std::integral_constant<int, 1>());
    else if (experts <= 64)
        by_steps(std::integral_constant<int, 2>());
    else if (experts <= 128)
        by_steps(std::integral_constant<int, 4>());
    else if (experts <= 256)
        by_steps(std::integral_constant<int, 8>());
    else
        go(grad_x_many_kernel<T, W>, 16, 16);
}

template <int T, int W>
void launch_grad_weight(const float* grad, const void* x, void* grad_weight, float* workspace, int64_t tokens,
                        int64_t hidden, int64_t experts, hipStream_t st) {
    const int64_t n = grad_parts(tokens, hidden, experts);
    auto go = [&](auto kernel, int et) {
        const dim3 grid(static_cast<unsigned>(up(hidden, 64 * 16 / Elem<T>::kBytes)),
                        static_cast<unsigned>(up(experts, 16 * et)), static_cast<unsigned>(n));
        hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, st, grad, static_cast<const char*>(x), workspace, tokens,
                           hidden, experts);
    };
    if (experts <= 16)
        go(grad_weight_kernel<T, W, 1>, 1);
    else if (experts <= 32)
        go(grad_weight_kernel<T, W, 2>, 2);
    else
        go(grad_weight_kernel<T, W, 4>, 4);
    const int64_t all = experts * hidden, blocks = up(all, kBlock);
    hipLaunchKernelGGL(add_weight_parts_kernel<W>, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)),
                       dim3(kBlock), 0, st, workspace, grad_weight, static_cast<int>(n), all);
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
    if (!sizes_ok(tokens, hidden, experts)) return -1;
    const int64_t n = logits_parts(tokens, hidden, experts);
    return n > 1 ? n * tokens * experts * 4 : 0;
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
        launch_logits<decltype(t)::value, decltype(w)::value>(x, weight, logits, static_cast<float*>(workspace), tokens,
                                                              hidden, experts, as_stream(stream));
    });
    return launch_status();
}

extern "C" int64_t moe_router_logits_bwd_workspace_bytes(int64_t tokens, int64_t hidden, int64_t experts) {
    if (!sizes_ok(tokens, hidden, experts)) return -1;
    return grad_parts(tokens, hidden, experts) * experts * hidden * 4;
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
            launch_grad_x<T, W>(grad_logits, weight, grad_x, tokens, hidden, experts, st);
        if (grad_weight)
            launch_grad_weight<T, W>(grad_logits, x, grad_weight, static_cast<float*>(workspace), tokens, hidden, experts,
                                     st);
    });
    return launch_status();
}
