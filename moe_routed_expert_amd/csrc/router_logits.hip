// The router's product and its gradients (gfx950).
//
//   logits = x weight^T,  grad_x = grad_logits weight,  grad_weight = grad_logits^T x
//
// With tens to hundreds of experts all three are bound by reading or writing
// rows of x once (131072 x 7168 x 64 bf16: 1.9 GB, 120 GFLOP), and the matrix
// instructions wait for memory. What costs is how rows become operands: an
// operand has its 16 rows in 16 consecutive lanes, a load straight into it
// touches 64 cache lines, and the L1 takes one of them a cycle. So
//   logits       rows are read 128 bytes by 8 lanes and turned in LDS: 333 us,
//                5.7 TB/s; straight into operands 381;
//   grad_x       the weight's columns lie in LDS as operands, each wavefront
//                takes its tokens through all of them, and results go through
//                LDS to be stored by rows: 65536 x 7168 x 64 201 us, 5.4 TB/s;
//   grad_weight  8 tokens' elements are turned into operands in registers; the
//                tokens are split over parts, which a second launch adds: 212
//                us, 5.3 TB/s (with two pieces of grad_logits 171, see below).
// A block has at most 64 experts (grad_x: as many columns of hidden as fit in 64
// KB with all of them), so that with more of them the tokens or grad_logits are
// read more often: 65536 x 2048 x 256 bf16 167 us, of which 69 are the bytes'.
#include <type_traits>

#include "bf16_pieces.h"
#include "epi_common.h"
#include "moe_prologue.h"
#include "router_map.h"

namespace moe_epi {
namespace {

constexpr int kBlock = 256;
constexpr int64_t kMostExperts = 1024;
constexpr int64_t kMostHidden = 1 << 24;  // 32 rows of it have 32-bit offsets

// ---- logits ---------------------------------------------------------------------

constexpr int kStep = 64;       // of hidden, in one pass of the loop
constexpr int kTileRows = 128;  // tokens of a block
constexpr int64_t kMostRows = 1 << 24;  // tokens of a launch
constexpr int kFewWaves = 8;
constexpr int64_t kFewHidden = 8192;

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

constexpr int kTileWaves = 8;

// Where chunk c (8 elements) of a row lies in its 8 places of LDS, so that 16
// rows' chunks c, one for each lane, are in all banks alike.
__device__ __forceinline__ int place(int row, int c) { return c ^ (row & 7); }

// 16 tokens x 16 NT experts for each of 8 wavefronts, over the steps [steps z / n,
// steps (z + 1) / n) of hidden, kDeep - 1 of which are on their way. Rows are
// read by 8 lanes each, 128 bytes together, and become operands in LDS: a load
// whose lanes lie in rows of their own takes the L1 a cycle for each lane.
template <int T, int W, int NT, int kDeep>
__global__ __launch_bounds__(64 * kTileWaves, T == MOE_EPI_F32 ? 2 : 4) void logits_tile_kernel(const char* __restrict__ x,
                                                                         const char* __restrict__ weight,
                                                                         float* __restrict__ out, int64_t tokens,
                                                                         int64_t hidden, int64_t experts) {
    typedef Pieces<T, W> P;
    typedef Piece8<T> X;
    typedef Piece8<W> Y;
    static_assert(2 * NT <= kTileWaves && kDeep % 2 == 0, "");
    __shared__ u32x4 xs[2][X::kWords][kTileRows][8], ws[2][P::kW][16 * NT][8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, g = lane / 16, chunk = lane % 8, row = threadIdx.x / 8;  // row: 0 .. 63
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTileRows, e0 = blockIdx.y * 16 * NT;
    const int64_t steps = (hidden + kStep - 1) / kStep;
    const int64_t first = steps * blockIdx.z / gridDim.z, last = steps * (blockIdx.z + 1) / gridDim.z;
    const bool staging = wave < 2 * NT;  // of the weight, 8 rows a wavefront
    const int w_row = row % (16 * NT);
    const char* px[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t t = t0 + row + 64 * j;
        px[j] = x + ((t < tokens ? t : tokens - 1) * hidden + 8 * chunk) * X::kBytes;
    }
    const int64_t e = e0 + w_row;
    const char* pw = weight + ((e < experts ? e : experts - 1) * hidden + 8 * chunk) * Y::kBytes;
    f32x4 d[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) d[n] = f32x4{0, 0, 0, 0};

    struct Ahead {
        typename X::Raw x[2];
        typename Y::Raw w;
    };
    auto load = [&](int64_t step, Ahead& a) {
        const int64_t k = step * kStep;
        a.w = Y::load(pw + k * Y::kBytes);
#pragma unroll
        for (int j = 0; j < 2; ++j) a.x[j] = X::load(px[j] + k * X::kBytes);
    };
    auto stage = [&](const Ahead& a, int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < X::kWords; ++i) xs[buf][i][row + 64 * j][place(row, chunk)] = a.x[j].w[i];
        if (!staging) return;
        u32x4 piece[P::kW];
        cut_raw<W, P::kW>(a.w, piece);
#pragma unroll
        for (int p = 0; p < P::kW; ++p) ws[buf][p][w_row][place(w_row, chunk)] = piece[p];
    };
    auto multiply = [&](int buf) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = place(of16, 4 * h + g);
            typename X::Raw raw;
            u32x4 wp[NT][P::kW], xp[P::kX];
#pragma unroll
            for (int i = 0; i < X::kWords; ++i) raw.w[i] = xs[buf][i][16 * wave + of16][at];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < P::kW; ++p) wp[n][p] = ws[buf][p][16 * n + of16][at];
            cut_raw<T, P::kX>(raw, xp);
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n] = mfma_pieces<P::kF16>(wp[n], xp, d[n]);
        }
    };
    const int64_t whole = hidden / kStep < last ? hidden / kStep : last;  // the last step may have fewer than 64
    if (first < whole) {
        Ahead a[kDeep];
        // Loads past the last step repeat it: a load that stands in a branch makes the compiler wait for the newest
        // one where an older one is used.
        auto ahead = [&](int64_t s) { return s < whole ? s : whole - 1; };
#pragma unroll
        for (int i = 0; i < kDeep - 1; ++i) load(ahead(first + i), a[i]);
        stage(a[0], 0);
        __syncthreads();
        for (int64_t s = first; s < whole; s += kDeep)
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                if (s + i >= whole) break;
                load(ahead(s + i + kDeep - 1), a[(i + kDeep - 1) % kDeep]);
                multiply(i & 1);
                stage(a[(i + 1) % kDeep], (i + 1) & 1);
                __syncthreads();
            }
    }
    if (whole < last) {
        Ahead a;
        const int64_t k = whole * kStep, left = hidden - k - 8 * chunk;
        a.w = Y::load_first(pw + k * Y::kBytes, left);
#pragma unroll
        for (int j = 0; j < 2; ++j) a.x[j] = X::load_first(px[j] + k * X::kBytes, left);
        stage(a, 0);
        __syncthreads();
        multiply(0);
    }
    const int64_t t = t0 + 16 * wave + of16;
    if (t >= tokens) return;
    float* to = out + (blockIdx.z * tokens + t) * experts;
#pragma unroll
    for (int n = 0; n < NT; ++n) put4(to, e0 + 16 * n + lane / 16 * 4, experts, d[n]);
}

// 16 tokens x 16 experts: 8 wavefronts share the steps of hidden that
// the block has, and their sums are added in their order. Rows are read as above,
// and become operands in LDS that a wavefront has for itself.
template <int T, int W>
__global__ __launch_bounds__(64 * kFewWaves) void logits_few_kernel(const char* __restrict__ x,
                                                                    const char* __restrict__ weight,
                                                                    float* __restrict__ out, int64_t tokens,
                                                                    int64_t hidden, int64_t experts) {
    typedef Pieces<T, W> P;
    typedef Piece8<T> X;
    typedef Piece8<W> Y;
    constexpr int kWords = X::kWords + Y::kWords;  // 2 KB each
    __shared__ u32x4 rows[kFewWaves][kWords][16][8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, g = lane / 16, chunk = lane % 8, row = lane / 8;  // row, and row + 8
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 16;
    auto(*mine)[16][8] = rows[wave];
    const char *pw[2], *px[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t e = blockIdx.x * 16 + row + 8 * j;
        pw[j] = weight + ((e < experts ? e : experts - 1) * hidden + 8 * chunk) * Y::kBytes;
        const int64_t t = row0 + row + 8 * j;
        px[j] = x + ((t < tokens ? t : tokens - 1) * hidden + 8 * chunk) * X::kBytes;
    }
    f32x4 d = {0, 0, 0, 0};
    const int64_t steps = (hidden + kStep - 1) / kStep, all = static_cast<int64_t>(gridDim.z) * kFewWaves;
    const int64_t me = blockIdx.z * kFewWaves + wave;
    const int64_t first = steps * me / all, last = steps * (me + 1) / all;
    const int64_t whole = hidden / kStep < last ? hidden / kStep : last;  // the last step may have fewer than 64
    struct Ahead {
        typename Y::Raw w[2];
        typename X::Raw x[2];
    };
    auto load = [&](int64_t step, Ahead& a) {
        const int64_t k = step * kStep;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            a.w[j] = Y::load(pw[j] + k * Y::kBytes);
            a.x[j] = X::load(px[j] + k * X::kBytes);
        }
    };
    auto multiply = [&](const Ahead& a) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = row + 8 * j, at = place(r, chunk);
#pragma unroll
            for (int i = 0; i < Y::kWords; ++i) mine[i][r][at] = a.w[j].w[i];
#pragma unroll
            for (int i = 0; i < X::kWords; ++i) mine[Y::kWords + i][r][at] = a.x[j].w[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = place(of16, 4 * h + g);
            typename Y::Raw w;
            typename X::Raw v;
            u32x4 wp[P::kW], xp[P::kX];
#pragma unroll
            for (int i = 0; i < Y::kWords; ++i) w.w[i] = mine[i][of16][at];
#pragma unroll
            for (int i = 0; i < X::kWords; ++i) v.w[i] = mine[Y::kWords + i][of16][at];
            cut_raw<W, P::kW>(w, wp);
            cut_raw<T, P::kX>(v, xp);
            d = mfma_pieces<P::kF16>(wp, xp, d);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    constexpr int kDeep = 4;
    if (first < whole) {
        Ahead a[kDeep];
        auto ahead = [&](int64_t s) { return s < whole ? s : whole - 1; };
#pragma unroll
        for (int i = 0; i < kDeep - 1; ++i) load(ahead(first + i), a[i]);
        for (int64_t s = first; s < whole; s += kDeep)
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                if (s + i >= whole) break;
                load(ahead(s + i + kDeep - 1), a[(i + kDeep - 1) % kDeep]);
                multiply(a[i]);
            }
    }
    if (whole < last) {
        Ahead a;
        const int64_t k = whole * kStep, left = hidden - k - 8 * chunk;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            a.w[j] = Y::load_first(pw[j] + k * Y::kBytes, left);
            a.x[j] = X::load_first(px[j] + k * X::kBytes, left);
        }
        multiply(a);
    }
    // the wavefronts' sums take the place of their rows
    f32x4* part = reinterpret_cast<f32x4*>(&rows[0][0][0][0]);
    __syncthreads();
    part[wave * 64 + lane] = d;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) d += part[i * 64 + lane];
    const int64_t t = row0 + of16;
    if (t < tokens) put4(out + (blockIdx.z * tokens + t) * experts, blockIdx.x * 16 + lane / 16 * 4, experts, d);
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

// Few tokens: as many blocks of 16 tokens x 16 experts as the chip has CUs. 1024 x 7168 x 64 11.6 us so, 12.6 by
// tiles of 128 tokens; 2048 19.7 and 14.9; 1024 x 2048 x 256, four blocks a CU, 11.7 and 10.9.
bool few(int64_t tokens, int64_t experts) { return up(experts, 16) * up(tokens, 16) <= 256; }

// Parts that hidden is shared by. A launch that adds them up is not worth it up to 8192 of hidden for few tokens (32
// x 7168 x 64 7.5 us, in two parts 9.0); tiles have two blocks per CU and about 8 steps each, 4 at
// least.
int64_t logits_parts(int64_t tokens, int64_t hidden, int64_t experts) {
    if (tokens == 0) return 1;
    if (few(tokens, experts)) return up(hidden, kFewHidden) < 16 ? up(hidden, kFewHidden) : 16;
    const int64_t blocks = up(tokens, kTileRows) * up(experts, 64), wanted = 512 / blocks, most = up(hidden, 8 * kStep);
    const int64_t n = wanted < most ? wanted : most;
    return n < 1 ? 1 : (n > 16 ? 16 : n);
}

// ---- gradients ----------------------------------------------------------------------

// Pieces of the factors: all bits of both, also where the result has 16. The
// terms of a sum may cancel (gradients of a softmax's logits add up to 0 over a
// token's experts), and then what two pieces of a float32 leave out is more than
// the result's rounding. The third piece of grad_logits takes 416 us instead of
// 381 (both gradients, 65536 x 7168 x 64 bf16), that of a float32 weight also
// 87 instead of 57 (grad_x, 16384 x 7168 x 64).
template <int T>
struct GradPieces {
    static constexpr int kGrad = 3;
    static constexpr int kOther = T == MOE_EPI_BF16 ? 1 : (T == MOE_EPI_F16 ? 2 : 3);
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
    typedef GradPieces<W> P;
    typedef Piece8<MOE_EPI_F32> G;
    constexpr int V = 16 / Elem<W>::kBytes;  // weights of a 16-byte load
    constexpr int kTileBytes = 16 * Elem<T>::kBytes;  // of 16 hidden elements of a token
    __shared__ u32x4 lds[HT * KS * P::kOther][64], results[kBlock / 64][MT][16][8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t h0 = static_cast<int64_t>(blockIdx.x) * 16 * HT;
    // Operand row m of tile j is the hidden element that makes a lane's results
    // neighbours in memory: with 16-bit results two tiles give 8 of them.
    constexpr bool kPairs = T != MOE_EPI_F32;
    auto tile_of = [&](int h, int& tile, int& m) {  // of hidden element h0 + h
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
            tile_of(hv + j, tile, m);
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
        // kAtOnce tiles of results, 128 bytes of each token or what the block has of them, go through LDS, from which
        // 8 lanes store a token's: stores whose lanes lie in rows of their own take a cycle for each lane.
        constexpr int kAtOnce = HT < 128 / kTileBytes ? HT : 128 / kTileBytes, kChunks = kAtOnce * kTileBytes / 16;
        constexpr int kEach = 16 / Elem<T>::kBytes;  // elements of a chunk
#pragma unroll 1
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
                    for (int m = 0; m < MT; ++m) d[a][m] = mfma_pieces<false>(w, g[m][k], d[a][m]);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                u32x4(*turn)[8] = results[wave][m];
                if constexpr (kPairs) {
#pragma unroll
                    for (int a = 0; a < kAtOnce; a += 2) {
                        const float f[8] = {d[a][m][0], d[a][m][1], d[a][m][2], d[a][m][3],
                                            d[a + 1][m][0], d[a + 1][m][1], d[a + 1][m][2], d[a + 1][m][3]};
                        turn[of16][place(of16, 2 * a + lane / 16)] = Elem<T>::pack(f);
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < kAtOnce; ++a)
                        turn[of16][place(of16, 4 * a + lane / 16)] = __builtin_bit_cast(u32x4, d[a][m]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 16 * kChunks / 64; ++i) {
                    typedef u32x4 loose __attribute__((aligned(2)));
                    const int at = lane + 64 * i, row = at / kChunks, c = at % kChunks;
                    const u32x4 v = results[wave][m][row][place(row, c)];
                    const int64_t t = t0 + 16 * m + row, h = h0 + 16 * j + kEach * c;
                    if (t >= end || h >= hidden) continue;
                    char* to = grad_x + (t * hidden + h) * Elem<T>::kBytes;
                    if (h + kEach <= hidden) {
                        __builtin_nontemporal_store(v, reinterpret_cast<loose*>(to));
                    } else {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            if (h + e >= hidden) continue;
                            if constexpr (T == MOE_EPI_F32)
                                reinterpret_cast<uint32_t*>(to)[e] = v[e];
                            else
                                reinterpret_cast<uint16_t*>(to)[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e % 2)));
                        }
                    }
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// As above for more than 256 experts, 16 hidden a block: all experts' operands lie in LDS, and a wavefront reads and
// cuts the gradients of 32 experts at a time.
template <int T, int W>
__global__ __launch_bounds__(kBlock) void grad_x_many_kernel(const float* __restrict__ grad,
                                                             const char* __restrict__ weight,
                                                             char* __restrict__ grad_x, int64_t tokens, int64_t hidden,
                                                             int64_t experts, int64_t tokens_a_block) {
    typedef GradPieces<W> P;
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
            d = mfma_pieces<false>(w, g, d);
        }
        if (t >= end) continue;
        const int64_t h = h0 + lane / 16 * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (h + i < hidden) Elem<T>::store1(grad_x, t * hidden + h + i, d[i]);
    }
}

// 8 bytes of a row, of which `left` elements exist.
template <int T>
__device__ __forceinline__ u32x2 load8(const char* p, int64_t left) {
    u32x2 r = {0, 0};
#pragma unroll
    for (int i = 0; i < 8 / Elem<T>::kBytes; ++i) {
        if (i >= left) continue;
        if constexpr (T == MOE_EPI_F32)
            r[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else
            r[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    }
    return r;
}

// As turn_rows for rows of 8 bytes.
template <int T, int P>
__device__ __forceinline__ void turn_short_rows(const u32x2 (&r)[8], u32x4 (&piece)[8 / Elem<T>::kBytes][P]) {
    if constexpr (T == MOE_EPI_F32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i][j]);
            cut<P>(f, piece[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 t;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[i] = __builtin_amdgcn_perm(r[2 * i + 1][j / 2], r[2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
            cut_raw<T, P>(typename Piece8<T>::Raw{{t}}, piece[j]);
        }
    }
}

constexpr int kGradWaves = 8;

// 16 ET experts x 16 HT hidden for each of 8 wavefronts, over the tokens of part
// z: the tokens are the inner dimension. A wavefront reads 8 tokens' elements of
// its hidden, 8 bytes a lane and token, and turns them into operands in
// registers; the operands of grad are made once a block. kOnce: no other block
// reads the same elements, which then need not stay in the caches (65536 x 7168
// x 64 251 -> 211 us; 16384 x 2048 x 256, read by four blocks, 54 -> 59).
template <int T, int W, int ET, bool kOnce>
__global__ __launch_bounds__(64 * kGradWaves) void grad_weight_kernel(const float* __restrict__ grad, const char* __restrict__ x,
                                                             float* __restrict__ parts, int64_t tokens, int64_t hidden,
                                                             int64_t experts) {
    typedef GradPieces<T> P;
    constexpr int HT = 8 / Elem<T>::kBytes;  // hidden of a lane
    __shared__ u32x4 lds[2][ET][P::kGrad][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of16 = lane % 16, k8 = lane / 16 * 8;
    const int64_t h = static_cast<int64_t>(blockIdx.x) * 16 * kGradWaves * HT + wave * 16 * HT + of16 * HT;
    // the operands of grad: tile wave % ET, 4 of a lane's 8 tokens in each of two wavefronts
    const int tile = wave % ET, half = wave / ET % 2;
    const bool staging = wave < 2 * ET;
    const int64_t e0 = blockIdx.y * 16 * ET, mine = e0 + 16 * tile + of16;
    const int64_t steps = (tokens + kGradStep - 1) / kGradStep;
    const int64_t first = steps * blockIdx.z / gridDim.z, last = steps * (blockIdx.z + 1) / gridDim.z;
    const int64_t left = hidden - h;
    f32x4 d[ET][HT];
#pragma unroll
    for (int e = 0; e < ET; ++e)
#pragma unroll
        for (int j = 0; j < HT; ++j) d[e][j] = f32x4{0, 0, 0, 0};
    struct Ahead {
        u32x2 x[8];
        float g[4];
    };
    // Columns past the last hidden element or expert are loaded from what comes after, or from the first ones, and
    // not stored; the last steps, whose tokens have too little after them, load by bounds (router_map.h).
    // A load's address is that of a token, which the wavefront shares, and the lane's 32-bit place from there.
    const uint32_t at = static_cast<uint32_t>((k8 * hidden + (left > 0 ? h : 0)) * Elem<T>::kBytes);
    const uint32_t at_g = static_cast<uint32_t>(((k8 + 4 * half) * experts + (mine < experts ? mine : experts - 1)) * 4);
    auto token_x = [&](int64_t t) { return x + t * hidden * Elem<T>::kBytes; };
    auto token_g = [&](int64_t t) { return reinterpret_cast<const char*>(grad + t * experts); };
    auto load = [&](int64_t s, Ahead& a) {
        typedef u32x2 loose __attribute__((aligned(2)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const loose* p = reinterpret_cast<const loose*>(token_x(s * kGradStep + i) + at);
            if constexpr (kOnce)
                a.x[i] = __builtin_nontemporal_load(p);
            else
                a.x[i] = *p;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) a.g[i] = *reinterpret_cast<const float*>(token_g(s * kGradStep + i) + at_g);
    };
    auto stage = [&](Ahead& a, int buf) {
        if (!staging) return;
        u32x2 piece[P::kGrad];
        cut4<P::kGrad>(a.g, piece);
#pragma unroll
        for (int p = 0; p < P::kGrad; ++p) reinterpret_cast<u32x2*>(&lds[buf][tile][p][lane])[half] = piece[p];
    };
    auto multiply = [&](Ahead& now, int buf) {
        u32x4 v[HT][P::kOther], g[ET][P::kGrad];
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int p = 0; p < P::kGrad; ++p) g[e][p] = lds[buf][e][p][lane];
        __builtin_amdgcn_sched_barrier(0);
        turn_short_rows<T, P::kOther>(now.x, v);
#pragma unroll
        for (int e = 0; e < ET; ++e)
#pragma unroll
            for (int j = 0; j < HT; ++j) d[e][j] = mfma_pieces<false>(g[e], v[j], d[e][j]);
    };
    const int64_t inside = steps_inside(tokens, hidden, HT), whole = inside < last ? inside : last;
    constexpr int kDeep = 4;
    if (first < whole) {
        Ahead a[kDeep];
        // Loads past the last step repeat it: a load that stands in a branch makes the compiler wait for the newest
        // one where an older one is used.
        auto ahead = [&](int64_t s) { return s < whole ? s : whole - 1; };
#pragma unroll
        for (int i = 0; i < kDeep - 1; ++i) load(ahead(first + i), a[i]);
        stage(a[0], 0);
        __syncthreads();
        for (int64_t s = first; s < whole; s += kDeep)
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                if (s + i >= whole) break;
                load(ahead(s + i + kDeep - 1), a[(i + kDeep - 1) % kDeep]);
                multiply(a[i], i & 1);
                stage(a[(i + 1) % kDeep], (i + 1) & 1);
                __syncthreads();
            }
    }
#pragma unroll 1
    for (int64_t s = whole < first ? first : whole; s < last; ++s) {
        Ahead a;
        const int64_t t = s * kGradStep + k8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a.x[i] = t + i < tokens && left > 0 ? load8<T>(token_x(s * kGradStep + i) + at, left) : u32x2{0, 0};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a.g[i] = t + 4 * half + i < tokens ? *reinterpret_cast<const float*>(token_g(s * kGradStep + i) + at_g) : 0.0f;
        stage(a, s & 1);
        __syncthreads();
        multiply(a, s & 1);
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
    const int64_t blocks = up(hidden, 512) * up(experts, 64), wanted = 256 / blocks, most = up(tokens, 4 * kGradStep);
    const int64_t n = wanted < most ? wanted : most;
    return n < 1 ? 1 : n;
}

bool sizes_ok(int64_t tokens, int64_t hidden, int64_t experts) {
    int64_t a;
    return tokens >= 0 && tokens <= INT32_MAX && experts >= 1 && experts <= kMostExperts && hidden <= kMostHidden &&
           bytes_ok(tokens, hidden, 4, &a) && bytes_ok(experts, hidden, 4, &a) && bytes_ok(tokens, experts, 4, &a);
}

template <int T, int W>
void launch_logits(const void* x, const void* weight, float* logits, float* workspace, int64_t tokens, int64_t hidden,
                   int64_t experts, hipStream_t st) {
    const int64_t n = logits_parts(tokens, hidden, experts);
    float* to = n > 1 ? workspace : logits;
    const char *px = static_cast<const char*>(x), *pw = static_cast<const char*>(weight);
    if (few(tokens, experts)) {
        const dim3 grid(static_cast<unsigned>(up(experts, 16)), static_cast<unsigned>(up(tokens, 16)), static_cast<unsigned>(n)),
            block(64 * kFewWaves);
        hipLaunchKernelGGL((logits_few_kernel<T, W>), grid, block, 0, st, px, pw, to, tokens, hidden, experts);
    } else {
        constexpr int kDeep = 4;
        auto go = [&](auto kernel, int nt) {
            // a grid has fewer than 2^32 work-items; calls of so many tokens have one part
            for (int64_t t = 0; t < tokens; t += kMostRows) {
                const int64_t here = tokens - t < kMostRows ? tokens - t : kMostRows;
                const dim3 grid(static_cast<unsigned>(up(here, kTileRows)), static_cast<unsigned>(up(experts, 16 * nt)),
                                static_cast<unsigned>(n));
                hipLaunchKernelGGL(kernel, grid, dim3(64 * kTileWaves), 0, st, px + t * hidden * Elem<T>::kBytes, pw,
                                   to + t * experts, here, hidden, experts);
            }
        };
        if (experts <= 16)
            go(logits_tile_kernel<T, W, 1, kDeep>, 1);
        else if (experts <= 32)
            go(logits_tile_kernel<T, W, 2, kDeep>, 2);
        else
            go(logits_tile_kernel<T, W, 4, kDeep>, 4);
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
        const int64_t columns = up(hidden, width), wanted = columns < 512 ? 512 / columns : 1;  // two blocks per CU
        int64_t each = up(up(tokens, wanted), 4 * wave_tokens) * 4 * wave_tokens;
        if (up(tokens, each) > 65535) each = up(up(tokens, 65535), 4 * wave_tokens) * 4 * wave_tokens;
        const dim3 grid(static_cast<unsigned>(columns), static_cast<unsigned>(up(tokens, each)));
        hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, st, grad, static_cast<const char*>(weight),
                           static_cast<char*>(grad_x), tokens, hidden, experts, each);
    };
    // hidden of a block: as many as 64 KB of LDS hold, up to 512
    constexpr int kW = GradPieces<W>::kOther;
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
        const dim3 grid(static_cast<unsigned>(up(hidden, 16 * kGradWaves * 8 / Elem<T>::kBytes)),
                        static_cast<unsigned>(up(experts, 16 * et)), static_cast<unsigned>(n));
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kGradWaves), 0, st, grad, static_cast<const char*>(x), workspace, tokens,
                           hidden, experts);
    };
    if (experts <= 16)
        go(grad_weight_kernel<T, W, 1, true>, 1);
    else if (experts <= 32)
        go(grad_weight_kernel<T, W, 2, true>, 2);
    else if (experts <= 64)
        go(grad_weight_kernel<T, W, 4, true>, 4);
    else
        go(grad_weight_kernel<T, W, 4, false>, 4);
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
