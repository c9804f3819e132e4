// Grouped products of the routed experts in 8-bit integers (gfx950): int8 rows
// with one scale each times int8 weights with one scale per output channel,
// summed exactly in int32 by v_mfma_i32_16x16x64_i8.
//
//   gate_up: y[r, j] = bf16(silu(min(g, L)) * clamp(u, -L, L) * p[r]),
//            g = sum_h a[t, h] wg[e, j, h] * sa[t] * sg[e, j], u likewise,
//            t = slot_of[r] / top_k: the tokens are read in place, a row of
//            each for every expert that takes it, with no gathered copy;
//   down:    out[r, n] = round(sum_i h[r, i] wd[e, n, i] * sh[r] * p[r] * sd[e, n]).
//
// The integer sums carry no rounding, so their order is free: tiles, steps
// and wavefronts may be arranged at will without changing a bit.
//
// Three kernels, by rows / experts, the mean number of rows of an expert where the
// buffers hold no more than the rows there are (launch_int8):
//   few rows    the weights are read once and set the time (below);
//   tiles       a block covers BM rows of one expert and BN columns of each of
//               two weight tiles (gate and up of the same columns; two
//               neighbouring column ranges of the down weights). Steps of 128
//               along K: a row of a tile is then 128 bytes, eight 16-byte
//               chunks, XOR-swizzled so that a fragment read (one chunk of each
//               of 16 rows) takes 16 different bank groups. Memory goes
//               straight to LDS in two or three stages; the next stages' loads
//               are in flight while this one's products run. Blocks of 64 x 64
//               and 128 x 64 tiles fill each other's waits where a CU has
//               several; where it has about one, the third stage does (gate_up
//               as below, 48 rows an expert 58.9 -> 44.2 us, 64 rows 62.5 ->
//               47.1), which with several would keep some of them out;
//   large tiles 256 x 128 x 2, eight wavefronts of 64 x 64 x 2, 128
//               accumulators a lane, one block per CU, with the loop written
//               out so that fragment reads and loads go between the matrix
//               instructions in a fixed order. The matrix units are busy 61%
//               of the cycles, at the 1.9 GHz that the power limit leaves under
//               this load (2.4 without), the LDS 24%; the rest waits at the
//               barrier for a step's loads, which have less than one step to
//               arrive, and for a tile's first loads.
//               65536 rows over 8 experts: gate_up (7168 -> 2 x 2048) 1570 us,
//               2452 TOP/s, down (2048 -> 7168, bf16 out) 927 us, 2076 TOP/s,
//               float32 out 1029 us: its shorter K gives the output a larger
//               share; a library product of 16384^3 in int8 runs at 2341 TOP/s
//               on this part. On the way there, gate_up / down: the plain loop
//               1695 / 1010; the loop written out 1609 / 960; the first two
//               steps' loads issued together, the scales asked for at the start
//               and the output staged in one piece 1590 / 940; nontemporal
//               stores of the output 1570 / 927. Eight loading wavefronts
//               against four: gate_up 1609 / 1641, down 947 / 940; row tiles
//               per group: gate_up 1: 1691, 2: 1641, 4: 1648, 8: 1689; down 8:
//               977, 16: 972, 32: 983, 128: 1002; steps of 64 with two blocks
//               per CU (128 x 128 x 2 or 256 x 64 x 2): gate_up 1935, down 1099;
//               128 x 128 x 2 in steps of 128 with three stages 1933 / 1141 (and
//               at 128 rows an expert, gate_up 69 against 76 for the tiles above,
//               down 46 against 35);
//               blocks that stay for several tiles and load the next one's first
//               step under the stores: gate_up 1570 against 1591, down 989
//               against 932 (registers spill, and the loads wait for the stores);
//               output stored from registers, without LDS: 1580 against 1591,
//               957 against 932.
#include <type_traits>

#include "epi_common.h"
#include "grouped_map.h"
#include "moe_routed.h"
#include "swiglu_math.h"

namespace moe_epi {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;            // bytes (elements) of K per step
constexpr int kChunks = kStep / 16;   // 16-byte chunks of a tile row
constexpr int64_t kMaxK = 131072;     // below it |sum| < 2^31 even for -128 * -128

// Rows of a that the rows of an expert read: row r itself, or the token of its slot.
struct Rows {
    const float* scale;
    const int32_t* slot_of;  // NULL: rows are their own
    uint32_t top_k;
    int64_t slots;
    // The row of a for row r; -1 for a slot out of range (read row 0, count it as zeros).
    __device__ __forceinline__ int64_t of(int64_t r) const {
        if (!slot_of) return r;
        const int32_t s = slot_of[r];
        return s >= 0 && s < slots ? static_cast<int64_t>(static_cast<uint32_t>(s) / top_k) : -1;
    }
};

enum class Out { kSwiglu, kBf16, kF32 };

// BM rows and BN columns of each weight by WM x WN wavefronts; GM row tiles to
// a group of the tile order; kLoadWaves wavefronts load; S stages of LDS; kRoll:
// the main loop that keeps one block per CU busy (below), otherwise the plain one.
template <int BM_, int BN_, int WM_, int WN_, int GM_, int LW_, int S_, bool kRoll_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, GM = GM_, kLoadWaves = LW_, S = S_;
    static constexpr bool kRoll = kRoll_;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MI = BM / (16 * WM), NI = BN / (16 * WN);
    static constexpr int kABytes = BM * kStep, kWBytes = BN * kStep, kStage = kABytes + 2 * kWBytes;
    static constexpr int kLoadThreads = 64 * kLoadWaves;
    static constexpr int kALoads = BM * kChunks / kLoadThreads, kWLoads = BN * kChunks / kLoadThreads;
    static constexpr int kLoads = kALoads + 2 * kWLoads;  // of a step, per loading wavefront
    static constexpr int kMfmas = 2 * MI * NI;            // of a sub-step of 64
    static constexpr int kEvery = kMfmas / kLoads;        // matrix instructions per load
    static constexpr int kLds = S * kStage;
    static_assert(BM * BN * 4 <= kLds, "a staged output tile fits: both halves in bf16, one in float32");
    static_assert(S == 2 || (!kRoll && S == 3 && kLoadWaves == WM * WN), "stages of the two loops");
    static_assert(BM + 2 * BN <= kThreads, "a thread per row and per column of the scales");
    static_assert(kALoads >= 1 && kWLoads >= 1 && BM * kChunks % kLoadThreads == 0 && BN * kChunks % kLoadThreads == 0,
                  "whole chunks per lane");
    static_assert(kEvery >= 1, "a load per matrix instruction at most");
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && BM <= kThreads, "whole MFMA tiles");
    static_assert(WM * WN >= kLoadWaves && BM * BN % (8 * kThreads) == 0, "loading wavefronts; whole output chunks");
};

__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) only (gfx9 encoding)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// This wavefront's loads but the last kLeft and its LDS accesses are done, then the block meets.
template <int kLeft>
__device__ __forceinline__ void stage_barrier() {
    static_assert(kLeft < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt((kLeft & 0xF) | 0x0070 | (kLeft >> 4) << 14);  // vmcnt(kLeft) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Inclusive scan of one value per lane over the wavefront, by lane shifts:
// within rows of 16 lanes by 1, 2, 4 and 8, then lane 15 of a row into the
// next row and lane 31 into the upper half. Lanes that receive nothing get `none`.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp(int none, int v) {
    return __builtin_amdgcn_update_dpp(none, v, kCtrl, kRows, 0xF, false);
}
template <class F>
__device__ __forceinline__ int scan(int v, int none, F&& op) {
    v = op(v, dpp<0x111, 0xF>(none, v));  // row_shr 1, 2, 4, 8
    v = op(v, dpp<0x112, 0xF>(none, v));
    v = op(v, dpp<0x114, 0xF>(none, v));
    v = op(v, dpp<0x118, 0xF>(none, v));
    v = op(v, dpp<0x142, 0xA>(none, v));  // row_bcast 15, 31
    return op(v, dpp<0x143, 0xC>(none, v));
}

// The mt-th row tile of bm rows over all experts in order (rows == 0: there is
// none). The whole wavefront takes 64 experts at a time: with the running
// maximum of offs as the clamped end of each expert and the running sum of
// their tiles, the expert is the first whose sum passes mt. One expert after
// the other, as many dependent reads as experts, would take longer than a
// short product.
struct RowTile {
    int row0, rows, expert;
};
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ offs, int rows, int experts, int mt, int bm) {
    const int lane = static_cast<int>(threadIdx.x & 63u);
    int carry = 0, before = 0;  // end of the last expert, and tiles, of earlier groups of 64
    for (int e0 = 0; e0 < experts; e0 += 64) {
        int end = e0 + lane < experts ? offs[e0 + lane] : 0;
        end = end > rows ? rows : (end < carry ? carry : end);
        end = scan(end, 0, [](int x, int y) { return x > y ? x : y; });
        const int start = dpp<0x138, 0xF>(carry, end);  // wave_shr 1: the expert before
        const int n = end - start, tiles = n > 0 ? (n - 1) / bm + 1 : 0;
        const int sum = scan(tiles, 0, [](int x, int y) { return x + y; });
        const uint64_t past = __ballot(before + sum > mt);
        if (past) {
            const int hit = __builtin_ctzll(past);
            const int row0 = __builtin_amdgcn_readlane(start + (mt - before - (sum - tiles)) * bm, hit);
            const int left = __builtin_amdgcn_readlane(end, hit) - row0;
            return RowTile{row0, left < bm ? left : bm, e0 + hit};
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        carry = __builtin_amdgcn_readlane(end, 63);
    }
    return RowTile{0, 0, 0};
}

template <class C, Out kOut, bool kWide>
__device__ __forceinline__ void grouped_int8_tile(
    uint8_t* lds, const int8_t* __restrict__ a, const Rows& rows_of, const int8_t* __restrict__ w1,
    const float* __restrict__ s1, const int8_t* __restrict__ w2, const float* __restrict__ s2,
    const int32_t* __restrict__ offs, const float* __restrict__ probs, void* __restrict__ out, int rows, int k_dim,
    int64_t n_dim, int experts, float limit, int64_t n_tiles, int64_t n_blocks) {
    constexpr bool kPair = kOut == Out::kSwiglu;  // two weights of the same columns
    constexpr int MI = C::MI, NI = C::NI;
    float* const row_scale = reinterpret_cast<float*>(lds + C::kLds);
    float* const row_prob = row_scale + C::BM;
    float* const col_scale = row_prob + C::BM;  // of the two weight tiles

    int64_t mt, nt;
    tile_of(blockIdx.x, n_blocks / n_tiles, n_tiles, C::GM, &mt, &nt);
    const RowTile tr = find_tile(offs, rows, experts, static_cast<int>(mt), C::BM);
    if (tr.rows == 0) return;
    const int64_t col1 = nt * (kPair ? C::BN : 2 * C::BN), col2 = kPair ? col1 : col1 + C::BN;
    const int n1 = static_cast<int>(n_dim - col1 < C::BN ? n_dim - col1 : C::BN);
    const int n2 = static_cast<int>(n_dim - col2 <= 0 ? 0 : (n_dim - col2 < C::BN ? n_dim - col2 : C::BN));

    const int tid = static_cast<int>(threadIdx.x), lane = tid % 64;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const bool loads = wave < C::kLoadWaves;

    // The scales of a row and its probability, or of a column, one thread each:
    // asked for now, kept in LDS once the products are done.
    const int64_t wrow = static_cast<int64_t>(tr.expert) * n_dim;
    float scale = 0.0f, prob = 1.0f;
    if (tid < C::BM) {
        const int r = tr.row0 + (tid < tr.rows ? tid : tr.rows - 1);
        const int64_t u = rows_of.of(r);
        if (u >= 0) scale = rows_of.scale[u];
        if (probs) prob = probs[r];
    } else if (tid < C::BM + 2 * C::BN) {
        const int c = tid - C::BM, second = c >= C::BN;
        if (c - second * C::BN < (second ? n2 : n1))
            scale = (second ? s2 : s1)[wrow + (second ? col2 - C::BN : col1) + c];
    }

    // This lane's 16-byte chunks of a stage: slot row * 8 + (chunk ^ swizzle(row))
    // holds chunk `chunk` of tile row `row`. The rows of a lane's loads are a
    // multiple of 16 apart, so all of them take the same chunk of their row. Rows
    // past the tile repeat its last one. Loads go by a base in scalar registers,
    // the lane's 32-bit offset from it, and the step's offset in a scalar; only
    // the rows of a tensor of 2 GiB and more, read in place, need 64-bit addresses.
    constexpr int kFlags = 0x00020000;  // raw buffer, 32-bit data format
    const int lrow = (wave % C::kLoadWaves * 64 + lane) / kChunks;
    const int kq = ((lane % kChunks) ^ swizzle(lrow)) * 16;
    const int8_t* const abase = rows_of.slot_of ? a : a + static_cast<int64_t>(tr.row0) * k_dim;
    const int8_t* const t1 = w1 + (wrow + col1) * k_dim;
    const int8_t* const t2 = w2 + (wrow + (n2 > 0 ? col2 : col1)) * k_dim;
    auto buffer = [](const int8_t* p) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p), 0, 0x7FFFFFFF, kFlags);
    };
    const __amdgpu_buffer_rsrc_t ra = buffer(abase), r1 = buffer(t1), r2 = buffer(t2);
    int va[C::kALoads], v1[C::kWLoads], v2[C::kWLoads];
    const int8_t* pa[kWide ? C::kALoads : 1];
    if (loads) {
#pragma unroll
        for (int i = 0; i < C::kALoads; ++i) {
            const int row = i * (C::kLoadThreads / kChunks) + lrow, r = row < tr.rows ? row : tr.rows - 1;
            int64_t u = r;
            if (rows_of.slot_of) {
                u = rows_of.of(tr.row0 + r);
                u = u >= 0 ? u : 0;
            }
            if constexpr (kWide)
                pa[i] = abase + u * k_dim + kq;
            else
                va[i] = static_cast<int>(u * k_dim) + kq;
        }
        const int m2 = n2 > 0 ? n2 : n1;
#pragma unroll
        for (int i = 0; i < C::kWLoads; ++i) {
            const int row = i * (C::kLoadThreads / kChunks) + lrow;
            v1[i] = (row < n1 ? row : n1 - 1) * k_dim + kq;
            v2[i] = (row < m2 ? row : m2 - 1) * k_dim + kq;
        }
    }
    // Load number i of step kt: the rows' chunks first, then the weights' in
    // pairs. A step that crosses the end of K takes the start of the row for
    // the chunks past it.
    const int nk = (k_dim + kStep - 1) / kStep;
    const int last = k_dim % kStep ? nk - 1 : -1;  // the step that crosses, if one does
    auto issue_one = [&](int kt, int i) {
        uint8_t* st = lds + static_cast<unsigned>(kt) % C::S * C::kStage;
        int k = kt * kStep, more = 0;
        if (kt == last) {
            more = k + kq < k_dim ? k : -kq;
            k = 0;
        }
        auto bl = [&](__amdgpu_buffer_rsrc_t r, int v, uint8_t* dst) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, v + more, k,
                                                     0, 0);
        };
        if (i < C::kALoads) {
            uint8_t* dst = st + (i * C::kLoadThreads + wave * 64) * 16;
            if constexpr (kWide)
                __builtin_amdgcn_global_load_lds(pa[i] + k + more, (__attribute__((address_space(3))) void*)dst, 16, 0,
                                                 0);
            else
                bl(ra, va[i], dst);
        } else {
            const int j = (i - C::kALoads) / 2;
            uint8_t* dst = st + C::kABytes + (j * C::kLoadThreads + wave * 64) * 16;
            if ((i - C::kALoads) % 2 == 0)
                bl(r1, v1[j], dst);
            else
                bl(r2, v2[j], dst + C::kWBytes);
        }
    };
    auto issue = [&](int kt) {
        if (loads)
#pragma unroll
            for (int i = 0; i < C::kLoads; ++i) issue_one(kt, i);
    };
    // Step kt has landed (`left` later loads may be on their way) and nobody reads
    // the stage of the step before any more. In the step that crosses the end of K
    // the rows' chunks past it are cleared, so that whatever the weights hold there
    // counts 0.
    auto meet = [&](int kt, auto left) {
        stage_barrier<decltype(left)::value>();
        if (kt == last) {
            uint8_t* const st = lds + static_cast<unsigned>(kt) % C::S * C::kStage;
            if (loads && kt * kStep + kq >= k_dim)
#pragma unroll
                for (int i = 0; i < C::kALoads; ++i)
                    *reinterpret_cast<i32x4*>(st + (i * C::kLoadThreads + tid) * 16) = i32x4{0, 0, 0, 0};
            lds_barrier();
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    i32x4 acc1[MI][NI], acc2[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc1[mi][ni] = acc2[mi][ni] = i32x4{0, 0, 0, 0};

    // Fragments of one sub-step of 64: 16 rows, a 16-byte chunk of each per group
    // of 16 lanes. Which group takes which chunk is free as long as rows and
    // weights agree; lanes l and l + 32 on neighbouring chunks keep the LDS less
    // busy than lanes l and l + 16. Each fragment is read again for the next
    // sub-step right after the last matrix instruction that uses it.
    i32x4 fa[MI], f1[NI], f2[NI];
    const int chunk0 = ((lane / 16) & 1) * 2 + lane / 32;
    auto fragment = [&](const uint8_t* tile, int row, int kk) {
        return *reinterpret_cast<const i32x4*>(tile + (row * kChunks + ((4 * kk + chunk0) ^ swizzle(row))) * 16);
    };
    auto read_a = [&](const uint8_t* st, int kk, int mi) {
        fa[mi] = fragment(st, wm * (C::BM / C::WM) + mi * 16 + lane % 16, kk);
    };
    auto read_w = [&](const uint8_t* st, int kk, int ni) {
        const int row = wn * (C::BN / C::WN) + ni * 16 + lane % 16;
        f1[ni] = fragment(st + C::kABytes, row, kk);
        f2[ni] = fragment(st + C::kABytes + C::kWBytes, row, kk);
    };
    auto mfma = [&](int i) {
        const int ni = i / (2 * MI), mi = i / 2 % MI;
        if (i % 2 == 0)
            acc1[mi][ni] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f1[ni], fa[mi], acc1[mi][ni], 0, 0, 0);
        else
            acc2[mi][ni] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f2[ni], fa[mi], acc2[mi][ni], 0, 0, 0);
    };
    auto reads_after = [&](int i, const uint8_t* st, int kk) {
        if (i >= 2 * MI * (NI - 1) && i % 2 == 1) read_a(st, kk, i / 2 % MI);
        if (i % (2 * MI) == 2 * MI - 1) read_w(st, kk, i / (2 * MI));
    };
    auto substep = [&](const uint8_t* next, int kk) {  // with the reads of `next`, sub-step kk, in this order
#pragma unroll
        for (int i = 0; i < C::kMfmas; ++i) {
            mfma(i);
            reads_after(i, next, kk);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    const std::integral_constant<int, 0> none;
    if constexpr (C::kRoll) {
        // From the middle of one step to the middle of the next: after the barrier the
        // next step is complete and this one's stage is free, so the step after next
        // is loaded into it, a load after every kEvery-th matrix instruction.
        issue(0);
        if (nk > 1) {
            issue(1);
            stage_barrier<C::kLoads>();  // not the step that crosses the end of K
        } else {
            meet(0, none);
        }
#pragma unroll
        for (int i = 0; i < C::kMfmas; ++i) reads_after(i, lds, 0);
        substep(lds, 1);
        meet(1, none);
        for (int kt = 0; kt + 1 < nk; ++kt) {
            const uint8_t* next = lds + ((kt + 1) & 1) * C::kStage;
#pragma unroll
            for (int i = 0; i < C::kMfmas; ++i) {
                mfma(i);
                if (i % C::kEvery == 0 && i / C::kEvery < C::kLoads && loads && kt + 2 < nk)
                    issue_one(kt + 2, i / C::kEvery);
                reads_after(i, next, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            substep(next, 1);
            meet(kt + 2, none);
        }
#pragma unroll
        for (int i = 0; i < C::kMfmas; ++i) mfma(i);
        __builtin_amdgcn_sched_barrier(0);
    } else {
        // S - 1 steps are on their way; few rows give too few blocks to fill each
        // other's waits.
#pragma unroll
        for (int i = 0; i < C::S - 1; ++i)
            if (i < nk) issue(i);
        for (int kt = 0; kt < nk; ++kt) {
            if (C::S > 2 && kt + 1 < nk)
                meet(kt, std::integral_constant<int, (C::S - 2) * C::kLoads>());
            else
                meet(kt, none);
            if (kt + C::S - 1 < nk) issue(kt + C::S - 1);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const uint8_t* const st = lds + static_cast<unsigned>(kt) % C::S * C::kStage;
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) read_a(st, kk, mi);
#pragma unroll
                for (int ni = 0; ni < NI; ++ni) read_w(st, kk, ni);
#pragma unroll
                for (int i = 0; i < C::kMfmas; ++i) mfma(i);
            }
        }
    }
    if (tid < C::BM) {
        row_scale[tid] = scale;
        row_prob[tid] = prob;
    } else if (tid < C::BM + 2 * C::BN) {
        col_scale[tid - C::BM] = scale;
    }
    lds_barrier();  // all fragment reads done before the stages become the output tile

    // Lane l holds, in register j of tile (mi, ni), row mi * 16 + l % 16 and
    // column ni * 16 + 4 * (l / 16) + j of the wavefront's part.
    auto col_of = [&](int ni) { return wn * (C::BN / C::WN) + ni * 16 + 4 * (lane / 16); };
    auto row_of = [&](int mi) { return wm * (C::BM / C::WM) + mi * 16 + lane % 16; };
    if constexpr (kOut != Out::kF32) {
        // The whole output tile in bf16, the two column ranges of down side by side,
        // so that a row is stored in one run. 16-byte chunks of a row are swizzled by
        // the row: 16 rows of one chunk take 16 different bank groups.
        constexpr int kCols = kPair ? C::BN : 2 * C::BN, kRowChunks = kCols / 8;
        constexpr int kWrap = kRowChunks < 16 ? kRowChunks : 16, kEach = 16 / kWrap;
        uint8_t* const stage = lds;
        auto at = [](int row, int c) {
            return (row * kRowChunks + ((c / 8) ^ (row / kEach % kWrap))) * 16 + c % 8 * 2;
        };
#pragma unroll
        for (int half = 0; half < (kPair ? 1 : 2); ++half)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) {
                const int c = half * C::BN + col_of(ni);
                const f32x4 sc1 = *reinterpret_cast<const f32x4*>(col_scale + c);
                f32x4 sc2{};
                if constexpr (kPair) sc2 = *reinterpret_cast<const f32x4*>(col_scale + C::BN + c);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const int r = row_of(mi);
                    const float sa = row_scale[r], p = row_prob[r];
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (kPair) {
                            const float g = static_cast<float>(acc1[mi][ni][j]) * sa * sc1[j];
                            const float u = static_cast<float>(acc2[mi][ni][j]) * sa * sc2[j];
                            v[j] = fwd_elem(g, u, p, limit);
                        } else {
                            const int q = half == 0 ? acc1[mi][ni][j] : acc2[mi][ni][j];
                            v[j] = static_cast<float>(q) * sa * sc1[j] * p;
                        }
                    }
                    *reinterpret_cast<u32x2*>(stage + at(r, c)) =
                        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                }
            }
        lds_barrier();
        uint16_t* o = static_cast<uint16_t*>(out) + col1;
        const int n = kPair ? n1 : n1 + n2;
#pragma unroll
        for (int i = 0; i < C::BM * kRowChunks / C::kThreads; ++i) {
            const int s = i * C::kThreads + tid, row = s / kRowChunks, c = s % kRowChunks * 8;
            if (row < tr.rows && c < n)
                store_nt16(o + static_cast<int64_t>(tr.row0 + row) * n_dim + c,
                           *reinterpret_cast<const u32x4*>(stage + at(row, c)));
        }
    } else {
        // float32, one weight tile at a time; 16-byte chunks of a row swizzled by the row
        float* stage = reinterpret_cast<float*>(lds);
        float* o = static_cast<float*>(out);
        auto at = [](int row, int c) { return row * C::BN + (c ^ ((row & 15) << 2)); };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t c0 = half == 0 ? col1 : col2;
            const int n = half == 0 ? n1 : n2;
            if (half == 1) lds_barrier();
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) {
                const int c = col_of(ni);
                const f32x4 sc = *reinterpret_cast<const f32x4*>(col_scale + half * C::BN + c);
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const int r = row_of(mi);
                    const float sa = row_scale[r], p = row_prob[r];
                    f32x4 v;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int q = half == 0 ? acc1[mi][ni][j] : acc2[mi][ni][j];
                        v[j] = static_cast<float>(q) * sa * sc[j] * p;
                    }
                    *reinterpret_cast<f32x4*>(stage + at(r, c)) = v;
                }
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < C::BM * C::BN / 4 / C::kThreads; ++i) {
                const int s = i * C::kThreads + tid, row = s / (C::BN / 4), c = s % (C::BN / 4) * 4;
                if (row < tr.rows && c < n)
                    store_nt16(o + static_cast<int64_t>(tr.row0 + row) * n_dim + c0 + c,
                               *reinterpret_cast<const u32x4*>(stage + at(row, c)));
            }
        }
    }
}

template <class C, Out kOut, bool kWide>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(2))) void grouped_int8_kernel(
    const int8_t* __restrict__ a, Rows rows_of, const int8_t* __restrict__ w1, const float* __restrict__ s1,
    const int8_t* __restrict__ w2, const float* __restrict__ s2, const int32_t* __restrict__ offs,
    const float* __restrict__ probs, void* __restrict__ out, int rows, int k_dim, int64_t n_dim, int experts,
    float limit, int64_t n_tiles, int64_t n_blocks) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds + 8 * (C::BM + C::BN)];
    grouped_int8_tile<C, kOut, kWide>(lds, a, rows_of, w1, s1, w2, s2, offs, probs, out, rows, k_dim, n_dim, experts,
                                      limit, n_tiles, n_blocks);
}

// ---- few rows per expert ---------------------------------------------------------------
//
// Bound by reading the weights of the experts that have rows, once. A block
// takes one row tile of 16 * MT rows and 16 * NT columns of each of two
// weights (gate and up; two neighbouring column ranges of down); its W
// wavefronts share K in pieces of 256 and meet in LDS at the end (whole
// numbers: any order).
//
// A load instruction takes 256 consecutive bytes of each of 4 weight rows,
// and the wavefront passes them through its own part of LDS into the order
// the matrix instruction wants. Loaded straight into that order, 64 bytes of
// each of 16 rows, the same kernel ran at 4.1-4.6 TB/s of weights instead of
// 6.4 (gate_up of 32 rows, 8 experts of 7168 -> 2 x 2048: 57.5 and 51.6 us
// without and with the weights kept in the caches, against 36.6). The next
// piece is on its way while the present one is multiplied; weights are read
// once (nontemporal: 42.0 us without), the rows' bytes stay in L2.

constexpr int kPiece = 256;                 // bytes of K of a weight row that a wavefront takes at a time
constexpr int kPieceChunks = kPiece / 16;   // 16: a load instruction covers 4 rows of 256 bytes

template <int MT, int NT, int W, Out kOut>
__global__ __launch_bounds__(64 * W) void grouped_int8_few_kernel(
    const int8_t* __restrict__ a, Rows rows_of, const int8_t* __restrict__ w1, const float* __restrict__ s1,
    const int8_t* __restrict__ w2, const float* __restrict__ s2, const int32_t* __restrict__ offs,
    const float* __restrict__ probs, void* __restrict__ out, int rows, int k_dim, int64_t n_dim, int experts,
    float limit, int n_tiles) {
    constexpr bool kPair = kOut == Out::kSwiglu;
    constexpr int T = 2 * NT;  // weight tiles of 16 rows: the first NT of w1, the others of w2
    constexpr int kStageVecs = T * 16 * kPieceChunks, kPartVecs = MT * T * 64;
    __shared__ i32x4 lds[W * (kStageVecs > kPartVecs ? kStageVecs : kPartVecs)];
    const int lane = static_cast<int>(threadIdx.x & 63u);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int mt = static_cast<int>(blockIdx.x) / n_tiles, nt = static_cast<int>(blockIdx.x) % n_tiles;
    const RowTile tr = find_tile(offs, rows, experts, mt, 16 * MT);
    if (tr.rows == 0) return;
    const int64_t col1 = static_cast<int64_t>(nt) * (kPair ? 16 : 32) * NT, col2 = kPair ? col1 : col1 + 16 * NT;
    const int64_t wrow = static_cast<int64_t>(tr.expert) * n_dim;

    // loads: lane l takes chunk l % 16 of rows l / 16 + 4 i
    const int lc = lane % 16 * 16, lr = lane / 16;
    const int8_t* pw[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int64_t c = (t < NT ? col1 + t * 16 : col2 + (t - NT) * 16) + lr + 4 * i;
            c = c < n_dim ? c : n_dim - 1;
            pw[t][i] = (t < NT ? w1 : w2) + (wrow + c) * k_dim;
        }
    const int at = lane / 16 * 16;
    const int8_t* pa[MT];
    float sa[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = m * 16 + lane % 16;
        const int64_t u = rows_of.of(tr.row0 + (i < tr.rows ? i : tr.rows - 1));
        pa[m] = a + (u >= 0 ? u : 0) * k_dim;
        sa[m] = u >= 0 ? rows_of.scale[u] : 0.0f;
    }
    i32x4 acc[MT][T];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[m][t] = i32x4{0, 0, 0, 0};

    // The wavefront's own part of LDS: row r's chunk c at 16 r + (c ^ r), so that the 16
    // rows of a fragment read take 16 different bank groups. No other wavefront touches
    // it, and a wavefront's LDS accesses stay in order, so no barrier is needed.
    i32x4* const mine = lds + wave * (kStageVecs > kPartVecs ? kStageVecs : kPartVecs);
    i32x4 rw[T][4], ra[MT][4];  // the next piece, on its way
    // Past the end of K any bytes will do: the rows' are replaced by zeros below.
    auto fetch = [&](int k0) {
        const int k = k0 + lc < k_dim ? k0 + lc : 0;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rw[t][i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pw[t][i] + k));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int ka = k0 + s * 64 + at < k_dim ? k0 + s * 64 + at : 0;
#pragma unroll
            for (int m = 0; m < MT; ++m) ra[m][s] = *reinterpret_cast<const i32x4*>(pa[m] + ka);
        }
    };
    int k0 = wave * kPiece;
    if (k0 < k_dim) fetch(k0);
    for (; k0 < k_dim; k0 += W * kPiece) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = lr + 4 * i;
                mine[(t * 16 + row) * 16 + ((lane % 16) ^ row)] = rw[t][i];
            }
        i32x4 fa[MT][4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m) fa[m][s] = k0 + s * 64 + at < k_dim ? ra[m][s] : i32x4{0, 0, 0, 0};
        if (k0 + W * kPiece < k_dim) fetch(k0 + W * kPiece);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const i32x4 f = mine[(t * 16 + lane % 16) * 16 + ((4 * s + lane / 16) ^ (lane % 16))];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[m][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f, fa[m][s], acc[m][t], 0, 0, 0);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if constexpr (W > 1) __syncthreads();  // the parts of the sum take the place of the pieces
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t) lds[((wave * MT + m) * T + t) * 64 + lane] = acc[m][t];
    __syncthreads();
    // Lane l of row tile m has row m * 16 + l % 16 and columns 4 * (l / 16) .. + 3 of each weight tile.
#pragma unroll
    for (int mn = 0; mn < MT * NT; ++mn) {
        const int m = mn / NT, n = mn % NT;
        if (mn % W != wave) continue;
        const int i = m * 16 + lane % 16;
        if (i >= tr.rows) continue;
        i32x4 q1{0, 0, 0, 0}, q2{0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < W; ++v) {
            q1 += lds[((v * MT + m) * T + n) * 64 + lane];
            q2 += lds[((v * MT + m) * T + NT + n) * 64 + lane];
        }
        const int64_t r = tr.row0 + i;
        const float p = probs ? probs[r] : 1.0f;
#pragma unroll
        for (int half = 0; half < (kPair ? 1 : 2); ++half) {
            const int64_t c = (half == 0 ? col1 : col2) + n * 16 + 4 * (lane / 16);
            if (c >= n_dim) continue;  // n_dim is a multiple of 8: four columns are in or out
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float t1 = s1[wrow + c + j];
                if constexpr (kPair) {
                    const float g = static_cast<float>(q1[j]) * sa[m] * t1;
                    const float u = static_cast<float>(q2[j]) * sa[m] * s2[wrow + c + j];
                    v[j] = fwd_elem(g, u, p, limit);
                } else {
                    v[j] = static_cast<float>(half == 0 ? q1[j] : q2[j]) * sa[m] * t1 * p;
                }
            }
            if constexpr (kOut == Out::kF32)
                *reinterpret_cast<f32x4*>(static_cast<float*>(out) + r * n_dim + c) = f32x4{v[0], v[1], v[2], v[3]};
            else
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + r * n_dim + c) =
                    u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
    }
}

template <int MT, int W, Out kOut>
void launch_few_waves(unsigned grid, const int8_t* a, const Rows& rows_of, const int8_t* w1, const float* s1,
                      const int8_t* w2, const float* s2, const int32_t* offs, const float* probs, void* out,
                      int64_t rows, int64_t k_dim, int64_t n_dim, int64_t experts, float limit, int64_t n_tiles,
                      hipStream_t st) {
    hipLaunchKernelGGL((grouped_int8_few_kernel<MT, 1, W, kOut>), dim3(grid), dim3(64 * W), 0, st, a, rows_of, w1, s1,
                       w2, s2, offs, probs, out, static_cast<int>(rows), static_cast<int>(k_dim), n_dim,
                       static_cast<int>(experts), limit, static_cast<int>(n_tiles));
}

template <int MT, Out kOut>
int launch_few(const int8_t* a, const Rows& rows_of, const int8_t* w1, const float* s1, const int8_t* w2,
               const float* s2, const int32_t* offs, const float* probs, void* out, int64_t rows, int64_t k_dim,
               int64_t n_dim, int64_t experts, float limit, hipStream_t st) {
    // row tiles: no more than rows, and one partial one per expert
    const int64_t most = (rows + 16 * MT - 1) / (16 * MT) + experts, m_tiles = most < rows ? most : rows;
    const int64_t cols = kOut == Out::kSwiglu ? 16 : 32, n_tiles = (n_dim + cols - 1) / cols;
    const int64_t blocks = m_tiles * n_tiles;
    if (blocks >= (int64_t{1} << 31)) return MOE_EPI_ERR_BAD_SHAPE;
    // Wavefronts that share K: as many as keep the grid near 4096 wavefronts, 16
    // per CU. One GPU, us with 1 / 2 / 4: 32 rows 2048 -> 7168 on 8 experts (1792
    // blocks) 19.7 / 19.6 / 21.0; 8 rows 2048 -> 2 x 768 on 64 (384 blocks)
    // 9.8 / 8.3 / 7.4.
    auto go = [&](auto launch) {
        (void)hipGetLastError();
        launch(static_cast<unsigned>(blocks), a, rows_of, w1, s1, w2, s2, offs, probs, out, rows, k_dim, n_dim,
               experts, limit, n_tiles, st);
        return launch_status();
    };
    if (blocks <= 1024) return go(launch_few_waves<MT, 4, kOut>);
    if (blocks <= 2048) return go(launch_few_waves<MT, 2, kOut>);
    return go(launch_few_waves<MT, 1, kOut>);
}

// ---- launches ------------------------------------------------------------------------

// Three tile sizes. The large one has the fewest bytes per product and takes a
// CU by itself; the smaller ones give few rows more blocks. The middle one has
// two stages where several blocks share a CU, and three where there is about
// one block per CU, so that more of the weights are on their way.
template <Out kOut> struct Tiles {
    static constexpr int kGroup = kOut == Out::kSwiglu ? 2 : 16;  // row tiles per group of the tile order
    typedef Tile<256, 128, 4, 2, kGroup, kOut == Out::kSwiglu ? 8 : 4, 2, true> Large;
    typedef Tile<128, 64, 2, 2, kGroup, 4, 2, false> Middle;
    typedef Tile<128, 64, 2, 2, kGroup, 4, 3, false> MiddleDeep;
    typedef Tile<64, 64, 2, 2, kGroup, 4, 3, false> Small;
};

template <class C, Out kOut>
int launch_tiles(const int8_t* a, const Rows& rows_of, int64_t tokens, const int8_t* w1, const float* s1,
                 const int8_t* w2, const float* s2, const int32_t* offs, const float* probs, void* out, int64_t rows,
                 int64_t k_dim, int64_t n_dim, int64_t experts, float limit, hipStream_t st) {
    int64_t n_tiles, n_blocks;
    const int64_t grid =
        grouped_grid(rows, n_dim, kOut == Out::kSwiglu ? C::BN : 2 * C::BN, experts, C::BM, &n_tiles, &n_blocks);
    if (grid == 0) return MOE_EPI_ERR_BAD_SHAPE;
    auto go = [&](auto kernel) {
        (void)hipGetLastError();
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), 0, st, a, rows_of, w1, s1, w2,
                           s2, offs, probs, out, static_cast<int>(rows), static_cast<int>(k_dim), n_dim,
                           static_cast<int>(experts), limit, n_tiles, n_blocks);
        return launch_status();
    };
    if constexpr (kOut == Out::kSwiglu) {
        // the rows of a are read in place: their offsets pass 31 bits in a large enough tensor
        if (rows_of.slot_of && tokens * k_dim > INT32_MAX) return go(grouped_int8_kernel<C, kOut, true>);
    }
    return go(grouped_int8_kernel<C, kOut, false>);
}

template <Out kOut>
int launch_int8(const int8_t* a, const Rows& rows_of, int64_t tokens, const int8_t* w1, const float* s1,
                const int8_t* w2, const float* s2, const int32_t* offs, const float* probs, void* out, int64_t rows,
                int64_t k_dim, int64_t n_dim, int64_t experts, float limit, hipStream_t st) {
    auto few = [&](auto launch) {
        return launch(a, rows_of, w1, s1, w2, s2, offs, probs, out, rows, k_dim, n_dim, experts, limit, st);
    };
    auto tiles = [&](auto launch) {
        return launch(a, rows_of, tokens, w1, s1, w2, s2, offs, probs, out, rows, k_dim, n_dim, experts, limit, st);
    };
    // By rows / experts, as many as the buffers hold: how many of them there are
    // stands in offs, on the device. A larger tile reads the weights fewer times,
    // a smaller one wastes fewer rows of a partial tile; and a tile size is taken
    // only where it gives half of the CUs a block. Buffers larger than the rows
    // get a larger tile than the rows need: 267 rows on 8 experts in buffers of
    // 267 / of 2048 rows (256 tokens, 8 choices, 8 of 64 experts here) gate_up
    // 37.8 / 74.5, down 22.8 / 50.8; 28 in 28 / 256 37.5 / 37.0, 19.9 / 21.4; 2124
    // in 2124 / 16384 102.8 / 99.9, 63.9 / 62.8. Measured with exact buffers (us, 8 experts, gate_up 7168 -> 2 x 2048 / down 2048 ->
    // 7168; few rows by 16 and by 32, small, middle, middle with three stages,
    // large):
    //   rows an expert  16          32          small       middle      deep        large
    //     8             39.2/19.8   41.1/20.9   43/24       63/26       46/30       96/34
    //    16             56.5/26.4   42.7/23.0   43.0/24.3   63.2/26.6   45.6/30.4   94.9/34.3
    //    24             71.6/32.4   49.1/25.6   43.5/24.1   64.8/27.3   46.3/31.0   95.1/34.4
    //    48                         96.9/47.7   44.2/25.9   62.1/27.4   47.1/40.9   94.1/34.8
    //    64                          112/59.5   65.2/41.1   62.5/27.1   47.1/31.1   93.9/35.6
    //    96                          168/77.1   69.7/40.0   63.9/29.4   49.4/31.8   95.3/57.8
    //   128                          211/99.4   85.0/55.9   76.5/49.9   83.0/56.8   94.6/39.1
    //   192                          291/142     101/67.3   78.2/53.2   85.8/57.5   99.3/38.1
    //   256                          378/185     124/84.5    126/74.5    119/84.8    106/66.5
    // and where the grid is small (4 experts, 1024 -> 2 x 512):
    //   100              6.6         6.7         8.2        10.3        10.3        18.9
    //   400             15.6        15.1         8.6        11.4        11.1        19.7
    //  1500             43.1        37.3        17.0        14.0        20.4        20.3
    auto grid_of = [&](int bm, int cols) { return (rows / bm + experts / 2) * ((n_dim + cols - 1) / cols); };
    constexpr int kCols = kOut == Out::kSwiglu ? 1 : 2;  // column ranges of a tile
    typedef typename Tiles<kOut>::Large Large;
    typedef typename Tiles<kOut>::Middle Middle;
    typedef typename Tiles<kOut>::Small Small;
    const int64_t middle = grid_of(Middle::BM, kCols * Middle::BN);
    if (rows <= 10 * experts) return few(launch_few<1, kOut>);
    if (rows <= 18 * experts || grid_of(Small::BM, kCols * Small::BN) < 128) return few(launch_few<2, kOut>);
    if (rows <= 56 * experts || middle < 128) return tiles(launch_tiles<Small, kOut>);
    if (rows <= (kCols == 1 ? 192 : 112) * experts || grid_of(Large::BM, kCols * Large::BN) < 128)
        return middle <= 320 ? tiles(launch_tiles<typename Tiles<kOut>::MiddleDeep, kOut>)
                             : tiles(launch_tiles<Middle, kOut>);
    return tiles(launch_tiles<Large, kOut>);
}

bool shape_ok(int64_t rows, int64_t k_dim, int64_t n_dim, int64_t experts) {
    return rows >= 0 && rows <= INT32_MAX && k_dim > 0 && k_dim < kMaxK && k_dim % 16 == 0 && n_dim > 0 &&
           n_dim % 8 == 0 && experts > 0 && experts <= INT32_MAX && n_dim <= INT64_MAX / 4 / experts;
}

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int grouped_gate_up_swiglu_int8_fwd(const int8_t* a, const float* a_scale, const int32_t* slot_of,
                                               const int8_t* w_gate, const float* w_gate_scale, const int8_t* w_up,
                                               const float* w_up_scale, const int32_t* offs, const float* probs,
                                               uint16_t* y, int64_t rows, int64_t tokens, int64_t top_k,
                                               int64_t hidden, int64_t inter, int64_t experts, float limit,
                                               void* stream) {
    if (!shape_ok(rows, hidden, inter, experts) || tokens < 0 || top_k < 1 || tokens > INT32_MAX / top_k)
        return MOE_EPI_ERR_BAD_SHAPE;
    if (!slot_of && (top_k != 1 || tokens != rows)) return MOE_EPI_ERR_BAD_SHAPE;
    int64_t ab, wb, yb, tb, rb, sb, ob;
    if (!bytes_ok(tokens, hidden, 1, &ab) || !bytes_ok(experts * inter, hidden, 1, &wb) ||
        !bytes_ok(rows, inter, 2, &yb) || !bytes_ok(tokens, 1, 4, &tb) || !bytes_ok(rows, 1, 4, &rb) ||
        !bytes_ok(experts, inter, 4, &sb) || !bytes_ok(experts, 1, 4, &ob))
        return MOE_EPI_ERR_BAD_SHAPE;
    if (!(limit > 0.0f) || !isfinite(limit)) return MOE_EPI_ERR_BAD_LIMIT;
    if (rows == 0) return MOE_EPI_SUCCESS;
    if ((tokens > 0 && (!a || !a_scale)) || !w_gate || !w_gate_scale || !w_up || !w_up_scale || !offs || !y)
        return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(a, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(y, 16) || !aligned(a_scale, 4) ||
        !aligned(slot_of, 4) || !aligned(w_gate_scale, 4) || !aligned(w_up_scale, 4) || !aligned(offs, 4) ||
        !aligned(probs, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range ry = range_of(y, yb);
    for (const Range& r : {range_of(a, ab), range_of(a_scale, tb), range_of(slot_of, slot_of ? rb : 0),
                           range_of(w_gate, wb), range_of(w_up, wb), range_of(w_gate_scale, sb),
                           range_of(w_up_scale, sb), range_of(offs, ob), range_of(probs, probs ? rb : 0)})
        if (overlaps(ry, r)) return MOE_EPI_ERR_ALIAS;
    // Without tokens no slot is in range. The kernels read row 0 of a for such a slot, times a scale of 0, and
    // any `hidden` bytes will do for it: a row of the weights.
    if (tokens == 0) a = w_gate;
    const Rows rows_of{a_scale, slot_of, static_cast<uint32_t>(top_k), tokens * top_k};
    return launch_int8<Out::kSwiglu>(a, rows_of, tokens, w_gate, w_gate_scale, w_up, w_up_scale, offs, probs, y, rows,
                                     hidden, inter, experts, limit, as_stream(stream));
}

extern "C" int grouped_down_router_int8_fwd(const int8_t* h, const float* h_scale, const int8_t* w_down,
                                            const float* w_down_scale, const int32_t* offs, const float* probs,
                                            void* out, int out_dtype, int64_t rows, int64_t inter, int64_t hidden,
                                            int64_t experts, void* stream) {
    if (out_dtype != MOE_EPI_BF16 && out_dtype != MOE_EPI_F32) return MOE_EPI_ERR_BAD_DTYPE;
    if (!shape_ok(rows, inter, hidden, experts)) return MOE_EPI_ERR_BAD_SHAPE;
    int64_t hb, wb, ob, rb, sb, fb;
    if (!bytes_ok(rows, inter, 1, &hb) || !bytes_ok(experts * hidden, inter, 1, &wb) ||
        !bytes_ok(rows, hidden, elem_bytes(out_dtype), &ob) || !bytes_ok(rows, 1, 4, &rb) ||
        !bytes_ok(experts, hidden, 4, &sb) || !bytes_ok(experts, 1, 4, &fb))
        return MOE_EPI_ERR_BAD_SHAPE;
    if (rows == 0) return MOE_EPI_SUCCESS;
    if (!h || !h_scale || !w_down || !w_down_scale || !offs || !out) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(h, 16) || !aligned(w_down, 16) || !aligned(out, 16) || !aligned(h_scale, 4) ||
        !aligned(w_down_scale, 4) || !aligned(offs, 4) || !aligned(probs, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range ro = range_of(out, ob);
    for (const Range& r : {range_of(h, hb), range_of(h_scale, rb), range_of(w_down, wb), range_of(w_down_scale, sb),
                           range_of(offs, fb), range_of(probs, probs ? rb : 0)})
        if (overlaps(ro, r)) return MOE_EPI_ERR_ALIAS;
    const Rows rows_of{h_scale, nullptr, 1u, rows};
    const hipStream_t st = as_stream(stream);
    if (out_dtype == MOE_EPI_F32)
        return launch_int8<Out::kF32>(h, rows_of, rows, w_down, w_down_scale, w_down, w_down_scale, offs, probs, out,
                                      rows, inter, hidden, experts, 1.0f, st);
    return launch_int8<Out::kBf16>(h, rows_of, rows, w_down, w_down_scale, w_down, w_down_scale, offs, probs, out, rows,
                                   inter, hidden, experts, 1.0f, st);
}
