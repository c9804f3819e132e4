// Order of the routed rows (gfx950): a stable counting sort of the slots by
// local expert.
//
// A slot s = t * top_k + j names an expert; with first <= expert < first +
// experts its bucket is expert - first, otherwise it has no row. With
//   start[b] = number of slots in buckets below b,
//   rank[s]  = number of slots s' < s in s's own bucket,
// the row of s is start[b] + rank[s]. Both are counts of whole numbers, so
// the result does not depend on the order in which they are formed.
//
// Ranks within a wavefront come from ballots: one per bit of the bucket gives
// each lane the mask of the lanes in its own bucket, the bits below the lane
// are its rank, and the lowest lane of each mask adds the mask's count to the
// wavefront's counter of that bucket. The counters are private to a
// wavefront, so no atomic operation is needed.
//
// Short calls are bound by their chain of reads, counts and writes, and a call
// of up to 2048 slots is one block (32 x 8 slots over 64 experts 2.9 us, 1 x 8
// over 256 experts 3.8; 256 x 8 over 64 4.5, against 6.0 by two launches, but
// 512 x 8 over 256 8.1 against 7.5). Longer ones count tiles of slots first: two launches,
// 131072 x 8 slots over 8 local experts 10.0 us, of which the 12 MB that are
// read and written need 2; with more than 8192 counts a third launch sums them,
// since every block would read them all (131072 x 8 over 256 experts 20.3 us
// against 40.2; 32768 x 8 over 128, 8192 counts, 12.7 without it against 14.8).
#include <type_traits>

#include "epi_common.h"
#include "moe_routed.h"

namespace moe_epi {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxSlotsPerToken = 1024;
constexpr int kTileThreads = 1024;
constexpr int kTileWaves = kTileThreads / 64;
constexpr int kMostGroups = 4;                   // groups of 64 slots per wavefront of a tile, at most
constexpr int kOneGroups = 2;                    // and of a call's only tile
constexpr int64_t kTiles = 256;                  // tiles that a call aims at: one per CU
constexpr int kDirect = 8;                       // counts per thread that a block reads of all tiles

inline int bits_for(int64_t experts) {           // buckets 0 .. experts (experts: no row)
    int n = 0;
    while ((experts >> n) != 0) ++n;
    return n;
}

// The bucket of slot s; `experts` for a slot without a row or past the end.
template <class Id>
__device__ __forceinline__ uint32_t bucket_of(const Id* __restrict__ ids, int64_t s, int64_t slots, int64_t first,
                                              int experts) {
    if (s >= slots) return static_cast<uint32_t>(experts);
    const uint64_t b = static_cast<uint64_t>(static_cast<int64_t>(ids[s])) - static_cast<uint64_t>(first);
    return b < static_cast<uint64_t>(experts) ? static_cast<uint32_t>(b) : static_cast<uint32_t>(experts);
}

// The lanes of the wavefront whose bucket equals the calling lane's.
__device__ __forceinline__ uint64_t same_bucket(uint32_t b, int nbits) {
    uint64_t mask = ~uint64_t{0};
    for (int i = 0; i < nbits; ++i) {
        const bool on = (b >> i) & 1u;
        const uint64_t v = __ballot(on);
        mask &= on ? v : ~v;
    }
    return mask;
}

__device__ __forceinline__ int rank_in(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
}

__device__ __forceinline__ bool is_lowest(uint64_t mask) {
    return __builtin_ctzll(mask) == static_cast<int>(threadIdx.x & 63u);
}

// Exclusive scan of n counts in LDS by the calling wavefront, in place; returns the total.
__device__ __forceinline__ int wave_scan(int* v, int n) {
    const int lane = static_cast<int>(threadIdx.x & 63u);
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int c = i0 + lane < n ? v[i0 + lane] : 0;
        int x = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(x, d, 64);
            if (lane >= d) x += y;
        }
        if (i0 + lane < n) v[i0 + lane] = carry + x - c;
        carry += __shfl(x, 63, 64);
    }
    return carry;
}

// Counts of one tile's slots per bucket: hist[tile * experts + b].
template <class Id, int kGroups>
__global__ __launch_bounds__(kTileThreads) void moe_sort_count(const Id* __restrict__ ids, int* __restrict__ hist,
                                                               int64_t slots, int64_t first, int experts) {
    __shared__ int count[kMaxExperts];
    for (int e = threadIdx.x; e < experts; e += kTileThreads) count[e] = 0;
    __syncthreads();
    const int64_t s0 = static_cast<int64_t>(blockIdx.x) * (kTileThreads * kGroups) + threadIdx.x;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const uint32_t b = bucket_of(ids, s0 + g * kTileThreads, slots, first, experts);
        if (b < static_cast<uint32_t>(experts)) atomicAdd(&count[b], 1);  // whole numbers: any order, one sum
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kTileThreads)
        hist[static_cast<int64_t>(blockIdx.x) * experts + e] = count[e];
}

// The counts of 64 experts (one a lane) become the slots of earlier tiles, and
// their totals go to totals[e]: each wavefront sums a run of tiles, then
// replaces its counts from the sum of the runs before.
__global__ __launch_bounds__(kTileThreads) void moe_sort_scan(int* __restrict__ hist, int* __restrict__ totals,
                                                              int64_t tiles, int experts) {
    __shared__ int run[kTileWaves][64];
    const int lane = static_cast<int>(threadIdx.x & 63u), wave = static_cast<int>(threadIdx.x >> 6);
    const int e = static_cast<int>(blockIdx.x) * 64 + lane;
    const int64_t per = (tiles + kTileWaves - 1) / kTileWaves, t0 = wave * per;
    const int64_t t1 = t0 + per < tiles ? t0 + per : tiles;
    int n = 0;
    if (e < experts)
#pragma unroll 8
        for (int64_t t = t0; t < t1; ++t) n += hist[t * experts + e];
    run[wave][lane] = n;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += run[w][lane];
    if (e >= experts) return;
#pragma unroll 8
    for (int64_t t = t0; t < t1; ++t) {
        const int c = hist[t * experts + e];
        hist[t * experts + e] = before;
        before += c;
    }
    if (wave == kTileWaves - 1) totals[e] = before;
}

// Rows of one tile's slots, kThreads * kGroups of them. A single tile's own
// counts are the totals (kMany false: hist and totals are not read); of many,
// hist holds every tile's counts, or, where totals are given, the slots of
// earlier tiles (moe_sort_scan).
template <class Id, int kThreads, int kGroups, bool kMany>
__global__ __launch_bounds__(kThreads) void moe_sort_place(const Id* __restrict__ ids,
                                                           const int* __restrict__ hist,
                                                           const int* __restrict__ totals, int* __restrict__ offs,
                                                           int* __restrict__ row_of, int* __restrict__ slot_of,
                                                           int64_t slots, int64_t first, int experts, int nbits,
                                                           int tiles) {
    // counts per wavefront and bucket (a tile has up to 4096 slots), earlier tiles' slots and start per bucket
    constexpr int kWaves = kThreads / 64;
    extern __shared__ uint16_t wave_count[];  // [kWaves][experts]
    __shared__ int before[kMaxExperts];
    __shared__ int start[kMaxExperts];
    __shared__ int total_rows;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int tile = static_cast<int>(blockIdx.x);

    const int64_t s0 = static_cast<int64_t>(tile) * (kThreads * kGroups) + wave * (64 * kGroups) + lane;
    uint32_t b[kGroups];
    uint64_t mask[kGroups];
    uint16_t* mine = wave_count + wave * experts;
    // everything that is read is asked for at once
#pragma unroll
    for (int g = 0; g < kGroups; ++g) b[g] = bucket_of(ids, s0 + g * 64, slots, first, experts);
    int count[kMany ? kDirect : 1];
    if constexpr (kMany) {
#pragma unroll
        for (int k = 0; k < kDirect; ++k) {
            const int i = tid + k * kThreads;
            count[k] = !totals && i < tiles * experts ? hist[i] : 0;
        }
    }
    for (int i = lane; i < experts; i += 64) mine[i] = 0;
    for (int e = tid; e < experts; e += kThreads) {
        start[e] = kMany && totals ? totals[e] : 0;
        before[e] = kMany && totals ? hist[static_cast<int64_t>(tile) * experts + e] : 0;
    }
    if constexpr (kMany) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDirect; ++k) {
            if (count[k] == 0) continue;
            const uint32_t i = tid + k * kThreads, t = i / static_cast<uint32_t>(experts), e = i - t * experts;
            atomicAdd(&start[e], count[k]);  // whole numbers: any order, one sum
            if (static_cast<int>(t) < tile) atomicAdd(&before[e], count[k]);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        mask[g] = same_bucket(b[g], nbits);
        if (b[g] < static_cast<uint32_t>(experts) && is_lowest(mask[g])) mine[b[g]] += __popcll(mask[g]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    // the wavefronts' counts become the slots of the bucket in the tile's earlier wavefronts
    for (int e = tid; e < experts; e += kThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = wave_count[w * experts + e];
            wave_count[w * experts + e] = static_cast<uint16_t>(n);
            n += c;
        }
        if constexpr (!kMany) start[e] = n;
    }
    __syncthreads();
    if (wave == 0) {
        const int n = wave_scan(start, experts);
        if (lane == 0) total_rows = n;
    }
    __syncthreads();
    const int rows = total_rows;
    if (tile == 0)
        for (int e = tid; e < experts; e += kThreads) offs[e] = e + 1 < experts ? start[e + 1] : rows;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int64_t s = s0 + g * 64;
        int row = -1;
        if (b[g] < static_cast<uint32_t>(experts)) {
            row = start[b[g]] + before[b[g]] + mine[b[g]] + rank_in(mask[g]);
            slot_of[row] = static_cast<int>(s);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (b[g] < static_cast<uint32_t>(experts) && is_lowest(mask[g])) mine[b[g]] += __popcll(mask[g]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (s < slots) {
            row_of[s] = row;
            if (s >= rows) slot_of[s] = -1;  // past the last row
        }
    }
}

__global__ void moe_sort_empty(int* __restrict__ offs, int experts) {
    for (int e = threadIdx.x; e < experts; e += blockDim.x) offs[e] = 0;
}

bool sizes_ok(int64_t tokens, int64_t top_k, int64_t experts) {
    return tokens >= 0 && top_k >= 1 && top_k <= kMaxSlotsPerToken && experts >= 1 && experts <= kMaxExperts &&
           tokens <= INT32_MAX / top_k;
}

// Groups per wavefront: the fewest that make no more than kTiles tiles. Each
// group of a wavefront comes after the one before (32 x 8 slots over 64 experts
// 2.9 us with one, 3.4 with two, 4.5 with four; 4096 x 8 slots 6.6, 7.7, 9.7),
// but every tile adds counts that all others read (131072 x 8 slots over 8 local
// experts 16.8, 10.8, 10.0).
// Two groups give way to four where that spares the third launch (40000 x 8 slots
// over 64 experts 13.2, 11.3).
int64_t tiles_of(int64_t slots, int groups) {
    const int64_t tile = kTileThreads * groups;
    return (slots + tile - 1) / tile;
}
// Every block of moe_sort_place reads all counts, kDirect a thread, while they
// are that few; beyond that a third launch sums them first.
bool scans(int64_t tiles, int64_t experts) { return tiles * experts > kDirect * kTileThreads; }

int groups_of(int64_t slots, int64_t experts) {
    if (slots <= kTileThreads * kOneGroups) return slots <= kTileThreads ? 1 : kOneGroups;
    int g = 1;
    while (g < kMostGroups && tiles_of(slots, g) > kTiles) g *= 2;
    if (g == 2 && scans(tiles_of(slots, 2), experts) && !scans(tiles_of(slots, 4), experts)) g = 4;
    return g;
}

template <class Id>
void launch_sort(const void* ids, int64_t first, int* offs, int* row_of, int* slot_of, int* hist, int64_t slots,
                 int experts, hipStream_t st) {
    const int groups = groups_of(slots, experts), tiles = static_cast<int>(tiles_of(slots, groups));
    const Id* p = static_cast<const Id*>(ids);
    int* totals = nullptr;
    auto place = [&](int threads, auto kernel) {
        const int lds = threads / 64 * experts * static_cast<int>(sizeof(uint16_t));
        hipLaunchKernelGGL(kernel, dim3(tiles), dim3(threads), lds, st, p, hist, totals, offs, row_of, slot_of,
                           slots, first, experts, bits_for(experts), tiles);
    };
    if (slots <= 256) return place(256, moe_sort_place<Id, 256, 1, false>);
    if (tiles == 1)
        return groups == 1 ? place(kTileThreads, moe_sort_place<Id, kTileThreads, 1, false>)
                           : place(kTileThreads, moe_sort_place<Id, kTileThreads, kOneGroups, false>);
    auto many = [&](auto groups) {
        constexpr int G = decltype(groups)::value;
        hipLaunchKernelGGL((moe_sort_count<Id, G>), dim3(tiles), dim3(kTileThreads), 0, st, p, hist, slots, first,
                           experts);
        if (scans(tiles, experts)) {
            totals = hist + static_cast<int64_t>(tiles) * experts;
            hipLaunchKernelGGL(moe_sort_scan, dim3((experts + 63) / 64), dim3(kTileThreads), 0, st, hist, totals,
                               tiles, experts);
        }
        place(kTileThreads, moe_sort_place<Id, kTileThreads, G, true>);
    };
    switch (groups) {
        case 1: return many(std::integral_constant<int, 1>());
        case 2: return many(std::integral_constant<int, 2>());
        default: return many(std::integral_constant<int, kMostGroups>());
    }
}

}  // namespace
}  // namespace moe_epi

using namespace moe_epi;

extern "C" int64_t moe_sort_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts) {
    if (!sizes_ok(tokens, top_k, experts)) return -1;
    const int64_t slots = tokens * top_k, tiles = tiles_of(slots, groups_of(slots, experts));
    return tiles > 1 ? (tiles + 1) * experts * 4 : 0;
}

extern "C" int moe_sort_fwd(const void* expert_of, int id_bytes, int64_t first_expert, int32_t* offs, int32_t* row_of,
                            int32_t* slot_of, void* workspace, int64_t workspace_bytes, int64_t tokens, int64_t top_k,
                            int64_t experts, void* stream) {
    if (id_bytes != 4 && id_bytes != 8) return MOE_EPI_ERR_BAD_DTYPE;
    const int64_t need = moe_sort_workspace_bytes(tokens, top_k, experts);
    if (need < 0 || workspace_bytes < need) return MOE_EPI_ERR_BAD_SHAPE;
    const int64_t slots = tokens * top_k;
    if (!offs || (need > 0 && !workspace)) return MOE_EPI_ERR_NULL_POINTER;
    if (slots > 0 && (!expert_of || !row_of || !slot_of)) return MOE_EPI_ERR_NULL_POINTER;
    if (!aligned(expert_of, id_bytes) || !aligned(offs, 4) || !aligned(row_of, 4) || !aligned(slot_of, 4) ||
        !aligned(workspace, 4))
        return MOE_EPI_ERR_MISALIGNED;
    const Range in = range_of(expert_of, slots * id_bytes),
                out[4] = {range_of(offs, experts * 4), range_of(row_of, slots * 4), range_of(slot_of, slots * 4),
                          range_of(workspace, need)};
    for (int i = 0; i < 4; ++i) {
        if (overlaps(out[i], in)) return MOE_EPI_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out[j])) return MOE_EPI_ERR_ALIAS;
    }
    (void)hipGetLastError();
    const hipStream_t st = as_stream(stream);
    if (slots == 0)
        hipLaunchKernelGGL(moe_sort_empty, dim3(1), dim3(256), 0, st, offs, static_cast<int>(experts));
    else if (id_bytes == 4)
        launch_sort<int32_t>(expert_of, first_expert, offs, row_of, slot_of, static_cast<int*>(workspace), slots,
                             static_cast<int>(experts), st);
    else
        launch_sort<int64_t>(expert_of, first_expert, offs, row_of, slot_of, static_cast<int*>(workspace), slots,
                             static_cast<int>(experts), st);
    return launch_status();
}
