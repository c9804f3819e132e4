// Which steps of the router's weight gradient load without bounds (host and device).
#pragma once

#include <stdint.h>

namespace moe_epi {

constexpr int kGradStep = 32;  // tokens of a step

// The step's lanes load `width` elements of a token's row at a multiple of
// `width` below hidden, so the last lane's go up to width - 1 past the row, into
// the next tokens' rows: one of them, or several where rows are shorter than that.
// These are the steps before the first whose loads may leave the tensor.
__host__ __device__ __forceinline__ int64_t steps_inside(int64_t tokens, int64_t hidden, int width) {
    const int64_t after = (width - 1 + hidden - 1) / hidden;
    return tokens > after ? (tokens - after) / kGradStep : 0;
}

}  // namespace moe_epi
