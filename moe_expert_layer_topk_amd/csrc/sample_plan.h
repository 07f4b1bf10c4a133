// What moe_sample makes of top_k (sample.hip). Plain C++, constexpr, so that the
// kernels and a test on the host take the same functions.
#pragma once

#include "moe.h"

namespace moe {

// The number of tokens that a row's top_k keeps, 0: all. No row has more than
// MOE_SAMPLE_MAX_COLS, and sums with larger numbers would not fit an int.
constexpr int kept_by_count(int top_k) { return top_k <= 0 ? 0 : top_k < MOE_SAMPLE_MAX_COLS ? top_k : MOE_SAMPLE_MAX_COLS; }

// Whether a chunk with so many candidates looks for the k-th first.
constexpr bool worth_parts(int candidates, int k) { return k && candidates > 2 * k + 64; }

}  // namespace moe
