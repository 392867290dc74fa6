// ep_count.h -- how many blocks and steps the rows of an expert take.  Row
// counts go up to 2^31 - 1, so nothing is added to one before it is divided.
#pragma once

#include <stdint.h>

namespace ep {

// Blocks of `size` rows that n rows take, the last perhaps in part.
constexpr int blocks_of(int n, int size) { return n > 0 ? (n - 1) / size + 1 : 0; }

// Whether step s of 64 rows lies within n rows (0 <= 64 s <= n).
constexpr bool whole_step(int s, int n) { return n - s * 64 >= 64; }

// Blocks of `size` rows there can be at most: one for every full block of rows
// and a part of one for every expert that holds rows.
constexpr int64_t max_row_blocks(int64_t num_rows, int num_experts, int size)
{
    return num_rows / size + (num_rows < num_experts ? num_rows : num_experts);
}

}  // namespace ep
