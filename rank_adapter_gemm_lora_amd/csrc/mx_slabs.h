// mx_slabs.h -- how many rows one launch of a microscaled kernel takes.  Host
// arithmetic alone, so that it can be checked without a GPU.
#pragma once

#include <stdint.h>

namespace lora {

// HIP takes fewer than 2^32 threads along a dimension of a launch.
constexpr int64_t kLaunchThreads = ((int64_t)1 << 32) - 1;

// Most rows of a launch in which every `tile` rows are `blocks` workgroups of
// `threads`: whole groups of eight tiles where a group fits (the kernels that
// tile rows walk them in bands of eight).
constexpr int64_t slab_rows(int tile, int64_t blocks, int threads)
{
    const int64_t tiles = kLaunchThreads / threads / blocks;
    return (tiles >= 8 ? tiles & ~(int64_t)7 : tiles) * tile;
}

// go(first row, rows) over slabs of at most `most` rows.
template <class F> void for_slabs(int64_t n_rows, int64_t most, F go)
{
    for (int64_t r = 0; r < n_rows; r += most)
        go(r, n_rows - r < most ? n_rows - r : most);
}

}  // namespace lora
