// moe.h -- the grouping of a batch's (row, choice) pairs by expert: the plan
// object, and the launchers of the router, the grouping and the combination.
// Not part of the public ABI (include/lora.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx.h"

namespace lora {

constexpr int kMoeMaxChunks = 256;     // chunks of rows that the larger batches are counted in: one a CU
constexpr int kMoeSmallPairs = 2048;   // batches of at most so many pairs: one workgroup, one launch
constexpr int64_t kMoeMaxPairs = (int64_t)1 << 30;

// Heights of the row tiles that the experts' products work in.
constexpr int kMoeHeights = 4;
constexpr int moe_height_shift(int i) { return 4 + i; }   // 16, 32, 64, 128 rows

// One row tile: positions [first, end) of the grouped order, all of one expert.
struct alignas(16) MoeTile {
    int32_t expert, first, end, none;
};

// Pair p = row * top_k + choice.  Positions: the pairs sorted by expert, in
// their own order inside a group, those without an expert last.
struct MoeLists {
    int32_t *order;                 // [pairs] pair at a position
    int32_t *place;                 // [pairs] position of a pair, -1 without an expert
    int32_t *n_tiles;               // [kMoeHeights]
    MoeTile *tiles[kMoeHeights];
};

// Row tiles of 2^shift rows that `pairs` pairs of at most `experts` experts can need.
inline int64_t moe_tile_bound(int64_t pairs, int experts, int shift)
{
    const int64_t used = pairs < experts ? pairs : experts;
    const int64_t most = (pairs >> shift) + used;
    return most < pairs ? most : pairs;
}

struct MoeRouteArgs {
    const void *logits;      // null: ids are given
    int64_t ldl;
    const int32_t *ids_in;
    int32_t *ids;            // routed: written
    float *weights;          // routed: written
    int64_t n_rows;
    int experts, top_k;
    int score, renorm;
    float scale;
    int32_t *order;          // the caller's copy, or null
    int32_t *offsets;        // or null: [experts + 1] first position of a group; the last: pairs with an expert
    MoeLists l;
    int32_t *hist;           // [chunks + 1][experts + 1]
    int64_t chunk_rows;
    int n_chunks;
};
hipError_t launch_moe_route(int dtype, const MoeRouteArgs &a, hipStream_t s);

struct MoeCombineArgs {
    void *out;
    int64_t ldo;
    const void *y;
    int64_t ldy;
    int y_dtype;
    const float *weights;
    const void *res;         // or null
    int64_t ldr;
    const int32_t *place;
    int64_t n_rows;
    int64_t d;
    int top_k;
    int64_t row0;            // first row of this launch
    int64_t rows;            // of this launch
};
hipError_t launch_moe_combine(int dtype, const MoeCombineArgs &a, hipStream_t s);

}  // namespace lora

struct lora_moe_plan {
    int device;
    int experts, top_k;
    int64_t max_rows;
    int64_t n_rows;          // of the last grouping, -1 before the first
    void *memory;
    lora::MoeLists l;
    int32_t *hist;
};
