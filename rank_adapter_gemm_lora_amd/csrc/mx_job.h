// mx_job.h -- arguments of the products with an epilogue, and their launchers.
#pragma once

#include "moe.h"
#include "mx.h"

namespace lora {

// The job's arguments; outputs, bias and residual in dtype.
struct MxEpilogue {
    const void *bias;        // [d] (gated: [2 d]; grouped: one after the other), or null
    const void *res;         // or null
    int64_t ldr;
    void *y;                 // or null
    int64_t ldy;
    MxBlocks b;              // b.q null: not wanted
    int64_t d;               // outputs of a row
    int dtype, act;
    // grouped by expert
    const MoeTile *tiles;
    const int32_t *n_tiles;
    int tile0;               // first tile of this launch
    const int32_t *rows;     // row of X at a position; null: X is in grouped order
    int64_t code_stride, scale_stride;   // bytes from one expert's image to the next
};

hipError_t launch_mx_linear_fused(int format, const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s);

}  // namespace lora
