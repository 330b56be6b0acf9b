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
    const int32_t *order;    // pair at a position, whose row is X's; null: X is in grouped order
    MxDiv by_top_k;
    int pairs, in_rows;      // rows of the outputs and of X: nothing beyond is touched,
                             // whatever grouping the plan holds by now
    int64_t code_stride, scale_stride;   // bytes from one expert's image to the next
};

// The batch's grouping, from which the products take their row tiles.
struct MxGroups {
    MoeLists l;
    int64_t pairs;
    int experts, top_k;
    bool by_row;         // X is in the batch's own rows
};
hipError_t launch_mx_experts(int format, bool gated, const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s);
hipError_t launch_mx_linear_fused(int format, const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s);

}  // namespace lora

struct lora_mx_experts {
    int device;
    int n_cu;
    int experts;
    int gated;
    int64_t rows;        // of an expert's weight: outputs, or twice as many where gated
    int64_t d;           // outputs
    lora::MxImage w;     // the first expert's image
    int64_t code_stride, scale_stride;
    int n_loaded;
    unsigned char loaded[LORA_MAX_EXPERTS];
};
