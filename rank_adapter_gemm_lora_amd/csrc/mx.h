// mx.h -- host-side structures of the microscaled (MX) operators and the
// launchers of their kernels.  Not part of the public ABI (include/lora.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "mx_slabs.h"

namespace lora {

constexpr int64_t kMxMaxK = (int64_t)1 << 20;       // inputs of a row in blocks
constexpr int64_t kMxMaxNormK = (int64_t)1 << 16;   // a norm's row stays in one workgroup's registers
constexpr int64_t kMxMaxBlockNormK = (int64_t)1 << 15;   // the same, in 64 bits
constexpr int64_t kMxMaxD = (int64_t)1 << 22;
constexpr int64_t kMxMaxRows = (int64_t)1 << 30;

constexpr int kMxChunk = 128;   // k of one matrix-core product; code rows are padded to it
constexpr int kMxPadRows = 256; // weight images are padded to this many output features

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as one 64-bit multiply and a shift:
// with 2^(s-1) < d <= 2^s and m = floor(2^(31+s) / d) + 1 (32 bits), m d
// exceeds 2^(31+s) by at most d <= 2^s, so n m / 2^(31+s) exceeds n / d by less
// than 2^31 2^s / (2^(31+s) d) = 1 / d, which never carries past an integer.
struct MxDiv {
    uint32_t m, d;
    int sh;
};
inline MxDiv mx_div(uint32_t d)
{
    int s = 0;
    while (((uint64_t)1 << s) < d)
        ++s;
    return MxDiv{(uint32_t)(((uint64_t)1 << (31 + s)) / d + 1), d, 31 + s};
}

// One matrix in blocks: rows of codes and of scales.
struct MxBlocks {
    uint8_t *q;
    int64_t ldq;
    uint8_t *s;
    int64_t lds;
};

// The elementwise kernels: thread i of a launch takes 8 elements, unit i % units
// of row i / units; a row has units = (k rounded up to 128) / 8 of them.
struct MxRowArgs {
    const void *x;       // quantise: [rows][ldx]; swiglu: gate and up; dequantise: not read
    int64_t ldx;
    void *out;           // dense output (dequantise, swiglu), or null
    int64_t ldo;
    MxBlocks b;          // blocks written (dequantise: read); b.q null: none
    int64_t k;
    int64_t row0;        // first row of this launch
    uint32_t n_units;    // rows of this launch * units
    MxDiv div;           // by units
};
hipError_t launch_mx_quantize(int dtype, int format, MxRowArgs a, int64_t n_rows, hipStream_t s);
hipError_t launch_mx_dequantize(int dtype, int format, MxRowArgs a, int64_t n_rows, hipStream_t s);
hipError_t launch_swiglu_mx(int dtype, MxRowArgs a, int64_t n_rows, hipStream_t s);

struct MxNormArgs {
    const void *x;
    int64_t ldx;
    const void *res;     // or null
    int64_t ldr;
    const void *weight;
    double eps;
    double inv_k;        // 1 / k
    void *h;             // or null
    int64_t ldh;
    void *out;           // or null
    int64_t ldo;
    MxBlocks b;          // b.q null: not wanted
    int64_t row0;        // first row of this launch
    int64_t n_rows;
    int64_t k;
};
hipError_t launch_rmsnorm_mx(int dtype, const MxNormArgs &a, hipStream_t s);

struct MxBlockNormArgs {
    const void *y;
    int64_t ldy;
    const void *res;     // or null
    int64_t ldr;
    const void *post;    // or null: y stands as it is
    const void *gate;    // or null
    int64_t ldg;         // 0: one row for all
    const void *pre;     // or null: h alone
    double scale, eps;
    double inv_k;        // 1 / k
    void *h;             // or null
    int64_t ldh;
    void *out;           // or null
    int64_t ldo;
    MxBlocks b;          // b.q null: not wanted
    int64_t row0;        // first row of this launch
    int64_t n_rows;
    int64_t k;
};
hipError_t launch_block_norm_mx(int dtype, const MxBlockNormArgs &a, hipStream_t s);

// The weight image.  Output features are cut into tiles of 16, k into chunks of
// 128; per (tile, chunk) the codes are one kilobyte in matrix-core operand
// order: lane l = 16 g + r holds the 32 codes of k 32 g .. + 31 (16 bytes) of
// the feature in row r, which is block g of the chunk.  A pair of tiles shares
// 32 features: row 4 g + i of tile 2 p + h is feature 32 p + 8 g + 4 h + i, so
// that the lane that gets rows 4 g .. + 3 of both tiles' results has eight
// neighbouring features of a row.  The scales of four chunks are 256
// bytes: byte j of lane l's word is the scale of that lane's block in chunk j.
// Both are padded with zeros: features to kMxPadRows, scales to four chunks.
// All tiles of a chunk lie together, so that workgroups at the same k read
// neighbouring addresses (64 x 4096 x 28672 in 4 bits 13.8 us; with all chunks
// of a tile together, a power of two apart, 14.5 us).
struct MxImage {
    uint8_t *codes;      // [chunks][tiles][64][16]
    uint8_t *scales;     // [chunks / 4, rounded up][tiles][64][4]
    int64_t d;           // features of the image
    int64_t k;
    int64_t half;        // 0; or outputs of a gated weight, whose rows are the gates' and then the others'
    int tiles;
    int chunks;
};
// Features of a gated weight's image: 32 gates and the 32 values that they
// gate by turns, so that a lane that has the sums of eight gates has those of
// their values in the next pair of tiles.
inline int64_t mx_gated_features(int64_t half) { return (half + 31) / 32 * 64; }
// From dense rows (src: dtype) or from rows in e2m1 blocks (dtype < 0: b).
hipError_t launch_mx_image(int dtype, const void *src, int64_t ldw, const MxBlocks &b,
                           const MxImage &w, hipStream_t s);

struct MxLinearArgs {
    MxImage w;
    const uint8_t *q;
    int64_t ldq;
    const uint8_t *s;
    int64_t lds;
    void *y;
    int64_t ldy;
    int64_t n_rows;
    int n_cu;
};
hipError_t launch_mx_linear(int dtype, int format, const MxLinearArgs &a, hipStream_t s);

}  // namespace lora

struct lora_mx_weight {
    int device;
    int n_cu;
    int loaded;
    lora::MxImage w;
};
