// mx_experts.hip -- launches of the experts' products: rows grouped by expert,
// groups of any sizes, one launch.  The kernels are those of the plain product;
// a workgroup takes its row tile from the plan's list of tiles of its height,
// so that a tile has rows of one expert, and the rows of X from the pairs at its
// positions.  The grid is the most tiles that so many pairs can need; how many
// there are is read on the device, and workgroups without a tile end at once.
#include "mx_linear_kernels.h"
#include "mx_slabs.h"

namespace lora {

namespace {

// Launch `go` over slabs of row tiles of 16 << height rows.
template <class JOB, class F>
void tile_slabs(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, int height, int tiles, int threads, F go)
{
    const int64_t cols = (a.w.d + 16 * tiles - 1) / (16 * tiles);
    for_slabs(moe_tile_bound(g.pairs, g.experts, moe_height_shift(height)), slab_rows(1, cols, threads), [&](int64_t t, int64_t n) {
        JOB j;
        static_cast<MxEpilogue &>(j) = e;
        j.tiles = g.l.tiles[height];
        j.n_tiles = g.l.n_tiles + height;
        j.tile0 = (int)t;
        j.order = g.by_row ? g.l.order : nullptr;
        j.by_top_k = mx_div((uint32_t)g.top_k);
        j.pairs = (int)g.pairs;
        j.in_rows = (int)(g.pairs / g.top_k);
        go(mx_grid((int)n, (int)cols), j);
    });
}

template <bool GATED, int FMT, int MT, int NW>
void experts_direct(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    typedef MxFused<true, GATED> Job;
    tile_slabs<Job>(a, e, g, MT - 1, 4, 64 * NW, [&](const MxGrid &grid, const Job &j) {
        mx_linear_direct_kernel<Job, 0, FMT, MT, 4, NW><<<dim3((uint32_t)grid.rows * grid.cols), 64 * NW, 0, s>>>(a, grid, j);
    });
}

template <bool GATED, int FMT, int RW, int MT, int FW, int NT, int KW>
void experts_tiles(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    typedef MxFused<true, GATED> Job;
    typedef MxTile<0, FMT, RW, MT, FW, NT, KW> T;
    constexpr int kThreads = 64 * T::kSet * KW, kHeight = T::kRows == 64 ? 2 : 3;
    static_assert(T::kRows == 16 << kHeight, "a height that the plan lists");
    tile_slabs<Job>(a, e, g, kHeight, T::kTiles, kThreads, [&](const MxGrid &grid, const Job &j) {
        mx_linear_tile_kernel<Job, 0, FMT, RW, MT, FW, NT, KW><<<dim3((uint32_t)grid.rows * grid.cols), kThreads, 0, s>>>(a, grid, j);
    });
}

// How the rows fall to the experts is not known here, so the tile is chosen for
// equal groups: `mean` rows each, of as many experts as can have any.
//
// Few rows an expert: the stream of their weights is what counts.  Straight into
// registers, 16 or 32 rows, and of the wavefronts that split k as few as keep
// the chip full, so that each has a long run of k; from some 24 rows on, 64x128
// through LDS, whose wavefronts without rows leave the matrix cores to others
// (us, on weights past the last-level cache; rows of the batch, top 8 of 64; 4096
// -> 2 x 1024 gated, e4m3):
//     rows  mean    16x64 of 8 / 4 / 2      32x64 of 4 / 2       64x128
//     1     1       10.5  11.0  12.1        10.5  11.1            20.7
//     16    2       49.0  39.2  40.2        37.8  40.4            46.3
//     64    8         -   51.1  49.4        46.1  49.4            48.8
//     128   16        -   65.4  62.0        55.1  57.3            64.4
//     192   24        -   81.3  77.1        66.4  69.8            72.4
//     256   32        -   94.1  86.8        73.8  77.6            72.9
//     320   40        -  111.3  99.3        86.1  87.7            78.6
// (64 rows, 285 MB of weights: 5.6 TB/s by the kernel taken, 16x64 of 4, and 6.2 by the
// 32x64 beside it: up to a mean of 8 the rule takes 16x64, which these figures, of k =
// 4096 in 8 bits alone, do not bear out there; top 2 of 8, 4096 -> 2 x 14336, mean 32: 140
// and 107); and with k = 1024, two groups of four chunks, 1024 -> 4096:
//     64    8         -   35.2  27.5        34.5  31.9            29.2
//     128   16        -   47.3  34.2        41.0  36.8            32.1
//     256   32        -   72.8  50.1        56.6  45.9            38.3
// (2048 -> 2 x 512, top 4, 8 rows: 16x64 of 4 6.4, 32x64 of 4 7.9).
//
// Small grids (few experts): the smallest tile that leaves every CU at most
// half a workgroup, as groups are uneven (4 experts, top 2, 4096 -> 2 x 1024):
//     rows  mean    16x64 of 8   32x64 of 4   64x64, k in 4   64x128, k in 2   64x128
//     32    16       7.8          8.6         12.0              -                -
//     64    32      13.2         10.0         12.2            17.4             20.7
//     128   64        -          14.4         12.6            17.6             20.8
//     256   128       -          20.4         22.0            18.1             21.2
//     512   256       -          30.3         31.3            25.6             24.1
// (top 2 of 8, 14336 -> 4096, mean 32: 32x64 66.7, 64x128 with k in 2 80.5).
//
// Beyond, 64x128; and in grids that stay full with them the larger tile (128x256, in 4
// bits 128x128), whose unfilled tiles cost more the fewer rows an expert has: from 512
// rows an expert on, in 4 bits from 256 (64x128 / larger):
//     mean                      256        384        512        640        768        1024       2048
//     top 8 of 64, 4096 -> 2 x 1024
//       e4m3                 212 / 221  294 / 291  377 / 371  466 / 454  550 / 536  721 / 694  1404 / 1354
//       e2m1                 135 / 135  181 / 178  232 / 220  284 / 265  333 / 304  423 / 400   812 / 755
//     top 8 of 64, 1024 -> 4096, fp32
//       e4m3                 120 / 133  171 / 171  223 / 224  276 / 267  326 / 318  429 / 414   874 / 816
//       e2m1                  84 /  80  114 / 108  146 / 137  181 / 169  215 / 198  283 / 266   554 / 505
// and under eight of its workgroups a CU (e4m3, top 2 of 16; the last column has them):
//     2048 -> 4096            53 /  68   76 /  86   98 / 107  120 / 125  144 / 149  190 / 192   371 / 364
//     4096 -> 2 x 1024        59 /  81   81 /  84  102 / 124  122 / 125  144 / 154  186 / 199   354 / 352
template <bool GATED, int FMT> void experts_pick(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    const int64_t cu = a.n_cu, used = g.pairs < g.experts ? g.pairs : g.experts, mean = (g.pairs + used - 1) / used;
    const int groups = (a.w.chunks + 3) / 4;   // of four chunks, what a wavefront takes at a time
    auto grid = [&](int rows, int features) {
        return used * ((mean + rows - 1) / rows) * ((a.w.d + features - 1) / features);
    };
    if (mean <= 8 || (mean <= 12 && groups < 4) || (mean <= 16 && grid(16, 64) <= cu) || grid(16, 64) <= cu / 2) {
        if (groups >= 8 && grid(16, 64) <= cu)
            return experts_direct<GATED, FMT, 1, 8>(a, e, g, s);
        if (groups >= 4)
            return experts_direct<GATED, FMT, 1, 4>(a, e, g, s);
        return experts_direct<GATED, FMT, 1, 2>(a, e, g, s);
    }
    if ((mean <= 24 && groups >= 4) || (mean <= 32 && grid(64, 128) <= cu) || grid(32, 64) <= cu / 2) {
        if (groups >= 4)
            return experts_direct<GATED, FMT, 2, 4>(a, e, g, s);
        return experts_direct<GATED, FMT, 2, 2>(a, e, g, s);
    }
    if (grid(64, 64) <= cu / 2)
        return experts_tiles<GATED, FMT, 4, 1, 1, 4, 4>(a, e, g, s);
    if (grid(64, 128) <= cu / 2)
        return experts_tiles<GATED, FMT, 4, 1, 1, 8, 2>(a, e, g, s);
    if constexpr (FMT == LORA_MX_E4M3) {
        if (mean >= 512 && grid(128, 256) >= 8 * cu)
            return experts_tiles<GATED, FMT, 2, 4, 2, 8, 1>(a, e, g, s);
    } else {
        if (mean >= 256 && grid(128, 128) >= 8 * cu)
            return experts_tiles<GATED, FMT, 8, 1, 1, 8, 1>(a, e, g, s);
    }
    experts_tiles<GATED, FMT, 4, 1, 1, 8, 1>(a, e, g, s);
}

}  // namespace

hipError_t launch_mx_experts(int format, bool gated, const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    if (gated && format == LORA_MX_E4M3)
        experts_pick<true, LORA_MX_E4M3>(a, e, g, s);
    else if (gated)
        experts_pick<true, LORA_MX_E2M1>(a, e, g, s);
    else if (format == LORA_MX_E4M3)
        experts_pick<false, LORA_MX_E4M3>(a, e, g, s);
    else
        experts_pick<false, LORA_MX_E2M1>(a, e, g, s);
    return hipGetLastError();
}

}  // namespace lora
