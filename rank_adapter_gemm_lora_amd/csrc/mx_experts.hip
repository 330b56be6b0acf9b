// mx_experts.hip -- launches of the experts' products: rows grouped by expert,
// groups of any sizes, one launch.  The kernels are those of the plain product;
// a workgroup takes its row tile from the plan's list of tiles of its height,
// so that a tile has rows of one expert, and the rows of X through the plan's
// row numbers.  The grid is the most tiles that so many pairs can need; how many
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
        j.rows = g.by_row ? g.l.row : nullptr;
        go(mx_grid((int)n, (int)cols), j);
    });
}

template <bool GATED, int FMT, int MT, int NT>
void experts_direct(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    typedef MxFused<true, GATED> Job;
    constexpr int kThreads = 64 * kDirectWaves;
    tile_slabs<Job>(a, e, g, MT - 1, NT, kThreads, [&](const MxGrid &grid, const Job &j) {
        mx_linear_direct_kernel<Job, 0, FMT, MT, NT><<<dim3((uint32_t)grid.rows * grid.cols), kThreads, 0, s>>>(a, grid, j);
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

template <bool GATED, int FMT> void experts_pick(const MxLinearArgs &a, const MxEpilogue &e, const MxGroups &g, hipStream_t s)
{
    const int64_t cu = a.n_cu, used = g.pairs < g.experts ? g.pairs : g.experts, mean = (g.pairs + used - 1) / used;
    auto grid = [&](int rows, int features) {
        return used * ((mean + rows - 1) / rows) * ((a.w.d + features - 1) / features);
    };
    if (mean <= 16)
        return experts_direct<GATED, FMT, 1, 4>(a, e, g, s);
    if (mean <= 32)
        return experts_direct<GATED, FMT, 2, 4>(a, e, g, s);
    if (grid(64, 128) <= cu)
        return experts_tiles<GATED, FMT, 4, 1, 1, 8, FMT == LORA_MX_E4M3 ? 4 : 2>(a, e, g, s);
    if constexpr (FMT == LORA_MX_E4M3) {
        if (mean >= 256 && grid(128, 256) >= 2 * cu)
            return experts_tiles<GATED, FMT, 2, 4, 2, 8, 1>(a, e, g, s);
    } else {
        if (mean >= 256 && grid(128, 128) >= 2 * cu)
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
