// mx_fused.hip -- launches of the product of blocks and a 4-bit weight with an
// epilogue.
#include "mx_linear_kernels.h"
#include "mx_slabs.h"

namespace lora {

namespace {

typedef MxFused<false, false> Job;

// Launch `go` over slabs of rows: row tiles of `rows` rows by column tiles of
// `tiles` times 16 features, one workgroup of `threads` each.
template <class F>
void fused_slabs(const MxLinearArgs &a, const MxEpilogue &e, int rows, int tiles, int threads, F go)
{
    const int64_t cols = (a.w.d + 16 * tiles - 1) / (16 * tiles), size = e.dtype == DT_F32 ? 4 : 2;
    for_slabs(a.n_rows, slab_rows(rows, cols, threads), [&](int64_t r, int64_t n) {
        MxLinearArgs b = a;
        b.n_rows = n;
        b.q = a.q + r * a.ldq;
        b.s = a.s + r * a.lds;
        Job j;
        static_cast<MxEpilogue &>(j) = e;
        if (e.y)
            j.y = static_cast<char *>(e.y) + r * e.ldy * size;
        if (e.res)
            j.res = static_cast<const char *>(e.res) + r * e.ldr * size;
        if (e.b.q) {
            j.b.q = e.b.q + r * e.b.ldq;
            j.b.s = e.b.s + r * e.b.lds;
        }
        go(b, mx_grid((int)((n + rows - 1) / rows), (int)cols), j);
    });
}

template <int FMT, int MT, int NT> void fused_direct(const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s)
{
    constexpr int kThreads = 64 * kDirectWaves;
    fused_slabs(a, e, 16 * MT, NT, kThreads, [&](const MxLinearArgs &b, const MxGrid &g, const Job &j) {
        mx_linear_direct_kernel<Job, 0, FMT, MT, NT><<<dim3((uint32_t)g.rows * g.cols), kThreads, 0, s>>>(b, g, j);
    });
}

template <int FMT, int RW, int MT, int FW, int NT, int KW>
void fused_tiles(const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s)
{
    typedef MxTile<0, FMT, RW, MT, FW, NT, KW> T;
    constexpr int kThreads = 64 * T::kSet * KW;
    fused_slabs(a, e, T::kRows, T::kTiles, kThreads, [&](const MxLinearArgs &b, const MxGrid &g, const Job &j) {
        mx_linear_tile_kernel<Job, 0, FMT, RW, MT, FW, NT, KW><<<dim3((uint32_t)g.rows * g.cols), kThreads, 0, s>>>(b, g, j);
    });
}

// The tile by the same rule as the plain product's (linear_pick, with both
// sides' times), whose sums these are, bit for bit; 16 features alone would
// part a block of 32 outputs, so the smallest tile is 16 x 32.  With weights past
// the last-level cache (us; picked, and the nearest other tile):
//   1 x 4096 x 6144       16x32 5.8          16x64 7.0
//   64 x 4096 x 14336     64x64 15.3         32x64 18.2
//   512 x 4096 x 14336    64x128 50.2        128x256 54.0   (gelu into blocks 57)
//   2048 x 4096 x 14336   64x128 165         128x256 168
//   16384 x 14336 x 4096  128x256 1110 - 1150, 1.7 PFLOP/s, the matrix cores busy 78 %
//                         of the cycles at the clock that the card's power leaves
template <int FMT> void fused_pick(const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s)
{
    const int64_t cu = a.n_cu;
    auto grid = [&](int rows, int features) {
        return (a.n_rows + rows - 1) / rows * ((a.w.d + features - 1) / features);
    };
    const int64_t few = a.n_rows <= 16 ? 2 * cu : cu;
    if (grid(16, 32) <= few)
        return fused_direct<FMT, 1, 2>(a, e, s);
    if (grid(16, 64) <= few)
        return fused_direct<FMT, 1, 4>(a, e, s);
    if (grid(32, 64) <= cu)
        return fused_direct<FMT, 2, 4>(a, e, s);
    if (grid(64, 64) <= cu)
        return fused_tiles<FMT, 4, 1, 1, 4, 4>(a, e, s);
    if constexpr (FMT == LORA_MX_E4M3) {
        if (grid(64, 128) <= cu)
            return fused_tiles<FMT, 4, 1, 1, 8, 4>(a, e, s);
        const int64_t n = grid(128, 256), rounds = n / (2 * cu), left = n % (2 * cu);
        const int64_t sevenths = 7 * rounds + (left > cu ? 7 : left > 0 ? 4 : 0);
        if (rounds > 0 && n * 7 * 100 >= sevenths * 2 * cu * 82)
            return fused_tiles<FMT, 2, 4, 2, 8, 1>(a, e, s);
    } else {
        if (grid(64, 128) <= cu)
            return fused_tiles<FMT, 4, 1, 1, 8, 2>(a, e, s);
        const int64_t n = grid(256, 256);
        if (n * 100 >= (n + cu - 1) / cu * cu * 70)
            return fused_tiles<FMT, 4, 4, 2, 8, 1>(a, e, s);
        if (grid(128, 128) >= 2 * cu)
            return fused_tiles<FMT, 8, 1, 1, 8, 1>(a, e, s);
    }
    fused_tiles<FMT, 4, 1, 1, 8, 1>(a, e, s);
}

}  // namespace

hipError_t launch_mx_linear_fused(int format, const MxLinearArgs &a, const MxEpilogue &e, hipStream_t s)
{
    if (format == LORA_MX_E4M3)
        fused_pick<LORA_MX_E4M3>(a, e, s);
    else
        fused_pick<LORA_MX_E2M1>(a, e, s);
    return hipGetLastError();
}

}  // namespace lora
