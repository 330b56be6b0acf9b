// mx_linear.hip -- launches of the product of blocks and a 4-bit weight.
#include "mx_linear_kernels.h"
#include "mx_slabs.h"

namespace lora {

namespace {

// Launch `go` over slabs of rows: row tiles of `rows` rows by column tiles of
// `tiles` times 16 features, `per` workgroups of `threads` each.
template <int DT, class F>
void by_row_slabs(const MxLinearArgs &a, int rows, int tiles, int per, int threads, F go)
{
    const int64_t cols = (a.w.d + 16 * tiles - 1) / (16 * tiles);
    for_slabs(a.n_rows, slab_rows(rows, cols * per, threads), [&](int64_t r, int64_t n) {
        MxLinearArgs b = a;
        b.n_rows = n;
        b.q = a.q + r * a.ldq;
        b.s = a.s + r * a.lds;
        b.y = static_cast<char *>(a.y) + r * a.ldy * (DT == DT_F32 ? 4 : 2);
        go(b, (int)((n + rows - 1) / rows), (int)cols);
    });
}

template <int DT, int FMT, int MT, int NT> void linear_direct(const MxLinearArgs &a, hipStream_t s)
{
    // one tile a workgroup: both of every pair
    constexpr int kPer = NT == 1 ? 2 : 1;
    constexpr int kThreads = 64 * kDirectWaves;
    by_row_slabs<DT>(a, 16 * MT, NT * kPer, kPer, kThreads, [&](const MxLinearArgs &b, int rows, int cols) {
        mx_linear_direct_kernel<MxPlain, DT, FMT, MT, NT>
            <<<dim3((uint32_t)rows * cols * kPer), kThreads, 0, s>>>(b, mx_grid(rows, cols * kPer), MxPlain{});
    });
}

template <int DT, int FMT, int RW, int MT, int FW, int NT, int KW>
void linear_tiles(const MxLinearArgs &a, hipStream_t s)
{
    typedef MxTile<DT, FMT, RW, MT, FW, NT, KW> T;
    constexpr int kThreads = 64 * T::kSet * KW;
    by_row_slabs<DT>(a, T::kRows, T::kTiles, 1, kThreads, [&](const MxLinearArgs &b, int rows, int cols) {
        mx_linear_tile_kernel<MxPlain, DT, FMT, RW, MT, FW, NT, KW>
            <<<dim3((uint32_t)rows * cols), kThreads, 0, s>>>(b, mx_grid(rows, cols), MxPlain{});
    });
}

// The smallest tile that gives every CU at most one workgroup: fewer, larger
// workgroups leave CUs idle, more of them repeat reads (us, 1024 wavefronts'
// worth of k splits on either side; e4m3 on 256 CUs):
//   24 x 4096 x 4096     16x16 (512 workgroups) 7.2    16x32 (256)  5.6   16x64 (128)  6.1
//   64 x 4096 x 4096     16x32 (512)            8.1    16x64 (256)  6.6   64x64  (64) 10.0
//   96 x 4096 x 4096     16x64 (384)           11.2    32x64 (192)  8.2   64x64 (128) 10.1
//   128 x 4096 x 6144    32x64 (384)           15.2    64x64 (192) 10.6   64x128 (96) 13.9
//   512 x 14336 x 4096   64x64 (512)           57      64x128 (256) 44    128x256 (64) 147
// (up to 16 rows twice as many: larger tiles only add features there;
//   8 x 4096 x 28672     16x64 (448)           12.2    64x128 (224) 15.3).
// Beyond one round, 64x128 with k in one piece, four workgroups a CU (three in 4
// bits, whose two chunks a stage take 51 KB of LDS), until the largest tile's
// rounds (two workgroups a CU in 8 bits, one in 4 bits) are well filled (a CU left
// with one of two runs it in 4/7 of the pair's time):
//   1024 x 4096 x 6144   64x128 39.0   128x256 (192 workgroups) 47.6
//   20000 x 1024 x 1024  64x128 35.7   128x256 (628)            38.8
//   4096 x 4096 x 6144   64x128 134    128x256 (768)            126
//   35422 x 4096 x 6144  64x128 1169   128x256 (6672)           1035
// and in 4 bits
//   35422 x 512 x 512    64x128 20.5   256x256 (278) 27.3
//   2048 x 4096 x 6144   64x128 43.2   256x256 (192) 38.0
//   2048 x 4096 x 4096   64x128 33.9   256x256 (128) 36.2   128x128 (512) 28.7
template <int DT, int FMT> void linear_pick(const MxLinearArgs &a, hipStream_t s)
{
    const int64_t cu = a.n_cu;
    auto grid = [&](int rows, int features) {
        return (a.n_rows + rows - 1) / rows * ((a.w.d + features - 1) / features);
    };
    const int64_t few = a.n_rows <= 16 ? 2 * cu : cu;
    if (grid(16, 16) <= few)
        return linear_direct<DT, FMT, 1, 1>(a, s);
    if (grid(16, 32) <= few)
        return linear_direct<DT, FMT, 1, 2>(a, s);
    if (grid(16, 64) <= few)
        return linear_direct<DT, FMT, 1, 4>(a, s);
    if (grid(32, 64) <= cu)
        return linear_direct<DT, FMT, 2, 4>(a, s);
    if (grid(64, 64) <= cu)
        return linear_tiles<DT, FMT, 4, 1, 1, 4, 4>(a, s);
    if constexpr (FMT == LORA_MX_E4M3) {
        if (grid(64, 128) <= cu)
            return linear_tiles<DT, FMT, 4, 1, 1, 8, 4>(a, s);
        const int64_t n = grid(128, 256), rounds = n / (2 * cu), left = n % (2 * cu);
        const int64_t sevenths = 7 * rounds + (left > cu ? 7 : left > 0 ? 4 : 0);
        if (rounds > 0 && n * 7 * 100 >= sevenths * 2 * cu * 82)
            return linear_tiles<DT, FMT, 2, 4, 2, 8, 1>(a, s);
    } else {
        if (grid(64, 128) <= cu)   // two chunks a stage: four sets' slots would not fit LDS
            return linear_tiles<DT, FMT, 4, 1, 1, 8, 2>(a, s);
        const int64_t n = grid(256, 256);
        if (n * 100 >= (n + cu - 1) / cu * cu * 70)
            return linear_tiles<DT, FMT, 4, 4, 2, 8, 1>(a, s);
        if (grid(128, 128) >= 2 * cu)
            return linear_tiles<DT, FMT, 8, 1, 1, 8, 1>(a, s);
    }
    linear_tiles<DT, FMT, 4, 1, 1, 8, 1>(a, s);
}

}  // namespace

hipError_t launch_mx_linear(int dtype, int format, const MxLinearArgs &a, hipStream_t s)
{
    if (dtype == DT_F32 && format == LORA_MX_E4M3)
        linear_pick<DT_F32, LORA_MX_E4M3>(a, s);
    else if (dtype == DT_F32)
        linear_pick<DT_F32, LORA_MX_E2M1>(a, s);
    else if (format == LORA_MX_E4M3)
        linear_pick<DT_BF16, LORA_MX_E4M3>(a, s);
    else
        linear_pick<DT_BF16, LORA_MX_E2M1>(a, s);
    return hipGetLastError();
}

}  // namespace lora
