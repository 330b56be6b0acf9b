// mx_linear_kernels.h -- the kernels of y = X W^T with X in e4m3 or e2m1 blocks and W in e2m1 blocks
// (the weight image).  W is the row operand of the matrix instruction and X the
// column operand, so a lane's four results are four neighbouring outputs of one
// row of X: D row 4 g + i, column m in lane l = 16 g + m.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes codes and scales as they are.  Of a
// chunk of 128 k, lane l holds the 32 codes k 32 g .. + 31 of an e2m1 operand
// (its block g), or k 16 g .. + 15 and 64 + 16 g .. + 15 of an e4m3 operand; in
// both cases its scale byte is that of block g.
//
// The instruction aligns the products of each group of eight k to the largest
// exponent sum E (of the two elements' exponents) in the group and drops what
// lies below 2^(E - 13) (probed: 448 * 6 keeps 2^-3 and loses 2^-4, 256 * 1
// keeps 2^-5 and loses 2^-6); group sums and the accumulator meet in fp32.
// e2m1 times e2m1 spans 2^-2 .. 36, so every bit is kept.  e4m3 times e2m1
// spans 2^-10 .. 2688, so up to 5e-5 of the result would be lost.  Sums here
// are held in fp32, so an e4m3 operand is taken as the sum of two, split at
// bit 6 of the code: |x| >= 2 (last bit 2^-2, E <= 10: products keep 2^-3) and
// |x| < 2 (last bit 2^-9, E <= 2: products keep 2^-11, need 2^-10).  Each of the
// two products is exact inside its groups; two instructions of 32 cycles cost
// what the four bf16 instructions on widened codes do, at a quarter of the LDS
// traffic and with no widening of W.
//
// What becomes of the sums is the job's: stored as they are (MxPlain), or taken
// through an epilogue, of one weight or of a batch's experts (mx_epilogue.h).
#pragma once

#include <type_traits>
#include <utility>

#include "mx_device.h"
#include "mx_epilogue.h"

namespace lora {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFp8 = 0, kFp4 = 4;   // operand format codes of the instruction

// One X operand of a chunk: a lane's codes as the instruction takes them.
template <int FMT> struct MxOperand;
template <> struct MxOperand<LORA_MX_E2M1> {
    i32x8_t v;
    __device__ __forceinline__ void set(u32x4_t c, u32x4_t)
    {
        v = i32x8_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
    }
};
template <> struct MxOperand<LORA_MX_E4M3> {
    i32x8_t v, lo;   // codes of |x| >= 2 and of the rest, zeros in the other's places
    __device__ __forceinline__ void set_word(int i, u32x4_t a, u32x4_t b)
    {
        const uint32_t c = i < 4 ? a[i & 3] : b[i & 3];
        // byte masks from bit 6: moved to the sign of bytes 1, 3, 5 and 7,
        // which selectors 8 .. 11 of the byte permutation spread
        const uint32_t h = c & __builtin_amdgcn_perm(c << 1, c << 9, 0x0b090a08u);
        v[i] = (int)h;
        lo[i] = (int)(c ^ h);
    }
    __device__ __forceinline__ void set(u32x4_t a, u32x4_t b)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            set_word(i, a, b);
    }
};

// acc += W tile x X codes; J: the byte of the W scale word that holds the
// chunk's scale (X's is in byte 0).  Scales have to be in vector registers of
// their lanes: both come from per-lane loads.
template <int FMT, int J>
__device__ __forceinline__ f32x4_t mx_mfma(u32x4_t w, uint32_t sw, i32x8_t x, uint32_t sx, f32x4_t acc)
{
    const i32x8_t a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        a, x, acc, kFp4, FMT == LORA_MX_E4M3 ? kFp8 : kFp4, J, (int)sw, 0, (int)sx);
}

// Neighbouring outputs of one row.
template <int DT>
__device__ __forceinline__ void mx_store4(void *y, int64_t idx, f32x4_t v)
{
    if constexpr (DT == DT_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + idx) = make_float4(v.x, v.y, v.z, v.w);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + idx) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}
template <int DT>
__device__ __forceinline__ void mx_store8(void *y, int64_t idx, f32x4_t u, f32x4_t v)
{
    const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    Vec8<DT>::store(y, idx, f);
}

// Row and column tile of a workgroup.  Workgroups of one XCD walk bands of eight
// row tiles, so that its L2 serves the X rows and W tiles that they share; the
// divisions' multipliers come from the host.
struct MxGrid {
    int rows, cols;
    MxDiv band;   // by 8 cols
    MxDiv last;   // by the last band's row tiles, where they are fewer than eight
    MxDiv by_cols;
};
inline MxGrid mx_grid(int rows, int cols)
{
    return MxGrid{rows, cols, mx_div(8u * cols), mx_div(rows % 8 ? rows % 8 : 8), mx_div(cols)};
}
struct MxPlace {
    int row, col;
};
__device__ __forceinline__ MxPlace mx_place(const MxGrid &g)
{
    const uint32_t id = (uint32_t)xcd_major(blockIdx.x, gridDim.x);
    const uint32_t band = mx_div_of(id, g.band), in = id - band * g.band.d;
    if ((int)band * 8 + 8 <= g.rows)
        return MxPlace{(int)(band * 8 + (in & 7)), (int)(in >> 3)};
    const uint32_t col = mx_div_of(in, g.last);
    return MxPlace{(int)(band * 8 + in - col * g.last.d), (int)col};
}

// The same of one expert's row tile: how many there are is the batch's, so the
// place is taken among the workgroups that have one; the others have no work
// (row < 0).  The workgroups with work then lie on all XCDs.
__device__ __forceinline__ MxPlace mx_place_among(const MxGrid &g, int rows)
{
    const uint32_t n = (uint32_t)rows * g.cols;
    if (blockIdx.x >= n)
        return MxPlace{-1, 0};
    const uint32_t id = (uint32_t)xcd_major(blockIdx.x, n);
    const uint32_t band = mx_div_of(id, g.band), in = id - band * g.band.d;
    if ((int)band * 8 + 8 <= rows)
        return MxPlace{(int)(band * 8 + (in & 7)), (int)(in >> 3)};
    const uint32_t last = rows & 7, col = in / last;
    return MxPlace{(int)(band * 8 + in - col * last), (int)col};
}

// A workgroup's work: rows [row0, end) of the batch, from image column `col` of
// the weight at w.
struct MxWork {
    int row0, end, col, expert;
    bool none;
};
// BANDS: the place is taken in bands, among the tiles that there are; otherwise
// all columns of a tile come one after the other, whatever their number, so that
// the tile and the number are read at once (few rows: an expert's weights are
// read by one or two tiles, and the start counts).
template <bool BANDS, class JOB>
__device__ __forceinline__ MxWork mx_work(MxLinearArgs &a, const MxGrid &grid, const JOB &job, int tile_rows)
{
    if constexpr (JOB::kGrouped) {
        const int first = job.tile0;
        MxPlace at;
        MoeTile t;
        if constexpr (BANDS) {
            at = mx_place_among(grid, max(min(*job.n_tiles - first, grid.rows), 0));
            if (at.row < 0)
                return MxWork{0, 0, 0, 0, true};
            t = job.tiles[first + at.row];
        } else {
            const int row = (int)mx_div_of(blockIdx.x, grid.by_cols);
            at = MxPlace{row, (int)(blockIdx.x - row * grid.cols)};
            t = job.tiles[first + row];
            if (first + row >= *job.n_tiles)
                return MxWork{0, 0, 0, 0, true};
        }
        a.w.codes += t.expert * job.code_stride;
        a.w.scales += t.expert * job.scale_stride;
        return MxWork{t.first, min(t.end, job.pairs), at.col, t.expert, t.first >= job.pairs};
    } else {
        const MxPlace at = mx_place(grid);
        return MxWork{at.row * tile_rows, (int)a.n_rows, at.col, 0, false};
    }
}
// Row of X that stands at a position; rows past the end repeat the last one.
template <class JOB> __device__ __forceinline__ uint32_t mx_source(const JOB &job, const MxWork &work, int r)
{
    const int at = min(r, work.end - 1);
    if constexpr (JOB::kGrouped)
        return job.order ? min(mx_div_of((uint32_t)job.order[at], job.by_top_k), (uint32_t)job.in_rows - 1) : (uint32_t)at;
    else
        return (uint32_t)at;
}

template <class F, int... I> __device__ __forceinline__ void mx_for(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void mx_for(F f)
{
    mx_for(f, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------ few rows, small grids
//
// One workgroup: 16 MT rows x 16 NT features; its wavefronts take groups of
// four chunks in turn, each for the whole tile, and are summed in wavefront
// order through LDS.  Operands go straight into registers (W in operand order,
// X as 16 rows' pieces of 16 bytes): nothing is shared between wavefronts, so
// there is no LDS traffic and no barrier in the loop.  A wavefront holds four
// chunks; each is refilled with the next group's as soon as it is multiplied.
// Bound by the stream of W and by what a launch costs: 1 x 4096 x 6144 4.1 us with
// its 13.4 MB in the caches and 5.9 us where 64 weights take turns (857 MB);
// 1 x 14336 x 4096 7.2 us (31 MB at 4.3 TB/s), 64 x 4096 x 4096 6.3 us, in the caches.
constexpr int kDirectWaves = 8;

template <int FMT, int MT, int NT> struct MxChunk {
    u32x4_t w[NT], x[MT][FMT == LORA_MX_E4M3 ? 2 : 1];
};

template <class JOB, int DT, int FMT, int MT, int NT, int NW = kDirectWaves>
__global__ __launch_bounds__(64 * NW, 2) void mx_linear_direct_kernel(MxLinearArgs a, MxGrid grid, JOB job)
{
    static_assert(!JOB::kFused || NT == 4 || (NT == 2 && !JOB::kGated), "blocks of 32 outputs lie in one workgroup");
    constexpr int kPair = NT > 1 ? 2 : 1, kParts = MT * NT / kPair;
    __shared__ f32x4_t part[NW][MT * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, m = lane & 15;
    const MxWork work = mx_work<false>(a, grid, job, 16 * MT);
    if (work.none)
        return;
    const int n_rows = work.end, row0 = work.row0;
    const int64_t tile0 = (int64_t)work.col * NT;
    const int chunks = a.w.chunks, groups = (chunks + 3) / 4;
    const uint8_t *xq[MT], *xs[MT], *wc[NT];
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const uint32_t r = mx_source(job, work, row0 + 16 * t + m);
        xq[t] = a.q + r * a.ldq + 16 * g;
        xs[t] = a.s + r * a.lds;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[t][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        wc[n] = a.w.codes + ((tile0 + n) * 64 + lane) * 16;
    const uint8_t *ws = a.w.scales + (tile0 * 64 + lane) * 4;

    MxChunk<FMT, MT, NT> ring[4];
    u32x4_t sx[MT], sxn[MT];
    uint32_t sw[NT], swn[NT];
    auto load = [&](auto J, int grp) {
        constexpr int j = decltype(J)::value;
        // past the end: the last chunk again, not multiplied
        const int64_t c = min(4 * grp + j, chunks - 1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            ring[j].w[n] = *reinterpret_cast<const u32x4_t *>(wc[n] + c * ((int64_t)a.w.tiles * 1024));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            ring[j].x[t][0] = *reinterpret_cast<const u32x4_t *>(xq[t] + c * (FMT == LORA_MX_E4M3 ? 128 : 64));
            if constexpr (FMT == LORA_MX_E4M3)
                ring[j].x[t][1] = *reinterpret_cast<const u32x4_t *>(xq[t] + c * 128 + 64);
        }
    };
    auto load_scales = [&](int grp) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
            sxn[t] = *reinterpret_cast<const u32x4_t *>(xs[t] + (int64_t)grp * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            swn[n] = *reinterpret_cast<const uint32_t *>(ws + ((int64_t)grp * a.w.tiles + n) * 256);
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int t = 0; t < MT; ++t)
            sx[t] = sxn[t];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            sw[n] = swn[n];
    };
    // products of one chunk; the next X tile's codes are split between them
    auto multiply = [&](auto J) {
        constexpr int j = decltype(J)::value;
        MxOperand<FMT> x, next;
        auto tile = [&](MxOperand<FMT> &o, int t, int i) {
            if constexpr (FMT == LORA_MX_E4M3)
                o.set_word(i, ring[j].x[t][0], ring[j].x[t][1]);
            else if (i == 0)
                o.set(ring[j].x[t][0], ring[j].x[t][0]);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i)
            tile(x, 0, i);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint32_t s = sx[t][j] >> (8 * g);
            constexpr int kParts = FMT == LORA_MX_E4M3 ? 2 * NT : NT;
#pragma unroll
            for (int n = 0; n < kParts; ++n) {
                if constexpr (FMT == LORA_MX_E4M3)
                    acc[t][n % NT] = mx_mfma<FMT, j>(ring[j].w[n % NT], sw[n % NT], n < NT ? x.v : x.lo, s, acc[t][n % NT]);
                else
                    acc[t][n] = mx_mfma<FMT, j>(ring[j].w[n], sw[n], x.v, s, acc[t][n]);
                if (t + 1 < MT) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 8 * n / kParts; i < 8 * (n + 1) / kParts; ++i)
                        tile(next, t + 1, i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            x = next;
        }
    };
    int grp = wave;
    if (grp < groups) {
        load_scales(grp);
        mx_for<4>([&](auto J) { load(J, grp); });
        for (; grp + NW < groups; grp += NW) {
            take_scales();
            load_scales(grp + NW);
            mx_for<4>([&](auto J) {
                multiply(J);
                load(J, grp + NW);
            });
        }
        take_scales();
        mx_for<4>([&](auto J) {
            if (4 * grp + decltype(J)::value < chunks)
                multiply(J);
        });
    }
    if constexpr (JOB::kFused) {
#pragma unroll
        for (int i = 0; i < MT * NT; ++i)
            part[wave][i][lane] = acc[i / NT][i % NT];
        __syncthreads();
        // unit u of a row's U: 8 outputs, four neighbouring lanes a block of 32
        constexpr int U = JOB::kGated ? NT : 2 * NT;
        static_assert(64 * NW % U == 0, "a thread's unit is the same in all of its rows");
        const int u = threadIdx.x % U;
        MxFinish<JOB> finish(job, work.expert, tile0 * 16 / (JOB::kGated ? 2 : 1) + 8 * u);
#pragma unroll 1
        for (int r = threadIdx.x / U; r < 16 * MT; r += 64 * NW / U) {
            auto sums = [&](int pair, float (&f)[8]) {
                f32x4_t v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        v[h] += part[w][(r >> 4) * NT + 2 * pair + h][16 * (u & 3) + (r & 15)];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = v[e >> 2][e & 3];
            };
            float f[8], up[8];
            if constexpr (JOB::kGated) {
                sums(u >> 2 << 1, f);
                sums((u >> 2 << 1) + 1, up);
            } else {
                sums(u >> 2, f);
            }
            finish.row(row0 + r, row0 + r < n_rows, f, up);
        }
        return;
    }
    // wavefront p % NW finishes part p: it keeps its own sums of it
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        if (p % NW == wave)
            continue;
#pragma unroll
        for (int i = kPair * p; i < kPair * (p + 1); ++i)
            part[wave][i][lane] = acc[i / NT][i % NT];
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        if (p % NW != wave)
            continue;
        f32x4_t v[kPair];
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
            const int f = kPair * p + i;
            v[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w)
                v[i] += w == p % NW ? acc[f / NT][f % NT] : part[w][f][lane];
        }
        const int r = row0 + 16 * (kPair * p / NT) + m;
        if constexpr (kPair == 2) {
            const int64_t o = (tile0 + kPair * p % NT) * 16 + 8 * g;
            if (r < n_rows && o < a.w.d)
                mx_store8<DT>(a.y, (int64_t)r * a.ldy + o, v[0], v[1]);
        } else {
            const int64_t o = (tile0 >> 1) * 32 + 8 * g + 4 * (tile0 & 1);
            if (r < n_rows && o < a.w.d)
                mx_store4<DT>(a.y, (int64_t)r * a.ldy + o, v[0]);
        }
    }
}

// ---------------------------------------------------------------- tiles
//
// One workgroup: RW x FW wavefronts of 16 MT rows x 16 NT features each, KW
// times over (each set of wavefronts takes a contiguous run of k; the sets'
// sums are added in a fixed order at the end).  k advances in stages of 128
// bytes of an X row: one chunk of e4m3, two of e2m1.  A stage's X rows and W
// tiles go global -> LDS directly into one of two slots, while the other is
// multiplied:
//   X: 16-byte unit u of a row sits at u ^ (row / 2 % 8), applied to the source
//      address, so that the operand reads (16 rows of one unit) spread over all
//      banks; the units of one row are one 128-byte line;
//   W: the image's kilobytes as they are.
// Slots are separate shared objects, named at compile time in each step: the
// compiler then sees that the copies in flight do not feed the reads.  One wait
// and one barrier a stage: the wait is for this wavefront's copies of the stage,
// the barrier for everybody's, and for everybody's reads of the slot refilled
// next (consumed by products issued before it).  The scales of four chunks are
// copied alike into a slot of their own, read at the first of their stages and
// refilled at the second (loaded into registers per chunk they cost every row's
// line again: 35422 x 4096 x 6144 1080 us for 1039).
//
// 35422 x 4096 x 6144 in e4m3: 1040 - 1100 us (1.6 - 1.7 PFLOP/s; torch's bf16
// product 1220), the matrix cores busy 78 % of the cycles, the clock held by the
// card's power: 890 us on zeros.  512 x 14336 x 4096 in e2m1: 28 us, of which
// the copies alone take 27 (14 TB/s from L2, whose lines are first touched in
// the stage that copies them).
template <int DT, int FMT, int RW, int MT, int FW, int NT, int KW>
struct MxTile {
    static constexpr int kSC = FMT == LORA_MX_E4M3 ? 1 : 2;   // chunks of a stage
    static constexpr int kSet = RW * FW;                      // wavefronts of a set
    static constexpr int kRows = 16 * RW * MT;
    static constexpr int kTiles = FW * NT;                    // of 16 features
    static constexpr int kXUnits = kRows * 8;                 // 16 bytes each
    static constexpr int kWUnits = kTiles * kSC * 64;
    static constexpr int kXCopies = kXUnits / 64 / kSet;      // of a wavefront, a stage
    static constexpr int kWCopies = kWUnits / 64 / kSet;
    static constexpr int kXScaleCopies = kRows / 64;          // of the set, four chunks
    static constexpr int kScaleCopies = kXScaleCopies + kTiles / 4;
    static_assert(kXUnits % (64 * kSet) == 0 && kWUnits % (64 * kSet) == 0, "whole copies");
    static_assert(kRows % 64 == 0 && kTiles % 4 == 0, "whole copies of scales");
    static_assert(NT % 2 == 0, "features come in pairs of tiles");
    static_assert(KW == 1 || FW * NT <= 8, "half the sets' sums fit the X slots, even tiles one and odd ones the other");
};

__device__ __forceinline__ void mx_copy16(const uint8_t *src, u32x4_t *dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

template <class JOB, int DT, int FMT, int RW, int MT, int FW, int NT, int KW>
__global__ __launch_bounds__(64 * RW * FW * KW, 2) void mx_linear_tile_kernel(MxLinearArgs a, MxGrid grid, JOB job)
{
    typedef MxTile<DT, FMT, RW, MT, FW, NT, KW> T;
    __shared__ u32x4_t x0[KW * T::kXUnits], x1[KW * T::kXUnits];
    __shared__ u32x4_t w0[KW * T::kWUnits], w1[KW * T::kWUnits];
    __shared__ u32x4_t scales[KW * T::kScaleCopies * 64];   // of four chunks: X rows, W tiles
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int set = wave / T::kSet, wv = wave % T::kSet;
    const int wr = wv / FW, wf = wv % FW;
    const int g = lane >> 4, m = lane & 15;
    const MxWork work = mx_work<true>(a, grid, job, T::kRows);
    if (work.none)
        return;
    const int n_rows = work.end, row0 = work.row0;
    const int64_t tile0 = (int64_t)work.col * T::kTiles;
    const int chunks = a.w.chunks, groups = (chunks + 3) / 4;
    // this set's groups of four chunks
    const int per = (groups + KW - 1) / KW;
    const int c_begin = 4 * per * set, c_end = min(chunks, c_begin + 4 * per);

    const uint8_t *xsrc[T::kXCopies];
    int xunit[T::kXCopies];
#pragma unroll
    for (int i = 0; i < T::kXCopies; ++i) {
        const int r = (i * T::kSet + wv) * 8 + (lane >> 3);
        const uint32_t row = mx_source(job, work, row0 + r);
        xunit[i] = (lane & 7) ^ ((r >> 1) & 7);
        xsrc[i] = a.q + row * a.ldq;
    }
    const uint8_t *wsrc = a.w.codes + tile0 * 1024 + lane * 16;
    // a set's copies of scales are dealt out to its wavefronts
    constexpr int kDeal = (T::kScaleCopies + T::kSet - 1) / T::kSet;
    const uint8_t *ssrc[kDeal];
#pragma unroll
    for (int i = 0; i < kDeal; ++i) {
        const int n = i * T::kSet + wv;   // X: a row a lane; W: four tiles of 16 lanes
        const uint32_t row = mx_source(job, work, row0 + 64 * n + lane);
        const int64_t tile = tile0 + 4 * (n - T::kXScaleCopies) + (lane >> 4);
        ssrc[i] = n < T::kXScaleCopies ? a.s + row * a.lds : a.w.scales + tile * 256 + (lane & 15) * 16;
    }

    // Groups end anywhere in a tile: a wavefront without rows only copies (512 rows
    // top 8 of 64, 1024 -> 4096: 57 us, then 53).
    const bool idle = JOB::kGrouped && row0 + 16 * wr * MT >= n_rows;

    u32x4_t sx[MT];
    uint32_t sw[NT];
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[t][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // copies of the stage that starts at chunk c
    auto fetch = [&](int c, u32x4_t *xd, u32x4_t *wd) {
        const bool half = FMT == LORA_MX_E2M1 && c + 1 >= chunks;   // the row ends inside the stage
#pragma unroll
        for (int i = 0; i < T::kXCopies; ++i) {
            const int u = half ? xunit[i] & 3 : xunit[i];
            mx_copy16(xsrc[i] + (int64_t)c * (128 / T::kSC) + u * 16,
                      xd + set * T::kXUnits + (i * T::kSet + wv) * 64);
        }
#pragma unroll
        for (int i = 0; i < T::kWCopies; ++i) {
            const int b = i * T::kSet + wv, h = b / T::kTiles, tile = b % T::kTiles;
            mx_copy16(wsrc + ((int64_t)min(c + h, chunks - 1) * a.w.tiles + tile) * 1024,
                      wd + set * T::kWUnits + b * 64);
        }
    };
    auto fetch_scales = [&](int grp) {
#pragma unroll
        for (int i = 0; i < kDeal; ++i) {
            const int n = i * T::kSet + wv;
            if (n < T::kScaleCopies)
                mx_copy16(ssrc[i] + (int64_t)grp * (n < T::kXScaleCopies ? 16 : (int64_t)a.w.tiles * 256),
                          scales + (set * T::kScaleCopies + n) * 64);
        }
    };
    // One chunk, H the half of its stage: the W tiles' codes and the first X
    // tile's are read (load), then multiplied tile by tile (multiply), each X
    // tile read one ahead; the split of the next X tile's codes is spread over
    // the products of this one's lower part.
    u32x4_t w[NT], xa, xb;
    auto read_x = [&](int t, int h, const u32x4_t *xd) {
        const u32x4_t *xp = xd + set * T::kXUnits + (wr * MT * 16 + 16 * t + m) * 8;
        if constexpr (FMT == LORA_MX_E4M3) {
            xa = xp[g ^ (m >> 1)];
            xb = xp[(4 + g) ^ (m >> 1)];
        } else {
            xa = xp[(4 * h + g) ^ (m >> 1)];
        }
    };
    auto load = [&](int h, const u32x4_t *xd, const u32x4_t *wd) {
        const u32x4_t *wp = wd + set * T::kWUnits + (h * T::kTiles + wf * NT) * 64 + lane;
        read_x(0, h, xd);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            w[n] = wp[64 * n];
    };
    auto multiply = [&](auto J, int h, const u32x4_t *xd) {
        constexpr int j = decltype(J)::value;
        MxOperand<FMT> x, next;
        x.set(xa, xb);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint32_t s = sx[t][j] >> (8 * g);
            if (t + 1 < MT)
                read_x(t + 1, h, xd);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (FMT == LORA_MX_E4M3)
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[t][n] = mx_mfma<FMT, j>(w[n], sw[n], x.v, s, acc[t][n]);
            if constexpr (FMT == LORA_MX_E4M3) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[t][n] = mx_mfma<FMT, j>(w[n], sw[n], x.lo, s, acc[t][n]);
                    if (t + 1 < MT) {
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 8 * n / NT; i < 8 * (n + 1) / NT; ++i)
                            next.set_word(i, xa, xb);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                x = next;
                __builtin_amdgcn_s_setprio(0);
            } else if (t + 1 < MT) {
                x.set(xa, xb);
            }
        }
    };
    auto step = [&](auto S, int c) {
        constexpr int st = decltype(S)::value;   // stage of the group
        u32x4_t *xc = st & 1 ? x1 : x0, *wc = st & 1 ? w1 : w0;
        u32x4_t *xn = st & 1 ? x0 : x1, *wn = st & 1 ? w0 : w1;
        __builtin_amdgcn_s_waitcnt(7 << 4);   // vmcnt 0, lgkmcnt 0
        asm volatile("s_barrier" ::: "memory");
        if constexpr (st == 0) {
            // this group's scales; their slot is refilled behind the next barrier
            const u32x4_t *sp = scales + set * T::kScaleCopies * 64;
#pragma unroll
            for (int t = 0; t < MT; ++t)
                sx[t] = sp[16 * (wr * MT + t) + m];
            const uint32_t *swp = reinterpret_cast<const uint32_t *>(sp + T::kXScaleCopies * 64);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sw[n] = swp[64 * (wf * NT + n) + lane];
        }
        // With several row tiles a wavefront, this stage's first operands are on
        // their way while the next stage's copies are issued; with one the
        // stages are short, and the copies go first.
        if constexpr (MT > 1) {
            if (!idle)
                load(0, xc, wc);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (c + T::kSC < c_end)
            fetch(c + T::kSC, xn, wn);
        if (st == 1 && c + 4 - T::kSC < c_end)
            fetch_scales((c - T::kSC) / 4 + 1);
        __builtin_amdgcn_sched_barrier(0);
        if (idle)
            return;
        if constexpr (MT == 1)
            load(0, xc, wc);
        if (c < c_end)
            multiply(std::integral_constant<int, st * T::kSC>{}, 0, xc);
        if constexpr (T::kSC == 2) {
            if (c + 1 < c_end) {
                load(1, xc, wc);
                multiply(std::integral_constant<int, st * 2 + 1>{}, 1, xc);
            }
        }
    };
    if (c_begin < c_end)
    {
        fetch(c_begin, x0, w0);
        fetch_scales(c_begin / 4);
    }
    for (int i = 0; i < per; ++i) {
        const int c = c_begin + 4 * i;
        step(std::integral_constant<int, 0>{}, c);
        step(std::integral_constant<int, 1>{}, c + T::kSC);
        if constexpr (T::kSC == 1) {
            step(std::integral_constant<int, 2>{}, c + 2);
            step(std::integral_constant<int, 3>{}, c + 3);
        }
    }
    // sets pairwise: the upper half hands its sums to the lower
    if constexpr (KW > 1) {
#pragma unroll
        for (int half = KW / 2; half > 0; half /= 2) {
            __syncthreads();
            if (set >= half && set < 2 * half) {
                const int at = ((set - half) * T::kSet + wv) * (MT * NT / 2 * 64) + lane;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        reinterpret_cast<f32x4_t *>(n & 1 ? x1 : x0)[at + (t * NT + n) / 2 * 64] = acc[t][n];
            }
            __syncthreads();
            if (set < half) {
                const int at = (set * T::kSet + wv) * (MT * NT / 2 * 64) + lane;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[t][n] += reinterpret_cast<const f32x4_t *>(n & 1 ? x1 : x0)[at + (t * NT + n) / 2 * 64];
            }
        }
        if constexpr (JOB::kFused)
            __syncthreads();   // the sums' slots are staged over below
        if (set > 0)
            return;
    }
    if constexpr (JOB::kFused) {
        // A wavefront's 16 rows at a time go through a part of the slots of its
        // own (8192 rows x 8 of 1024 -> 4096 in fp32 497 us; stored from the sums'
        // own lanes, half lines at a time, 534) and come back as units of 8 outputs, four neighbouring lanes a
        // block of 32 and whole lines of a row together; 16-byte unit c of row r
        // sits at c ^ r, which spreads the writes over all banks.
        static_assert(T::kSet == 4 || T::kSet == 8, "wavefronts share the four slots evenly");
        static_assert(sizeof(x0) >= T::kSet / 4 * 1024 * NT && sizeof(w0) >= T::kSet / 4 * 1024 * NT, "one part a wavefront");
        if constexpr (KW == 1)
            __syncthreads();   // everybody has read the last stage
        f32x4_t *stage = reinterpret_cast<f32x4_t *>((wv & 2) ? ((wv & 1) ? w1 : w0) : ((wv & 1) ? x1 : x0)) + (wv >> 2) * 64 * NT;
        constexpr int U = JOB::kGated ? NT : 2 * NT;   // units of a row
        const int64_t o0 = (tile0 + wf * NT) * 16 / (JOB::kGated ? 2 : 1);
        const int u = lane % U;
        MxFinish<JOB> finish(job, work.expert, o0 + 8 * u);
        // sums that are stored as they are, in fp32: 16 bytes a lane, side by side
        const bool as_they_are = !JOB::kGated && !job.bias && job.act == LORA_ACT_NONE && (JOB::kGrouped || !job.res) &&
                                 !job.b.q && job.dtype == DT_F32;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int first = row0 + 16 * (wr * MT + t);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                stage[m * 4 * NT + ((8 * (n / 2) + 2 * g + (n & 1)) ^ m)] = acc[t][n];
            mx_wave_fence();
            if (as_they_are) {
                const int c = lane % (4 * NT);
                float *y = static_cast<float *>(job.y) + o0 + 4 * c;
                if (o0 + 4 * c < job.d) {
#pragma unroll
                    for (int r = lane / (4 * NT); r < 16; r += 16 / NT)   // not kept in L2: 8192 rows x 8 of 1024 -> 4096 497 us, 525 if kept
                        if (first + r < n_rows)
                            __builtin_nontemporal_store(stage[r * 4 * NT + (c ^ r)], reinterpret_cast<f32x4_t *>(y + (first + r) * job.ldy));
                }
            } else {
#pragma unroll 1
                for (int r = lane / U; r < 16; r += 64 / U) {
                    auto unit = [&](int c, float (&f)[8]) {
                        const f32x4_t p = stage[r * 4 * NT + (c ^ r)], q = stage[r * 4 * NT + ((c + 1) ^ r)];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[e] = p[e];
                            f[4 + e] = q[e];
                        }
                    };
                    float f[8], up[8];
                    if constexpr (JOB::kGated) {
                        unit(16 * (u >> 2) + 2 * (u & 3), f);
                        unit(16 * (u >> 2) + 8 + 2 * (u & 3), up);
                    } else {
                        unit(2 * u, f);
                    }
                    finish.row(first + r, first + r < n_rows, f, up);
                }
            }
            mx_wave_fence();
        }
        return;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int r = row0 + 16 * (wr * MT + t) + m;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            const int64_t o = (tile0 + wf * NT + n) * 16 + 8 * g;
            if (r < n_rows && o < a.w.d)
                mx_store8<DT>(a.y, (int64_t)r * a.ldy + o, acc[t][n], acc[t][n + 1]);
        }
    }
}

}  // namespace

}  // namespace lora
