// mx_linear.hip -- y = X W^T with X in e4m3 or e2m1 blocks and W in e2m1 blocks
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
#include <type_traits>

#include "mx_device.h"

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
    __device__ __forceinline__ explicit MxOperand(u32x4_t c)
        : v{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0}
    {
    }
};
template <> struct MxOperand<LORA_MX_E4M3> {
    i32x8_t hi, lo;   // codes of |x| >= 2 and of the rest, zeros in the other's places
    __device__ __forceinline__ MxOperand(u32x4_t a, u32x4_t b)
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // byte masks from bit 6: moved to the sign of bytes 1, 3, 5 and 7,
            // which selectors 8 .. 11 of the byte permutation spread
            const uint32_t h = w[i] & __builtin_amdgcn_perm(w[i] << 1, w[i] << 9, 0x0b090a08u);
            hi[i] = (int)h;
            lo[i] = (int)(w[i] ^ h);
        }
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

// ---------------------------------------------------------------- few rows
//
// One workgroup: 16 features x 16 MT rows; its NW wavefronts take groups of
// four chunks in turn and are summed in wavefront order through LDS.  W is
// streamed once, straight into registers in operand order; all of a group's
// loads are issued before its first product, and the next group's before that.
template <int FMT, int MT> struct MxGroup {
    u32x4_t w[4];
    uint32_t sw;
    u32x4_t x[MT][4][FMT == LORA_MX_E4M3 ? 2 : 1];
    u32x4_t sx[MT];
    // wc, ws: this lane's words of the tile; xq, xs: its rows
    __device__ __forceinline__ void load(int grp, int chunks, const uint8_t *wc, const uint8_t *ws,
                                         const uint8_t *const (&xq)[MT], const uint8_t *const (&xs)[MT])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = min(4 * grp + j, chunks - 1);   // past the end: not multiplied
            w[j] = *reinterpret_cast<const u32x4_t *>(wc + c * 1024);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                x[t][j][0] = *reinterpret_cast<const u32x4_t *>(
                    xq[t] + c * (FMT == LORA_MX_E4M3 ? 128 : 64));
                if constexpr (FMT == LORA_MX_E4M3)
                    x[t][j][1] = *reinterpret_cast<const u32x4_t *>(xq[t] + c * 128 + 64);
            }
        }
        sw = *reinterpret_cast<const uint32_t *>(ws + (int64_t)grp * 256);
#pragma unroll
        for (int t = 0; t < MT; ++t)
            sx[t] = *reinterpret_cast<const u32x4_t *>(xs[t] + (int64_t)grp * 16);
    }
    template <int J>
    __device__ __forceinline__ void chunk(int g, f32x4_t (&acc)[MT])
    {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint32_t s4 = J == 0 ? sx[t].x : J == 1 ? sx[t].y : J == 2 ? sx[t].z : sx[t].w;
            const uint32_t s = s4 >> (8 * g);
            if constexpr (FMT == LORA_MX_E4M3) {
                const MxOperand<FMT> o(x[t][J][0], x[t][J][1]);
                acc[t] = mx_mfma<FMT, J>(w[J], sw, o.hi, s, acc[t]);
                acc[t] = mx_mfma<FMT, J>(w[J], sw, o.lo, s, acc[t]);
            } else {
                acc[t] = mx_mfma<FMT, J>(w[J], sw, MxOperand<FMT>(x[t][J][0]).v, s, acc[t]);
            }
        }
    }
    __device__ __forceinline__ void multiply(int n, int g, f32x4_t (&acc)[MT])
    {
        chunk<0>(g, acc);
        if (n > 1)
            chunk<1>(g, acc);
        if (n > 2)
            chunk<2>(g, acc);
        if (n > 3)
            chunk<3>(g, acc);
    }
};

template <int DT, int FMT, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void mx_linear_few_kernel(MxLinearArgs a)
{
    __shared__ f32x4_t part[NW][MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, m = lane & 15;
    const int64_t tile = blockIdx.x;
    const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);
    const int chunks = a.w.chunks, groups = (chunks + 3) / 4;
    const uint8_t *wc = a.w.codes + (tile * chunks * 64 + lane) * 16;
    const uint8_t *ws = a.w.scales + (tile * groups * 64 + lane) * 4;
    const uint8_t *xq[MT], *xs[MT];
    f32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        int64_t r = row0 + 16 * t + m;   // rows past the end repeat the last one
        r = r < a.n_rows ? r : a.n_rows - 1;
        xq[t] = a.q + r * a.ldq + 16 * g;
        xs[t] = a.s + r * a.lds;
        acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    MxGroup<FMT, MT> cur, nxt;
    if (wave < groups)
        cur.load(wave, chunks, wc, ws, xq, xs);
    for (int grp = wave; grp < groups; grp += NW) {
        if (grp + NW < groups)
            nxt.load(grp + NW, chunks, wc, ws, xq, xs);
        cur.multiply(chunks - 4 * grp, g, acc);
        cur = nxt;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
        part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += NW) {
        f32x4_t v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            v += part[w][t][lane];
        const int64_t r = row0 + 16 * t + m;
        const int64_t o = (tile >> 1) * 32 + 8 * g + 4 * (tile & 1);
        if (r < a.n_rows && o < a.w.d)
            mx_store4<DT>(a.y, r * a.ldy + o, v);
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
// next (consumed by products issued before it).
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
    static_assert(kXUnits % (64 * kSet) == 0 && kWUnits % (64 * kSet) == 0, "whole copies");
    static_assert(NT % 2 == 0, "features come in pairs of tiles");
    static_assert(KW == 1 || (MT % 2 == 0 && KW / 2 * kSet * MT / 2 * NT * 64 <= KW * kXUnits),
                  "half the sets' sums fit the X slots, even row tiles one and odd ones the other");
};

__device__ __forceinline__ void mx_copy16(const uint8_t *src, u32x4_t *dst)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

template <int DT, int FMT, int RW, int MT, int FW, int NT, int KW>
__global__ __launch_bounds__(64 * RW * FW * KW, 2) void mx_linear_tile_kernel(MxLinearArgs a, int row_tiles,
                                                                              int col_tiles)
{
    typedef MxTile<DT, FMT, RW, MT, FW, NT, KW> T;
    __shared__ u32x4_t x0[KW * T::kXUnits], x1[KW * T::kXUnits];
    __shared__ u32x4_t w0[KW * T::kWUnits], w1[KW * T::kWUnits];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int set = wave / T::kSet, wv = wave % T::kSet;
    const int wr = wv / FW, wf = wv % FW;
    const int g = lane >> 4, m = lane & 15;
    // workgroups of one XCD walk bands of eight row tiles, so that its L2 serves
    // the X rows and W tiles that they share
    const int id = xcd_major(blockIdx.x, gridDim.x);
    const int band = id / (8 * col_tiles), in = id % (8 * col_tiles);
    const int tall = min(8, row_tiles - 8 * band);
    const int64_t row0 = (int64_t)(8 * band + in % tall) * T::kRows;
    const int64_t tile0 = (int64_t)(in / tall) * T::kTiles;
    const int chunks = a.w.chunks, groups = (chunks + 3) / 4;
    // this set's groups of four chunks
    const int per = (groups + KW - 1) / KW;
    const int c_begin = 4 * per * set, c_end = min(chunks, c_begin + 4 * per);

    const uint8_t *xsrc[T::kXCopies];
    int xunit[T::kXCopies];
#pragma unroll
    for (int i = 0; i < T::kXCopies; ++i) {
        const int r = (i * T::kSet + wv) * 8 + (lane >> 3);
        const int64_t row = min(row0 + r, a.n_rows - 1);   // rows past the end repeat the last one
        xunit[i] = (lane & 7) ^ ((r >> 1) & 7);
        xsrc[i] = a.q + row * a.ldq;
    }
    const uint8_t *wsrc = a.w.codes + tile0 * chunks * 1024 + lane * 16;
    const uint8_t *xss[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xss[t] = a.s + min(row0 + 16 * (wr * MT + t) + m, a.n_rows - 1) * a.lds;
    const uint8_t *wss = a.w.scales + (tile0 + wf * NT) * groups * 256 + lane * 4;

    uint32_t sx[MT][T::kSC], sxn[MT][T::kSC], sw[NT], swn[NT];
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[t][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // copies of the stage that starts at chunk c, and its scales into registers
    auto fetch = [&](int c, u32x4_t *xd, u32x4_t *wd, bool group) {
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
            mx_copy16(wsrc + ((int64_t)tile * chunks + min(c + h, chunks - 1)) * 1024,
                      wd + set * T::kWUnits + b * 64);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < T::kSC; ++h)
                sxn[t][h] = *reinterpret_cast<const uint32_t *>(xss[t] + 4 * (c + h));
        if (group) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                swn[n] = *reinterpret_cast<const uint32_t *>(wss + ((int64_t)n * groups + (c >> 2)) * 256);
        }
    };
    // one chunk, H the half of its stage
    auto multiply = [&](auto J, auto H, const u32x4_t *xd, const u32x4_t *wd) {
        constexpr int j = decltype(J)::value, h = decltype(H)::value;
        const u32x4_t *wp = wd + set * T::kWUnits + (h * T::kTiles + wf * NT) * 64 + lane;
        const u32x4_t *xp = xd + set * T::kXUnits + (wr * MT * 16 + m) * 8;
        u32x4_t w[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            w[n] = wp[64 * n];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint32_t s = sx[t][h] >> (8 * g);
            if constexpr (FMT == LORA_MX_E4M3) {
                const MxOperand<FMT> o(xp[128 * t + (g ^ (m >> 1))], xp[128 * t + ((4 + g) ^ (m >> 1))]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[t][n] = mx_mfma<FMT, j>(w[n], sw[n], o.hi, s, acc[t][n]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[t][n] = mx_mfma<FMT, j>(w[n], sw[n], o.lo, s, acc[t][n]);
            } else {
                const MxOperand<FMT> o(xp[128 * t + ((4 * h + g) ^ (m >> 1))]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[t][n] = mx_mfma<FMT, j>(w[n], sw[n], o.v, s, acc[t][n]);
            }
        }
    };
    auto step = [&](auto S, int c) {
        constexpr int st = decltype(S)::value;   // stage of the group
        u32x4_t *xc = st & 1 ? x1 : x0, *wc = st & 1 ? w1 : w0;
        u32x4_t *xn = st & 1 ? x0 : x1, *wn = st & 1 ? w0 : w1;
        __builtin_amdgcn_s_waitcnt(7 << 4);   // vmcnt 0, lgkmcnt 0
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < T::kSC; ++h)
                sx[t][h] = sxn[t][h];
        if constexpr (st == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sw[n] = swn[n];
        }
        if (c + T::kSC < c_end)
            fetch(c + T::kSC, xn, wn, (st + 1) * T::kSC == 4);
        if (c < c_end)
            multiply(std::integral_constant<int, st * T::kSC>{}, std::integral_constant<int, 0>{}, xc, wc);
        if constexpr (T::kSC == 2)
            if (c + 1 < c_end)
                multiply(std::integral_constant<int, st * 2 + 1>{}, std::integral_constant<int, 1>{}, xc, wc);
    };
    if (c_begin < c_end)
        fetch(c_begin, x0, w0, true);
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
                const int at = ((set - half) * T::kSet + wv) * (MT / 2 * NT * 64) + lane;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        reinterpret_cast<f32x4_t *>(t & 1 ? x1 : x0)[at + (t / 2 * NT + n) * 64] = acc[t][n];
            }
            __syncthreads();
            if (set < half) {
                const int at = (set * T::kSet + wv) * (MT / 2 * NT * 64) + lane;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[t][n] += reinterpret_cast<const f32x4_t *>(t & 1 ? x1 : x0)[at + (t / 2 * NT + n) * 64];
            }
        }
        if (set > 0)
            return;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t r = row0 + 16 * (wr * MT + t) + m;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            const int64_t o = (tile0 + wf * NT + n) * 16 + 8 * g;
            if (r < a.n_rows && o < a.w.d)
                mx_store8<DT>(a.y, r * a.ldy + o, acc[t][n], acc[t][n + 1]);
        }
    }
}

template <int DT, int FMT, int RW, int MT, int FW, int NT, int KW>
void linear_tiles(const MxLinearArgs &a, hipStream_t s)
{
    typedef MxTile<DT, FMT, RW, MT, FW, NT, KW> T;
    const int64_t cols = (a.w.d + 16 * T::kTiles - 1) / (16 * T::kTiles);
    const int64_t most = (((int64_t)1 << 30) / cols) & ~7;   // row tiles of one launch
    for (int64_t t = 0; t * T::kRows < a.n_rows; t += most) {
        const int64_t r = t * T::kRows;
        MxLinearArgs b = a;
        b.n_rows = a.n_rows - r < most * T::kRows ? a.n_rows - r : most * T::kRows;
        b.q = a.q + r * a.ldq;
        b.s = a.s + r * a.lds;
        b.y = static_cast<char *>(a.y) + r * a.ldy * (DT == DT_F32 ? 4 : 2);
        const int64_t rows = (b.n_rows + T::kRows - 1) / T::kRows;
        mx_linear_tile_kernel<DT, FMT, RW, MT, FW, NT, KW>
            <<<dim3((uint32_t)(rows * cols)), 64 * T::kSet * KW, 0, s>>>(b, (int)rows, (int)cols);
    }
}

template <int DT, int FMT> void linear_pick(const MxLinearArgs &a, hipStream_t s)
{
    const uint32_t tiles = (uint32_t)((a.w.d + 31) / 32 * 2);   // both of a pair
    if (a.n_rows <= 16)
        mx_linear_few_kernel<DT, FMT, 1, 8><<<dim3(tiles, 1), 512, 0, s>>>(a);
    else if (a.n_rows <= 32)
        mx_linear_few_kernel<DT, FMT, 2, 8><<<dim3(tiles, 1), 512, 0, s>>>(a);
    else if ((a.n_rows + 127) / 128 * ((a.w.d + 255) / 256) >= a.n_cu)
        linear_tiles<DT, FMT, 2, 4, 2, 8, 1>(a, s);
    else if ((a.n_rows + 127) / 128 * ((a.w.d + 127) / 128) >= a.n_cu)
        linear_tiles<DT, FMT, 2, 4, 2, 4, 2>(a, s);
    else
        linear_tiles<DT, FMT, 2, 2, 2, 2, 4>(a, s);
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
