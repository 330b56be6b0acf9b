// mx_linear.hip -- y = X W^T with X in e4m3 or e2m1 blocks and W in e2m1 blocks
// (the weight image).  W is the row operand of the matrix instructions and X the
// column operand, so a lane's four results are four neighbouring outputs
// (features 4 g .. + 3, lane l = 16 g + m) of X row m.  In both forms lane l
// holds, of a chunk of 128 k, the 32 codes of block g (k 32 g .. + 31) of its
// row and that block's scale.
//
// e2m1 X: v_mfma_scale_f32_16x16x128_f8f6f4 takes codes and scales as they are;
// a product has 4 significant bits and its sums are exact to fp32 rounding.
//
// e4m3 X: the same instruction on e4m3 aligns the products of each group of
// eight k to the largest of the group and drops what lies more than 13 binary
// places below it (measured: 1 + 2^-14 inside a group gives 1, across groups
// 1 + 2^-23 is kept), up to 5e-5 of the result where a block spans e4m3's whole
// range.  Sums here are held in fp32, so codes are widened to bf16 with their
// scale instead (exact: 4 significant bits, the same exponents as fp32) and
// multiplied by v_mfma_f32_16x16x32_bf16, four per chunk: instruction j takes
// codes 8 j .. 8 j + 7 of every lane, the same k in both operands.
#include "mx_device.h"

namespace lora {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;   // operand format code of the instruction

// The codes of one lane's block: 16 bytes of e2m1 or 32 of e4m3.
template <int FMT> struct MxLane;
template <> struct MxLane<LORA_MX_E2M1> {
    uint4 c;
    __device__ __forceinline__ void load(const uint8_t *p) { c = *reinterpret_cast<const uint4 *>(p); }
};
template <> struct MxLane<LORA_MX_E4M3> {
    uint4 lo, hi;
    __device__ __forceinline__ void load(const uint8_t *p)
    {
        lo = *reinterpret_cast<const uint4 *>(p);
        hi = *reinterpret_cast<const uint4 *>(p + 16);
    }
};

// A scale byte as the float 2^(b - 127).  The widening conversions read only its
// exponent field, 0 as 2^-127; 255 is passed as a NaN.
__device__ __forceinline__ float mx_scale_f32(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7fc00000u : b << 23);
}

// Eight e2m1 codes (one word) or e4m3 codes (two) and their scale -> bf16.
__device__ __forceinline__ bf16x8_t mx_widen_e2m1(uint32_t c, float s)
{
    bf16x8_t r;
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
    r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
    r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
    return r;
}
__device__ __forceinline__ bf16x8_t mx_widen_e4m3(uint32_t c0, uint32_t c1, float s)
{
    bf16x8_t r;
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, false);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, true);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, false);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, true);
    r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
    r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
    return r;
}

// One chunk: c[t] += W tile x X tile t; sw / sx: the lanes' scale bytes.
template <int FMT, int MT>
__device__ __forceinline__ void mx_chunk(uint4 w, uint32_t sw, const MxLane<FMT> (&x)[MT],
                                         const uint32_t (&sx)[MT], f32x4_t (&c)[MT])
{
    if constexpr (FMT == LORA_MX_E2M1) {
        const i32x8_t a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint4 v = x[t].c;
            const i32x8_t b = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
            c[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c[t], kFp4, kFp4, 0,
                                                                    (int)sw, 0, (int)sx[t]);
        }
    } else {
        const float fw = mx_scale_f32(sw);
        const bf16x8_t a0 = mx_widen_e2m1(w.x, fw), a1 = mx_widen_e2m1(w.y, fw);
        const bf16x8_t a2 = mx_widen_e2m1(w.z, fw), a3 = mx_widen_e2m1(w.w, fw);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const float fx = mx_scale_f32(sx[t]);
            const uint4 l = x[t].lo, h = x[t].hi;
            c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, mx_widen_e4m3(l.x, l.y, fx), c[t], 0, 0, 0);
            c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, mx_widen_e4m3(l.z, l.w, fx), c[t], 0, 0, 0);
            c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a2, mx_widen_e4m3(h.x, h.y, fx), c[t], 0, 0, 0);
            c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a3, mx_widen_e4m3(h.z, h.w, fx), c[t], 0, 0, 0);
        }
    }
}

// Four neighbouring outputs of one row.
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

// One workgroup: 16 features x 16 MT rows; its NW wavefronts split the chunks of
// k and are summed in wavefront order through LDS.
template <int DT, int FMT, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void mx_linear_split_kernel(MxLinearArgs a)
{
    __shared__ f32x4_t part[NW][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, m = lane & 15;
    const int64_t tile = blockIdx.x;
    const int64_t row0 = (int64_t)blockIdx.y * (16 * MT);
    const int chunks = a.w.chunks;
    const int c0 = chunks * wave / NW, c1 = chunks * (wave + 1) / NW;
    const uint8_t *wc = a.w.codes + (tile * chunks * 64 + lane) * 16;
    const uint8_t *ws = a.w.scales + (tile * ((chunks + 3) / 4) * 64 + lane) * 4;
    constexpr int kLane = FMT == LORA_MX_E4M3 ? 32 : 16;   // bytes of a lane's codes
    const uint8_t *xq[MT], *xs[MT];
    f32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        int64_t r = row0 + 16 * t + m;   // rows past the end repeat the last one
        r = r < a.n_rows ? r : a.n_rows - 1;
        xq[t] = a.q + r * a.ldq + kLane * g;
        xs[t] = a.s + r * a.lds;
        acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int c = c0; c < c1; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(wc + (int64_t)c * 1024);
        const uint32_t sw = ws[(int64_t)(c >> 2) * 256 + (c & 3)];
        MxLane<FMT> x[MT];
        uint32_t sx[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            x[t].load(xq[t] + (int64_t)c * (4 * kLane));
            sx[t] = xs[t][4 * c + g];
        }
        mx_chunk<FMT, MT>(w, sw, x, sx, acc);
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
        const int64_t r = row0 + 16 * t + m, o = tile * 16 + 4 * g;
        if (r < a.n_rows && o < a.w.d)
            mx_store4<DT>(a.y, r * a.ldy + o, v);
    }
}

template <int DT, int FMT> void linear_pick(const MxLinearArgs &a, hipStream_t s)
{
    const uint32_t tiles = (uint32_t)((a.w.d + 15) / 16);
    if (a.n_rows <= 16) {
        mx_linear_split_kernel<DT, FMT, 1, 8><<<dim3(tiles, 1), 512, 0, s>>>(a);
        return;
    }
    // slabs of rows: the second grid dimension is at most 65535
    const int64_t most = (int64_t)65535 * 64;
    for (int64_t r = 0; r < a.n_rows; r += most) {
        MxLinearArgs b = a;
        b.n_rows = a.n_rows - r < most ? a.n_rows - r : most;
        b.q = a.q + r * a.ldq;
        b.s = a.s + r * a.lds;
        b.y = static_cast<char *>(a.y) + r * a.ldy * (DT == DT_F32 ? 4 : 2);
        mx_linear_split_kernel<DT, FMT, 4, 8>
            <<<dim3(tiles, (uint32_t)((b.n_rows + 63) / 64)), 512, 0, s>>>(b);
    }
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
