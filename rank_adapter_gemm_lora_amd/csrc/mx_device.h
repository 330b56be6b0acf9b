// mx_device.h -- gfx950 device helpers of the microscaled operators: one block
// of 32 held by four neighbouring lanes of a wavefront, 8 values a lane.
#pragma once

#include "device_common.h"
#include "mx.h"

namespace lora {

__device__ __forceinline__ uint32_t mx_div_of(uint32_t n, const MxDiv &d)
{
    return (uint32_t)(((uint64_t)n * d.m) >> d.sh);
}

template <int FMT> struct MxFmt;
template <> struct MxFmt<LORA_MX_E4M3> {
    static constexpr int emax = 8;
    static constexpr int unit_bytes = 8;   // codes of 8 elements
    typedef uint2 unit_t;
};
template <> struct MxFmt<LORA_MX_E2M1> {
    static constexpr int emax = 2;
    static constexpr int unit_bytes = 4;
    typedef uint32_t unit_t;
};

// Value of a lane's neighbour in its group of four (quad permutation 1 0 3 2,
// then 2 3 0 1: a move inside the register file, no LDS).
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
}

// Scale byte of the block that this lane's 8 values and those of its three
// quad neighbours make up.  The magnitudes are compared as integers, which
// orders finite floats and puts infinities and then NaNs above them, so the
// exponent field of the largest gives every case: 255 (not finite) stays 255,
// the rest is floor(log2 m) + 127 - emax, at least 0 (subnormal floats have
// field 0 and a true exponent further below the clamp).
template <int FMT> __device__ __forceinline__ uint32_t mx_block_scale(const float (&f)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    m = max(m, quad_xor1(m));
    m = max(m, quad_xor2(m));
    const int e = (int)(m >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - MxFmt<FMT>::emax, 0);
}

// The lane's 8 codes under that scale.  The product with a power of two is
// exact or, below the smallest normal float, far under half a code step; the
// conversion rounds to nearest even.  e4m3's conversion turns what is beyond
// its range into NaN, so its input is clamped; e2m1's saturates.
template <int FMT>
__device__ __forceinline__ typename MxFmt<FMT>::unit_t mx_codes(const float (&f)[8], uint32_t sb)
{
    const float inv = __uint_as_float((254u - min(sb, 253u)) << 23);   // 2^(127 - sb)
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        u[i] = sb == 255u ? 0.f : f[i] * inv;
    if constexpr (FMT == LORA_MX_E4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = fminf(fmaxf(u[i], -448.f), 448.f);
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], hi, true);
        return make_uint2((uint32_t)lo, (uint32_t)hi);
    } else {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u[0], u[1], 1.f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u[2], u[3], 1.f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u[4], u[5], 1.f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, u[6], u[7], 1.f, 3);
        return w;
    }
}

// g / (1 + exp(-g)) * u, in the values that fp32 operations one by one give (none of
// 7.3 M bf16 or 2.9 M fp32 outputs differs), so that codes are those of an
// unfused fp32 computation, also beside a border.  The quotient is g times the
// hardware's reciprocal and one correction by what is left of g.  The reciprocal
// of a denominator past 2^126 would be flushed, so past 2^64 it is taken of a
// scaled one.
__device__ __forceinline__ float mx_silu_mul(float g, float u)
{
    const float d = 1.f + expf(-g);
    const float k = d > 0x1p64f ? 0x1p-64f : 1.f;
    const float rc = __builtin_amdgcn_rcpf(d * k), q = g * rc;
    const float left = fmaf(-(d * k), q, g);   // NaN where g or d is not finite: q stands
    return (left == left ? fmaf(left, rc, q) : q) * k * u;
}

// Write this lane's unit of a row in blocks: 8 codes, and from the first lane
// of each 16 (128 elements, four blocks) the four scale bytes as one word; the
// row's last such lane also writes the padding words.  unit: 0 .. units - 1, a
// row's 16-unit groups never straddle the 16-lane groups of a wavefront
// (units is a multiple of 16 and so is unit - lane).
template <int FMT>
__device__ __forceinline__ void mx_store_unit(uint8_t *q, uint8_t *s, int unit, int units,
                                              const float (&f)[8])
{
    const uint32_t sb = mx_block_scale<FMT>(f);
    *reinterpret_cast<typename MxFmt<FMT>::unit_t *>(q + (int64_t)unit * MxFmt<FMT>::unit_bytes) =
        mx_codes<FMT>(f, sb);
    // lanes 0, 4, 8, 12 of the group -> one word: shift by quad, or together
    const int quad = (unit >> 2) & 3;
    uint32_t word = sb << (8 * quad);
    word |= (uint32_t)__shfl_xor((int)word, 4);
    word |= (uint32_t)__shfl_xor((int)word, 8);
    if ((unit & 15) == 0) {
        uint32_t *sw = reinterpret_cast<uint32_t *>(s);
        const int n = unit >> 4, chunks = units >> 4;
        sw[n] = word;
        if (n == chunks - 1)
            for (int p = chunks; p < ((chunks + 3) & ~3); ++p)
                sw[p] = 0;
    }
}

}  // namespace lora
