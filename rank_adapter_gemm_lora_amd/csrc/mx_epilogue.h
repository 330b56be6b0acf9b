// mx_epilogue.h -- what a fused product does with its sums: bias, activation
// (or gate), residual, and the two forms of the result.
#pragma once

#include "mx_device.h"
#include "mx_job.h"

namespace lora {

// The sums as they are, in the kernel's own dtype.
struct MxPlain {
    static constexpr bool kFused = false, kGrouped = false, kGated = false;
};

template <bool GROUPED, bool GATED> struct MxFused : MxEpilogue {
    static constexpr bool kFused = true, kGrouped = GROUPED, kGated = GATED;
};

// Orders a wavefront's own LDS writes ahead of its lanes' reads of each other's.
__device__ __forceinline__ void mx_wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

__device__ __forceinline__ void mx_load8(int dtype, const void *p, int64_t at, float (&f)[8])
{
    if (dtype == DT_F32) {
        Vec8<DT_F32> v;
        v.load(p, at);
        v.to_f32(f);
    } else {
        Vec8<DT_BF16> v;
        v.load(p, at);
        v.to_f32(f);
    }
}

// v / (1 + exp(-z)): exp as the hardware's power of two, with what its argument's
// rounding loses brought in behind it, and the hardware's reciprocal; some five
// roundings in all.  A denominator past 2^126 gives 0.
__device__ __forceinline__ float mx_logistic_mul(float v, float z)
{
    constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.925963033e-8f, kLn2 = 0.693147181f;
    constexpr int kPositive = 0x180;   // finite, not zero; the others stand
    const float t = z * -kLog2E, lost = fmaf(z, -kLog2E, -t) - z * kLog2ELow;
    const float e = __builtin_amdgcn_exp2f(t);
    return v * __builtin_amdgcn_rcpf(1.f + (__builtin_amdgcn_classf(e, kPositive) ? fmaf(e, lost * kLn2, e) : e));
}

// v Phi(v), Phi the normal distribution: with x = |v|, Phi(-x) = exp(-x^2 / 2) r(x),
// r(x) = erfcx(x / sqrt 2) / 2, which falls slowly: a polynomial in 1 / (1 + 0.3 x),
// fitted here to r on 0 <= x <= 14.5 by weighted least squares until its largest
// relative error was least (5.8e-8).  Nothing cancels for negative v, as 1 + erf
// would.  x^2's and its multiple's rounding are brought in behind the power of two.
// Over all v within 8 roundings of the value (rms 1.3), in some 30 instructions
// (512 x 4096 x 14336 with blocks 54.1 us; with the library's erfc, in branches over
// its ranges, 56.9).
__device__ __forceinline__ float mx_gelu(float v)
{
    constexpr float kC[9] = {7.37266964e-06f, 0.119484201f, 0.121945299f, 0.0945857242f, 0.142765597f,
                             -0.0768401325f, 0.228952199f, -0.169307664f, 0.0384074338f};
    constexpr float kHalfLog2E = 0.721347511f, kHalfLog2ELow = 9.62981517e-9f, kLn2 = 0.693147181f;
    constexpr int kPositive = 0x180;   // finite, not zero; the others stand
    const float x = fabsf(v), t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.f));
    float r = kC[8];
#pragma unroll
    for (int i = 7; i >= 0; --i)
        r = fmaf(r, t, kC[i]);
    const float s = x * x, low = fmaf(x, x, -s), a = s * -kHalfLog2E;
    const float lost = fmaf(s, -kHalfLog2E, -a) - fmaf(low, kHalfLog2E, s * kHalfLog2ELow);
    const float e = __builtin_amdgcn_exp2f(a);
    const float below = r * (__builtin_amdgcn_classf(e, kPositive) ? fmaf(e, lost * kLn2, e) : e);   // Phi(-x)
    return v * (v < 0.f ? below : 1.f - below);
}

// Activations in fp32.  The tanh form of GELU as v / (1 + exp(-2 z)), the same
// expression without its cancellation.
__device__ __forceinline__ void mx_activate(int act, float (&f)[8])
{
    if (act == LORA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = f[e] < 0.f ? 0.f : f[e];
    } else if (act == LORA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_logistic_mul(f[e], f[e]);
    } else if (act == LORA_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_gelu(f[e]);
    } else if (act == LORA_ACT_GELU_TANH) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_logistic_mul(f[e], 1.5957691216057308f * fmaf(0.044715f * f[e] * f[e], f[e], f[e]));
    }
}

// Outputs o .. o + 7 of some rows.  Four neighbouring lanes hold the units of one
// block of 32 of a row and come here together; o is a multiple of 8, that of the
// first of them of 32.
template <class JOB> struct MxFinish {
    const JOB &job;
    int64_t o;
    bool some, live;        // the block, this unit has outputs
    float bias[8], up_bias[8];

    __device__ __forceinline__ MxFinish(const JOB &j, int expert, int64_t first) : job(j), o(first)
    {
        some = (o & ~(int64_t)31) < job.d;
        live = o < job.d;
        if (job.bias && live) {
            const int64_t at = expert * (JOB::kGated ? 2 * job.d : job.d) + o;
            mx_load8(job.dtype, job.bias, at, bias);
            if constexpr (JOB::kGated)
                mx_load8(job.dtype, job.bias, at + job.d, up_bias);
        }
    }

    // One row's unit from its sums (gated: f the gate's, up the other's).
    __device__ __forceinline__ void row(int row, bool in, float (&f)[8], float (&up)[8])
    {
        if (!in || !some)
            return;
        if (live) {
            if (job.bias) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] += bias[e];
                    if constexpr (JOB::kGated)
                        up[e] += up_bias[e];
                }
            }
            if constexpr (JOB::kGated) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = mx_logistic_mul(f[e], f[e]) * up[e];
            } else {
                mx_activate(job.act, f);
            }
            if (!JOB::kGrouped && job.res) {
                float r[8];
                mx_load8(job.dtype, job.res, row * job.ldr + o, r);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] += r[e];
            }
            if (job.y) {
                if (job.dtype == DT_F32)
                    Vec8<DT_F32>::store(job.y, row * job.ldy + o, f);
                else
                    Vec8<DT_BF16>::store(job.y, row * job.ldy + o, f);
            }
        }
        if (!job.b.q)
            return;
        if (!live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = 0.f;
        }
        const uint32_t sb = mx_block_scale<LORA_MX_E4M3>(f);
        uint8_t *q = job.b.q + row * job.b.ldq, *s = job.b.s + row * job.b.lds;
        *reinterpret_cast<uint2 *>(q + o) = mx_codes<LORA_MX_E4M3>(f, sb);
        const int part = (int)(o >> 3) & 3;
        const int64_t block = o >> 5, blocks = (job.d + 31) >> 5;
        if (part == 0)
            s[block] = (uint8_t)sb;
        if (block == blocks - 1) {   // zeros to the ends of the row's codes and scales
            for (int64_t at = 32 * blocks + 8 * part; at < ((job.d + 127) & ~(int64_t)127); at += 32)
                *reinterpret_cast<uint2 *>(q + at) = make_uint2(0, 0);
            for (int64_t at = blocks + part; at < ((job.d + 511) >> 9) * 16; at += 4)
                s[at] = 0;
        }
    }
};

}  // namespace lora
