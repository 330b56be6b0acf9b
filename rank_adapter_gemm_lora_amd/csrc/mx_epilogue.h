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

// Activations in fp32.  GELU by the complementary error function, whose value for
// negative arguments loses nothing where 1 + erf would cancel; its tanh form
// as v / (1 + exp(-2 z)), the same expression without the cancellation.
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
            f[e] = 0.5f * f[e] * erfcf(f[e] * -0.70710678118654752f);
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
