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

// v times the logistic function of z, z of v's sign, from t + lost = -|z| log2(e), lost what
// rounding t has left: with e = 2^(t + lost), max(v, -0) - |v| e / (1 + e).  The
// power of two is the hardware's, with the lost part brought in behind it, the quotient
// by the hardware's reciprocal and one correction by what is left of e.  Large values
// are rounded once, at the end (v / (1 + e) would round 1 + e too, and the error's root mean
// square over a product's results is then 5.0e-8 instead of 3.8e-8).  Under 2^-64, e and
// with it the quotient are held times 2^64, so that neither leaves fp32 before the result
// does (a SiLU of -87.4 is -1e-36).  Within 6 roundings, each operation counted at its worst.
__device__ __forceinline__ float mx_times_logistic(float v, float t, float lost)
{
#pragma clang fp contract(off)   // t + 64 joined to t's product would not have lost what is brought in
    constexpr float kLn2 = 0.693147181f;
    constexpr int kPositive = 0x180;   // finite, not zero; the others stand
    const bool far = t < -64.f;
    const float k = far ? 0x1p-64f : 1.f;
    const float p = __builtin_amdgcn_exp2f(far ? t + 64.f : t);
    const float e = __builtin_amdgcn_classf(p, kPositive) ? fmaf(p, lost * kLn2, p) : p;
    const float d = fmaf(e, k, 1.f), rc = __builtin_amdgcn_rcpf(d), q = e * rc;
    const float tail = fmaf(fmaf(-d, q, e), rc, q);
    const float b = v > 0x1p100f ? 0x1p100f : fabsf(v);   // infinity has no tail: not infinity times 0
    return fmaf(-(b * tail), k, v < 0.f ? -0.f : v);
}

// v / (1 + exp(-v))
__device__ __forceinline__ float mx_silu(float v)
{
#pragma clang fp contract(off)
    constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.925963033e-8f;
    const float x = fabsf(v), t = x * -kLog2E;
    return mx_times_logistic(v, t, fmaf(-x, kLog2ELow, fmaf(x, -kLog2E, -t)));
}

// v (1 + tanh z) / 2, z = sqrt(2 / pi) (v + 0.044715 v^3), as v times the logistic function of
// 2 z: the same expression without its cancellation, within 3 |2 z| roundings more for 2 z's
// own (v^2, the sum of products and its constants; the product with |v| is brought in).
__device__ __forceinline__ float mx_gelu_tanh(float v)
{
#pragma clang fp contract(off)
    constexpr float kOne = -2.30220819f, kCube = -0.102943242f;   // -sqrt(8 / pi) log2(e), and 0.044715 times it
    const float x = fabsf(v), w = fmaf(v * v, kCube, kOne), t = x * w;
    return mx_times_logistic(v, t, fmaf(x, w, -t));
}

// v Phi(v), Phi the normal distribution: max(v, -0) - x Phi(-x) with x = |v|, and Phi(-x) =
// exp(-x^2 / 2) r(x), r(x) = erfcx(x / sqrt 2) / 2, which falls slowly: a polynomial in
// 1 / (1 + 0.3f x), fitted here to r on 0 <= x <= 13.3, where the power of two ends, by
// weighted least squares until its largest relative error was least (5.9e-8 with the
// coefficients as they are held).  Nothing cancels for negative v, as 1 + erf would, and
// x r, near 0.4 where exp(-x^2 / 2) is smallest, keeps the tail's product normal as long as
// the result is.  x^2's and its multiple's rounding are brought in behind the power of two.
// Within 18 roundings, each operation counted at its worst (the polynomial's variable 3 at
// a slope of 2.7, its sums 4.2, the power of two 3), and 6.8 over 59 thousand values down
// to results of 2^-126, in some 30 instructions (512 x 4096 x 14336 with blocks 55 us a pass).
__device__ __forceinline__ float mx_gelu(float v)
{
    constexpr float kC[9] = {6.6857497e-06f, 0.1194959f, 0.12186197f, 0.09491117f, 0.14200212f,
                             -0.07573549f, 0.2279869f, -0.16884065f, 0.03831141f};
    constexpr float kHalfLog2E = 0.721347511f, kHalfLog2ELow = 9.62981517e-9f, kLn2 = 0.693147181f;
    constexpr int kPositive = 0x180;   // finite, not zero; the others stand
    const float x = fabsf(v), t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.f));
    float r = kC[8];
#pragma unroll
    for (int i = 7; i >= 0; --i)
        r = fmaf(r, t, kC[i]);
    const float s = x * x, low = fmaf(x, x, -s), a = s * -kHalfLog2E;
    const float lost = fmaf(s, -kHalfLog2E, -a) - fmaf(low, kHalfLog2E, s * kHalfLog2ELow);
    const float p = __builtin_amdgcn_exp2f(a);
    const float e = __builtin_amdgcn_classf(p, kPositive) ? fmaf(p, lost * kLn2, p) : p;
    const float b = v > 0x1p100f ? 0x1p100f : x;   // infinity has no tail: not infinity times 0
    return fmaf(-(b * r), e, v < 0.f ? -0.f : v);
}

// Activations in fp32.
__device__ __forceinline__ void mx_activate(int act, float (&f)[8])
{
    if (act == LORA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = f[e] < 0.f ? 0.f : f[e];
    } else if (act == LORA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_silu(f[e]);
    } else if (act == LORA_ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_gelu(f[e]);
    } else if (act == LORA_ACT_GELU_TANH) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_gelu_tanh(f[e]);
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
                    f[e] = mx_silu(f[e]) * up[e];
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
