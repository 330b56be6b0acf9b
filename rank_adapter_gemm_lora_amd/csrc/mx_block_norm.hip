// mx_block_norm.hip -- what stands between two blocks of a layer: the norm of
// the finished block's output, its gate and residual scale, the residual sum,
// and the next block's norm with block outputs, from one pass.  Bound by HBM
// traffic: y, the residual and a gate by rows are read once, h, n and the
// blocks of n written once.
#include <type_traits>

#include "mx_device.h"

namespace lora {

namespace {

// Sum over a wavefront, the same in every lane: butterflies inside rows of 16 by
// register moves (neighbours, pairs, then the row's halves mirrored), then the
// four rows' sums in row order.
__device__ __forceinline__ double wave_sum(double v)
{
    auto moved = [](double x, auto ctrl) {
        const int64_t b = __double_as_longlong(x);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, decltype(ctrl)::value, 0xF, 0xF, true);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), decltype(ctrl)::value, 0xF, 0xF, true);
        return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
    };
    v += moved(v, std::integral_constant<int, 0xB1>{});    // quad permutation 1 0 3 2
    v += moved(v, std::integral_constant<int, 0x4E>{});    // quad permutation 2 3 0 1
    v += moved(v, std::integral_constant<int, 0x141>{});   // halves of a row mirrored
    v += moved(v, std::integral_constant<int, 0x140>{});   // rows mirrored
    const int64_t b = __double_as_longlong(v);
    double s = 0.;
#pragma unroll
    for (int r = 0; r < 64; r += 16) {
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, r);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), r);
        s += __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
    }
    return s;
}

// The same over the workgroup's T threads; part: T / 64 values of this sum alone.
template <int T> __device__ __forceinline__ double block_sum(double v, double *part)
{
    v = wave_sum(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.;
#pragma unroll
        for (int w = 0; w < T / 64; ++w)
            v += part[w];
    }
    return v;
}

// v as a float that rounds to bf16 or a code as v itself does: 21 bits of v, the
// last one set where anything below it is (rounded to odd), which a float holds
// exactly (under 2^-126 the float's own rounding comes first).
__device__ __forceinline__ float mx_odd_of(double v)
{
    const int64_t b = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32) | min(lo, 1u);
    float f = (float)__longlong_as_double((int64_t)((uint64_t)hi << 32));
    asm("" : "+v"(f));   // or the compiler joins the two conversions into a longer one of its own
    return f;
}

// One row per workgroup of T threads, NU units of 8 elements a thread (unit t +
// T j).  All of a row is loaded before anything is written, so outputs may
// replace inputs.  Everything between the loads and the stores is in 64 bits
// (the vector units run 64-bit products and sums at the 32-bit ones' rate): h and n
// then differ from their exact values by some 2^-50, and each output is that value
// rounded once.  A weight times a gate is exact there, where in fp32 it could leave
// the range of both (35422 x 4096 with either: 318 us a pass).  Up to two units a
// thread the weights come with the row, ahead of the sums; beyond, the registers
// would not hold them.
//
// 35422 x 4096 bf16 with a channel's gate: 245 us, 1.31 GB at 5.3 TB/s, the vector
// units issuing 73 % of the time (a pass with the blocks' inverse 322 us; weights
// loaded where they are used 344, one unit of 512 threads 350, four of 128 327).
// 1 x 4096: 3.7 us.  Rows past 16384 go over the 128 registers of a lane of 1024
// threads: 28 bytes of each in bf16, 228 in fp32, are kept in scratch (a call of 64 x
// 32768 15.9 and 46 us, of 64 x 16384 8.6 and 10.1).
template <int DT, int NU, int T>
__global__ __launch_bounds__(T) void block_norm_mx_kernel(MxBlockNormArgs a)
{
    __shared__ double part[2][T / 64];
    constexpr bool kEarly = NU <= 2;
    const int tid = threadIdx.x;
    const int64_t row = a.row0 + blockIdx.x;
    const int units = (int)((a.k + kMxChunk - 1) / kMxChunk) * (kMxChunk / 8);
    Vec8<DT> vy[NU], vr[NU], vg[NU], vpost[NU], vpre[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int64_t c = (int64_t)(tid + T * j) * 8;
        if (c < a.k) {
            vy[j].load(a.y, row * a.ldy + c);
            if (a.res)
                vr[j].load(a.res, row * a.ldr + c);
            else
                vr[j].zero();
            if (a.gate)
                vg[j].load(a.gate, row * a.ldg + c);
            if (kEarly && a.post)
                vpost[j].load(a.post, c);
            if (kEarly && a.pre)
                vpre[j].load(a.pre, c);
        }
    }
    double h[NU][8];   // y first
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        float f[8];
        vy[j].to_f32(f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[j][e] = (double)f[e];
    }
    double by = a.scale;   // what y is multiplied by next to its weight and gate
    if (a.post) {
        double sum = 0.;
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            if ((int64_t)(tid + T * j) * 8 < a.k) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum = fma(h[j][e], h[j][e], sum);
            }
        }
        by *= rsqrt(block_sum<T>(sum, part[0]) * a.inv_k + a.eps);
    }
    double sum = 0.;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int64_t c = (int64_t)(tid + T * j) * 8;
        if (c < a.k) {
            if (!kEarly && a.post)
                vpost[j].load(a.post, c);
            float r[8];
            vr[j].to_f32(r);
            if (a.post && a.gate) {
                float g[8], w[8];
                vg[j].to_f32(g);
                vpost[j].to_f32(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double m = (double)w[e] * (double)g[e];
                    h[j][e] = fma(by * h[j][e], m, (double)r[e]);
                }
            } else if (a.post || a.gate) {
                float w[8];
                if (a.post)
                    vpost[j].to_f32(w);
                else
                    vg[j].to_f32(w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] = fma(by * h[j][e], (double)w[e], (double)r[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[j][e] = fma(by, h[j][e], (double)r[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = fma(h[j][e], h[j][e], sum);
        }
    }
    double inv = 0.;
    if (a.pre)
        inv = rsqrt(block_sum<T>(sum, part[1]) * a.inv_k + a.eps);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int unit = tid + T * j;
        const int64_t c = (int64_t)unit * 8;
        float n[8];
        if (c < a.k) {
            float f[8], w[8];
            if (a.h) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = DT == DT_F32 ? (float)h[j][e] : mx_odd_of(h[j][e]);
                Vec8<DT>::store(a.h, row * a.ldh + c, f);
            }
            if (a.pre) {
                if (!kEarly)
                    vpre[j].load(a.pre, c);
                vpre[j].to_f32(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double v = h[j][e] * inv * (double)w[e];
                    n[e] = mx_odd_of(v);
                    f[e] = DT == DT_F32 ? (float)v : n[e];
                }
                if (a.out)
                    Vec8<DT>::store(a.out, row * a.ldo + c, f);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                n[e] = 0.f;
        }
        if (a.b.q && unit < units)   // whole 16-lane groups
            mx_store_unit<LORA_MX_E4M3>(a.b.q + row * a.b.ldq, a.b.s + row * a.b.lds, unit, units, n);
    }
}

template <int DT, int NU, int T> void block_norm_go(MxBlockNormArgs a, hipStream_t s)
{
    for_slabs(a.n_rows, slab_rows(1, 1, T), [&](int64_t row0, int64_t rows) {
        a.row0 = row0;
        block_norm_mx_kernel<DT, NU, T><<<dim3((uint32_t)rows), dim3(T), 0, s>>>(a);
    });
}

template <int DT> void block_norm_pick(const MxBlockNormArgs &a, hipStream_t s)
{
    const int64_t units = (a.k + 7) / 8;
    if (units <= 64)
        block_norm_go<DT, 1, 64>(a, s);
    else if (units <= 256)
        block_norm_go<DT, 1, 256>(a, s);
    else if (units <= 512)
        block_norm_go<DT, 2, 256>(a, s);
    else if (units <= 1024)
        block_norm_go<DT, 2, 512>(a, s);
    else if (units <= 2048)
        block_norm_go<DT, 4, 512>(a, s);
    else
        block_norm_go<DT, 4, 1024>(a, s);
}

}  // namespace

hipError_t launch_block_norm_mx(int dtype, const MxBlockNormArgs &a, hipStream_t s)
{
    if (dtype == DT_F32)
        block_norm_pick<DT_F32>(a, s);
    else
        block_norm_pick<DT_BF16>(a, s);
    return hipGetLastError();
}

}  // namespace lora
