// mx_rows.hip -- the row-wise microscaled operators: quantisation and its
// inverse, the weight image, the gated activation and the RMS norm with their
// block outputs.  All are bound by HBM traffic: each input element is read
// once and each output written once.
#include "mx_device.h"

namespace lora {

namespace {

constexpr int kRowThreads = 256;

// Units of 8 elements that a thread takes, kRowThreads apart; their loads are
// all issued before the first is used (14336 x 4096 bf16 to e2m1: 30.1 us, 148
// MB at 4.9 TB/s; with one unit 31.4 us).
constexpr int kRowUnits = 2;

struct MxUnitAt {
    int64_t row;
    int unit;
    bool in;   // of this launch (whole groups of 16 lanes: n_units is a multiple of 16)
};
__device__ __forceinline__ MxUnitAt mx_unit_at(const MxRowArgs &a, int j)
{
    const uint32_t i = blockIdx.x * (kRowThreads * kRowUnits) + kRowThreads * j + threadIdx.x;
    const uint32_t r = mx_div_of(i, a.div);
    return MxUnitAt{a.row0 + r, (int)(i - r * a.div.d), i < a.n_units};
}

// x -> blocks.  Per element: the input's 2 or 4 bytes in, 33/32 (e4m3) or
// 17/32 (e2m1) bytes out.
template <int DT, int FMT>
__global__ __launch_bounds__(kRowThreads) void mx_quantize_kernel(MxRowArgs a)
{
    MxUnitAt at[kRowUnits];
    Vec8<DT> v[kRowUnits];
#pragma unroll
    for (int j = 0; j < kRowUnits; ++j) {
        at[j] = mx_unit_at(a, j);
        v[j].zero();
        if (at[j].in && (int64_t)at[j].unit * 8 < a.k)
            v[j].load(a.x, at[j].row * a.ldx + at[j].unit * 8);
    }
#pragma unroll
    for (int j = 0; j < kRowUnits; ++j) {
        if (!at[j].in)
            return;
        float f[8];
        v[j].to_f32(f);
        mx_store_unit<FMT>(a.b.q + at[j].row * a.b.ldq, a.b.s + at[j].row * a.b.lds, at[j].unit,
                           (int)a.div.d, f);
    }
}

// silu(g) * u -> a dense row and blocks (512 x 14336 bf16: 14.0 us, 52 MB at 3.7
// TB/s, bound by its instructions; 15.0 us with a true division.  The hardware's
// exponential with its error carried takes 13.3 us at the same error, 3.6e-8 -
// 4.5e-8 in the root mean square, but one code in some millions then differs from
// the elementary operations').
template <int DT>
__global__ __launch_bounds__(kRowThreads) void swiglu_mx_kernel(MxRowArgs a)
{
    MxUnitAt at[kRowUnits];
    Vec8<DT> vg[kRowUnits], vu[kRowUnits];
#pragma unroll
    for (int j = 0; j < kRowUnits; ++j) {
        at[j] = mx_unit_at(a, j);
        vg[j].zero();
        vu[j].zero();
        if (at[j].in && (int64_t)at[j].unit * 8 < a.k) {
            vg[j].load(a.x, at[j].row * a.ldx + at[j].unit * 8);
            vu[j].load(a.x, at[j].row * a.ldx + a.k + at[j].unit * 8);
        }
    }
#pragma unroll
    for (int j = 0; j < kRowUnits; ++j) {
        if (!at[j].in)
            return;
        float g[8], u[8], f[8];
        vg[j].to_f32(g);
        vu[j].to_f32(u);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = mx_silu_mul(g[e], u[e]);
        if (a.out && (int64_t)at[j].unit * 8 < a.k)
            Vec8<DT>::store(a.out, at[j].row * a.ldo + at[j].unit * 8, f);
        if (a.b.q)
            mx_store_unit<LORA_MX_E4M3>(a.b.q + at[j].row * a.b.ldq, a.b.s + at[j].row * a.b.lds,
                                        at[j].unit, (int)a.div.d, f);
    }
}

// e4m3 / e2m1 codes of 8 elements -> fp32 (the conversions are exact).
template <int FMT>
__device__ __forceinline__ void mx_values(typename MxFmt<FMT>::unit_t c, float (&f)[8])
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    f32x2_t p[4];
    if constexpr (FMT == LORA_MX_E4M3) {
        p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false);
        p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
        p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false);
        p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        f[2 * m] = p[m].x;
        f[2 * m + 1] = p[m].y;
    }
}

// 2^(sb - 127) as a float; 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t sb)
{
    return __uint_as_float(sb == 0 ? 0x00400000u : sb == 255 ? 0x7fc00000u : sb << 23);
}

// blocks -> values
template <int DT, int FMT>
__global__ __launch_bounds__(kRowThreads) void mx_dequantize_kernel(MxRowArgs a)
{
    const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x;
    if (i >= a.n_units)
        return;
    const uint32_t r = mx_div_of(i, a.div);
    const int unit = (int)(i - r * a.div.d);
    const int64_t row = a.row0 + r;
    if ((int64_t)unit * 8 >= a.k)
        return;
    const auto c = *reinterpret_cast<const typename MxFmt<FMT>::unit_t *>(
        a.b.q + row * a.b.ldq + (int64_t)unit * MxFmt<FMT>::unit_bytes);
    const float sc = mx_scale_value(a.b.s[row * a.b.lds + (unit >> 2)]);
    float f[8];
    mx_values<FMT>(c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] *= sc;
    Vec8<DT>::store(a.out, row * a.ldo + unit * 8, f);
}

// Where the image keeps output feature o.
__device__ __forceinline__ int64_t mx_image_tile(int64_t o) { return (o >> 5) * 2 + ((o >> 2) & 1); }
__device__ __forceinline__ int mx_image_row(int64_t o) { return (int)(((o >> 3) & 3) * 4 + (o & 3)); }

// The weight's row that image feature j holds; -1 where it is padding.
__device__ __forceinline__ int64_t mx_image_source(const MxImage &w, int64_t j)
{
    if (w.half == 0)
        return j < w.d ? j : -1;
    const int64_t o = (j >> 6) * 32 + (j & 31);
    return o < w.half ? ((j >> 5) & 1) * w.half + o : -1;
}

// Dense rows -> weight image: thread = (feature, unit of 8 k).  Runs once per
// weight, not tuned beyond reading whole 16-byte units.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void mx_image_dense_kernel(const void *src, int64_t ldw,
                                                                     MxImage w)
{
    const int units = w.chunks * 16, groups = (w.chunks + 3) / 4;
    const int unit = blockIdx.y * kRowThreads + threadIdx.x;
    const int64_t o = blockIdx.x, row = mx_image_source(w, o);
    if (unit >= units)
        return;
    Vec8<DT> v;
    v.zero();
    if (row >= 0 && (int64_t)unit * 8 < w.k)
        v.load(src, row * ldw + unit * 8);
    float f[8];
    v.to_f32(f);
    const uint32_t sb = mx_block_scale<LORA_MX_E2M1>(f);
    const int chunk = unit >> 4, lane = 16 * ((unit >> 2) & 3) + mx_image_row(o);
    const int64_t tile = mx_image_tile(o);
    *reinterpret_cast<uint32_t *>(w.codes + (((int64_t)chunk * w.tiles + tile) * 64 + lane) * 16 +
                                  4 * (unit & 3)) = mx_codes<LORA_MX_E2M1>(f, sb);
    if ((unit & 3) == 0) {
        uint8_t *sc = w.scales + (((int64_t)(chunk >> 2) * w.tiles + tile) * 64 + lane) * 4;
        sc[chunk & 3] = (uint8_t)sb;
        if (chunk == w.chunks - 1)
            for (int j = w.chunks; j < groups * 4; ++j)
                sc[j & 3] = 0;
    }
}

// Rows in e2m1 blocks -> weight image: thread = (feature, block of 32).  Codes
// and scales past k are replaced by zeros (k is a multiple of 8: whole words).
__global__ __launch_bounds__(kRowThreads) void mx_image_packed_kernel(MxBlocks b, MxImage w)
{
    const int blocks = w.chunks * 4, groups = (w.chunks + 3) / 4;
    const int blk = blockIdx.y * kRowThreads + threadIdx.x;
    const int64_t o = blockIdx.x, row = mx_image_source(w, o);
    if (blk >= blocks)
        return;
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t sb = 0;
    const int64_t k0 = (int64_t)blk * 32;
    if (row >= 0 && k0 < w.k) {
        c = *reinterpret_cast<const uint4 *>(b.q + row * b.ldq + (int64_t)blk * 16);
        sb = b.s[row * b.lds + blk];
        c.y = k0 + 8 < w.k ? c.y : 0u;
        c.z = k0 + 16 < w.k ? c.z : 0u;
        c.w = k0 + 24 < w.k ? c.w : 0u;
    }
    const int chunk = blk >> 2, lane = 16 * (blk & 3) + mx_image_row(o);
    const int64_t tile = mx_image_tile(o);
    *reinterpret_cast<uint4 *>(w.codes + (((int64_t)chunk * w.tiles + tile) * 64 + lane) * 16) = c;
    uint8_t *sc = w.scales + (((int64_t)(chunk >> 2) * w.tiles + tile) * 64 + lane) * 4;
    sc[chunk & 3] = (uint8_t)sb;
    if (chunk == w.chunks - 1)
        for (int j = w.chunks; j < groups * 4; ++j)
            sc[j & 3] = 0;
}

// (x + y) 2^e = 1 / sqrt(m): the hardware's reciprocal root (within 2^-23), one
// Newton step on m's high and low parts, and what rounding that step loses.  An m
// that is, or whose root is, near the ends of fp32's range is brought to [1/4, 1) by
// an even power of two first; its root's power is left for h (a mean square of 2^250
// has a root, but no fp32 square).  y and e are 0 where m is 0 or not finite.
struct MxRoot {
    float x, y;
    int e;
};
__device__ __forceinline__ MxRoot mx_inv_sqrt(double m)
{
    int e = 0;
    if (!(m >= 0x1p-96 && m < 0x1p96)) {
        e = -((__builtin_amdgcn_frexp_exp(m) + 1) >> 1);
        m = __builtin_ldexp(m, 2 * e);
    }
    const float hi = (float)m, lo = (float)(m - hi);
    const float r = __builtin_amdgcn_rsqf(hi);
    float x = r, y = 0.f;
    if (hi > 0.f && hi < INFINITY) {
        const float t = hi * r, tl = fmaf(hi, r, -t);
        const float left = fmaf(-t, r, 1.f) - fmaf(lo * r, r, tl * r);   // 1 - m r^2
        x = fmaf(0.5f * r, left, r);
        y = fmaf(0.5f * r, left, -(x - r));
    }
    return MxRoot{x, y, e};
}

// n + l (l under half a step of n) rounded to odd: towards zero, then the last
// bit set; n itself if l is 0 or not finite.  Rounding that to a shorter format
// gives what n + l itself rounds to, which n would not on a border (l decides).
// l is 0 where n is: the sign's subtraction never passes 0.
__device__ __forceinline__ float mx_to_odd(float n, float l)
{
    constexpr int kFiniteNotZero = 0x198;   // normals and subnormals of either sign
    const int b = __float_as_int(n);
    const int odd = (b + ((__float_as_int(l) ^ b) >> 31)) | 1;
    return __int_as_float(__builtin_amdgcn_classf(l, kFiniteNotZero) ? odd : b);
}

// One row per workgroup of T threads; the row stays in registers, NU units of 8
// a thread (unit t + T j), so x and the residual are read once and nothing is
// written before the whole row is in.  (fp32 rows past 32768, eight units a thread
// of 1024, go over the 128 registers of a lane: 64 bytes of each are kept in
// scratch.  64 x 65536: 27 us.)
// The squares are summed in 64 bits, so that the codes of n + lost are the exact
// value's but for its last bits: none of 4.3 M differed (fp32 sums: 4, and codes
// of the rounded n: 7).  35422 x 4096 bf16: 225 - 228 us, 1.3 GB at 5.7 TB/s,
// and as long with fp32 sums and codes; 300 x 14336, one to two rows a CU and bound
// by their instructions: 11.2 us (a pass with its inverse 16.0 us; with fp32 sums
// and codes 14.9).
template <int DT, int NU, int T>
__global__ __launch_bounds__(T) void rmsnorm_mx_kernel(MxNormArgs a)
{
    __shared__ double part[T / 64];
    const int tid = threadIdx.x;
    const int64_t row = a.row0 + blockIdx.x;
    const int units = (int)((a.k + kMxChunk - 1) / kMxChunk) * (kMxChunk / 8);
    Vec8<DT> vx[NU], vr[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int64_t c = (int64_t)(tid + T * j) * 8;
        vx[j].zero();
        vr[j].zero();
        if (c < a.k) {
            vx[j].load(a.x, row * a.ldx + c);
            if (a.res)
                vr[j].load(a.res, row * a.ldr + c);
        }
    }
    float f[NU][8];
    double sum = 0.;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        float r[8];
        vx[j].to_f32(f[j]);
        vr[j].to_f32(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[j][e] += r[e];
            sum = fma((double)f[j][e], (double)f[j][e], sum);
        }
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1)
        sum += __shfl_xor(sum, m);
    if (T > 64) {
        if ((tid & 63) == 0)
            part[tid >> 6] = sum;
        __syncthreads();
        sum = 0.;
#pragma unroll
        for (int w = 0; w < T / 64; ++w)
            sum += part[w];
    }
    const MxRoot inv = mx_inv_sqrt(sum * a.inv_k + a.eps);
    const int far = __builtin_amdgcn_readfirstlane(inv.e);   // the same in every lane
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int unit = tid + T * j;
        const int64_t c = (int64_t)unit * 8;
        if (c < a.k) {
            if (a.h)
                Vec8<DT>::store(a.h, row * a.ldh + c, f[j]);
            Vec8<DT> vw;
            vw.load(a.weight, c);
            float w[8], n[8];
            vw.to_f32(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // h inv w and what its roundings lose: n is near the once-rounded
                // value, and its codes are taken of n + lost, not of n.  (A product
                // that is not finite stands without the lost part.)
                const float fj = __builtin_ldexpf(f[j][e], far);
                const float p = fj * inv.x, pw = p * w[e];
                const float l = fmaf(fj, inv.x, -p) + fj * inv.y;
                n[e] = fabsf(pw) < INFINITY ? fmaf(p, w[e], l * w[e]) : pw;
                f[j][e] = mx_to_odd(n[e], fmaf(l, w[e], fmaf(p, w[e], -n[e])));
            }
            if (a.out)
                Vec8<DT>::store(a.out, row * a.ldo + c, n);
        }
        if (a.b.q && unit < units)   // whole 16-lane groups
            mx_store_unit<LORA_MX_E4M3>(a.b.q + row * a.b.ldq, a.b.s + row * a.b.lds, unit, units,
                                        f[j]);
    }
}

// Launch `go` over slabs of rows whose units fit 31 bits.
template <class F> hipError_t by_slabs(MxRowArgs a, int64_t n_rows, int per_thread, F go)
{
    const int64_t units = (a.k + kMxChunk - 1) / kMxChunk * (kMxChunk / 8);
    a.div = mx_div((uint32_t)units);
    const int64_t most = ((int64_t)1 << 30) / units;
    for (int64_t r = 0; r < n_rows; r += most) {
        a.row0 = r;
        a.n_units = (uint32_t)((n_rows - r < most ? n_rows - r : most) * units);
        const uint32_t per = kRowThreads * per_thread;
        go(a, dim3((a.n_units + per - 1) / per));
    }
    return hipGetLastError();
}

template <int DT, int NU, int T> void norm_go(MxNormArgs a, hipStream_t s)
{
    for_slabs(a.n_rows, slab_rows(1, 1, T), [&](int64_t row0, int64_t rows) {
        a.row0 = row0;
        rmsnorm_mx_kernel<DT, NU, T><<<dim3((uint32_t)rows), dim3(T), 0, s>>>(a);
    });
}

template <int DT> void norm_pick(const MxNormArgs &a, hipStream_t s)
{
    const int64_t units = (a.k + 7) / 8;
    if (units <= 64)
        norm_go<DT, 1, 64>(a, s);
    else if (units <= 256)
        norm_go<DT, 1, 256>(a, s);
    else if (units <= 512)
        norm_go<DT, 2, 256>(a, s);
    else if (units <= 1024)
        norm_go<DT, 4, 256>(a, s);
    else if (units <= 2048)
        norm_go<DT, 4, 512>(a, s);
    else if (units <= 4096)
        norm_go<DT, 4, 1024>(a, s);
    else
        norm_go<DT, 8, 1024>(a, s);
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, int format, MxRowArgs a, int64_t n_rows, hipStream_t s)
{
    return by_slabs(a, n_rows, kRowUnits, [&](const MxRowArgs &b, dim3 grid) {
        if (dtype == DT_F32 && format == LORA_MX_E4M3)
            mx_quantize_kernel<DT_F32, LORA_MX_E4M3><<<grid, kRowThreads, 0, s>>>(b);
        else if (dtype == DT_F32)
            mx_quantize_kernel<DT_F32, LORA_MX_E2M1><<<grid, kRowThreads, 0, s>>>(b);
        else if (format == LORA_MX_E4M3)
            mx_quantize_kernel<DT_BF16, LORA_MX_E4M3><<<grid, kRowThreads, 0, s>>>(b);
        else
            mx_quantize_kernel<DT_BF16, LORA_MX_E2M1><<<grid, kRowThreads, 0, s>>>(b);
    });
}

hipError_t launch_mx_dequantize(int dtype, int format, MxRowArgs a, int64_t n_rows, hipStream_t s)
{
    return by_slabs(a, n_rows, 1, [&](const MxRowArgs &b, dim3 grid) {
        if (dtype == DT_F32 && format == LORA_MX_E4M3)
            mx_dequantize_kernel<DT_F32, LORA_MX_E4M3><<<grid, kRowThreads, 0, s>>>(b);
        else if (dtype == DT_F32)
            mx_dequantize_kernel<DT_F32, LORA_MX_E2M1><<<grid, kRowThreads, 0, s>>>(b);
        else if (format == LORA_MX_E4M3)
            mx_dequantize_kernel<DT_BF16, LORA_MX_E4M3><<<grid, kRowThreads, 0, s>>>(b);
        else
            mx_dequantize_kernel<DT_BF16, LORA_MX_E2M1><<<grid, kRowThreads, 0, s>>>(b);
    });
}

hipError_t launch_swiglu_mx(int dtype, MxRowArgs a, int64_t n_rows, hipStream_t s)
{
    return by_slabs(a, n_rows, kRowUnits, [&](const MxRowArgs &b, dim3 grid) {
        if (dtype == DT_F32)
            swiglu_mx_kernel<DT_F32><<<grid, kRowThreads, 0, s>>>(b);
        else
            swiglu_mx_kernel<DT_BF16><<<grid, kRowThreads, 0, s>>>(b);
    });
}

hipError_t launch_rmsnorm_mx(int dtype, const MxNormArgs &a, hipStream_t s)
{
    if (dtype == DT_F32)
        norm_pick<DT_F32>(a, s);
    else
        norm_pick<DT_BF16>(a, s);
    return hipGetLastError();
}

hipError_t launch_mx_image(int dtype, const void *src, int64_t ldw, const MxBlocks &b,
                           const MxImage &w, hipStream_t s)
{
    const uint32_t rows = (uint32_t)w.tiles * 16;
    const uint32_t per = dtype < 0 ? w.chunks * 4 : w.chunks * 16;
    const dim3 grid(rows, (per + kRowThreads - 1) / kRowThreads);
    if (dtype < 0)
        mx_image_packed_kernel<<<grid, kRowThreads, 0, s>>>(b, w);
    else if (dtype == DT_F32)
        mx_image_dense_kernel<DT_F32><<<grid, kRowThreads, 0, s>>>(src, ldw, w);
    else
        mx_image_dense_kernel<DT_BF16><<<grid, kRowThreads, 0, s>>>(src, ldw, w);
    return hipGetLastError();
}

}  // namespace lora
