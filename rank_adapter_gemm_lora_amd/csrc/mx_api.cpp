// mx_api.cpp -- host side of the microscaled operators: argument checks, the
// 4-bit weight object and the kernel launches.  Every entry point returns a
// status; no exception leaves this file.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "mx.h"

using namespace lora;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(lora_dtype t) { return t == LORA_F32 || t == LORA_BF16; }
bool format_ok(lora_mx_format f) { return f == LORA_MX_E4M3 || f == LORA_MX_E2M1; }
int dt_of(lora_dtype t) { return t == LORA_F32 ? DT_F32 : DT_BF16; }
hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Widths and rows: negative or uneven ones are wrong, large ones unsupported.
lora_status check_shape(int64_t n_rows, int64_t k, int64_t k_max)
{
    if (n_rows < 0 || k < 8 || k % 8 != 0)
        return LORA_E_ARG;
    return n_rows >= kMxMaxRows || k > k_max ? LORA_E_UNSUPPORTED : LORA_OK;
}

// A dense matrix of n_rows x width elements with row stride ld; its last
// element's byte offset must fit 62 bits.
bool dense_ok(const void *p, int64_t ld, int64_t width, int64_t n_rows)
{
    return ld >= width && ld % 8 == 0 && ld < ((int64_t)1 << 58) / (n_rows + 1) &&
           (n_rows == 0 || (p && aligned16(p)));
}

bool blocks_ok(const void *q, int64_t ldq, const void *s, int64_t lds, lora_mx_format f, int64_t k,
               int64_t n_rows)
{
    return ldq >= LORA_MX_CODE_BYTES(k, f) && ldq % 16 == 0 && lds >= LORA_MX_SCALE_BYTES(k) &&
           lds % 16 == 0 && ldq < ((int64_t)1 << 60) / (n_rows + 1) &&
           lds < ((int64_t)1 << 60) / (n_rows + 1) &&
           (n_rows == 0 || (q && s && aligned16(q) && aligned16(s)));
}

MxBlocks blocks_of(const void *q, int64_t ldq, const void *s, int64_t lds)
{
    return MxBlocks{static_cast<uint8_t *>(const_cast<void *>(q)), ldq,
                    static_cast<uint8_t *>(const_cast<void *>(s)), lds};
}

bool on_device(const lora_mx_weight *w)
{
    int cur = -1;
    return hipGetDevice(&cur) == hipSuccess && cur == w->device;
}

}  // namespace

lora_status lora_mx_quantize(void *q, int64_t ldq, void *s, int64_t lds, lora_mx_format format,
                             const void *x, int64_t ldx, lora_dtype dtype, int64_t n_rows,
                             int64_t k, void *stream)
{
    if (!dtype_ok(dtype) || !format_ok(format))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, k, kMxMaxK);
    if (st != LORA_OK)
        return st;
    if (!dense_ok(x, ldx, k, n_rows) || !blocks_ok(q, ldq, s, lds, format, k, n_rows))
        return LORA_E_ARG;
    if (n_rows == 0)
        return LORA_OK;
    MxRowArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.b = blocks_of(q, ldq, s, lds);
    a.k = k;
    return status_of(launch_mx_quantize(dt_of(dtype), format, a, n_rows, stream_of(stream)));
}

lora_status lora_mx_dequantize(void *x, int64_t ldx, lora_dtype dtype, const void *q, int64_t ldq,
                               const void *s, int64_t lds, lora_mx_format format, int64_t n_rows,
                               int64_t k, void *stream)
{
    if (!dtype_ok(dtype) || !format_ok(format))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, k, kMxMaxK);
    if (st != LORA_OK)
        return st;
    if (!dense_ok(x, ldx, k, n_rows) || !blocks_ok(q, ldq, s, lds, format, k, n_rows))
        return LORA_E_ARG;
    if (n_rows == 0)
        return LORA_OK;
    MxRowArgs a{};
    a.out = x;
    a.ldo = ldx;
    a.b = blocks_of(q, ldq, s, lds);
    a.k = k;
    return status_of(launch_mx_dequantize(dt_of(dtype), format, a, n_rows, stream_of(stream)));
}

lora_status lora_mx_weight_create(lora_mx_weight **out, int64_t d, int64_t k)
{
    if (!out)
        return LORA_E_ARG;
    *out = nullptr;
    if (d < 8 || d % 8 != 0 || k < 8 || k % 8 != 0)
        return LORA_E_ARG;
    if (d > kMxMaxD || k > kMxMaxK)
        return LORA_E_UNSUPPORTED;
    lora_mx_weight *w = new (std::nothrow) lora_mx_weight();
    if (!w)
        return LORA_E_NOMEM;
    std::memset(w, 0, sizeof *w);
    w->w.d = d;
    w->w.k = k;
    w->w.tiles = (int)((d + kMxPadRows - 1) / kMxPadRows * (kMxPadRows / 16));
    w->w.chunks = (int)((k + kMxChunk - 1) / kMxChunk);
    hipError_t e = hipGetDevice(&w->device);
    if (e == hipSuccess)
        e = hipDeviceGetAttribute(&w->n_cu, hipDeviceAttributeMultiprocessorCount, w->device);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&w->w.codes), (size_t)w->w.tiles * w->w.chunks * 1024);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&w->w.scales),
                      (size_t)w->w.tiles * ((w->w.chunks + 3) / 4) * 256);
    if (e != hipSuccess) {
        (void)hipFree(w->w.codes);
        delete w;
        return status_of(e);
    }
    *out = w;
    return LORA_OK;
}

lora_status lora_mx_weight_destroy(lora_mx_weight *w)
{
    if (!w)
        return LORA_OK;
    const hipError_t e = hipDeviceSynchronize();
    (void)hipFree(w->w.codes);
    (void)hipFree(w->w.scales);
    delete w;
    return status_of(e);
}

lora_status lora_mx_weight_load(lora_mx_weight *w, const void *W, int64_t ldw, lora_dtype dtype,
                                void *stream)
{
    if (!w || !dtype_ok(dtype) || !dense_ok(W, ldw, w->w.k, w->w.d) || !on_device(w))
        return LORA_E_ARG;
    const lora_status st = status_of(
        launch_mx_image(dt_of(dtype), W, ldw, MxBlocks{}, w->w, stream_of(stream)));
    if (st == LORA_OK)
        w->loaded = 1;
    return st;
}

lora_status lora_mx_weight_load_packed(lora_mx_weight *w, const void *q, int64_t ldq,
                                       const void *s, int64_t lds, void *stream)
{
    if (!w || !blocks_ok(q, ldq, s, lds, LORA_MX_E2M1, w->w.k, w->w.d) || !on_device(w))
        return LORA_E_ARG;
    const lora_status st = status_of(
        launch_mx_image(-1, nullptr, 0, blocks_of(q, ldq, s, lds), w->w, stream_of(stream)));
    if (st == LORA_OK)
        w->loaded = 1;
    return st;
}

lora_status lora_mx_linear(const lora_mx_weight *w, void *y, int64_t ldy, lora_dtype dtype,
                           const void *q, int64_t ldq, const void *s, int64_t lds,
                           lora_mx_format format, int64_t n_rows, void *stream)
{
    if (!w || !dtype_ok(dtype) || !format_ok(format))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, w->w.k, kMxMaxK);
    if (st != LORA_OK)
        return st;
    if (!dense_ok(y, ldy, w->w.d, n_rows) || !blocks_ok(q, ldq, s, lds, format, w->w.k, n_rows) ||
        !on_device(w))
        return LORA_E_ARG;
    if (!w->loaded)
        return LORA_E_EMPTY;
    if (n_rows == 0)
        return LORA_OK;
    MxLinearArgs a{};
    a.w = w->w;
    a.q = static_cast<const uint8_t *>(q);
    a.ldq = ldq;
    a.s = static_cast<const uint8_t *>(s);
    a.lds = lds;
    a.y = y;
    a.ldy = ldy;
    a.n_rows = n_rows;
    a.n_cu = w->n_cu;
    return status_of(launch_mx_linear(dt_of(dtype), format, a, stream_of(stream)));
}

lora_status lora_rmsnorm_mx(void *out, int64_t ldo, void *q, int64_t ldq, void *s, int64_t lds,
                            void *h_out, int64_t ldh, const void *x, int64_t ldx,
                            const void *residual, int64_t ldr, const void *weight, float eps,
                            lora_dtype dtype, int64_t n_rows, int64_t k, void *stream)
{
    if (!dtype_ok(dtype) || !(eps >= 0.f) || !std::isfinite(eps))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, k, kMxMaxNormK);
    if (st != LORA_OK)
        return st;
    if ((!out && !q && !h_out) || !q != !s || !dense_ok(x, ldx, k, n_rows) ||
        !dense_ok(weight, k, k, 1) || (residual && !dense_ok(residual, ldr, k, n_rows)) ||
        (h_out && !dense_ok(h_out, ldh, k, n_rows)) || (out && !dense_ok(out, ldo, k, n_rows)) ||
        (q && !blocks_ok(q, ldq, s, lds, LORA_MX_E4M3, k, n_rows)))
        return LORA_E_ARG;
    if (n_rows == 0)
        return LORA_OK;
    MxNormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.res = residual;
    a.ldr = ldr;
    a.weight = weight;
    a.eps = eps;
    a.inv_k = 1. / (double)k;
    a.h = h_out;
    a.ldh = ldh;
    a.out = out;
    a.ldo = ldo;
    a.b = blocks_of(q, ldq, s, lds);
    a.n_rows = n_rows;
    a.k = k;
    return status_of(launch_rmsnorm_mx(dt_of(dtype), a, stream_of(stream)));
}

lora_status lora_swiglu_mx(void *out, int64_t ldo, void *q, int64_t ldq, void *s, int64_t lds,
                           const void *gu, int64_t ldg, lora_dtype dtype, int64_t n_rows,
                           int64_t f, void *stream)
{
    if (!dtype_ok(dtype))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, f, kMxMaxK);
    if (st != LORA_OK)
        return st;
    if ((!out && !q) || !q != !s || !dense_ok(gu, ldg, 2 * f, n_rows) ||
        (out && !dense_ok(out, ldo, f, n_rows)) ||
        (q && !blocks_ok(q, ldq, s, lds, LORA_MX_E4M3, f, n_rows)))
        return LORA_E_ARG;
    if (n_rows == 0)
        return LORA_OK;
    MxRowArgs a{};
    a.x = gu;
    a.ldx = ldg;
    a.out = out;
    a.ldo = ldo;
    a.b = blocks_of(q, ldq, s, lds);
    a.k = f;
    return status_of(launch_swiglu_mx(dt_of(dtype), a, n_rows, stream_of(stream)));
}
