// mx_api.cpp -- host side of the microscaled operators: argument checks, the
// 4-bit weight object and the kernel launches.  Every entry point returns a
// status; no exception leaves this file.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "mx_checks.h"
#include "mx_job.h"

using namespace lora;

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
    if (!w || !dtype_ok(dtype) || !dense_ok(W, ldw, w->w.k, w->w.d) || !on_device(w->device))
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
    if (!w || !blocks_ok(q, ldq, s, lds, LORA_MX_E2M1, w->w.k, w->w.d) || !on_device(w->device))
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
        !on_device(w->device))
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

lora_status lora_mx_linear_fused(const lora_mx_weight *w, void *y, int64_t ldy, void *yq,
                                 int64_t ldyq, void *ys, int64_t ldys, lora_dtype dtype,
                                 const void *q, int64_t ldq, const void *s, int64_t lds,
                                 lora_mx_format format, const void *bias, lora_act act,
                                 const void *residual, int64_t ldr, int64_t n_rows, void *stream)
{
    if (!w || !dtype_ok(dtype) || !format_ok(format) || act < LORA_ACT_NONE || act >= LORA_ACT_SWIGLU)
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, w->w.k, kMxMaxK);
    if (st != LORA_OK)
        return st;
    if ((!y && !yq) || !yq != !ys || (y && !dense_ok(y, ldy, w->w.d, n_rows)) ||
        (yq && !blocks_ok(yq, ldyq, ys, ldys, LORA_MX_E4M3, w->w.d, n_rows)) ||
        !blocks_ok(q, ldq, s, lds, format, w->w.k, n_rows) || (bias && !aligned16(bias)) ||
        (residual && !dense_ok(residual, ldr, w->w.d, n_rows)) || !on_device(w->device))
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
    a.n_rows = n_rows;
    a.n_cu = w->n_cu;
    MxEpilogue e{};
    e.bias = bias;
    e.res = residual;
    e.ldr = ldr;
    e.y = y;
    e.ldy = ldy;
    e.b = blocks_of(yq, ldyq, ys, ldys);
    e.d = w->w.d;
    e.dtype = dt_of(dtype);
    e.act = act;
    return status_of(launch_mx_linear_fused(format, a, e, stream_of(stream)));
}

lora_status lora_mx_experts_create(lora_mx_experts **out, int n_experts, int64_t d, int64_t k,
                                   int gated)
{
    if (!out)
        return LORA_E_ARG;
    *out = nullptr;
    const int unit = gated ? 16 : 8;
    if (n_experts < 1 || d < unit || d % unit != 0 || k < 8 || k % 8 != 0)
        return LORA_E_ARG;
    if (n_experts > LORA_MAX_EXPERTS || d > kMxMaxD || k > kMxMaxK)
        return LORA_E_UNSUPPORTED;
    lora_mx_experts *x = new (std::nothrow) lora_mx_experts();
    if (!x)
        return LORA_E_NOMEM;
    std::memset(x, 0, sizeof *x);
    x->experts = n_experts;
    x->gated = gated != 0;
    x->rows = d;
    x->d = gated ? d / 2 : d;
    x->w.half = gated ? d / 2 : 0;
    x->w.d = gated ? mx_gated_features(d / 2) : d;
    x->w.k = k;
    x->w.tiles = (int)((x->w.d + kMxPadRows - 1) / kMxPadRows * (kMxPadRows / 16));
    x->w.chunks = (int)((k + kMxChunk - 1) / kMxChunk);
    x->code_stride = (int64_t)x->w.tiles * x->w.chunks * 1024;
    x->scale_stride = (int64_t)x->w.tiles * ((x->w.chunks + 3) / 4) * 256;
    hipError_t e = hipGetDevice(&x->device);
    if (e == hipSuccess)
        e = hipDeviceGetAttribute(&x->n_cu, hipDeviceAttributeMultiprocessorCount, x->device);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&x->w.codes), (size_t)n_experts * x->code_stride);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&x->w.scales), (size_t)n_experts * x->scale_stride);
    if (e != hipSuccess) {
        (void)hipFree(x->w.codes);
        delete x;
        return status_of(e);
    }
    *out = x;
    return LORA_OK;
}

lora_status lora_mx_experts_destroy(lora_mx_experts *x)
{
    if (!x)
        return LORA_OK;
    const hipError_t e = hipDeviceSynchronize();
    (void)hipFree(x->w.codes);
    (void)hipFree(x->w.scales);
    delete x;
    return status_of(e);
}

namespace {

lora_status experts_load(lora_mx_experts *x, int expert, int dtype, const void *W, int64_t ldw,
                         const MxBlocks &b, void *stream)
{
    if (expert < 0 || expert >= x->experts || !on_device(x->device))
        return LORA_E_ARG;
    MxImage w = x->w;
    w.codes += expert * x->code_stride;
    w.scales += expert * x->scale_stride;
    const lora_status st = status_of(launch_mx_image(dtype, W, ldw, b, w, stream_of(stream)));
    if (st == LORA_OK && !x->loaded[expert]) {
        x->loaded[expert] = 1;
        ++x->n_loaded;
    }
    return st;
}

}  // namespace

lora_status lora_mx_experts_load(lora_mx_experts *x, int expert, const void *W, int64_t ldw,
                                 lora_dtype dtype, void *stream)
{
    if (!x || !dtype_ok(dtype) || !dense_ok(W, ldw, x->w.k, x->rows))
        return LORA_E_ARG;
    return experts_load(x, expert, dt_of(dtype), W, ldw, MxBlocks{}, stream);
}

lora_status lora_mx_experts_load_packed(lora_mx_experts *x, int expert, const void *q, int64_t ldq,
                                        const void *s, int64_t lds, void *stream)
{
    if (!x || !blocks_ok(q, ldq, s, lds, LORA_MX_E2M1, x->w.k, x->rows))
        return LORA_E_ARG;
    return experts_load(x, expert, -1, nullptr, 0, blocks_of(q, ldq, s, lds), stream);
}

lora_status lora_mx_expert_linear(const lora_mx_experts *x, const lora_moe_plan *plan, void *y,
                                  int64_t ldy, void *yq, int64_t ldyq, void *ys, int64_t ldys,
                                  lora_dtype dtype, const void *q, int64_t ldq, const void *s,
                                  int64_t lds, lora_mx_format format, lora_moe_input input,
                                  const void *bias, lora_act act, void *stream)
{
    if (!x || !plan || !dtype_ok(dtype) || !format_ok(format) || act < LORA_ACT_NONE ||
        act > LORA_ACT_SWIGLU || (act == LORA_ACT_SWIGLU) != (x->gated != 0) ||
        (input != LORA_MOE_ROWS && input != LORA_MOE_PAIRS) || plan->experts != x->experts ||
        !on_device(x->device) || !on_device(plan->device))
        return LORA_E_ARG;
    if (plan->n_rows < 0 || x->n_loaded < x->experts)
        return LORA_E_EMPTY;
    const int64_t pairs = plan->n_rows * plan->top_k;
    const int64_t n_in = input == LORA_MOE_ROWS ? plan->n_rows : pairs;
    if ((!y && !yq) || !yq != !ys || (y && !dense_ok(y, ldy, x->d, pairs)) ||
        (yq && !blocks_ok(yq, ldyq, ys, ldys, LORA_MX_E4M3, x->d, pairs)) ||
        !blocks_ok(q, ldq, s, lds, format, x->w.k, n_in) || (bias && !aligned16(bias)))
        return LORA_E_ARG;
    if (pairs == 0)
        return LORA_OK;
    MxLinearArgs a{};
    a.w = x->w;
    a.q = static_cast<const uint8_t *>(q);
    a.ldq = ldq;
    a.s = static_cast<const uint8_t *>(s);
    a.lds = lds;
    a.n_cu = x->n_cu;
    MxEpilogue e{};
    e.bias = bias;
    e.y = y;
    e.ldy = ldy;
    e.b = blocks_of(yq, ldyq, ys, ldys);
    e.d = x->d;
    e.dtype = dt_of(dtype);
    e.act = act;
    e.code_stride = x->code_stride;
    e.scale_stride = x->scale_stride;
    const MxGroups g{plan->l, pairs, plan->experts, plan->top_k, input == LORA_MOE_ROWS};
    return status_of(launch_mx_experts(format, x->gated != 0, a, e, g, stream_of(stream)));
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

lora_status lora_block_norm_mx(void *out, int64_t ldo, void *q, int64_t ldq, void *s, int64_t lds,
                               void *h_out, int64_t ldh, const void *y, int64_t ldy,
                               const void *residual, int64_t ldr, const void *w_post,
                               const void *gate, int64_t ldg, float scale, const void *w_pre,
                               float eps, lora_dtype dtype, int64_t n_rows, int64_t k, void *stream)
{
    if (!dtype_ok(dtype) || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(scale))
        return LORA_E_ARG;
    const lora_status st = check_shape(n_rows, k, kMxMaxBlockNormK);
    if (st != LORA_OK)
        return st;
    if ((!out && !q && !h_out) || !q != !s || (!w_pre && (out || q)) ||
        !dense_ok(y, ldy, k, n_rows) || (residual && !dense_ok(residual, ldr, k, n_rows)) ||
        (w_post && !aligned16(w_post)) || (w_pre && !aligned16(w_pre)) ||
        (gate && !(ldg == 0 ? aligned16(gate) : dense_ok(gate, ldg, k, n_rows))) ||
        (h_out && !dense_ok(h_out, ldh, k, n_rows)) || (out && !dense_ok(out, ldo, k, n_rows)) ||
        (q && !blocks_ok(q, ldq, s, lds, LORA_MX_E4M3, k, n_rows)))
        return LORA_E_ARG;
    if (n_rows == 0)
        return LORA_OK;
    MxBlockNormArgs a{};
    a.y = y;
    a.ldy = ldy;
    a.res = residual;
    a.ldr = ldr;
    a.post = w_post;
    a.gate = gate;
    a.ldg = ldg;
    a.pre = w_pre;
    a.scale = scale;
    a.eps = eps;
    a.inv_k = 1. / (double)k;
    a.h = h_out;
    a.ldh = ldh;
    a.out = out;
    a.ldo = ldo;
    a.b = blocks_of(q, ldq, s, lds);
    a.n_rows = n_rows;
    a.k = k;
    return status_of(launch_block_norm_mx(dt_of(dtype), a, stream_of(stream)));
}
