// moe_api.cpp -- host side of the router, the grouping by expert and the
// combination: argument checks, the plan object and the kernel launches.  Every
// entry point returns a status; no exception leaves this file.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "moe.h"
#include "mx_checks.h"

using namespace lora;

namespace {

// Rows of a chunk and their number: at most kMoeMaxChunks, of whole 16 rows.
void chunks_of(int64_t n_rows, int64_t &rows, int &n)
{
    rows = ((n_rows + kMoeMaxChunks - 1) / kMoeMaxChunks + 15) / 16 * 16;
    n = rows > 0 ? (int)((n_rows + rows - 1) / rows) : 0;
}

lora_status group(lora_moe_plan *plan, int dtype, MoeRouteArgs a, void *stream)
{
    a.experts = plan->experts;
    a.top_k = plan->top_k;
    a.l = plan->l;
    a.hist = plan->hist;
    chunks_of(a.n_rows, a.chunk_rows, a.n_chunks);
    const lora_status st = status_of(launch_moe_route(dtype, a, stream_of(stream)));
    if (st == LORA_OK)
        plan->n_rows = a.n_rows;
    return st;
}

bool aligned_to(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

lora_status lora_moe_plan_create(lora_moe_plan **out, int64_t max_rows, int n_experts, int top_k)
{
    if (!out)
        return LORA_E_ARG;
    *out = nullptr;
    if (max_rows < 1 || n_experts < 1 || top_k < 1 || top_k > n_experts)
        return LORA_E_ARG;
    if (n_experts > LORA_MAX_EXPERTS || top_k > LORA_MAX_TOP_K || max_rows > kMoeMaxPairs / top_k)
        return LORA_E_UNSUPPORTED;
    lora_moe_plan *p = new (std::nothrow) lora_moe_plan();
    if (!p)
        return LORA_E_NOMEM;
    std::memset(p, 0, sizeof *p);
    p->experts = n_experts;
    p->top_k = top_k;
    p->max_rows = max_rows;
    p->n_rows = -1;
    const int64_t pairs = max_rows * top_k;
    // one allocation; every part starts on a 16-byte boundary
    int64_t bytes = 0;
    auto part = [&](int64_t n) {
        const int64_t at = bytes;
        bytes += (n + 15) / 16 * 16;
        return at;
    };
    const int64_t order = part(pairs * 4), place = part(pairs * 4);
    const int64_t n_tiles = part(kMoeHeights * 4);
    int64_t tiles[kMoeHeights];
    for (int i = 0; i < kMoeHeights; ++i)
        tiles[i] = part(moe_tile_bound(pairs, n_experts, moe_height_shift(i)) * (int64_t)sizeof(MoeTile));
    const int64_t chunks = (max_rows + 15) / 16 < kMoeMaxChunks ? (max_rows + 15) / 16 : kMoeMaxChunks;
    const int64_t hist = part((chunks + 1) * (n_experts + 1) * 4);
    hipError_t e = hipGetDevice(&p->device);
    if (e == hipSuccess)
        e = hipMalloc(&p->memory, (size_t)bytes);
    // no tiles, until a grouping has run
    if (e == hipSuccess)
        e = hipMemset(static_cast<char *>(p->memory) + n_tiles, 0, kMoeHeights * 4);
    if (e == hipSuccess)
        e = hipStreamSynchronize(nullptr);
    if (e != hipSuccess) {
        (void)hipFree(p->memory);
        delete p;
        return status_of(e);
    }
    char *m = static_cast<char *>(p->memory);
    p->l.order = reinterpret_cast<int32_t *>(m + order);
    p->l.place = reinterpret_cast<int32_t *>(m + place);
    p->l.n_tiles = reinterpret_cast<int32_t *>(m + n_tiles);
    for (int i = 0; i < kMoeHeights; ++i)
        p->l.tiles[i] = reinterpret_cast<MoeTile *>(m + tiles[i]);
    p->hist = reinterpret_cast<int32_t *>(m + hist);
    *out = p;
    return LORA_OK;
}

lora_status lora_moe_plan_destroy(lora_moe_plan *plan)
{
    if (!plan)
        return LORA_OK;
    const hipError_t e = hipDeviceSynchronize();
    (void)hipFree(plan->memory);
    delete plan;
    return status_of(e);
}

lora_status lora_moe_route(lora_moe_plan *plan, int32_t *ids, float *weights, int32_t *order,
                           int32_t *offsets, const void *logits, int64_t ldl, lora_dtype dtype,
                           int64_t n_rows, lora_moe_score score, int renormalize, float scale,
                           void *stream)
{
    if (!plan || !dtype_ok(dtype) || (score != LORA_MOE_SOFTMAX && score != LORA_MOE_SIGMOID) ||
        !std::isfinite(scale) || n_rows < 0 || n_rows > plan->max_rows || ldl < plan->experts ||
        ldl >= ((int64_t)1 << 58) / (n_rows + 1) || !on_device(plan->device))
        return LORA_E_ARG;
    if (n_rows > 0 && (!aligned_to(logits, dtype == LORA_F32 ? 4 : 2) || !aligned_to(ids, 4) ||
                       !aligned_to(weights, 4)))
        return LORA_E_ARG;
    if ((order && !aligned_to(order, 4)) || (offsets && !aligned_to(offsets, 4)))
        return LORA_E_ARG;
    MoeRouteArgs a{};
    a.logits = logits;
    a.ldl = ldl;
    a.ids = ids;
    a.weights = weights;
    a.n_rows = n_rows;
    a.score = score;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.order = order;
    a.offsets = offsets;
    return group(plan, dt_of(dtype), a, stream);
}

lora_status lora_moe_group(lora_moe_plan *plan, const int32_t *ids, int64_t n_rows, int32_t *order,
                           int32_t *offsets, void *stream)
{
    if (!plan || n_rows < 0 || n_rows > plan->max_rows || (n_rows > 0 && !aligned_to(ids, 4)) ||
        (order && !aligned_to(order, 4)) || (offsets && !aligned_to(offsets, 4)) ||
        !on_device(plan->device))
        return LORA_E_ARG;
    MoeRouteArgs a{};
    a.ids_in = ids;
    a.n_rows = n_rows;
    a.order = order;
    a.offsets = offsets;
    return group(plan, DT_F32, a, stream);
}

lora_status lora_moe_combine(const lora_moe_plan *plan, void *out, int64_t ldo, const void *y,
                             int64_t ldy, lora_dtype y_dtype, const float *weights,
                             const void *residual, int64_t ldr, lora_dtype dtype, int64_t d,
                             void *stream)
{
    if (!plan || !dtype_ok(dtype) || !dtype_ok(y_dtype) || !on_device(plan->device))
        return LORA_E_ARG;
    if (plan->n_rows < 0)
        return LORA_E_EMPTY;
    const int64_t n = plan->n_rows;   // at most kMoeMaxPairs, which the plan has checked
    if (d < 8 || d % 8 != 0)
        return LORA_E_ARG;
    if (d > kMxMaxD)
        return LORA_E_UNSUPPORTED;
    if (!dense_ok(out, ldo, d, n) || !dense_ok(y, ldy, d, n * plan->top_k) ||
        (residual && !dense_ok(residual, ldr, d, n)) || (n > 0 && !aligned_to(weights, 4)))
        return LORA_E_ARG;
    if (n == 0)
        return LORA_OK;
    MoeCombineArgs a{};
    a.out = out;
    a.ldo = ldo;
    a.y = y;
    a.ldy = ldy;
    a.y_dtype = dt_of(y_dtype);
    a.weights = weights;
    a.res = residual;
    a.ldr = ldr;
    a.place = plan->l.place;
    a.n_rows = n;
    a.d = d;
    a.top_k = plan->top_k;
    return status_of(launch_moe_combine(dt_of(dtype), a, stream_of(stream)));
}
