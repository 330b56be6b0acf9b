// mx_checks.h -- argument checks shared by the host sides of the microscaled
// operators and the mixture layer's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx.h"

namespace lora {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool dtype_ok(lora_dtype t) { return t == LORA_F32 || t == LORA_BF16; }
inline bool format_ok(lora_mx_format f) { return f == LORA_MX_E4M3 || f == LORA_MX_E2M1; }
inline int dt_of(lora_dtype t) { return t == LORA_F32 ? DT_F32 : DT_BF16; }
inline hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Widths and rows: negative or uneven ones are wrong, large ones unsupported.
inline lora_status check_shape(int64_t n_rows, int64_t k, int64_t k_max)
{
    if (n_rows < 0 || k < 8 || k % 8 != 0)
        return LORA_E_ARG;
    return n_rows >= kMxMaxRows || k > k_max ? LORA_E_UNSUPPORTED : LORA_OK;
}

// A dense matrix of n_rows x width elements with row stride ld; its last
// element's byte offset must fit 62 bits.
inline bool dense_ok(const void *p, int64_t ld, int64_t width, int64_t n_rows)
{
    return ld >= width && ld % 8 == 0 && ld < ((int64_t)1 << 58) / (n_rows + 1) &&
           (n_rows == 0 || (p && aligned16(p)));
}

inline bool blocks_ok(const void *q, int64_t ldq, const void *s, int64_t lds, lora_mx_format f,
                      int64_t k, int64_t n_rows)
{
    return ldq >= LORA_MX_CODE_BYTES(k, f) && ldq % 16 == 0 && lds >= LORA_MX_SCALE_BYTES(k) &&
           lds % 16 == 0 && ldq < ((int64_t)1 << 60) / (n_rows + 1) &&
           lds < ((int64_t)1 << 60) / (n_rows + 1) &&
           (n_rows == 0 || (q && s && aligned16(q) && aligned16(s)));
}

inline MxBlocks blocks_of(const void *q, int64_t ldq, const void *s, int64_t lds)
{
    return MxBlocks{static_cast<uint8_t *>(const_cast<void *>(q)), ldq,
                    static_cast<uint8_t *>(const_cast<void *>(s)), lds};
}

inline bool on_device(int device)
{
    int cur = -1;
    return hipGetDevice(&cur) == hipSuccess && cur == device;
}

}  // namespace lora
