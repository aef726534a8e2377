// Internal declarations of the 4-bit operators and the mixture-of-experts
// layer: launchers, called with arguments that ops.cpp has checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fo_ops.h"

namespace fo {

int launch_mx4_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, void *codes,
                        void *scales, hipStream_t s);
int launch_mx4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols, int32_t out_type,
                          void *out, hipStream_t s);
int launch_mx4_gemm(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                    int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t problems, const int32_t *row_ends,
                    hipStream_t s);

}  // namespace fo
