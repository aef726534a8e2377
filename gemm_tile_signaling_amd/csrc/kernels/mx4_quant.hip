// The 4-bit (MX) format: 16-bit rows to codes and scales, and back.
//
// One block of 32 values shares the scale 2^(byte - 127), byte = max(0, E - 2)
// with E the exponent field of its largest magnitude as fp32.  The division by
// the scale is exact (a power of two), so the rounding to E2M1 is the only one;
// v_cvt_scalef32_pk_fp4_f32 does both, rounding to nearest even and holding
// magnitudes above 6 as 6.
#include "../ops_internal.h"
#include "mx4.h"

namespace fo {
namespace {

constexpr int kThreads = 256;

// One thread per block of 32 values.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T *x, int64_t rows, int64_t cols, int64_t ld,
                                                            uint8_t *codes, uint8_t *scales) {
  const int64_t nb = (cols + 31) / 32, slots = (nb + 7) / 8 * 8;  // scale bytes of a row, whole panels
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= rows * slots) return;
  const int64_t row = i / slots, b = i % slots;
  uint8_t *scale = scales + ((b / 8) * rows + row) * 8 + b % 8;
  if (b >= nb) {
    *scale = 0;
    return;
  }
  float v[32];
  uint32_t top = 0;
  for (int j = 0; j < 32; ++j) {
    const int64_t c = b * 32 + j;
    v[j] = c < cols ? (float)x[row * ld + c] : 0.0f;
    top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
  const uint32_t byte = mx4_scale_byte(top);
  u32x4 out = {0, 0, 0, 0};
  if (byte != 255)
    for (int q = 0; q < 4; ++q)
      for (int j = 0; j < 4; ++j) out[q] |= mx4_pair(v[q * 8 + j * 2], v[q * 8 + j * 2 + 1], mx4_scale(byte)) << (8 * j);
  *reinterpret_cast<u32x4 *>(codes + (row * nb + b) * 16) = out;
  *scale = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *codes, const uint8_t *scales,
                                                              int64_t rows, int64_t cols, T *out) {
  const int64_t nb = (cols + 31) / 32;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= rows * nb) return;
  const int64_t row = i / nb, b = i % nb;
  const float s = mx4_scale(scales[((b / 8) * rows + row) * 8 + b % 8]);
  const u32x4 c = *reinterpret_cast<const u32x4 *>(codes + (row * nb + b) * 16);
  for (int j = 0; j < 32 && b * 32 + j < cols; ++j) {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j / 8] >> (4 * (j % 8 & 6)), s, 0);
    out[row * cols + b * 32 + j] = (T)v[j & 1];
  }
}

}  // namespace

int launch_mx4_quantize(const void *x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, void *codes,
                        void *scales, int cus, hipStream_t s) {
  const int64_t n = rows * (((cols + 31) / 32 + 7) / 8 * 8), grid = (n + kThreads - 1) / kThreads;
  if (grid > 0x7FFFFFFF) return FO_ERR_UNSUPPORTED;
  auto *c = static_cast<uint8_t *>(codes), *sc = static_cast<uint8_t *>(scales);
  if (dtype == FO_BF16)
    quantize_kernel<<<dim3(grid), kThreads, 0, s>>>(static_cast<const __bf16 *>(x), rows, cols, ld, c, sc);
  else
    quantize_kernel<<<dim3(grid), kThreads, 0, s>>>(static_cast<const _Float16 *>(x), rows, cols, ld, c, sc);
  return hipGetLastError() == hipSuccess ? FO_OK : FO_ERR_HIP;
}

int launch_mx4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols, int32_t out_type,
                          void *out, int cus, hipStream_t s) {
  const int64_t n = rows * ((cols + 31) / 32), grid = (n + kThreads - 1) / kThreads;
  if (grid > 0x7FFFFFFF) return FO_ERR_UNSUPPORTED;
  auto *c = static_cast<const uint8_t *>(codes), *sc = static_cast<const uint8_t *>(scales);
  if (out_type == FO_BF16)
    dequantize_kernel<<<dim3(grid), kThreads, 0, s>>>(c, sc, rows, cols, static_cast<__bf16 *>(out));
  else if (out_type == FO_FP16)
    dequantize_kernel<<<dim3(grid), kThreads, 0, s>>>(c, sc, rows, cols, static_cast<_Float16 *>(out));
  else
    dequantize_kernel<<<dim3(grid), kThreads, 0, s>>>(c, sc, rows, cols, static_cast<float *>(out));
  return hipGetLastError() == hipSuccess ? FO_OK : FO_ERR_HIP;
}

}  // namespace fo
