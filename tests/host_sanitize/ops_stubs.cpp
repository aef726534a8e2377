// Stand-ins for the launchers of the 4-bit operators and the mixture-of-experts
// layer, for the host-only sanitizer build (tests/test_host_sanitizers_ops.py).
// No GPU code is built or run.
#include "../../gemm_tile_signaling_amd/csrc/ops_internal.h"

namespace fo {

int launch_mx4_quantize(const void *, int64_t, int64_t, int64_t, int32_t, void *, void *, hipStream_t) {
  return FO_ERR_UNSUPPORTED;
}
int launch_mx4_dequantize(const void *, const void *, int64_t, int64_t, int32_t, void *, hipStream_t) {
  return FO_ERR_UNSUPPORTED;
}
int launch_mx4_gemm(const void *, const void *, const void *, const void *, void *, int64_t, int64_t, int64_t, int32_t,
                    int32_t, const int32_t *, int, hipStream_t) {
  return FO_ERR_UNSUPPORTED;
}
int launch_moe(const fo_moe_desc &d, int32_t, const void *, const void *, const void *, const void *, const void *,
               const void *, void *, int32_t *, float *, void *, int, hipStream_t) {
  return moe_layout(d).bytes > 0 ? FO_ERR_UNSUPPORTED : FO_ERR_INVALID;
}

}  // namespace fo
