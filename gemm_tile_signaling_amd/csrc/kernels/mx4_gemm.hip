// Product of two 4-bit (MX) operands: out = A . B^T, sums in fp32.
#include "../ops_internal.h"
#include "mx4.h"

namespace fo {
namespace {

struct Mx4Params {
  const uint8_t *a, *as, *b, *bs;
  uint16_t *out;
  int64_t M, N;
  int32_t nb;               // blocks of a row
  int32_t problems;
  const int32_t *row_ends;  // NULL: one problem
};

// Rows [begin, end) and problem of row tile i (tiles of BM rows, no tile spans
// two problems); false past the last tile.  Every lane gets the same answer.
__device__ __forceinline__ bool find_rows(const Mx4Params &p, int BM, int64_t i, int *problem, int64_t *begin,
                                          int64_t *end) {
  if (!p.row_ends) {
    *problem = 0;
    *begin = i * BM;
    *end = p.M;
    return *begin < p.M;
  }
  const int lane = threadIdx.x & 63;
  auto at = [&](int q) { return (int64_t)min(max(p.row_ends[q], 0), (int32_t)p.M); };
  for (int q0 = 0; q0 < p.problems; q0 += 64) {
    const int q = q0 + lane;
    const int64_t b = q > 0 && q < p.problems ? at(q - 1) : 0, e = q < p.problems ? at(q) : b;
    int32_t tiles = e > b ? (int32_t)((e - b + BM - 1) / BM) : 0, sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t other = __shfl_up(sum, d);
      if (lane >= d) sum += other;
    }
    const uint64_t past = __ballot(i < sum);
    if (past) {
      const int l = __builtin_ctzll(past);
      *problem = q0 + l;
      *begin = __shfl((int32_t)b, l) + (i - __shfl(sum - tiles, l)) * BM;
      *end = __shfl((int32_t)e, l);
      return true;
    }
    i -= __shfl(sum, 63);
  }
  return false;
}

// One wave per 16 x 16 tile, operands straight from memory.
template <typename T>
__global__ __launch_bounds__(64) void mx4_gemm_simple(Mx4Params p) {
  int problem;
  int64_t row0, row_end;
  const uint32_t tn = (uint32_t)((p.N + 15) / 16), tile_n = blockIdx.x % tn;
  if (!find_rows(p, 16, blockIdx.x / tn, &problem, &row0, &row_end)) return;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int64_t m = row0 + r, n = (int64_t)tile_n * 16 + r, bn = problem * p.N + n;
  const bool m_ok = m < row_end, n_ok = n < p.N;
  f32x4 acc = {};
  const int64_t b_rows = p.problems * p.N;
  for (int k = g; k - g < p.nb; k += 4) {  // block k of the row
    u32x4 a = {}, b = {};
    uint32_t sa = 0, sb = 0;
    if (m_ok && k < p.nb) {
      a = *reinterpret_cast<const u32x4 *>(p.a + (m * p.nb + k) * 16);
      sa = p.as[((k / 8) * p.M + m) * 8 + k % 8];
    }
    if (n_ok && k < p.nb) {
      b = *reinterpret_cast<const u32x4 *>(p.b + (bn * p.nb + k) * 16);
      sb = p.bs[((k / 8) * b_rows + bn) * 8 + k % 8];
    }
    acc = mx4_mma16<0, 0>(b, sb, a, sa, acc);
  }
  // lane: columns 4 g .. 4 g + 3 of row r
  if (m_ok)
    for (int i = 0; i < 4; ++i) {
      const int64_t c = (int64_t)tile_n * 16 + g * 4 + i;
      if (c < p.N) reinterpret_cast<T *>(p.out)[m * p.N + c] = (T)acc[i];
    }
}

}  // namespace

int launch_mx4_gemm(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                    int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t problems, const int32_t *row_ends,
                    hipStream_t s) {
  Mx4Params p{};
  p.a = static_cast<const uint8_t *>(a_codes);
  p.as = static_cast<const uint8_t *>(a_scales);
  p.b = static_cast<const uint8_t *>(b_codes);
  p.bs = static_cast<const uint8_t *>(b_scales);
  p.out = static_cast<uint16_t *>(out);
  p.M = M;
  p.N = N;
  p.nb = (int32_t)(K / 32);
  p.problems = problems;
  p.row_ends = row_ends;
  const int64_t grid = ((M + 15) / 16 + (problems - 1)) * ((N + 15) / 16);
  if (grid > 0x7FFFFFFF) return FO_ERR_UNSUPPORTED;
  if (dtype == FO_BF16)
    mx4_gemm_simple<__bf16><<<dim3((uint32_t)grid), 64, 0, s>>>(p);
  else
    mx4_gemm_simple<_Float16><<<dim3((uint32_t)grid), 64, 0, s>>>(p);
  return hipGetLastError() == hipSuccess ? FO_OK : FO_ERR_HIP;
}

}  // namespace fo
