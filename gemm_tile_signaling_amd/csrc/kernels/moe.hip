// Mixture-of-experts layer for a few tokens: three kernels.
//   router  logits of every expert, then (last workgroup to finish) the picks,
//           their weights, and each active expert's token mask;
//   up      h = silu(gate . x) * (up . x) for every (active expert, picked token);
//   down    out = sum over active experts of w * (down . h).
// The work is reading each active expert's weights once.  The weights' rows are
// one operand of the matrix instructions (16 rows per wave), the tokens the
// other (columns, 16 per tile), so a weight is read once for all its tokens.
#include <type_traits>

#include "../ops_internal.h"
#include "mx4.h"

namespace fo {
namespace {

constexpr int kMaxTokens = 64, kMaxTiles = kMaxTokens / 16, kMaxTopK = 16, kMaxExperts = 1024;

struct MoeParams {
  const uint16_t *x, *router;
  const uint8_t *gate_up, *gate_up_s, *down, *down_s;
  uint16_t *out;
  int32_t *ids_out;
  float *wts_out;
  uint32_t *counter;
  int32_t *head;
  uint64_t *masks;
  int32_t *ids;
  float *wts;
  float *logits;
  uint16_t *x_split;  // [2][tokens][D]
  uint16_t *h;        // [2][tokens * top_k][F]
  int32_t T, D, F, E, top_k, first, local, renorm, router_wgs;
};

template <typename T>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma16<__bf16>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma16<_Float16>(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                0);
}

// 8 values of a 4-bit block (one dword of codes) as bf16: exact from 2^-126 on.
__device__ __forceinline__ u32x4 mx4_to_bf16(uint32_t codes, float scale) {
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return v;
}

__device__ __forceinline__ u32x4 load16(const void *p) { return *reinterpret_cast<const u32x4 *>(p); }

// Order of the logits as unsigned integers: a NaN above every number, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Picks of token t by one wave: expert e of lane e % 64.
__device__ __forceinline__ void select_token(const MoeParams &p, int t, int lane, uint64_t *mask) {
  constexpr int R = kMaxExperts / 64;
  float l[R];
  uint32_t key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < p.E ? p.logits[(int64_t)t * p.E + e] : 0.0f;
    key[i] = e < p.E ? order_key(l[i]) : 0u;  // 0 is below the key of every logit
  }
  float top = 0, sum = 0, picked = 0, my_w = 0;
  int my_id = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 64 < p.E) {
        const uint64_t k = ((uint64_t)key[i] << 32) | (uint32_t)~(i * 64 + lane);
        best = k > best ? k : best;
      }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
      const uint64_t o = __shfl_xor((unsigned long long)best, d);
      best = o > best ? o : best;
    }
    const int e = (int)~(uint32_t)best;
    float le = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (e == i * 64 + lane) {
        le = l[i];
        key[i] = 0;
      }
    le = __shfl(le, e & 63);
    if (j == 0) {
      top = le;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i * 64 + lane < p.E) sum += __expf(l[i] - top);
      sum = wave_sum(sum);
    }
    const float w = __expf(le - top);
    picked += w;
    if (lane == j) {
      my_id = e;
      my_w = w;
    }
    const int here = e - p.first;
    if (lane == 0 && here >= 0 && here < p.local) atomicOr((unsigned long long *)&mask[here], 1ull << t);
  }
  if (lane < p.top_k) {
    const float w = my_w / (p.renorm ? picked : sum);
    p.ids[t * p.top_k + lane] = my_id;
    p.wts[t * p.top_k + lane] = w;
    if (p.ids_out) p.ids_out[t * p.top_k + lane] = my_id;
    if (p.wts_out) p.wts_out[t * p.top_k + lane] = w;
  }
}

// Router: 16 experts per workgroup, its waves each a share of the hidden size.
constexpr int kRouterWaves = 8;
template <typename T>
__global__ __launch_bounds__(64 * kRouterWaves) void moe_router(MoeParams p) {
  __shared__ float red[kRouterWaves][kMaxTiles][64][4];
  __shared__ uint64_t mask[kMaxExperts];
  __shared__ uint32_t ticket;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  if ((int)blockIdx.x >= p.router_wgs) {  // the workgroups that split fp16 tokens into two bf16 values
    const int64_t n = (int64_t)p.T * p.D, step = (int64_t)(gridDim.x - p.router_wgs) * blockDim.x;
    for (int64_t i = (int64_t)(blockIdx.x - p.router_wgs) * blockDim.x + tid; i < n; i += step) {
      const float v = (float)reinterpret_cast<const T *>(p.x)[i];
      const __bf16 hi = (__bf16)v;
      // an infinity or a NaN goes whole into the first part
      const __bf16 lo = fabsf(v) < __builtin_inff() ? (__bf16)(v - (float)hi) : (__bf16)0.0f;
      reinterpret_cast<__bf16 *>(p.x_split)[i] = hi;
      reinterpret_cast<__bf16 *>(p.x_split)[n + i] = lo;
    }
    return;
  }
  const int e = blockIdx.x * 16 + r, tiles = (p.T + 15) / 16;
  f32x4 acc[kMaxTiles] = {};
  for (int k0 = wave * 32; k0 < p.D; k0 += kRouterWaves * 32) {
    const int k = k0 + g * 8;
    u32x4 a = {};
    if (e < p.E && k < p.D) a = load16(p.router + (int64_t)e * p.D + k);
#pragma unroll
    for (int c = 0; c < kMaxTiles; ++c)
      if (c < tiles) {
        u32x4 b = {};
        if (c * 16 + r < p.T && k < p.D) b = load16(p.x + (int64_t)(c * 16 + r) * p.D + k);
        acc[c] = mma16<T>(a, b, acc[c]);
      }
  }
#pragma unroll
  for (int c = 0; c < kMaxTiles; ++c) *reinterpret_cast<f32x4 *>(red[wave][c][lane]) = acc[c];
  __syncthreads();
  for (int i = tid; i < tiles * 256; i += 64 * kRouterWaves) {
    const int c = i >> 8, l = (i >> 2) & 63, q = i & 3;
    float s = 0;
    for (int w = 0; w < kRouterWaves; ++w) s += red[w][c][l][q];
    const int t = c * 16 + (l & 15), ee = blockIdx.x * 16 + (l >> 4) * 4 + q;
    if (t < p.T && ee < p.E) p.logits[(int64_t)t * p.E + ee] = s;
  }
  // the last workgroup to arrive sees every logit and picks
  __threadfence();
  __syncthreads();
  if (tid == 0)
    ticket = __hip_atomic_fetch_add(p.counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < p.local; i += 64 * kRouterWaves) mask[i] = 0;
  __syncthreads();
  if (ticket != (uint32_t)p.router_wgs - 1) return;
  __threadfence();
  for (int t = wave; t < p.T; t += kRouterWaves) select_token(p, t, lane, mask);
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.local; e0 += 64) {
      const uint64_t m = e0 + lane < p.local ? mask[e0 + lane] : 0;
      const uint64_t any = __ballot(m != 0);
      if (m) {
        const int at = n + __popcll(any & ((1ull << lane) - 1));
        p.head[1 + at] = e0 + lane;
        p.masks[at] = m;
      }
      n += __popcll(any);
    }
    if (lane == 0) {
      p.head[0] = n;
      __hip_atomic_store(p.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

// Up: 16 values of h per workgroup and active expert, its waves each a share of the hidden size.
constexpr int kUpWaves = 4;
template <typename T, bool MX4>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up(MoeParams p) {
  using C = std::conditional_t<MX4, __bf16, T>;
  constexpr bool SPLIT = MX4 && std::is_same_v<T, _Float16>;
  __shared__ float red[kUpWaves][kMaxTiles][2][64][4];
  __shared__ int32_t token[kMaxTokens];
  const int slot = blockIdx.y;
  if (slot >= p.head[0]) return;
  const int e = p.head[1 + slot];
  const uint64_t mask = p.masks[slot];
  const int n = __popcll(mask), tiles = (n + 15) / 16;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  if (tid < 64 && (mask >> tid & 1)) token[__popcll(mask & ((1ull << tid) - 1))] = tid;
  __syncthreads();
  const int f = blockIdx.x * 16 + r;
  const bool f_ok = f < p.F;
  const int64_t rows = (int64_t)p.local * 2 * p.F, gate = (int64_t)e * 2 * p.F + f, up = gate + p.F;
  int64_t xt[kMaxTiles];  // offset of this lane's token in x, or -1
#pragma unroll
  for (int c = 0; c < kMaxTiles; ++c) xt[c] = c * 16 + r < n ? (int64_t)token[c * 16 + r] * p.D : -1;
  f32x4 acc[kMaxTiles][2] = {};
  if constexpr (MX4) {
    const int nb = p.D / 32;
    const uint16_t *x0 = SPLIT ? p.x_split : p.x, *x1 = p.x_split + (int64_t)p.T * p.D;
    for (int b0 = wave * 4; b0 < nb; b0 += kUpWaves * 4) {
      const int b = b0 + g;
      u32x4 cg = {}, cu = {};
      float sg = 1, su = 1;
      if (f_ok && b < nb) {
        cg = load16(p.gate_up + (gate * nb + b) * 16);
        cu = load16(p.gate_up + (up * nb + b) * 16);
        sg = mx4_scale(p.gate_up_s[((b / 8) * rows + gate) * 8 + b % 8]);
        su = mx4_scale(p.gate_up_s[((b / 8) * rows + up) * 8 + b % 8]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 ag = mx4_to_bf16(cg[j], sg), au = mx4_to_bf16(cu[j], su);
#pragma unroll
        for (int c = 0; c < kMaxTiles; ++c)
          if (c < tiles) {
            u32x4 v = {}, v1 = {};
            if (xt[c] >= 0 && b < nb) {
              v = load16(x0 + xt[c] + b * 32 + j * 8);
              if (SPLIT) v1 = load16(x1 + xt[c] + b * 32 + j * 8);
            }
            acc[c][0] = mma16<C>(ag, v, acc[c][0]);
            acc[c][1] = mma16<C>(au, v, acc[c][1]);
            if (SPLIT) {
              acc[c][0] = mma16<C>(ag, v1, acc[c][0]);
              acc[c][1] = mma16<C>(au, v1, acc[c][1]);
            }
          }
      }
    }
  } else {
    const uint16_t *w = reinterpret_cast<const uint16_t *>(p.gate_up);
    for (int k0 = wave * 32; k0 < p.D; k0 += kUpWaves * 32) {
      const int k = k0 + g * 8;
      u32x4 ag = {}, au = {};
      if (f_ok && k < p.D) {
        ag = load16(w + gate * p.D + k);
        au = load16(w + up * p.D + k);
      }
#pragma unroll
      for (int c = 0; c < kMaxTiles; ++c)
        if (c < tiles) {
          u32x4 v = {};
          if (xt[c] >= 0 && k < p.D) v = load16(p.x + xt[c] + k);
          acc[c][0] = mma16<C>(ag, v, acc[c][0]);
          acc[c][1] = mma16<C>(au, v, acc[c][1]);
        }
    }
  }
#pragma unroll
  for (int c = 0; c < kMaxTiles; ++c)
    for (int q = 0; q < 2; ++q) *reinterpret_cast<f32x4 *>(red[wave][c][q][lane]) = acc[c][q];
  __syncthreads();
  const int64_t plane = (int64_t)p.T * p.top_k * p.F;
  for (int i = tid; i < tiles * 256; i += 64 * kUpWaves) {
    const int c = i >> 8, l = (i >> 2) & 63, q = i & 3, col = c * 16 + (l & 15), ff = blockIdx.x * 16 + (l >> 4) * 4 + q;
    if (col >= n || ff >= p.F) continue;
    float a = 0, b = 0;
    for (int w = 0; w < kUpWaves; ++w) {
      a += red[w][c][0][l][q];
      b += red[w][c][1][l][q];
    }
    const float v = a / (1.0f + __expf(-a)) * b;
    const int t = token[col];
    int j = 0;
    while (j < p.top_k - 1 && p.ids[t * p.top_k + j] != p.first + e) ++j;
    const int64_t at = (int64_t)(t * p.top_k + j) * p.F + ff;
    const C hi = (C)v;
    const C lo = fabsf((float)hi) < __builtin_inff() ? (C)(v - (float)hi) : (C)0.0f;
    reinterpret_cast<C *>(p.h)[at] = hi;
    reinterpret_cast<C *>(p.h)[plane + at] = lo;
  }
}

// Down: 16 outputs of every token per workgroup; its waves share the active
// experts' ffn evenly (in units of 128 values, an expert after the other).
constexpr int kDownWaves = 8, kUnit = 128;
template <typename T, bool MX4>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down(MoeParams p) {
  using C = std::conditional_t<MX4, __bf16, T>;
  __shared__ float red[kDownWaves][kMaxTiles][64][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int d = blockIdx.x * 16 + r, tiles = (p.T + 15) / 16;
  const bool d_ok = d < p.D;
  const int units = (p.F + kUnit - 1) / kUnit;
  const int64_t total = (int64_t)p.head[0] * units, rows = (int64_t)p.local * p.D;
  int64_t u = total * wave / kDownWaves;
  const int64_t u_end = total * (wave + 1) / kDownWaves, plane = (int64_t)p.T * p.top_k * p.F;
  f32x4 sum[kMaxTiles] = {};
  while (u < u_end) {
    const int slot = (int)(u / units), first = (int)(u % units);
    const int last = (int)min((int64_t)units, first + (u_end - u));
    u += last - first;
    const int e = p.head[1 + slot];
    const uint64_t mask = p.masks[slot];
    const int64_t row = (int64_t)e * p.D + d;
    f32x4 acc[kMaxTiles] = {};
    int64_t ht[kMaxTiles];  // offset of this lane's token's h, or -1
    float wt[kMaxTiles];
#pragma unroll
    for (int c = 0; c < kMaxTiles; ++c) {
      const int t = c * 16 + r;
      ht[c] = -1;
      wt[c] = 0;
      if (mask >> t & 1) {
        int j = 0;
        while (j < p.top_k - 1 && p.ids[t * p.top_k + j] != p.first + e) ++j;
        ht[c] = (int64_t)(t * p.top_k + j) * p.F;
        wt[c] = p.wts[t * p.top_k + j];
      }
    }
    if constexpr (MX4) {
      const int nb = p.F / 32;
      for (int b0 = first * 4; b0 < last * 4; b0 += 4) {
        const int b = b0 + g;
        u32x4 cd = {};
        float sd = 1;
        if (d_ok && b < nb) {
          cd = load16(p.down + (row * nb + b) * 16);
          sd = mx4_scale(p.down_s[((b / 8) * rows + row) * 8 + b % 8]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 a = mx4_to_bf16(cd[j], sd);
#pragma unroll
          for (int c = 0; c < kMaxTiles; ++c)
            if (mask >> (c * 16) & 0xFFFF) {
              u32x4 hi = {}, lo = {};
              if (ht[c] >= 0 && b < nb) {
                hi = load16(p.h + ht[c] + b * 32 + j * 8);
                lo = load16(p.h + plane + ht[c] + b * 32 + j * 8);
              }
              acc[c] = mma16<C>(a, hi, acc[c]);
              acc[c] = mma16<C>(a, lo, acc[c]);
            }
        }
      }
    } else {
      const uint16_t *w = reinterpret_cast<const uint16_t *>(p.down);
      for (int k0 = first * kUnit; k0 < last * kUnit && k0 < p.F; k0 += 32) {
        const int k = k0 + g * 8;
        u32x4 a = {};
        if (d_ok && k < p.F) a = load16(w + row * p.F + k);
#pragma unroll
        for (int c = 0; c < kMaxTiles; ++c)
          if (mask >> (c * 16) & 0xFFFF) {
            u32x4 hi = {}, lo = {};
            if (ht[c] >= 0 && k < p.F) {
              hi = load16(p.h + ht[c] + k);
              lo = load16(p.h + plane + ht[c] + k);
            }
            acc[c] = mma16<C>(a, hi, acc[c]);
            acc[c] = mma16<C>(a, lo, acc[c]);
          }
      }
    }
    // only the expert's own tokens: a NaN or an infinity in its weights stays with them
#pragma unroll
    for (int c = 0; c < kMaxTiles; ++c)
      if (ht[c] >= 0)
        for (int q = 0; q < 4; ++q) sum[c][q] += wt[c] * acc[c][q];
  }
#pragma unroll
  for (int c = 0; c < kMaxTiles; ++c) *reinterpret_cast<f32x4 *>(red[wave][c][lane]) = sum[c];
  __syncthreads();
  for (int i = tid; i < tiles * 256; i += 64 * kDownWaves) {
    const int c = i >> 8, l = (i >> 2) & 63, q = i & 3, t = c * 16 + (l & 15), dd = blockIdx.x * 16 + (l >> 4) * 4 + q;
    if (t >= p.T || dd >= p.D) continue;
    float s = 0;
    for (int w = 0; w < kDownWaves; ++w) s += red[w][c][l][q];
    reinterpret_cast<T *>(p.out)[(int64_t)t * p.D + dd] = (T)s;
  }
}

template <typename T, bool MX4>
int launch_typed(const MoeParams &p, hipStream_t s) {
  constexpr bool SPLIT = MX4 && std::is_same_v<T, _Float16>;
  const int split = SPLIT ? (int)(((int64_t)p.T * p.D + 64 * kRouterWaves * 8 - 1) / (64 * kRouterWaves * 8)) : 0;
  moe_router<T><<<p.router_wgs + split, 64 * kRouterWaves, 0, s>>>(p);
  if (hipGetLastError() != hipSuccess) return FO_ERR_HIP;
  const int most = p.local < p.T * p.top_k ? p.local : p.T * p.top_k;  // experts that can be active
  moe_up<T, MX4><<<dim3((p.F + 15) / 16, most), 64 * kUpWaves, 0, s>>>(p);
  if (hipGetLastError() != hipSuccess) return FO_ERR_HIP;
  moe_down<T, MX4><<<(p.D + 15) / 16, 64 * kDownWaves, 0, s>>>(p);
  return hipGetLastError() == hipSuccess ? FO_OK : FO_ERR_HIP;
}

}  // namespace

int launch_moe(const fo_moe_desc &d, int32_t tokens, const void *x, const void *router, const void *gate_up,
               const void *gate_up_scales, const void *down, const void *down_scales, void *out, int32_t *ids,
               float *weights, void *workspace, int cus, hipStream_t s) {
  const MoeLayout l = moe_layout(d);
  char *ws = static_cast<char *>(workspace);
  MoeParams p{};
  p.x = static_cast<const uint16_t *>(x);
  p.router = static_cast<const uint16_t *>(router);
  p.gate_up = static_cast<const uint8_t *>(gate_up);
  p.gate_up_s = static_cast<const uint8_t *>(gate_up_scales);
  p.down = static_cast<const uint8_t *>(down);
  p.down_s = static_cast<const uint8_t *>(down_scales);
  p.out = static_cast<uint16_t *>(out);
  p.ids_out = ids;
  p.wts_out = weights;
  p.counter = reinterpret_cast<uint32_t *>(ws + l.counter);
  p.head = reinterpret_cast<int32_t *>(ws + l.head);
  p.masks = reinterpret_cast<uint64_t *>(ws + l.masks);
  p.ids = reinterpret_cast<int32_t *>(ws + l.ids);
  p.wts = reinterpret_cast<float *>(ws + l.wts);
  p.logits = reinterpret_cast<float *>(ws + l.logits);
  p.x_split = reinterpret_cast<uint16_t *>(ws + l.x_split);
  p.h = reinterpret_cast<uint16_t *>(ws + l.h);
  p.T = tokens;
  p.D = (int32_t)d.hidden;
  p.F = (int32_t)d.ffn;
  p.E = d.experts;
  p.top_k = d.top_k;
  p.first = d.first_expert;
  p.local = d.local_experts;
  p.renorm = d.renormalize;
  p.router_wgs = (d.experts + 15) / 16;
  if (d.weights == FO_MOE_MX4)
    return d.dtype == FO_BF16 ? launch_typed<__bf16, true>(p, s) : launch_typed<_Float16, true>(p, s);
  return d.dtype == FO_BF16 ? launch_typed<__bf16, false>(p, s) : launch_typed<_Float16, false>(p, s);
}

}  // namespace fo
