// dense_q4.hip - dense products with 4-bit weights (moe_q4_matmul): the
// attention projections, shared experts and output head around the routed
// experts, whose weights come in the same blocks.
//
//   y[t][n] = sum_b d[n][b] * sum_{j<32} (q[n][b][j] - 8) * x[t][32 b + j]
//
// The products run on the matrix cores as 16 tokens x 16 features x one block
// (v_mfma_f32_16x16x32), also for a single token: the weights' bytes bound
// few tokens, and the other rows of the tile cost nothing that is needed.
//
// Exactness. A block's weight operand is 16 + q, exact in both 16-bit types
// and formed by a shift and one v_bitop3 per two weights (q into the mantissa
// of 16.0: no subtraction, no conversion); the accumulator of a block's product
// starts at -24 * sum_j x_j, which makes it (q - 8), and comes from the same
// matrix instruction with a constant -24 operand, once for all features of a
// wave. The block's scale is applied to the sum in fp32. Activations enter
// unrounded: bf16 and fp16 as they are, fp32 (and scale * code of 8-bit
// activations) as three bf16 terms cut from the top, 8 bits each, whose sum
// is the value.
//
// Operand order: as in grouped_mfma.hip. Lane l covers row/column l % 16 and
// chunk c = l / 16 of a block, the elements 4c + {0, 2, 1, 3, 16, 18, 17, 19};
// the weights of chunk c are dword c of the block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"
#include "value_dev.h"

namespace moe {
namespace {

using namespace value_dev;

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// bf16 terms an activation is split into
template <int XT>
constexpr int terms_of() {
  return XT == MOE_F32 || XT == MOE_Q8_32 ? 3 : 1;
}

template <int XT>
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (XT == MOE_F16) {
    f16x8_t x, y;
    __builtin_memcpy(&x, &a, 16);
    __builtin_memcpy(&y, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
  } else {
    bf16x8_t x, y;
    __builtin_memcpy(&x, &a, 16);
    __builtin_memcpy(&y, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  }
}

// (x & m) | c in one v_bitop3 (truth table of S0 & S1 | S2)
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(x, m, c, 0xEA);
}

// the 8 weights 16 + q of a chunk from its dword: the nibble becomes the top
// four mantissa bits of 16.0 (bf16: bits 3..6, fp16: bits 6..9)
template <int XT>
__device__ __forceinline__ u32x4_t weights_of(uint32_t w) {
  if constexpr (XT == MOE_F16) {
    constexpr uint32_t M = 0x03C003C0u, C = 0x4C004C00u;
    return u32x4_t{and_or(w << 6, M, C), and_or(w >> 2, M, C), and_or(w << 2, M, C), and_or(w >> 6, M, C)};
  } else {
    constexpr uint32_t M = 0x00780078u, C = 0x41804180u;
    return u32x4_t{and_or(w << 3, M, C), and_or(w >> 5, M, C), and_or(w >> 1, M, C), and_or(w >> 9, M, C)};
  }
}
template <int XT>
__device__ __forceinline__ u32x4_t minus24() {
  const uint32_t v = XT == MOE_F16 ? 0xCE00CE00u : 0xC1C0C1C0u;
  return u32x4_t{v, v, v, v};
}

// (lane group g, dword d) -> (lane group d, dword g) within each 16-lane
// column: afterwards dword i of lane group c is the old dword c of group i
__device__ __forceinline__ void transpose4(u32x4_t& v) {
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v.x = c[0], v.y = c[1], v.z = d[0], v.w = d[1];
}
// each lane group's value in every lane of its 16-lane column
__device__ __forceinline__ void broadcast4(uint32_t x, uint32_t (&out)[4]) {
  const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  out[0] = lo[0], out[1] = lo[1], out[2] = hi[0], out[3] = hi[1];
}

// the upper halves of two words: low half from a, high half from b
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t lower_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// The operand of chunk c of a block of a row, from the row's values: elements
// 4c .. 4c + 3 and 16 + 4c .. 16 + 4c + 3, in the slots' order.
template <int XT>
__device__ __forceinline__ void chunk_of(const char* row, const float* scale, int64_t b, int c,
                                         u32x4_t (&t)[terms_of<XT>()]) {
  const int64_t i = 32 * b + 4 * c;
  if constexpr (XT == MOE_F16 || XT == MOE_BF16) {
    uint32_t lo[2], hi[2];
    __builtin_memcpy(lo, row + 2 * i, 8);
    __builtin_memcpy(hi, row + 2 * i + 32, 8);
    t[0] = u32x4_t{lower_halves(lo[0], lo[1]), upper_halves(lo[0], lo[1]), lower_halves(hi[0], hi[1]),
                   upper_halves(hi[0], hi[1])};
  } else {
    float v[8];
    if constexpr (XT == MOE_F32) {
      __builtin_memcpy(v, row + 4 * i, 16);
      __builtin_memcpy(v + 4, row + 4 * i + 64, 16);
    } else {
      uint32_t lo, hi;
      __builtin_memcpy(&lo, row + i, 4);
      __builtin_memcpy(&hi, row + i + 16, 4);
      const float s = scale[b];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = s * (float)(int8_t)(lo >> (8 * j));
        v[4 + j] = s * (float)(int8_t)(hi >> (8 * j));
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = __float_as_uint(v[j]);
        v[j] -= __uint_as_float(u[j] & 0xFFFF0000u);  // exact: the bits below
      }
      t[k] = u32x4_t{upper_halves(u[0], u[2]), upper_halves(u[1], u[3]), upper_halves(u[4], u[6]),
                     upper_halves(u[5], u[7])};
    }
  }
}

// y[t][f] = v, or += v
__device__ __forceinline__ void put(const Q4Args& a, int64_t t, int64_t f, float v) {
  const int64_t i = t * a.y_stride + f;
  if (a.y_type == MOE_F32)
    store1<MOE_F32>(a.y, i, a.accumulate ? load1<MOE_F32>(a.y, i) + v : v);
  else if (a.y_type == MOE_F16)
    store1<MOE_F16>(a.y, i, a.accumulate ? load1<MOE_F16>(a.y, i) + v : v);
  else
    store1<MOE_BF16>(a.y, i, a.accumulate ? load1<MOE_BF16>(a.y, i) + v : v);
}

// ---------------------------------------------------------------------------
// Up to 16 tokens per work-group (more: further work-groups): 16 NW features
// by 8 waves that share the reduction in steps of four blocks.

constexpr int kWaves = 8;

template <int XT, int NW>
__global__ __launch_bounds__(64 * kWaves) void q4_rows16_kernel(Q4Args a) {
  constexpr int TERMS = terms_of<XT>();
  __shared__ f32x4_t s_red[kWaves][NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, c = lane >> 4;
  const int64_t KB = a.K / 32, f0 = (int64_t)blockIdx.x * 16 * NW, t0 = (int64_t)blockIdx.y * 16;
  const int64_t trow = std::min<int64_t>(t0 + col, a.T - 1);  // past the last token: its row, never stored
  const char* xr = static_cast<const char*>(a.x) + trow * a.x_stride * value_size<XT>();
  const float* xs = XT == MOE_Q8_32 ? a.x_scales + trow * a.x_scales_stride : nullptr;
  f32x4_t acc[NW];
#pragma unroll
  for (int t = 0; t < NW; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t b0 = 4 * wave; b0 < KB; b0 += 4 * kWaves) {
    // lane (column, c) loads block b0 + c of its feature; past the row: its
    // last block with scale 0
    const int64_t b = std::min<int64_t>(b0 + c, KB - 1);
    u32x4_t w[NW];
    uint32_t d[NW][4];
#pragma unroll
    for (int t = 0; t < NW; ++t) {
      const int64_t f = std::min<int64_t>(f0 + 16 * t + col, a.N - 1);
      w[t] = static_cast<const u32x4_t*>(a.nibbles)[f * KB + b];
      const float s = b0 + c < KB ? half_to_float(a.w_scales[f * KB + b]) : 0.f;
      broadcast4(__float_as_uint(s), d[t]);
      transpose4(w[t]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4_t x[TERMS];
      chunk_of<XT>(xr, xs, std::min<int64_t>(b0 + i, KB - 1), c, x);
      f32x4_t base = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < TERMS; ++k) base = mfma<XT>(x[k], minus24<XT>(), base);
#pragma unroll
      for (int t = 0; t < NW; ++t) {
        const u32x4_t wt = weights_of<XT>(w[t][i]);
        f32x4_t p = base;
#pragma unroll
        for (int k = 0; k < TERMS; ++k) p = mfma<XT>(x[k], wt, p);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(__uint_as_float(d[t][i]), p[r], acc[t][r]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NW; ++t) s_red[wave][t][lane] = acc[t];
  __syncthreads();
  // lane (column, c) holds tokens 4c + i of its feature
  for (int e = threadIdx.x; e < 256 * NW; e += 64 * kWaves) {
    const int f = e % (16 * NW), r = e / (16 * NW);
    if (f0 + f >= a.N || t0 + r >= a.T) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_red[w][f / 16][16 * (r / 4) + f % 16][r % 4];
    put(a, t0 + r, f0 + f, v);
  }
}

template <int XT>
hipError_t launch_types(const Q4Args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 15) / 16));
  return launch(q4_rows16_kernel<XT, 1>, grid, dim3(64 * kWaves), Launch{s}, a);
}

}  // namespace

int64_t q4_workspace_bytes(int64_t T, int64_t N, int64_t K, int32_t x_type) { return 0; }

hipError_t launch_q4_matmul(const Q4Args& a, hipStream_t s) {
  switch (a.x_type) {
    case MOE_F32: return launch_types<MOE_F32>(a, s);
    case MOE_F16: return launch_types<MOE_F16>(a, s);
    case MOE_BF16: return launch_types<MOE_BF16>(a, s);
    default: return launch_types<MOE_Q8_32>(a, s);
  }
}

}  // namespace moe
