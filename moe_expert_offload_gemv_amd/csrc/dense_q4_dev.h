// dense_q4_dev.h - dense products with 4-bit weights (moe_q4_matmul, moe_q4_linear): the
// attention projections, shared experts and output head around the routed
// experts, whose weights come in the same blocks. Compiled by dense_q4.hip without and by
// dense_q4_linear.hip with an epilogue (kEpilogue, stated by the including file), so that the
// plain product carries nothing of it.
//
//   y[t][n] = sum_b d[n][b] * sum_{j<32} (q[n][b][j] - 8) * x[t][32 b + j]
//
// Three kernels, by the work of a call:
//   q4_dot_kernel   a few tokens: dot products on the vector unit, the tokens' values in
//                   registers. Bound by the weights' bytes (1 x 65537 x 4096 bf16, 151 MB, 28 us =
//                   5.4 TB/s, a streaming read) or, for few rows, by a launch and two trips to memory
//                   (1 x 2048 x 2048 fp32, 4.0 us).
//   q4_tile_kernel  up to 32 tokens or 2e9 products, and where the next would have too few tiles
//                   (wide_split): 16 tokens a work-group on the matrix cores, one launch (32 x 4096 x
//                   1536 fp32, 7.4 us; 201 x 1001 x 1056 fp16, 7.3: rounds of load, convert, barrier and
//                   product, 1 us each).
//   q4_wide_kernel  more: the activations are brought into operand form once, 64 x 64 tiles
//                   per wave (4096 x 5120 x 4096 bf16, 172 GFLOP, 264-300 us = 0.6 PFLOP/s, 17 of them the
//                   operand pass; the library's plain bf16 product of the same sizes would take 153). Per step of
//                   four blocks a wave issues 64 products and 460 vector instructions, 256 of them the scale
//                   FMAs that keep the weights exact; the two do not overlap on a SIMD
//                   (counters: vector unit 323, matrix cores 164 of 593 kcycles).
// The matrix cores take 16 tokens x 16 features x one block (v_mfma_f32_16x16x32).
//
// Exactness. A block's weight operand is 16 + q, exact in both 16-bit types
// and formed by a shift and one v_bitop3 per two weights (q into the mantissa
// of 16.0: no subtraction, no conversion); the accumulator of a block's product
// starts at -24 * sum_j x_j, which makes it (q - 8); these sums are formed with the
// activations' operand. The block's scale is applied to the sum in fp32. Activations enter
// unrounded: bf16 and fp16 as they are, 8-bit codes as whole numbers whose scale
// joins the block's, fp32 as three bf16 terms cut from the top, 8 bits each, whose
// sum is the value (down to bf16's last bit, 2^-133: the third term of a value below
// 2^-110 loses what lies under it).
//
// Operand order: as in grouped_mfma.hip. Lane l covers row/column l % 16 and
// chunk c = l / 16 of a block, the elements 4c + {0, 2, 1, 3, 16, 18, 17, 19};
// the weights of chunk c are dword c of the block.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"
#include "lane_dev.h"
#include "route_dev.h"
#include "value_dev.h"

namespace moe {
namespace {

using namespace lane_dev;
using namespace value_dev;

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Terms an activation is split into, and the operands' type: fp32 values are
// cut into three of bf16; 8-bit codes stay one exact fp16 term and their scales
// join the scale FMAs (880 x 3470 x 4992: 85 us, 160 as three terms of scale times code).
template <int XT>
constexpr int op_of() {
  return XT == MOE_F16 || XT == MOE_Q8_32 ? MOE_F16 : MOE_BF16;
}
template <int XT>
constexpr int terms_of() {
  return XT == MOE_F32 ? 3 : 1;
}
// runs of 16 floats beside a unit's operand: -24 sums, and the scales of codes
template <int XT>
constexpr int runs_of() {
  return XT == MOE_Q8_32 ? 2 : 1;
}

// OP: the 16-bit type of the products' operands, MOE_F16 or MOE_BF16
template <int OP>
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (OP == MOE_F16) {
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

// the 8 weights 16 + q of a chunk from its dword: the nibble becomes the top
// four mantissa bits of 16.0 (bf16: bits 3..6, fp16: bits 6..9)
template <int OP>
__device__ __forceinline__ uint32_t weights_part(uint32_t w, int i) {
  if constexpr (OP == MOE_F16) {
    constexpr uint32_t M = 0x03C003C0u, C = 0x4C004C00u;
    return and_or(i == 0 ? w << 6 : i == 1 ? w >> 2 : i == 2 ? w << 2 : w >> 6, M, C);
  } else {
    constexpr uint32_t M = 0x00780078u, C = 0x41804180u;
    return and_or(i == 0 ? w << 3 : i == 1 ? w >> 5 : i == 2 ? w >> 1 : w >> 9, M, C);
  }
}
template <int OP>
__device__ __forceinline__ u32x4_t weights_of(uint32_t w) {
  return u32x4_t{weights_part<OP>(w, 0), weights_part<OP>(w, 1), weights_part<OP>(w, 2), weights_part<OP>(w, 3)};
}

// 4 x 4 transpose within every quad of lanes: register i of lane j and
// register j of lane i change places
template <int CTRL>
__device__ __forceinline__ uint32_t from_quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ void transpose_quad(uint32_t (&v)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  constexpr int kXor1 = 0xB1, kXor2 = 0x4E;  // quad_perm [1,0,3,2], [2,3,0,1]
  // the moves stand before the selects: an arm of a conditional would run them
  // with half the lanes off, and they read the other half
  const uint32_t x0 = from_quad<kXor1>(v[0]), x1 = from_quad<kXor1>(v[1]);
  const uint32_t x2 = from_quad<kXor1>(v[2]), x3 = from_quad<kXor1>(v[3]);
  const uint32_t a0 = odd ? x1 : v[0], a1 = odd ? v[1] : x0, a2 = odd ? x3 : v[2], a3 = odd ? v[3] : x2;
  const uint32_t y0 = from_quad<kXor2>(a0), y1 = from_quad<kXor2>(a1);
  const uint32_t y2 = from_quad<kXor2>(a2), y3 = from_quad<kXor2>(a3);
  v[0] = high ? y2 : a0;
  v[1] = high ? y3 : a1;
  v[2] = high ? a2 : y0;
  v[3] = high ? a3 : y1;
}

// the upper halves of two words: low half from a, high half from b
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t lower_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// Four 8-bit codes as fp16, elements (0, 2) and (1, 3), exact: code + 128
// becomes the low mantissa byte of 1024 + code + 128, from which 1152 is taken.
__device__ __forceinline__ void codes_to_half(uint32_t codes, uint32_t& even, uint32_t& odd) {
  const uint32_t x = codes ^ 0x80808080u;
  const uint32_t u[2] = {__builtin_amdgcn_perm(0x64646464u, x, 0x04020400u),
                         __builtin_amdgcn_perm(0x64646464u, x, 0x04030401u)};
  f16x2_t h[2];
  __builtin_memcpy(h, u, 8);
  const f16x2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
  h[0] -= off, h[1] -= off;
  __builtin_memcpy(&even, &h[0], 4);
  __builtin_memcpy(&odd, &h[1], 4);
}

// The values of chunk c of a block of a row, elements 4c .. 4c + 3 and 16 + 4c
// .. 16 + 4c + 3, as loaded.
template <int XT>
struct RawChunk {
  uint32_t lo[XT == MOE_F32 ? 4 : XT == MOE_Q8_32 ? 1 : 2], hi[XT == MOE_F32 ? 4 : XT == MOE_Q8_32 ? 1 : 2];
};
template <int XT>
__device__ __forceinline__ RawChunk<XT> load_chunk(const char* row, int64_t b, int c) {
  RawChunk<XT> r;
  const char* p = row + (32 * b + 4 * c) * value_size<XT>();
  __builtin_memcpy(r.lo, p, 4 * value_size<XT>());
  __builtin_memcpy(r.hi, p + 16 * value_size<XT>(), 4 * value_size<XT>());
  return r;
}

// Its operand, in the slots' order: 16-bit values, codes as fp16, or fp32 values
// cut into bf16 terms.
template <int XT, int TERMS>
__device__ __forceinline__ void chunk_terms(const RawChunk<XT>& r, u32x4_t (&t)[TERMS]) {
  if constexpr (XT == MOE_F16 || XT == MOE_BF16) {
    t[0] = u32x4_t{lower_halves(r.lo[0], r.lo[1]), upper_halves(r.lo[0], r.lo[1]), lower_halves(r.hi[0], r.hi[1]),
                   upper_halves(r.hi[0], r.hi[1])};
  } else if constexpr (XT == MOE_Q8_32) {
    uint32_t h[4];
    codes_to_half(r.lo[0], h[0], h[1]);
    codes_to_half(r.hi[0], h[2], h[3]);
    t[0] = u32x4_t{h[0], h[1], h[2], h[3]};
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r.lo[j]), v[4 + j] = __uint_as_float(r.hi[j]);
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = __float_as_uint(v[j]);
        if (k + 1 < TERMS) v[j] -= __uint_as_float(u[j] & 0xFFFF0000u);  // exact: the bits below
      }
      t[k] = u32x4_t{upper_halves(u[0], u[2]), upper_halves(u[1], u[3]), upper_halves(u[4], u[6]),
                     upper_halves(u[5], u[7])};
    }
  }
}

// sum of a chunk's 8 values, small terms first
template <int XT, int TERMS>
__device__ __forceinline__ float chunk_sum(const u32x4_t (&t)[TERMS]) {
  float sum = 0.f;
#pragma unroll
  for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (op_of<XT>() == MOE_F16)
        sum += half_to_float((uint16_t)t[k][i]) + half_to_float((uint16_t)(t[k][i] >> 16));
      else
        sum += __uint_as_float(t[k][i] << 16) + __uint_as_float(t[k][i] & 0xFFFF0000u);
    }
  return sum;
}
// act(v) in fp32; exponentials and the error function to its last bits
__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case MOE_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays
    case MOE_ACT_SILU: return v / (1.0f + expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678f * v);
    case MOE_ACT_GELU_TANH: return v / (1.0f + expf(-1.59576912f * fmaf(0.044715f * v * v, v, v)));
    default: return v;
  }
}
__device__ __forceinline__ float load_value(const void* p, int type, int64_t i) {
  return type == MOE_F32 ? load1<MOE_F32>(p, i) : type == MOE_F16 ? load1<MOE_F16>(p, i) : load1<MOE_BF16>(p, i);
}
__device__ __forceinline__ float epilogue(const Q4Epilogue& e, int64_t t, int64_t f, float v) {
  if (e.bias) v += e.bias[f];
  v = activate(e.act, v);
  if (e.mul) v *= load_value(e.mul, e.mul_type, t * e.mul_stride + f);
  if (e.res) v += load_value(e.res, e.res_type, t * e.res_stride + f);
  return v;
}
// y[t][f] = v, or += v
__device__ __forceinline__ void put(const Q4Args& a, int64_t t, int64_t f, float v) {
  if constexpr (kEpilogue) v = epilogue(a.epi, t, f, v);
  const int64_t i = t * a.y_stride + f;
  if (a.y_type == MOE_F32)
    store1<MOE_F32>(a.y, i, a.accumulate ? load1<MOE_F32>(a.y, i) + v : v);
  else if (a.y_type == MOE_F16)
    store1<MOE_F16>(a.y, i, a.accumulate ? load1<MOE_F16>(a.y, i) + v : v);
  else
    store1<MOE_BF16>(a.y, i, a.accumulate ? load1<MOE_BF16>(a.y, i) + v : v);
}

// ---------------------------------------------------------------------------
// One token, or a few whose values fit the registers of a wave: dot products
// on the vector unit. LPR lanes share a weight row; lane l has its blocks l,
// l + LPR, ... (BPL of them) and keeps the activations of those blocks in
// registers for all rows the wave takes, NR at a time, the next NR being
// loaded meanwhile. A matrix tile would spend 140 instructions on 64 blocks,
// most of them to bring weights and scales to its lanes, and its products wait
// for each other; a lane's dot products take, per block of T tokens:
//   8-bit x   12 + 11 T  (v_dot4 on bytes: integers, exact)
//   16-bit x  32 + 18 T  (v_dot2 on 16 + q, sums starting at -24 sum x)
//   fp32 x    44 + 34 T  (v_cvt_f32_ubyte, FMA)

// the activations of one block of one token
template <int XT>
struct BlockX {
  static constexpr int WORDS = XT == MOE_F32 ? 32 : XT == MOE_Q8_32 ? 8 : 16;
  uint32_t v[WORDS];
  float base;   // what the sum starts from: -24 (-8: fp32, 8-bit codes) times the sum of the values
  float scale;  // 8-bit codes
};

template <int XT>
__device__ __forceinline__ void load_block_x(const char* row, const float* scale, int b, int KB, BlockX<XT>& x) {
  constexpr int S = value_size<XT>();
  uint32_t raw[8 * S];
  const bool inside = b < KB;  // past the row: zeros
  __builtin_memcpy(raw, row + (int64_t)min(b, KB - 1) * 32 * S, 32 * S);
#pragma unroll
  for (int i = 0; i < 8 * S; ++i) raw[i] = inside ? raw[i] : 0u;
  if constexpr (XT == MOE_F32) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x.v[i] = raw[i], sum += __uint_as_float(raw[i]);
    x.base = -8.0f * sum;
  } else if constexpr (XT == MOE_Q8_32) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = raw[i], sum = __builtin_amdgcn_sdot4((int)raw[i], 0x01010101, sum, false);
    x.base = __int_as_float(-8 * sum);  // an integer here
    x.scale = inside ? scale[b] : 0.f;
  } else {
    // pairs in the order of weights_part: chunk c, elements (0, 2), (1, 3), (16, 18), (17, 19)
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a = raw[8 * h + 2 * c], b2 = raw[8 * h + 2 * c + 1];
        x.v[4 * c + 2 * h] = lower_halves(a, b2);
        x.v[4 * c + 2 * h + 1] = upper_halves(a, b2);
#pragma unroll
        for (const uint32_t w : {a, b2})
          sum += XT == MOE_F16 ? half_to_float((uint16_t)w) + half_to_float((uint16_t)(w >> 16))
                               : __uint_as_float(w << 16) + __uint_as_float(w & 0xFFFF0000u);
      }
    x.base = -24.0f * sum;
  }
}

// sum over a block of (q - 8) x, times the block's scale
template <int XT, int T>
__device__ __forceinline__ void block_dots(u32x4_t w, float d, const BlockX<XT> (&x)[T], float (&acc)[T]) {
  if constexpr (XT == MOE_Q8_32) {
    int s[T];
#pragma unroll
    for (int t = 0; t < T; ++t) s[t] = __float_as_int(x[t].base);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t lo = w[c] & 0x0F0F0F0Fu, hi = (w[c] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        s[t] = __builtin_amdgcn_sdot4((int)lo, (int)x[t].v[c], s[t], false);
        s[t] = __builtin_amdgcn_sdot4((int)hi, (int)x[t].v[4 + c], s[t], false);
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = fmaf(d * x[t].scale, (float)s[t], acc[t]);
  } else if constexpr (XT == MOE_F32) {
    float s0[T], s1[T];
#pragma unroll
    for (int t = 0; t < T; ++t) s0[t] = x[t].base, s1[t] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // through v_bitop3 (S0 & S1): a plain AND is folded into an extract per element
      const uint32_t lo = __builtin_amdgcn_bitop3_b32(w[c], 0x0F0F0F0Fu, 0u, 0xC0);
      const uint32_t hi = __builtin_amdgcn_bitop3_b32(w[c] >> 4, 0x0F0F0F0Fu, 0u, 0xC0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = (float)((lo >> (8 * j)) & 0xFFu), b = (float)((hi >> (8 * j)) & 0xFFu);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          s0[t] = fmaf(a, __uint_as_float(x[t].v[4 * c + j]), s0[t]);
          s1[t] = fmaf(b, __uint_as_float(x[t].v[16 + 4 * c + j]), s1[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = fmaf(d, s0[t] + s1[t], acc[t]);
  } else {
    float s[T];
#pragma unroll
    for (int t = 0; t < T; ++t) s[t] = x[t].base;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = weights_part<XT>(w[c], i);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if constexpr (XT == MOE_F16) {
            f16x2_t a, b;
            __builtin_memcpy(&a, &p, 4);
            __builtin_memcpy(&b, &x[t].v[4 * c + i], 4);
            s[t] = __builtin_amdgcn_fdot2(a, b, s[t], false);
          } else {
            bf16x2_t a, b;
            __builtin_memcpy(&a, &p, 4);
            __builtin_memcpy(&b, &x[t].v[4 * c + i], 4);
            s[t] = __builtin_amdgcn_fdot2_f32_bf16(a, b, s[t], false);
          }
        }
      }
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = fmaf(d, s[t], acc[t]);
  }
}

// sum over the lanes at the same place of the wave's four 16-lane rows
__device__ __forceinline__ float across_rows(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// sum over the LPR lanes of a row, in every one of them
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor1>(__float_as_uint(v)));
  v += __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor2>(__float_as_uint(v)));
  v += __uint_as_float(route_dev::dpp32<route_dev::kDppRowHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(route_dev::dpp32<route_dev::kDppRowMirror>(__float_as_uint(v)));
  return LPR == 64 ? across_rows(v) : v;
}

// Sums of V values over the LPR lanes of a row: lane i (mod 4; 4 and above the
// second four) ends with value i. Two rounds in which a lane hands half of its
// values to its neighbour and keeps the other half, then plain sums over the
// lanes that keep the same one: 17 instructions for four values, 14 for one.
template <int LPR, int V>
__device__ __forceinline__ float row_sums(const float (&v)[V]) {
  static_assert(V <= 8, "two sets of four");
  if constexpr (V == 1) {
    return row_sum<LPR>(v[0]);
  } else {
    const int lane = threadIdx.x & 63;
    const bool odd = lane & 1, high = lane & 2;
    float out[V > 4 ? 2 : 1];
#pragma unroll
    for (int s = 0; s < (V > 4 ? 2 : 1); ++s) {
      float q[4], h[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = 4 * s + i < V ? v[4 * s + i < V ? 4 * s + i : 0] : 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float keep = odd ? q[2 * i + 1] : q[2 * i], send = odd ? q[2 * i] : q[2 * i + 1];
        h[i] = keep + __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor1>(__float_as_uint(send)));
      }
      const float keep = high ? h[1] : h[0], send = high ? h[0] : h[1];
      float r = keep + __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor2>(__float_as_uint(send)));
      r += __uint_as_float(route_dev::dpp32<0x124>(__float_as_uint(r)));  // row_ror:4, row_ror:8
      r += __uint_as_float(route_dev::dpp32<0x128>(__float_as_uint(r)));
      out[s] = LPR == 64 ? across_rows(r) : r;
    }
    if constexpr (V > 4) return lane & 4 ? out[1] : out[0];
    return out[0];
  }
}

constexpr int kDotWaves = 4;

// T: tokens held, at least those there are (the last one again, never stored).
// KS = 4: a row of more blocks than a wave's registers hold tokens for is shared
// by the work-group's waves, which add up through LDS (1 x 4096 x 14336 bf16: 9.1 us, 24.7 in tiles).
template <int XT, int LPR, int BPL, int T, int NR, int KS>
__global__ __launch_bounds__(64 * kDotWaves) void q4_dot_kernel(Q4Args a) {
  constexpr int RPW = 64 / LPR;  // rows side by side
  __shared__ float s_sum[KS > 1 ? 2 : 1][KS > 1 ? kDotWaves : 1][64];
  static_assert(KS == 1 || (KS == kDotWaves && LPR == 64), "a row's slices: the waves of its work-group");
  const int lane = threadIdx.x & 63, side = lane / LPR;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lb = (lane & (LPR - 1)) + (KS > 1 ? wave * LPR * BPL : 0);  // the lane's first block
  const int KB = (int)(a.K / 32), N = (int)a.N;
  const u32x4_t* nib = static_cast<const u32x4_t*>(a.nibbles);
  u32x4_t w[NR][BPL];
  uint16_t d[NR][BPL];
  auto issue = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = min((g * NR + r) * RPW + side, N - 1);  // past N: the last row, never stored
#pragma unroll
      for (int j = 0; j < BPL; ++j) {
        const int64_t at = (int64_t)row * KB + min(lb + LPR * j, KB - 1);
        w[r][j] = nib[at];
        d[r][j] = a.w_scales[at];
      }
    }
  };
  const int groups = (N + NR * RPW - 1) / (NR * RPW), stride = gridDim.x * (kDotWaves / KS);
  int g = KS > 1 ? blockIdx.x : blockIdx.x * kDotWaves + wave;
  int turn = 0;
  issue(g);
  BlockX<XT> x[BPL][T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t tok = std::min<int64_t>(t, a.T - 1);
    const char* row = static_cast<const char*>(a.x) + tok * a.x_stride * value_size<XT>();
    const float* scale = XT == MOE_Q8_32 ? a.x_scales + tok * a.x_scales_stride : nullptr;
#pragma unroll
    for (int j = 0; j < BPL; ++j) load_block_x<XT>(row, scale, lb + LPR * j, KB, x[j][t]);
  }
#pragma unroll 1
  for (; g < groups; g += stride) {
    float acc[NR][T];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int t = 0; t < T; ++t) acc[r][t] = 0.f;
#pragma unroll
      for (int j = 0; j < BPL; ++j) {
        // past the row the last block again, with zeros for x: its scale may be infinite
        const uint16_t scale = lb + LPR * j < KB ? d[r][j] : (uint16_t)0;
        block_dots<XT, T>(w[r][j], half_to_float(scale), x[j], acc[r]);
        // the row's registers are free: its loads of the next group
        const int row = min(((g + stride) * NR + r) * RPW + side, N - 1);
        const int64_t at = (int64_t)row * KB + min(lb + LPR * j, KB - 1);
        w[r][j] = nib[at];
        d[r][j] = a.w_scales[at];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // lane i of a row's lanes stores value i: token i / NR of row i % NR
    float flat[NR * T];
#pragma unroll
    for (int i = 0; i < NR * T; ++i) flat[i] = acc[i % NR][i / NR];
    float v = row_sums<LPR>(flat);
    if constexpr (KS > 1) {
      // every wave of the work-group has the same groups; a buffer is written again
      // only past the next barrier, when its reader has its values
      s_sum[turn][wave][lane] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int w = 0; w < KS; ++w) v += s_sum[turn][w][lane];
      turn ^= 1;
    }
    const int i = lane & (LPR - 1);
    const int64_t row = ((int64_t)g * NR + i % NR) * RPW + side;
    if (i < NR * (int)a.T && row < N && (KS == 1 || wave == 0)) put(a, i / NR, row, v);
  }
}

template <int XT, int LPR, int BPL, int T, int NR, int KS>
hipError_t launch_dot_rows(const Q4Args& a, hipStream_t s) {
  constexpr int RPW = 64 / LPR, GPW = kDotWaves / KS;  // rows side by side, groups of a work-group at a time
  static_assert(NR * T <= LPR && NR * T <= 8, "a lane per output of a row group");
  // as many work-groups as a CU holds at about this many registers, every wave
  // the same number of row groups
  constexpr int kRegs = 32 + BPL * T * (BlockX<XT>::WORDS + 2) + 7 * NR * BPL;
  constexpr int kGroups = 256 * GPW * std::max(1, std::min(8, 512 / kRegs));
  const int64_t groups = (a.N + NR * RPW - 1) / (NR * RPW), rounds = (groups + kGroups - 1) / kGroups;
  const dim3 grid((unsigned)((groups + GPW * rounds - 1) / (GPW * rounds)));
  return launch(q4_dot_kernel<XT, LPR, BPL, T, NR, KS>, grid, dim3(64 * kDotWaves), Launch{s}, a);
}
template <int XT, int LPR, int BPL, int T, int KS>
hipError_t launch_dot(const Q4Args& a, hipStream_t s) {
  // rows in flight: 64 bytes per lane; up to 8192 rows one at a time, so that every CU has some
  constexpr int kMany = std::max(1, std::min(4 / BPL, 8 / T));
  return a.N <= 8192 / KS ? launch_dot_rows<XT, LPR, BPL, T, 1, KS>(a, s)
                          : launch_dot_rows<XT, LPR, BPL, T, kMany, KS>(a, s);
}

// tokens times blocks per lane whose values the kernel keeps in registers
template <int XT, int KS>
constexpr int dot_limit() {
  return (XT == MOE_F32 ? 2 : XT == MOE_Q8_32 ? 12 : 4) * (KS > 1 && XT != MOE_Q8_32 ? 2 : 1);
}
template <int XT, int LPR, int BPL, int KS>
hipError_t launch_dot_tokens(const Q4Args& a, hipStream_t s) {
  constexpr int L = dot_limit<XT, KS>() / BPL;
  if constexpr (L >= 1)
    if (a.T <= 1) return launch_dot<XT, LPR, BPL, 1, KS>(a, s);
  if constexpr (L >= 2)
    if (a.T <= 2) return launch_dot<XT, LPR, BPL, 2, KS>(a, s);
  if constexpr (L >= 4)
    if (a.T <= 4) return launch_dot<XT, LPR, BPL, 4, KS>(a, s);
  if constexpr (L >= 6)
    if (a.T <= 6) return launch_dot<XT, LPR, BPL, 6, KS>(a, s);
  if constexpr (L >= 8 && KS > 1)
    if (a.T <= 8) return launch_dot<XT, LPR, BPL, 8, KS>(a, s);
  return hipErrorInvalidValue;
}
// blocks per lane, of a row of KB blocks shared by lanes of one wave, or by four
constexpr int kNoDot = 1 << 20;
constexpr int dot_blocks(int64_t KB) {
  return KB <= 16 ? 1 : KB <= 32 ? 2 : KB <= 64 ? 1 : KB <= 128 ? 2 : KB <= 256 ? 4 : kNoDot;
}
constexpr int split_blocks(int64_t KB) { return KB <= 64 ? kNoDot : KB <= 256 ? 1 : KB <= 512 ? 2 : KB <= 1024 ? 4 : kNoDot; }
// Slices of a row in the dot kernel; 0: the tile kernel. Four slices have 256 or
// more block places a row, of which KB are filled: with many rows they pay while
// places times a block's instructions stay below what the tiles take for the KB
// blocks, C instructions each (us, dots against tiles: 4 x 70000 x 2080 bf16, 73 against 31;
// 4 x 4096 x 14336, 14.6 against 24.7; 8 x 5120 x 4096, 15.5 against 12.4; fp32 4 x 5120 x 4096, 13.2
// against 16.6; codes 8 x 5120 x 4096, 11.2 against 12.3;
// bf16 4 x 5120 x 4096, 10.9 against 12.2). Up to 2048 rows both are
// latency, and the tiles have more of it (8 x 1018 x 6464: bf16 7.9 against 12.0, codes 5.5
// against 11.3; fp32 4 x 1018 x 6464, 9.4 against 18.9).
template <int XT>
int dot_slices(const Q4Args& a) {
  const int64_t T = a.T <= 2 ? a.T : (a.T + 1) / 2 * 2, KB = a.K / 32;
  if (T <= 6 && T * dot_blocks(KB) <= dot_limit<XT, 1>()) return 1;
  if (T > 8 || T * split_blocks(KB) > dot_limit<XT, 4>()) return 0;
  const int64_t instructions = XT == MOE_F32 ? 44 + 34 * T : XT == MOE_Q8_32 ? 12 + 11 * T : 32 + 18 * T;
  constexpr int C = XT == MOE_F32 ? 400 : XT == MOE_Q8_32 ? 200 : 208;
  return a.N <= 2048 || 256 * split_blocks(KB) * instructions <= KB * C ? 4 : 0;
}
template <int XT>
hipError_t launch_dot_types(const Q4Args& a, int slices, hipStream_t s) {
  const int64_t KB = a.K / 32;
  if (slices == 4) {
    if (KB <= 256) return launch_dot_tokens<XT, 64, 1, 4>(a, s);
    if (KB <= 512) return launch_dot_tokens<XT, 64, 2, 4>(a, s);
    return launch_dot_tokens<XT, 64, 4, 4>(a, s);
  }
  if (KB <= 16) return launch_dot_tokens<XT, 16, 1, 1>(a, s);
  if (KB <= 32) return launch_dot_tokens<XT, 16, 2, 1>(a, s);
  if (KB <= 64) return launch_dot_tokens<XT, 64, 1, 1>(a, s);
  if (KB <= 128) return launch_dot_tokens<XT, 64, 2, 1>(a, s);
  return launch_dot_tokens<XT, 64, 4, 1>(a, s);
}

// The weights of one step, four blocks of 16 features, as loaded: lane l has
// block l % 4 of row l / 4 of the tile and its scale. Sixteen neighbouring lanes so
// read four runs of 64 bytes (and of 8); the lanes of a product's column each
// reading its row would take a cache access per lane, 64 of them per load,
// and those bound the kernel.
struct StepWeights {
  u32x4_t w;
  uint32_t d;
};
// vector memory loads of a load_step: the waits of the wide kernel count them
constexpr int kStepLoads = 2;
// The products' column of a tile's feature and back: columns 4i + j and
// features 4j + i.
__device__ __forceinline__ constexpr int column_of(int f) { return 4 * (f & 3) + (f >> 2); }

// blocks 4s .. of the row whose first block is `row`; past the row: its last
// block, whose scale counts as 0 in step_ready. Nothing is done to the results
// here, which would wait for them. kStepLoads loads, one for each member of st.
__device__ __forceinline__ void load_step(const u32x4_t* nib, const uint16_t* scl, uint32_t row, int s, int lane, int KB,
                                          StepWeights& st) {
  const uint32_t at = row + (uint32_t)min(4 * s + (lane & 3), KB - 1);
  st.w = nib[at];
  st.d = scl[at];
}
// After the loads: w[i] of lane (column, c) holds chunk c of block 4s + i of
// the column's feature, d[i] that block's scale. With lane = 16 c + 4 h + l, the
// loaded word (c, h, l; dword) is wanted at (dword, h, c; register l): the swap
// rounds exchange c and dword, the quads l and the register. The scales take
// the same way from lane groups to registers by broadcasting.
__device__ __forceinline__ void step_ready(const StepWeights& st, int s, int lane, int KB, uint32_t (&w)[4], float (&d)[4]) {
  u32x4_t t = st.w;
  transpose4(t);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = t[i];
  transpose_quad(w);
  uint32_t b[4];
  broadcast4(4 * s + (lane & 3) < KB ? __float_as_uint(half_to_float((uint16_t)st.d)) : 0u, b);
  transpose_quad(b);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = __uint_as_float(b[i]);
}

// ---------------------------------------------------------------------------
// Some tokens, one launch: a work-group of W waves takes 16 tokens by 16 FW
// features; KW = W / FW waves share the reduction in steps of four blocks. A
// chunk of CB blocks of the activations at a time is brought into operand form
// in LDS by the whole work-group, read from memory in whole lines and converted
// once for all its features; the next chunk's values and the next two steps' weights
// are on their way meanwhile.
//
// 16 tokens a work-group: 32 or 64 would convert the weights once for more
// tokens, but leave CUs idle at the sizes that come here (128 tokens, bf16, 1024 x
// 1024: 7.0 us against 8.3 with 32; 5120 x 4096: 33 against 37; event times).

template <int XT, int W, int KW, int CB>
__global__ __launch_bounds__(64 * W, W / 4) void q4_tile_kernel(Q4Args a, int token_tiles) {
  constexpr int TERMS = terms_of<XT>(), OP = op_of<XT>(), FW = W / KW, ROWS = 16, THREADS = 64 * W;
  constexpr bool Q8 = XT == MOE_Q8_32;
  constexpr int UPB = 2 * value_size<XT>();               // 16-byte units of a block of x
  constexpr int UNITS = ROWS * CB * UPB / THREADS;        // a thread's units of a chunk
  constexpr int SCALES = (ROWS * CB + THREADS - 1) / THREADS;
  static_assert(ROWS * CB * UPB % THREADS == 0 && CB % (4 * KW) == 0, "whole rounds");
  // operand [term][block][slot][c] of 16 bytes. Token r of block b sits in slot
  // r + b (mod ROWS) and c is xor-ed by the slot, so that neither the stores (a row's
  // blocks side by side) nor a fragment's reads meet in a bank; -24 sums and
  // scales [block][token]
  constexpr int kTerm = CB * ROWS * 64, kBase = TERMS * kTerm, kScale = kBase + CB * ROWS * 4;
  constexpr int kLds = kScale + (Q8 ? CB * ROWS * 4 : 0), kSums = W * 64 * 16;
  __shared__ __attribute__((aligned(16))) uint8_t s_x[kLds > kSums ? kLds : kSums];
  float* s_base = reinterpret_cast<float*>(s_x + kBase);
  float* s_scale = reinterpret_cast<float*>(s_x + kScale);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c = lane >> 4, kw = wave % KW, fw = wave / KW;
  const int KB = (int)(a.K / 32), steps = (KB + 3) / 4;
  const int ftile = blockIdx.x / token_tiles;
  const int64_t t0 = (int64_t)(blockIdx.x - ftile * token_tiles) * ROWS;
  const int live = (int)std::min<int64_t>(a.T - t0, ROWS);
  const int f0 = (ftile * FW + fw) * 16, fb = min(f0, (int)a.N - 1);  // this wave's features
  const u32x4_t* nib = static_cast<const u32x4_t*>(a.nibbles) + (int64_t)fb * KB;
  const uint16_t* scl = a.w_scales + (int64_t)fb * KB;
  const uint32_t wrow = (uint32_t)(min(f0 + (lane >> 2), (int)a.N - 1) - fb) * KB;  // past N: the last row, never stored

  u32x4_t raw[UNITS];
  float rscale[SCALES];
  // unit u of this thread: 16 bytes v of block b of token slot r
  auto fetch = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int q = threadIdx.x + THREADS * u, r = q / (CB * UPB), b = min(b0 + q / UPB % CB, KB - 1), v = q % UPB;
      const char* p = static_cast<const char*>(a.x) + (t0 + min(r, live - 1)) * a.x_stride * value_size<XT>();
      __builtin_memcpy(&raw[u], p + (int64_t)b * 16 * UPB + 16 * v, 16);
    }
    if constexpr (Q8) {
#pragma unroll
      for (int u = 0; u < SCALES; ++u) {
        const int q = min((int)threadIdx.x + THREADS * u, ROWS * CB - 1);
        rscale[u] = a.x_scales[(t0 + min(q / CB, live - 1)) * a.x_scales_stride + min(b0 + q % CB, KB - 1)];
      }
    }
  };
  // into LDS, zeros for blocks past the row
  auto put8 = [&](int k, int b, int r, int cc, int half, uint32_t lo, uint32_t hi) __attribute__((always_inline)) {
    const int slot = (r + b) & (ROWS - 1);
    uint32_t* p =
        reinterpret_cast<uint32_t*>(s_x + k * kTerm + ((b * ROWS + slot) * 4 + (cc ^ ((slot >> 2) & 3))) * 16 + 8 * half);
    p[0] = lo, p[1] = hi;
  };
  auto store = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int q = threadIdx.x + THREADS * u, r = q / (CB * UPB), b = q / UPB % CB, v = q % UPB;
      u32x4_t x = b0 + b < KB ? raw[u] : u32x4_t{0, 0, 0, 0};
      float sum = 0.f;
      if constexpr (XT == MOE_F32) {  // elements 4v .. 4v + 3: chunk v % 4, half v / 4
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x[i]);
        sum = (f[0] + f[1]) + (f[2] + f[3]);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = __float_as_uint(f[i]);
            if (k < 2) f[i] -= __uint_as_float(w[i] & 0xFFFF0000u);  // exact: the bits below
          }
          put8(k, b, r, v & 3, v >> 2, upper_halves(w[0], w[2]), upper_halves(w[1], w[3]));
        }
      } else if constexpr (Q8) {  // elements 16 v .. : half v of every chunk
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t lo, hi;
          codes_to_half(x[i], lo, hi);
          n = __builtin_amdgcn_sdot4((int)x[i], 0x01010101, n, false);
          put8(0, b, r, i, v, lo, hi);
        }
        sum = (float)n;
      } else {  // elements 8 v .. : half v / 2 of chunks 2 (v % 2) and the next
#pragma unroll
        for (int i = 0; i < 2; ++i)
          put8(0, b, r, 2 * (v & 1) + i, v >> 1, lower_halves(x[2 * i], x[2 * i + 1]), upper_halves(x[2 * i], x[2 * i + 1]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum += XT == MOE_F16 ? half_to_float((uint16_t)x[i]) + half_to_float((uint16_t)(x[i] >> 16))
                               : __uint_as_float(x[i] << 16) + __uint_as_float(x[i] & 0xFFFF0000u);
      }
      // the block's other units are in the neighbouring lanes
      sum += __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor1>(__float_as_uint(sum)));
      if constexpr (UPB >= 4) sum += __uint_as_float(route_dev::dpp32<route_dev::kDppQuadXor2>(__float_as_uint(sum)));
      if constexpr (UPB >= 8) sum += __uint_as_float(route_dev::dpp32<route_dev::kDppRowHalfMirror>(__float_as_uint(sum)));
      if (v == 0) s_base[b * ROWS + r] = -24.0f * sum;
    }
    if constexpr (Q8) {
#pragma unroll
      for (int u = 0; u < SCALES; ++u) {
        const int q = threadIdx.x + THREADS * u;
        if (q < ROWS * CB) s_scale[q % CB * ROWS + q / CB] = rscale[u];
      }
    }
  };

  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int lb, const uint32_t (&w)[4], const float (&d)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4_t wt = weights_of<OP>(w[i]);
      const int slot = (col + lb + i) & (ROWS - 1), at = ((lb + i) * ROWS + slot) * 4 + (c ^ ((slot >> 2) & 3));
      f32x4_t p = *reinterpret_cast<const f32x4_t*>(s_base + (lb + i) * ROWS + 4 * c);
#pragma unroll
      for (int k = 0; k < TERMS; ++k) p = mfma<OP>(*reinterpret_cast<const u32x4_t*>(s_x + k * kTerm + 16 * at), wt, p);
      if constexpr (Q8) p *= *reinterpret_cast<const f32x4_t*>(s_scale + (lb + i) * ROWS + 4 * c);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = fmaf(d[i], p[r], acc[r]);
      __asm__ volatile("" : "+v"(acc));  // as in the wide kernel
    }
  };

  // A wave has one step of every chunk: kw, kw + KW, ... Its weights come two chunks
  // ahead, in two sets of registers (8 x 4096 x 14336 bf16: 20.0 us, 25.0 with one chunk ahead;
  // 16 x 5120 x 4096: 9.9 and 12.6).
  static_assert(CB == 4 * KW, "a step per wave and chunk");
  StepWeights st[2];
  fetch(0);
#pragma unroll
  for (int i = 0; i < 2; ++i) load_step(nib, scl, wrow, min(kw + i * KW, steps - 1), lane, KB, st[i]);
  auto chunk = [&](int b0, StepWeights& st) __attribute__((always_inline)) {
    if (b0) __syncthreads();  // every wave is done with the chunk before
    store(b0);
    __syncthreads();
    fetch(b0 + CB);  // past the row its last block, never stored: a branch would make the weights' wait cover it
    const int s = b0 / 4 + kw;
    uint32_t w[4];
    float d[4];
    step_ready(st, s, lane, KB, w, d);
    load_step(nib, scl, wrow, min(s + 2 * KW, steps - 1), lane, KB, st);  // past the last step: never used
    if (s < steps) compute(4 * kw, w, d);
  };
#pragma unroll 1
  for (int b0 = 0; b0 < KB; b0 += 2 * CB) {
    chunk(b0, st[0]);
    if (b0 + CB < KB) chunk(b0 + CB, st[1]);
  }
  // the KW partial sums, in wave order; lane (column, c) holds tokens 4c + r of its feature
  __syncthreads();
  f32x4_t* s_sum = reinterpret_cast<f32x4_t*>(s_x);
  s_sum[wave * 64 + lane] = acc;
  __syncthreads();
#pragma unroll 1
  for (int e = threadIdx.x; e < 16 * FW * live; e += THREADS) {
    const int f = e % (16 * FW), tok = e / (16 * FW);
    const float* p =
        reinterpret_cast<const float*>(s_sum) + (f / 16 * KW * 64 + 16 * (tok / 4) + column_of(f % 16)) * 4 + tok % 4;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) v += p[w * 256];
    if (ftile * 16 * FW + f < a.N) put(a, t0 + tok, ftile * 16 * FW + f, v);
  }
}

template <int XT, int W, int KW, int CB>
hipError_t launch_tile(const Q4Args& a, hipStream_t s) {
  constexpr int F = 16 * W / KW;
  const int64_t token_tiles = (a.T + 15) / 16, tiles = (a.N + F - 1) / F * token_tiles;
  return launch(q4_tile_kernel<XT, W, KW, CB>, dim3((unsigned)tiles), dim3(64 * W), Launch{s}, a, (int)token_tiles);
}
template <int XT>
hipError_t launch_tile_types(const Q4Args& a, hipStream_t s) {
  // As long as a work-group has a CU of its own it has all the waves that its features can use: 16
  // features and 8 waves, else 32 and 16 (rows long enough for their chunks of 32 blocks), else 32
  // and 8. us, bf16 and fp32: 16 x 4096 x 4096, 256 work-groups of 16 features, 8.1 and 12.3 against 9.9
  // and 14.3 in the last form; 16 x 5120 x 4096, 160 of 32, 9.5 and 12.6 in the second, 9.9 and 14.2 in
  // the last; 16 x 14336 x 4096, 448 of 32, 17.1 and 23.6 against 14.1 and 21.6; 32 x 4096 x 1536, fp32, 7.9
  // against 7.4.
  const int64_t tiles = (a.T + 15) / 16;
  if (tiles * ((a.N + 15) / 16) <= 256) return launch_tile<XT, 8, 8, 32>(a, s);
  if (tiles * ((a.N + 31) / 32) <= 256 && a.K > 2048) return launch_tile<XT, 16, 8, 32>(a, s);
  return launch_tile<XT, 8, 4, 16>(a, s);
}

// ---------------------------------------------------------------------------
// Operand form of the activations, for more tokens: per 16 tokens and block
// TERMS KiB in the lanes' order, and -24 * sum of the block for each of them.
// Tokens are padded to whole tiles and blocks to whole steps, both with zeros.


struct Operand {
  int64_t rows, KB, bytes;  // padded tokens, padded blocks, bytes with the sums
  uint8_t* terms;
  float* base;              // [rows / 16][KB][runs][16]
  __host__ __device__ static Operand make(uint8_t* ws, int64_t T, int64_t K, int n_terms, int runs, int tile_rows) {
    Operand o;
    o.rows = (T + tile_rows - 1) / tile_rows * tile_rows;
    o.KB = (K / 32 + 3) / 4 * 4;
    const int64_t units = o.rows / 16 * o.KB;
    o.terms = ws;
    o.base = reinterpret_cast<float*>(ws + units * n_terms * 1024);
    o.bytes = units * (n_terms * 1024 + runs * 64);
    return o;
  }
};

// a wave per 16 tokens and block
template <int XT>
__global__ __launch_bounds__(256) void q4_operand_kernel(Q4Args a, Operand o) {
  constexpr int TERMS = terms_of<XT>();
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= o.rows / 16 * o.KB) return;
  const int64_t b = unit % o.KB, row = unit / o.KB * 16 + r;
  u32x4_t t[TERMS];
  float sum;
#pragma unroll
  for (int k = 0; k < TERMS; ++k) t[k] = u32x4_t{0, 0, 0, 0};
  const bool in = row < a.T && b < a.K / 32;
  if (in)
    chunk_terms<XT>(load_chunk<XT>(static_cast<const char*>(a.x) + row * a.x_stride * value_size<XT>(), b, c), t);
  sum = chunk_sum<XT>(t);
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
#pragma unroll
  for (int k = 0; k < TERMS; ++k) reinterpret_cast<u32x4_t*>(o.terms)[(unit * TERMS + k) * 64 + lane] = t[k];
  if (c == 0) o.base[unit * 16 * runs_of<XT>() + r] = -24.0f * sum;
  if (XT == MOE_Q8_32 && c == 0) o.base[unit * 32 + 16 + r] = in ? a.x_scales[row * a.x_scales_stride + b] : 0.f;
}

// ---------------------------------------------------------------------------
// Many tokens: tiles of 64 tokens x 64 features per wave. The operand goes
// through LDS in a ring of stages of SB blocks, copied by the LDS-DMA loads; every
// wave loads its weights into registers one step (four blocks) ahead.
//   WK = 1: four waves make a tile of 128 x 128 and share two stages of four
//           blocks (one: fp32), with a barrier each.
//   WK = 4: four waves share one tile of 64 x 64 and split the reduction, step by
//           step; each has stages of its own, one block each, three copies ahead
//           (fp32: two) and no barrier; the sums are added at the end, in wave order.
//           Four times the work-groups, for calls with few tiles: those have a
//           wave per SIMD, whose copies nothing else covers.

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

// tokens, and features, of a work-group's tile
constexpr int wide_side(int WK) { return WK == 1 ? 128 : 64; }

// s_waitcnt immediate (GFX9 encoding) waiting for vmcnt <= n only
constexpr int waitcnt_vm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// What step_ready does, through LDS: a wave writes a tile's words and scales as
// loaded, lane (feature, block), and reads chunk c of every block back; the wave's
// own accesses are in order, no wait in between. Beside matrix products that take
// the place of register moves this saves 140 instructions a step
// (4096 x 5120 x 4096 bf16: 302 us with the moves, 285 so). Block b of feature f lies in
// quarter b ^ (f >> 2) of the feature's 64 bytes: without conflicts either way.
constexpr int kTurnBytes = 1024 + 256;
struct Turn {
  uint8_t *write_w, *write_d;
  const uint8_t *read_w[4], *read_d;
  static __device__ __forceinline__ Turn make(uint8_t* s, int lane) {
    const int col = lane & 15, c = lane >> 4;
    Turn t;
    t.write_w = s + (lane >> 2) * 64 + ((lane & 3) ^ (lane >> 4)) * 16;
    t.write_d = s + 1024 + lane * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.read_w[i] = s + col * 64 + (i ^ (col >> 2)) * 16 + c * 4;
    t.read_d = s + 1024 + col * 16;
    return t;
  }
  __device__ __forceinline__ void step(const StepWeights& st, int s, int lane, int KB, uint32_t (&w)[4], float (&d)[4]) const {
    exchange();  // the tile before has been read
    *reinterpret_cast<u32x4_t*>(write_w) = st.w;
    *reinterpret_cast<float*>(write_d) = 4 * s + (lane & 3) < KB ? half_to_float((uint16_t)st.d) : 0.f;
    exchange();
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(read_d);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(read_w[i]), d[i] = v[i];
  }
  // other lanes' words behind this point and before it: an order for the compiler, no
  // instruction, since a wave's LDS accesses are in order
  static __device__ __forceinline__ void exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
};

// A wave's tile of results on its way through the epilogue, [64 tokens][kTileRow]: the four lane groups write rows 4
// apart, 16 banks from each other
constexpr int kTileRow = 68;

// 4 values at i, of those before n
__device__ __forceinline__ f32x4_t load_values4(const void* p, int type, int64_t i, int n) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4 && type == MOE_F32) {
    __builtin_memcpy(&v, static_cast<const float*>(p) + i, 16);
  } else if (n >= 4) {
    uint32_t h[2];
    __builtin_memcpy(h, static_cast<const uint16_t*>(p) + i, 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint16_t b = (uint16_t)(h[j >> 1] >> (16 * (j & 1)));
      v[j] = type == MOE_F16 ? half_to_float(b) : bf16_to_float(b);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = load_value(p, type, i + j);
  }
  return v;
}
__device__ __forceinline__ void store_values4(void* p, int type, int64_t i, int n, f32x4_t v) {
  if (n >= 4 && type == MOE_F32) {
    __builtin_memcpy(static_cast<float*>(p) + i, &v, 16);
  } else if (n >= 4) {
    uint16_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = type == MOE_F16 ? float_to_half(v[j]) : float_to_bf16(v[j]);
    __builtin_memcpy(static_cast<uint16_t*>(p) + i, h, 8);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) {
        if (type == MOE_F32)
          store1<MOE_F32>(p, i + j, v[j]);
        else if (type == MOE_F16)
          store1<MOE_F16>(p, i + j, v[j]);
        else
          store1<MOE_BF16>(p, i + j, v[j]);
      }
  }
}
// The results of one wave's tile, tokens t0 .. t0 + 63 and features f0 .. f0 + 63, through the epilogue: four
// tokens at a time, a lane 4 features of one; the operands of the next four are on their way meanwhile
__device__ __forceinline__ void put_tile(const Q4Args& a, const float* s_y, int64_t t0, int f0, int lane) {
  const Q4Epilogue& e = a.epi;
  const int f = f0 + 4 * (lane & 15), n = (int)std::min<int64_t>(a.N - f, 4);
  if (n <= 0) return;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  const f32x4_t bias = e.bias ? load_values4(e.bias, MOE_F32, f, n) : zero;
  f32x4_t mul[2] = {zero, zero}, res[2] = {zero, zero};
  auto fetch = [&](int i, int to) __attribute__((always_inline)) {
    const int64_t t = t0 + 4 * i + (lane >> 4);
    if (t >= a.T) return;
    if (e.mul) mul[to] = load_values4(e.mul, e.mul_type, t * e.mul_stride + f, n);
    if (e.res) res[to] = load_values4(e.res, e.res_type, t * e.res_stride + f, n);
  };
  auto put4 = [&](int i, int from) __attribute__((always_inline)) {
    const int64_t t = t0 + 4 * i + (lane >> 4);
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(s_y + (4 * i + (lane >> 4)) * kTileRow + 4 * (lane & 15));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = activate(e.act, v[j] + bias[j]);
      if (e.mul) v[j] *= mul[from][j];
      if (e.res) v[j] += res[from][j];
    }
    if (t < a.T) store_values4(a.y, a.y_type, t * a.y_stride + f, n, v);
  };
  fetch(0, 0);
#pragma unroll 1
  for (int i = 0; i < 16; i += 2) {
    fetch(i + 1, 1);
    put4(i, 0);
    if (i + 2 < 16) fetch(i + 2, 0);
    put4(i + 1, 1);
  }
}

// two work-groups a CU, but for split fp32 tiles, whose stages of three terms leave room for one
template <int XT, int SB, int WK, int RING>
__global__ __launch_bounds__(256, WK > 1 && terms_of<XT>() == 3 ? 1 : 2) void q4_wide_kernel(Q4Args a, Operand o, int row_tiles, int col_tiles) {
  constexpr int TERMS = terms_of<XT>(), SIDE = wide_side(WK), MG = SIDE / 16;  // row tiles of 16 in the stages
  constexpr int RUNS = runs_of<XT>(), kBlockBase = 64 * RUNS;
  constexpr int kTermBytes = MG * SB * TERMS * 1024, kBaseBytes = MG * SB * kBlockBase, kStage = kTermBytes + kBaseBytes;
  constexpr int kSums = WK > 1 ? WK * 16 * 64 * 16 : kEpilogue ? 4 * 64 * kTileRow * 4 : 0;
  constexpr int kLds = RING * kStage * WK;
  static_assert(RING == 2 || SB == 1, "the ring's waits count blocks");
  static_assert(sizeof(StepWeights::w) == 16, "a load_step is one load of 16 bytes and one of a scale: kStepLoads");
  __shared__ __attribute__((aligned(1024))) uint8_t s_lds[kLds + 4 * kTurnBytes > kSums ? kLds + 4 * kTurnBytes : kSums];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c = lane >> 4;
  const Turn turn = Turn::make(s_lds + kLds + wave * kTurnBytes, lane);
  // work-groups go round the 8 XCDs: each XCD takes a run of the tiles, in
  // groups of 8 row tiles by all column tiles, so that the tiles it works on at
  // a time share operand rows and weights in its L2
  const int per = gridDim.x / 8, tile = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (tile >= row_tiles * col_tiles) return;
  const int group = tile / (8 * col_tiles), in_group = tile - group * 8 * col_tiles;
  const int group_rows = min(8, row_tiles - 8 * group);
  const int rt = 8 * group + in_group % group_rows, ct = in_group / group_rows;
  const int m0 = WK == 1 ? (wave & 1) * 4 : 0;                       // row tiles of 16 within the tile
  const int f0 = ct * SIDE + (WK == 1 ? (wave >> 1) * 64 : 0);       // this wave's features
  const int wk = WK == 1 ? 0 : wave;                                 // its share of the reduction
  const int KB = (int)(a.K / 32), steps = (int)(o.KB / 4);
  const int64_t u0 = (int64_t)rt * MG * o.KB;                        // first operand unit of the tile's rows
  uint8_t* s_x = s_lds + wk * RING * kStage;

  // block indexes of the lane's features (past N: the last one, never stored)
  // from the wave's first one: at most 63 rows of 2^15 blocks
  const int fb = min(f0, (int)a.N - 1);
  const u32x4_t* nib = static_cast<const u32x4_t*>(a.nibbles) + (int64_t)fb * KB;
  const uint16_t* scl = a.w_scales + (int64_t)fb * KB;
  uint32_t wrow[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) wrow[t] = (uint32_t)(min(f0 + 16 * t + (lane >> 2), (int)a.N - 1) - fb) * KB;
  StepWeights wn[4];
  auto issue_weights = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 4; ++t) load_step(nib, scl, wrow[t], s, lane, KB, wn[t]);
  };
  // blocks b0 .. b0 + SB - 1 into a buffer of the ring
  auto issue_stage = [&](int buf, int b0) __attribute__((always_inline)) {
    uint8_t* dst = s_x + buf * kStage;
    constexpr int kRun = SB * TERMS;              // KiB of a row tile
    constexpr int kMine = WK == 1 ? MG / 4 : MG;  // row tiles this wave copies
#pragma unroll
    for (int i = 0; i < kMine * kRun; ++i) {
      const int m = (WK == 1 ? kMine * wave : 0) + i / kRun, q = i % kRun;
      const uint8_t* src = o.terms + ((u0 + m * o.KB + b0) * TERMS + q) * 1024 + 16 * lane;
      __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + (m * kRun + q) * 1024), 16, 0, 0);
    }
    // the sums (and scales): 1 KiB per copy
    constexpr int kLanes = 4 * SB * RUNS;  // lanes of a row tile
#pragma unroll
    for (int i = 0; i < (kBaseBytes + 1023) / 1024; ++i) {
      if (WK == 1 && wave != i) continue;
      const int at = 64 * i + lane, m = at / kLanes;
      if (m < MG) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(o.base + (u0 + m * o.KB + b0) * 16 * RUNS) + 16 * (at % kLanes);
        __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + kTermBytes + 1024 * i), 16, 0, 0);
      }
    }
  };

  f32x4_t acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // Stage j of the wave (SB blocks of its steps in turn; four blocks of a step
  // are 4 / SB stages) lies in buffer j % RING and is copied RING - 1 stages ahead;
  // past the last step that one's blocks again, never read, so that every stage
  // is followed by the same number of loads.
  constexpr int NS = 4 / SB;                                             // stages of a step
  constexpr int kCopies = (WK == 1 ? MG / 4 : MG) * SB * TERMS + (WK == 1 ? 0 : (kBaseBytes + 1023) / 1024);
  const int last = wk < steps ? wk + (steps - 1 - wk) / WK * WK : wk;   // the wave's last step
  if (wk < steps) {
    issue_weights(wk);
#pragma unroll
    for (int j = 0; j < RING - 1; ++j) issue_stage(j, 4 * min(wk + WK * (j / NS), last) + SB * (j % NS));
  }
#pragma unroll 1
  for (int s = wk, n = 0; s < steps; s += WK, ++n) {
    uint32_t w[4][4];
    float d[4][4];
#pragma unroll
    for (int h = 0; h < NS; ++h) {
      const int j = n * NS + h, buf = NS % RING == 0 ? h % RING : j % RING;
      // Stage j is there (WK = 1: all waves' shares, and no wave reads stage j - 1 any more). Loads come
      // back in order: behind it are RING - 2 stages and, if they were issued in between, the step's weights.
      constexpr int kAfter = (RING - 2) * kCopies;
      if (RING > 2 && h >= 1 && h <= RING - 2)
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(kAfter + 4 * kStepLoads));
      else
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(kAfter));
      if constexpr (WK == 1) __syncthreads();
      // nothing moves above the wait: LDS reads would come too early, and uses of the weights
      // would be given a wait for every copy in flight
      __asm__ volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (h == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) turn.step(wn[t], s, lane, KB, w[t], d[t]);
        issue_weights(min(s + WK, last));
      }
      const int ahead = h + RING - 1;  // in stages from the step's first
      issue_stage(NS % RING == 0 ? ahead % RING : (j + RING - 1) % RING, 4 * min(s + WK * (ahead / NS), last) + SB * (ahead % NS));
      const uint8_t* st = s_x + buf * kStage;
      // One group per block and feature tile: the products of this tile (matrix
      // cores), beside them the scale FMAs of the tile before (VALU) and the
      // next tile's weights; the operand of the next block is read ahead.
      u32x4_t x[2][4][TERMS];
      f32x4_t base[2][4], p[2][4], dx[4];
      auto read_block = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int k = 0; k < TERMS; ++k)
            x[i & 1][m][k] = *reinterpret_cast<const u32x4_t*>(st + (((m0 + m) * SB + i) * TERMS + k) * 1024 + 16 * lane);
          base[i & 1][m] = *reinterpret_cast<const f32x4_t*>(st + kTermBytes + ((m0 + m) * SB + i) * kBlockBase + 16 * c);
        }
      };
      auto scale = [&](int g, int m) __attribute__((always_inline)) {
        const int t = g & 3;
        const float dt = d[t][SB * h + (g >> 2)];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[m][t][r] = fmaf(dt, XT == MOE_Q8_32 ? p[g & 1][m][r] * dx[m][r] : p[g & 1][m][r], acc[m][t][r]);
        // a use of the sums here: otherwise the compiler sinks the scale FMAs to the end of the
        // unrolled blocks and keeps all their products live
        __asm__ volatile("" : "+v"(acc[m][t]));
      };
      read_block(0);
      u32x4_t wt[2];
      wt[0] = weights_of<op_of<XT>()>(w[0][SB * h]);
#pragma unroll
      for (int g = 0; g < 4 * SB; ++g) {
        const int i = g >> 2;
        __builtin_amdgcn_sched_barrier(0);
        if ((g & 3) == 0 && i + 1 < SB) read_block(i + 1);
        // one product, a quarter of the next weights, the scale FMAs of one
        // product of the tile before, in this order: left to itself the compiler
        // issues the products back to back and the matrix cores idle beside the FMAs
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          p[g & 1][m] = base[i & 1][m];
#pragma unroll
          for (int k = 0; k < TERMS; ++k) p[g & 1][m] = mfma<op_of<XT>()>(x[i & 1][m][k], wt[g & 1], p[g & 1][m]);
          if (g + 1 < 4 * SB) wt[(g + 1) & 1][m] = weights_part<op_of<XT>()>(w[(g + 1) & 3][SB * h + ((g + 1) >> 2)], m);
          if (g > 0) scale(g - 1, m);
          if (XT == MOE_Q8_32 && (g & 3) == 0)  // wanted by the next tile's turn
            dx[m] = *reinterpret_cast<const f32x4_t*>(st + kTermBytes + ((m0 + m) * SB + i) * kBlockBase + 64 + 16 * c);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) scale(4 * SB - 1, m);
    }
  }
  if constexpr (WK == 1 && kEpilogue) {
    // Through LDS: the epilogue reads its operands and writes y in whole lines, 64 features of a token by
    // 16 lanes, in a loop (4096 x 4096 x 4096 bf16 with all of it: 260 us; 340 in the
    // lanes' own order, 2-byte accesses by 16 lanes).
    // Every wave is done with the stages and the copies behind the last one have landed; a wave's
    // 64 x 64 results are then its own.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    float* s_y = reinterpret_cast<float*>(s_lds) + wave * (64 * kTileRow);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) s_y[(16 * m + 4 * c + r) * kTileRow + 16 * t + col] = acc[m][t][r];
    Turn::exchange();
    put_tile(a, s_y, (int64_t)rt * SIDE + 16 * m0, f0, lane);
  } else if constexpr (WK == 1) {
    // lane (column, c) holds tokens 4c + r of its features
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = (int64_t)rt * SIDE + 16 * (m0 + m) + 4 * c + r;
        if (row >= a.T) continue;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int f = f0 + 16 * t + col;
          if (f < a.N) put(a, row, f, acc[m][t][r]);
        }
      }
  } else {
    // every wave is done with its stages, the copies behind the last one too
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    f32x4_t* s_sum = reinterpret_cast<f32x4_t*>(s_lds);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) s_sum[((wk * 4 + m) * 4 + t) * 64 + lane] = acc[m][t];
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < 64 * 64; e += 256) {
      const int f = e & 63, tok = e >> 6;
      const int64_t row = (int64_t)rt * SIDE + tok;
      if (row >= a.T || f0 + f >= a.N) continue;
      const float* p = reinterpret_cast<const float*>(s_sum) +
                       ((tok / 16 * 4 + f / 16) * 64 + 16 * (tok / 4 % 4) + f % 16) * 4 + tok % 4;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) v += p[w * 16 * 256];
      put(a, row, f0 + f, v);
    }
  }
}

template <int XT>
hipError_t launch_operand(const Q4Args& a, const Operand& o, hipStream_t s) {
  const int64_t waves = o.rows / 16 * o.KB;
  return launch(q4_operand_kernel<XT>, dim3((unsigned)((waves + 3) / 4)), dim3(256), Launch{s}, a, o);
}

// tokens of one pass: bounds the workspace and the grids (16384 tokens of
// k = 2^20 are 2^25 operand units; 128 row tiles of 2^22 features 2^22 tiles)
constexpr int64_t kPassTokens = 16384;

// 0: one launch without an operand pass; else the WK of the wide tiles. us on the GPU, one launch /
// split tiles / whole tiles:
//                                   bf16              fp32              codes
//   128 x 2048 x 4096, 1.1e9          16 /  24 /  71    24 /  37 / 111    16 /  29 /  89
//   1024 x 1024 x 1024, 1.1e9         17 /  15 /  28    27 /  19 /  38    17 /  17 /  32
// From 2e9 products on the operand pass pays, if every second CU or so has a tile of 64 x 64 to
// work on: each is one work-group and goes through the whole reduction by itself.
//   64 x 512 x 65536, 8 tiles         77 / 213 / 935   140 / 407 / 1627   76 / 292 / 1229
//   300 x 1024 x 8192, 80             35 /  39 / 129    62 /  65 / 210    35 /  48 / 166
//   64 x 6144 x 8192, 96              37 /  37 / 128    65 /  64 / 209    38 /  48 / 165
//   64 x 7168 x 8192, 112             47 /  37 / 128    78 /  64 / 209    47 /  48 / 165
//   512 x 1024 x 4096, 128            26 /  25 /  72    45 /  40 / 112    26 /  30 /  90
//   128 x 5120 x 4096, 160            32 /  25 /  71    57 /  39 / 111    33 /  30 /  89
// The pass reads and writes all activations, which a few features do not repay:
//   8192 x 256 x 1024                 30 /  24 /  33    52 /  46 /  53    30 /  26 /  38
//   16384 x 128 x 1024                31 /  31 /  40    55 /  64 /  68    30 /  32 /  45
//   100000 x 64 x 512                 62 / 140 / 196   105 / 227 / 279    58 / 151 / 219
// (beyond 2^20 tokens the one launch would have too many work-groups for a grid). Whole tiles of
// 128 x 128: two work-groups a CU, against one of split fp32 tiles, whose three terms fill the LDS.
//   512 x 5120 x 4096, 160           107 /  51 /  73   188 / 108 / 114   111 /  59 /  90
//   1024 x 4096 x 4096, 256          159 /  66 /  75   286 / 147 / 120   161 /  75 /  93
//   2048 x 5120 x 4096, 640          406 / 154 / 172   714 / 361 / 302   393 / 178 / 200
//   4096 x 4096 x 1024, 1024         199 /  86 /  70   341 / 208 / 119   198 /  98 /  80
//   48 x 65537 x 1024, 513 (of 48 tokens)  47 / 33 / 50  73 / 61 / 72     42 /  35 /  59
int wide_split(int64_t T, int64_t N, int64_t K, int32_t x_type) {
  if (T <= 32 || (double)T * (double)N * (double)K <= 2e9) return 0;
  const int64_t split = ((T + 63) / 64) * ((N + 63) / 64), whole = ((T + 127) / 128) * ((N + 127) / 128);
  if (split < (x_type == MOE_Q8_32 ? 160 : 112) || (N < 256 && T <= 1 << 20)) return 0;
  return whole >= (x_type == MOE_F32 && T > 256 ? 256 : 1024) ? 1 : 4;
}

template <int XT, int WK>
hipError_t launch_wide(const Q4Args& a, hipStream_t s) {
  constexpr int TERMS = terms_of<XT>(), SIDE = wide_side(WK), SB = TERMS == 3 || WK > 1 ? 1 : 4;
  constexpr int RING = WK == 1 ? 2 : TERMS == 3 ? 3 : 4;
  const int col_tiles = (int)((a.N + SIDE - 1) / SIDE);
  for (int64_t t0 = 0; t0 < a.T; t0 += kPassTokens) {
    Q4Args p = a;
    p.T = std::min(a.T - t0, kPassTokens);
    p.x = static_cast<const char*>(a.x) + t0 * a.x_stride * value_size<XT>();
    p.x_scales = a.x_scales ? a.x_scales + t0 * a.x_scales_stride : nullptr;
    p.y = static_cast<char*>(a.y) + t0 * a.y_stride * (a.y_type == MOE_F32 ? 4 : 2);
    if constexpr (kEpilogue) {
      if (a.epi.mul) p.epi.mul = static_cast<const char*>(a.epi.mul) + t0 * a.epi.mul_stride * (a.epi.mul_type == MOE_F32 ? 4 : 2);
      if (a.epi.res) p.epi.res = static_cast<const char*>(a.epi.res) + t0 * a.epi.res_stride * (a.epi.res_type == MOE_F32 ? 4 : 2);
    }
    const Operand o = Operand::make(a.ws, p.T, a.K, TERMS, runs_of<XT>(), SIDE);
    if (hipError_t e = launch_operand<XT>(p, o, s); e != hipSuccess) return e;
    const int row_tiles = (int)(o.rows / SIDE);
    const unsigned grid = (unsigned)(((int64_t)row_tiles * col_tiles + 7) / 8 * 8);
    hipError_t e = launch(q4_wide_kernel<XT, SB, WK, RING>, dim3(grid), dim3(256), Launch{s}, p, o, row_tiles, col_tiles);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int XT>
hipError_t launch_types(const Q4Args& a, hipStream_t s) {
  switch (wide_split(a.T, a.N, a.K, XT)) {
    case 1: return launch_wide<XT, 1>(a, s);
    case 4: return launch_wide<XT, 4>(a, s);
  }
  const int slices = dot_slices<XT>(a);
  return slices ? launch_dot_types<XT>(a, slices, s) : launch_tile_types<XT>(a, s);
}

hipError_t launch_q4(const Q4Args& a, hipStream_t s) {
  switch (a.x_type) {
    case MOE_F32: return launch_types<MOE_F32>(a, s);
    case MOE_F16: return launch_types<MOE_F16>(a, s);
    case MOE_BF16: return launch_types<MOE_BF16>(a, s);
    default: return launch_types<MOE_Q8_32>(a, s);
  }
}

}  // namespace
}  // namespace moe
