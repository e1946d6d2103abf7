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
__device__ __forceinline__ uint32_t weights_part(uint32_t w, int i) {
  if constexpr (XT == MOE_F16) {
    constexpr uint32_t M = 0x03C003C0u, C = 0x4C004C00u;
    return and_or(i == 0 ? w << 6 : i == 1 ? w >> 2 : i == 2 ? w << 2 : w >> 6, M, C);
  } else {
    constexpr uint32_t M = 0x00780078u, C = 0x41804180u;
    return and_or(i == 0 ? w << 3 : i == 1 ? w >> 5 : i == 2 ? w >> 1 : w >> 9, M, C);
  }
}
template <int XT>
__device__ __forceinline__ u32x4_t weights_of(uint32_t w) {
  return u32x4_t{weights_part<XT>(w, 0), weights_part<XT>(w, 1), weights_part<XT>(w, 2), weights_part<XT>(w, 3)};
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

// ---------------------------------------------------------------------------
// Operand form of the activations, for more tokens: per 16 tokens and block
// TERMS KiB in the lanes' order, and -24 * sum of the block for each of them.
// Tokens are padded to whole tiles and blocks to whole steps, both with zeros.

constexpr int kTileRows = 128;  // tokens of a wide tile

struct Operand {
  int64_t rows, KB, bytes;  // padded tokens, padded blocks, bytes with the sums
  uint8_t* terms;
  float* base;              // [rows / 16][KB][16]
  __host__ __device__ static Operand make(uint8_t* ws, int64_t T, int64_t K, int n_terms, int tile_rows) {
    Operand o;
    o.rows = (T + tile_rows - 1) / tile_rows * tile_rows;
    o.KB = (K / 32 + 3) / 4 * 4;
    const int64_t units = o.rows / 16 * o.KB;
    o.terms = ws;
    o.base = reinterpret_cast<float*>(ws + units * n_terms * 1024);
    o.bytes = units * (n_terms * 1024 + 64);
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
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < TERMS; ++k) t[k] = u32x4_t{0, 0, 0, 0};
  if (row < a.T && b < a.K / 32)
    chunk_of<XT>(static_cast<const char*>(a.x) + row * a.x_stride * value_size<XT>(),
                 XT == MOE_Q8_32 ? a.x_scales + row * a.x_scales_stride : nullptr, b, c, t);
#pragma unroll
  for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (XT == MOE_F16)
        sum += half_to_float((uint16_t)t[k][i]) + half_to_float((uint16_t)(t[k][i] >> 16));
      else
        sum += __uint_as_float(t[k][i] << 16) + __uint_as_float(t[k][i] & 0xFFFF0000u);
    }
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
#pragma unroll
  for (int k = 0; k < TERMS; ++k) reinterpret_cast<u32x4_t*>(o.terms)[(unit * TERMS + k) * 64 + lane] = t[k];
  if (c == 0) o.base[unit * 16 + r] = -24.0f * sum;
}

// ---------------------------------------------------------------------------
// Wide tiles: 128 tokens x 128 features by 4 waves of 64 x 64. The operand
// goes through LDS in stages of SB blocks, copied by the LDS-DMA loads two
// deep; every wave loads its weights into registers one step (four blocks)
// ahead.

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

constexpr int kWideN = 128;

template <int XT, int SB>
__global__ __launch_bounds__(256, 2) void q4_wide_kernel(Q4Args a, Operand o, int row_tiles, int col_tiles) {
  constexpr int TERMS = terms_of<XT>();
  constexpr int kTermBytes = 8 * SB * TERMS * 1024, kBaseBytes = 8 * SB * 64, kStage = kTermBytes + kBaseBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t s_x[2 * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c = lane >> 4;
  // work-groups go round the 8 XCDs: each XCD takes a run of the tiles, in
  // groups of 8 row tiles by all column tiles, so that the tiles it works on at
  // a time share operand rows and weights in its L2
  const int per = gridDim.x / 8, tile = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (tile >= row_tiles * col_tiles) return;
  const int group = tile / (8 * col_tiles), in_group = tile - group * 8 * col_tiles;
  const int group_rows = min(8, row_tiles - 8 * group);
  const int rt = 8 * group + in_group % group_rows, ct = in_group / group_rows;
  const int m0 = (wave & 1) * 4;                                     // row tiles of 16 within the tile
  const int f0 = ct * kWideN + (wave >> 1) * 64;                     // this wave's features
  const int KB = (int)(a.K / 32), steps = (int)(o.KB / 4);
  const int64_t u0 = (int64_t)rt * 8 * o.KB;                         // first operand unit of the tile's rows

  // block indexes of the lane's features (past N: the last one, never stored)
  // from the wave's first one: at most 63 rows of 2^15 blocks
  const int fb = min(f0, (int)a.N - 1);
  const u32x4_t* nib = static_cast<const u32x4_t*>(a.nibbles) + (int64_t)fb * KB;
  const uint16_t* scl = a.w_scales + (int64_t)fb * KB;
  uint32_t wrow[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) wrow[t] = (uint32_t)(min(f0 + 16 * t + col, (int)a.N - 1) - fb) * KB;
  u32x4_t wn[4];
  uint32_t dn[4];
  auto issue_weights = [&](int s) __attribute__((always_inline)) {
    const int b = 4 * s + c, bc = min(b, KB - 1);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      wn[t] = nib[wrow[t] + bc];
      dn[t] = scl[wrow[t] + bc];
    }
  };
  // stage j (blocks SB j ..) into buffer j % 2: SB TERMS 2 operand pieces of 1 KiB per wave
  auto issue_stage = [&](int j) __attribute__((always_inline)) {
    uint8_t* dst = s_x + (j & 1) * kStage;
    constexpr int kRun = SB * TERMS;  // KiB of a row tile
#pragma unroll
    for (int i = 0; i < 2 * kRun; ++i) {
      const int m = 2 * wave + i / kRun, q = i % kRun;
      const uint8_t* src = o.terms + ((u0 + m * o.KB + SB * j) * TERMS + q) * 1024 + 16 * lane;
      __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + (m * kRun + q) * 1024), 16, 0, 0);
    }
    // the sums: 64 SB bytes per row tile
    constexpr int kLanes = 4 * SB;  // lanes of a row tile
    if (wave < kBaseBytes / 1024 || (kBaseBytes < 1024 && wave == 0)) {
      const int at = 64 * wave + lane, m = at / kLanes;
      if (m < 8) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(o.base + (u0 + m * o.KB + SB * j) * 16) + 16 * (at % kLanes);
        __builtin_amdgcn_global_load_lds((glb_void_t*)src, (lds_void_t*)(dst + kTermBytes + 1024 * wave), 16, 0, 0);
      }
    }
  };

  f32x4_t acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  issue_weights(0);
  issue_stage(0);
  for (int s = 0; s < steps; ++s) {
    u32x4_t w[4];
    uint32_t d[4][4];
#pragma unroll
    for (int h = 0; h < 4 / SB; ++h) {
      const int j = s * (4 / SB) + h;
      // this wave's copies of stage j are done, then every wave's, and no wave reads stage j - 1 any more
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
      __syncthreads();
      if (h == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          w[t] = wn[t];
          transpose4(w[t]);
          // past the row: scale 0
          broadcast4(4 * s + c < KB ? __float_as_uint(half_to_float((uint16_t)dn[t])) : 0u, d[t]);
        }
        if (s + 1 < steps) issue_weights(s + 1);
      }
      if (SB * (j + 1) < o.KB) issue_stage(j + 1);
      const uint8_t* st = s_x + (j & 1) * kStage;
      // One group per block and feature tile: the products of this tile (matrix
      // cores), beside them the scale FMAs of the tile before (VALU) and the
      // next tile's weights; the operand of the next block is read ahead.
      u32x4_t x[2][4][TERMS];
      f32x4_t base[2][4], p[2][4];
      auto read_block = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int k = 0; k < TERMS; ++k)
            x[i & 1][m][k] = *reinterpret_cast<const u32x4_t*>(st + (((m0 + m) * SB + i) * TERMS + k) * 1024 + 16 * lane);
          base[i & 1][m] = *reinterpret_cast<const f32x4_t*>(st + kTermBytes + ((m0 + m) * SB + i) * 64 + 16 * c);
        }
      };
      auto scale = [&](int g, int m) __attribute__((always_inline)) {
        const int t = g & 3;
        const float dt = __uint_as_float(d[t][SB * h + (g >> 2)]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][t][r] = fmaf(dt, p[g & 1][m][r], acc[m][t][r]);
        // a use of the sums here: otherwise the compiler sinks the scale FMAs to the end of the
        // unrolled blocks and keeps all their products live
        __asm__ volatile("" : "+v"(acc[m][t]));
      };
      read_block(0);
      u32x4_t wt[2];
      wt[0] = weights_of<XT>(w[0][SB * h]);
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
          for (int k = 0; k < TERMS; ++k) p[g & 1][m] = mfma<XT>(x[i & 1][m][k], wt[g & 1], p[g & 1][m]);
          if (g + 1 < 4 * SB) wt[(g + 1) & 1][m] = weights_part<XT>(w[(g + 1) & 3][SB * h + ((g + 1) >> 2)], m);
          if (g > 0) scale(g - 1, m);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) scale(4 * SB - 1, m);
    }
  }
  // lane (column, c) holds tokens 4c + r of its features
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = (int64_t)rt * kTileRows + 16 * (m0 + m) + 4 * c + r;
      if (row >= a.T) continue;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int f = f0 + 16 * t + col;
        if (f < a.N) put(a, row, f, acc[m][t][r]);
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

bool wide(int64_t T) { return T > 256; }

template <int XT>
hipError_t launch_types(const Q4Args& a, hipStream_t s) {
  if (wide(a.T)) {
    constexpr int TERMS = terms_of<XT>();
    const int col_tiles = (int)((a.N + kWideN - 1) / kWideN);
    for (int64_t t0 = 0; t0 < a.T; t0 += kPassTokens) {
      Q4Args p = a;
      p.T = std::min(a.T - t0, kPassTokens);
      p.x = static_cast<const char*>(a.x) + t0 * a.x_stride * value_size<XT>();
      p.x_scales = a.x_scales ? a.x_scales + t0 * a.x_scales_stride : nullptr;
      p.y = static_cast<char*>(a.y) + t0 * a.y_stride * (a.y_type == MOE_F32 ? 4 : 2);
      const Operand o = Operand::make(a.ws, p.T, a.K, TERMS, kTileRows);
      if (hipError_t e = launch_operand<XT>(p, o, s); e != hipSuccess) return e;
      const int row_tiles = (int)(o.rows / kTileRows);
      const unsigned grid = (unsigned)(((int64_t)row_tiles * col_tiles + 7) / 8 * 8);
      hipError_t e = launch(q4_wide_kernel<XT, TERMS == 1 ? 4 : 1>, dim3(grid), dim3(256), Launch{s}, p, o, row_tiles,
                            col_tiles);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 15) / 16));
  return launch(q4_rows16_kernel<XT, 1>, grid, dim3(64 * kWaves), Launch{s}, a);
}

}  // namespace

int64_t q4_workspace_bytes(int64_t T, int64_t N, int64_t K, int32_t x_type) {
  if (!wide(T)) return 0;
  return Operand::make(nullptr, std::min(T, kPassTokens), K, x_type == MOE_F32 || x_type == MOE_Q8_32 ? 3 : 1, kTileRows).bytes;
}

hipError_t launch_q4_matmul(const Q4Args& a, hipStream_t s) {
  switch (a.x_type) {
    case MOE_F32: return launch_types<MOE_F32>(a, s);
    case MOE_F16: return launch_types<MOE_F16>(a, s);
    case MOE_BF16: return launch_types<MOE_BF16>(a, s);
    default: return launch_types<MOE_Q8_32>(a, s);
  }
}

}  // namespace moe
