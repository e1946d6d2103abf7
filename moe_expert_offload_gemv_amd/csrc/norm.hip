// norm.hip - residual add and RMS norm (moe_add_rmsnorm): the step between
// the residual stream and the layer's products.
//
//   s = x + residual, residual_out = s, v = s * weight / sqrt(mean(s^2) + eps)
//   out = v, or 8-bit codes with an fp32 scale per 32 values
//
// Bound by traffic: every value is read and written once. A row of up to
// 16384 values stays in the registers of one work-group between the sum of
// squares and the scaling (8 values per thread and chunk, one or two chunks: a
// work-group as small as holds the row, so that several rows' loads are in flight
// in a CU while one waits for its sum); longer rows are read twice. The sum of squares,
// the mean and the scaling are fp32; the norm uses the sum before its rounding to the
// residual's type. Squares leave fp32's range long before the values do: a row whose sum
// of squares is not finite, or whose mean is too small to have kept them all, is summed again
// scaled by a power of two.
//
// Measured (kernel alone): 12287 x 4096, fp32 x, bf16 residual and out, 504 MB, 89-91 us =
// 5.6 TB/s, above a streaming read (5.35) and a copy (4.95); 4096 x 2048 bf16 to codes, 60 MB,
// 12.5-13.1 us = 4.7 TB/s; one row of 2048 values 2.4-2.9 us, a launch and two trips to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"
#include "route_dev.h"
#include "value_dev.h"

namespace moe {
namespace {

using namespace value_dev;

constexpr int kNoResidual = -1;
// a group of codes whose largest magnitude is below 2^-100 is stored as
// zeros: 127 / a stays finite above it
constexpr uint32_t kMinGroupMax = (127u - 100u) << 23;
constexpr uint32_t kInfBits = 0x7F800000u;
// A square rounded below fp32's normal range is off by at most 2^-150: beside a mean
// of this size, or an eps of it, that is nothing
constexpr float kSmallMean = 0x1p-100f;

// s = x + residual of values i .. i + 7
template <int XT, int RT>
__device__ __forceinline__ void sum8(const void* x, const void* res, int64_t i, int64_t H, float (&s)[8]) {
  if (i + 8 <= H) {
    const Raw8<XT> xr = load8<XT>(x, i);
    if constexpr (RT != kNoResidual) {
      const Raw8<RT> rr = load8<RT>(res, i);
      float r[8];
      unpack8<RT>(rr, r);
      unpack8<XT>(xr, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += r[j];
    } else {
      unpack8<XT>(xr, s);
    }
  } else {
    load8_tail<XT>(x, i, H, s);
    if constexpr (RT != kNoResidual) {
      float r[8];
      load8_tail<RT>(res, i, H, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += r[j];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void put8(void* p, int64_t i, int64_t H, const float (&v)[8]) {
  if (i + 8 <= H)
    store8<TYPE>(p, i, v);
  else
    store8_tail<TYPE>(p, i, H, v);
}

// 8 codes of a group of 32 (four neighbouring threads, all of them or none
// inside the row); the group's first thread stores its scale
__device__ __forceinline__ void put_codes8(int8_t* out, float* scales, int64_t i, const float (&v)[8]) {
  uint32_t a = 0;
  // |v| as bits: ordered like the values, with inf and then NaN above them
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  a = max(a, route_dev::dpp32<route_dev::kDppQuadXor1>(a));
  a = max(a, route_dev::dpp32<route_dev::kDppQuadXor2>(a));
  const bool finite = a < kInfBits, none = a < kMinGroupMax;
  const float top = __uint_as_float(a);
  const float inv = finite && !none ? 127.0f / top : 0.f;
  const float scale = !finite ? __uint_as_float(0x7FC00000u) : none ? 0.f : top / 127.0f;
  uint32_t w[2] = {0, 0};
  if (finite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= ((uint32_t)(int)rintf(v[j] * inv) & 0xFFu) << (8 * (j & 3));
  }
  __builtin_memcpy(out + i, w, 8);
  if ((i & 31) == 0) scales[i >> 5] = scale;
}

// v = s * half * r * weight; half is 1 but for rows summed again
__device__ __forceinline__ void put_out8(const NormArgs& a, int64_t row, int64_t i, const float (&s)[8], float r,
                                         float half) {
  float v[8], w[8];
  if (a.weight) {
    if (i + 8 <= a.H)
      unpack8<MOE_F32>(load8<MOE_F32>(a.weight, i), w);
    else
      load8_tail<MOE_F32>(a.weight, i, a.H, w);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = a.weight ? s[j] * half * r * w[j] : s[j] * half * r;
  char* out = static_cast<char*>(a.out);
  if (a.out_type == MOE_F32)
    put8<MOE_F32>(out + 4 * row * a.out_stride, i, a.H, v);
  else if (a.out_type == MOE_F16)
    put8<MOE_F16>(out + 2 * row * a.out_stride, i, a.H, v);
  else if (a.out_type == MOE_BF16)
    put8<MOE_BF16>(out + 2 * row * a.out_stride, i, a.H, v);
  else
    put_codes8(reinterpret_cast<int8_t*>(out) + row * a.out_stride, a.scales + row * a.scales_stride, i, v);
}

// One work-group per row, rows in turn. NV > 0: the row's sums stay in NV
// chunks of 8 registers per thread; NV = 0: any length, read twice (the sums
// are formed again, so the residual may be updated in place).
template <int XT, int RT, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int W = THREADS / 64;
  __shared__ float s_sum[2][W], s_again[W];
  const float least = a.eps < kSmallMean ? kSmallMean * (float)a.H : 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    // Offsets within the row are formed anew for each: kept from row to row they would take more
    // than 64 registers with the values, and a CU then holds one work-group of 16 waves, not two
    // (4096 x 8192 bf16: 64 us, so 59.5; without residual, fp32 to bf16, 51 and 42).
    uint32_t tid = threadIdx.x;
    __asm__ volatile("" : "+v"(tid));
    const char* x = static_cast<const char*>(a.x) + row * a.x_stride * value_size<XT>();
    const char* res = nullptr;
    char* res_out = nullptr;
    if constexpr (RT != kNoResidual) {
      res = static_cast<const char*>(a.res) + row * a.res_stride * value_size<RT>();
      res_out = static_cast<char*>(a.res_out) + row * a.res_out_stride * value_size<RT>();
    }
    float s[NV > 0 ? NV : 1][8];
    float ss = 0.f;
    if constexpr (NV > 0) {
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int64_t i = 8 * ((int64_t)c * THREADS + tid);
        if (i < a.H) {
          sum8<XT, RT>(x, res, i, a.H, s[c]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) s[c][j] = 0.f;
        }
      }
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(s[c][j], s[c][j], ss);
    } else {
      for (int64_t i = 8 * (int64_t)tid; i < a.H; i += 8 * THREADS) {
        sum8<XT, RT>(x, res, i, a.H, s[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(s[0][j], s[0][j], ss);
      }
    }
    ss = route_dev::wave_sum(ss);
    if constexpr (W > 1) {
      // two sets in turn: a wave may reach the next row before the others have read this one's
      if ((threadIdx.x & 63) == 0) s_sum[turn][threadIdx.x >> 6] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) ss += s_sum[turn][w];
    }
    float r = 1.0f / sqrtf(ss / (float)a.H + a.eps), half = 1.0f;
    // the same for every thread of the work-group
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(!(ss >= least && ss < __builtin_inff())), 0)) {
      // 2^-80: values of any size and number stay below 2^120, a mean of 2^104, the least that
      // overflows, above 2^-56; 2^100: a mean below 2^-100 becomes 2^100 at most, the smallest square 2^-98
      const bool large = !(ss < __builtin_inff());
      const float k = large ? 0x1p-80f : 0x1p100f;
      float again = 0.f;
      auto add = [&](float v) __attribute__((always_inline)) { v *= k, again = fmaf(v, v, again); };
      if constexpr (NV > 0) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) add(s[c][j]);
      } else {
        for (int64_t i = 8 * (int64_t)tid; i < a.H; i += 8 * THREADS) {
          sum8<XT, RT>(x, res, i, a.H, s[0]);
#pragma unroll
          for (int j = 0; j < 8; ++j) add(s[0][j]);
        }
      }
      again = route_dev::wave_sum(again);
      if constexpr (W > 1) {
        const int lane = threadIdx.x & 63;
        if (lane == 0) s_again[threadIdx.x >> 6] = again;
        __syncthreads();  // written again past the next row's barrier at the earliest
        again = route_dev::wave_sum(lane < W ? s_again[lane & (W - 1)] : 0.f);
      }
      // 1 / sqrt(mean + eps) = k / sqrt(again / hidden + eps k^2), k as two factors so that neither
      // r (the root is 2^-61 at the least) nor s * half leaves the normal range before v does
      r = 1.0f / sqrtf(again / (float)a.H + a.eps * k * k) * (large ? 0x1p-40f : 0x1p66f);
      half = large ? 0x1p-40f : 0x1p34f;
    }
    if constexpr (NV > 0) {
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int64_t i = 8 * ((int64_t)c * THREADS + tid);
        if (i < a.H) {
          if constexpr (RT != kNoResidual) put8<RT>(res_out, i, a.H, s[c]);
          put_out8(a, row, i, s[c], r, half);
        }
      }
    } else {
      for (int64_t i = 8 * (int64_t)tid; i < a.H; i += 8 * THREADS) {
        sum8<XT, RT>(x, res, i, a.H, s[0]);
        if constexpr (RT != kNoResidual) put8<RT>(res_out, i, a.H, s[0]);
        put_out8(a, row, i, s[0], r, half);
      }
    }
  }
}

template <int XT, int RT>
hipError_t launch_types(const NormArgs& a, hipStream_t s) {
  // rows beyond the grid are taken in turn by the same work-groups
  const dim3 grid((unsigned)std::min<int64_t>(a.T, 1 << 16));
  const Launch l{s};
  if (a.H <= 512) return launch(add_rmsnorm_kernel<XT, RT, 64, 1>, grid, dim3(64), l, a);
  if (a.H <= 2048) return launch(add_rmsnorm_kernel<XT, RT, 256, 1>, grid, dim3(256), l, a);
  if (a.H <= 4096) return launch(add_rmsnorm_kernel<XT, RT, 256, 2>, grid, dim3(256), l, a);
  if (a.H <= 16384) return launch(add_rmsnorm_kernel<XT, RT, 1024, 2>, grid, dim3(1024), l, a);
  return launch(add_rmsnorm_kernel<XT, RT, 1024, 0>, grid, dim3(1024), l, a);
}

template <int XT>
hipError_t launch_res(const NormArgs& a, hipStream_t s) {
  if (!a.res) return launch_types<XT, kNoResidual>(a, s);
  if (a.res_type == MOE_F32) return launch_types<XT, MOE_F32>(a, s);
  if (a.res_type == MOE_F16) return launch_types<XT, MOE_F16>(a, s);
  return launch_types<XT, MOE_BF16>(a, s);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.x_type == MOE_F32) return launch_res<MOE_F32>(a, s);
  if (a.x_type == MOE_F16) return launch_res<MOE_F16>(a, s);
  return launch_res<MOE_BF16>(a, s);
}

}  // namespace moe
