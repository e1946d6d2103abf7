// heads_dev.h - device helpers of the norm and rotation of heads and its
// gradient (internal): how a head's values lie over lanes, angles, row sums.
//
// A head of D values is D / 2 slots of two values that turn together; the D - R
// values that do not turn are paired likewise, with angle 0. A lane holds NG groups
// of RUN slots, lanes 0 .. G - 1 of a row group the whole head, so that a pair never
// crosses lanes and the row's sum takes log2 G steps.
//   pairs   slot s: values 2s and 2s + 1
//   halves  slot s < R / 2: values s and s + R / 2; others: the first and the second
//           half of the values from R on
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "route_dev.h"
#include "value_dev.h"

namespace moe {
namespace heads_dev {

using namespace value_dev;

constexpr int kThreads = 256;

// RUN values as loaded
template <int TYPE, int RUN>
struct RawRun {
  uint32_t v[(RUN * value_size<TYPE>() + 3) / 4];
};
template <int TYPE, int RUN>
__device__ __forceinline__ RawRun<TYPE, RUN> load_run(const char* p) {
  RawRun<TYPE, RUN> r;
  if constexpr (RUN * value_size<TYPE>() == 2) {
    uint16_t h;
    __builtin_memcpy(&h, p, 2);
    r.v[0] = h;
  } else {
    __builtin_memcpy(r.v, p, RUN * value_size<TYPE>());
  }
  return r;
}
template <int TYPE, int RUN>
__device__ __forceinline__ float run_value(const RawRun<TYPE, RUN>& r, int i) {
  if constexpr (TYPE == MOE_F32) return __uint_as_float(r.v[i]);
  const uint32_t w = r.v[i >> 1];
  if constexpr (TYPE == MOE_F16) return half_to_float((uint16_t)(i & 1 ? w >> 16 : w));
  return i & 1 ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}
template <int TYPE, int RUN>
__device__ __forceinline__ void store_run(char* p, const float (&v)[RUN]) {
  if constexpr (TYPE == MOE_F32) {
    __builtin_memcpy(p, v, 4 * RUN);
  } else {
    uint16_t h[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) h[i] = TYPE == MOE_F16 ? float_to_half(v[i]) : float_to_bf16(v[i]);
    __builtin_memcpy(p, h, 2 * RUN);
  }
}

// where a group of slots lies in its head
struct Place {
  int a, b;  // first values of its two runs
  bool in;   // whether the head has it
};
template <int RUN, bool PAIRS>
__device__ __forceinline__ Place place_of(int group, int D, int R) {
  const int s = RUN * group;
  Place p;
  p.in = 2 * s < D;
  if (PAIRS)
    p.a = 2 * s, p.b = p.a + RUN;
  else if (2 * s < R)
    p.a = s, p.b = s + R / 2;
  else
    p.a = R / 2 + s, p.b = p.a + (D - R) / 2;
  if (!p.in) p.a = p.b = 0;
  return p;
}
// slot j of a group from its two runs, and back
template <bool PAIRS, int RUN>
__device__ __forceinline__ void to_slots(const float (&x)[2][RUN], float (&a)[RUN], float (&b)[RUN]) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    a[j] = PAIRS ? x[2 * j / RUN][2 * j % RUN] : x[0][j];
    b[j] = PAIRS ? x[(2 * j + 1) / RUN][(2 * j + 1) % RUN] : x[1][j];
  }
}
template <bool PAIRS, int RUN>
__device__ __forceinline__ void from_slots(const float (&a)[RUN], const float (&b)[RUN], float (&x)[2][RUN]) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    x[PAIRS ? 2 * j / RUN : 0][PAIRS ? 2 * j % RUN : j] = a[j];
    x[PAIRS ? (2 * j + 1) / RUN : 1][PAIRS ? (2 * j + 1) % RUN : j] = b[j];
  }
}
template <int TYPE, bool PAIRS, int RUN>
__device__ __forceinline__ void unpack_slots(const RawRun<TYPE, RUN> (&r)[2], float (&a)[RUN], float (&b)[RUN]) {
  float x[2][RUN];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < RUN; ++j) x[i][j] = run_value<TYPE, RUN>(r[i], j);
  to_slots<PAIRS, RUN>(x, a, b);
}
template <int TYPE, bool PAIRS, int RUN>
__device__ __forceinline__ void store_slots_as(char* row, const Place& p, const float (&a)[RUN], const float (&b)[RUN]) {
  float x[2][RUN];
  from_slots<PAIRS, RUN>(a, b, x);
  store_run<TYPE, RUN>(row + value_size<TYPE>() * p.a, x[0]);
  store_run<TYPE, RUN>(row + value_size<TYPE>() * p.b, x[1]);
}
template <bool PAIRS, int RUN>
__device__ __forceinline__ void store_slots(int type, char* row, const Place& p, const float (&a)[RUN], const float (&b)[RUN]) {
  if (type == MOE_F32)
    store_slots_as<MOE_F32, PAIRS, RUN>(row, p, a, b);
  else if (type == MOE_F16)
    store_slots_as<MOE_F16, PAIRS, RUN>(row, p, a, b);
  else
    store_slots_as<MOE_BF16, PAIRS, RUN>(row, p, a, b);
}

// sum over the G lanes of a row (a power of two), in every one of them; selects, not branches, within 16 lanes
__device__ __forceinline__ float lanes_sum(float v, int G) {
  using namespace route_dev;
  float w = v + __uint_as_float(dpp32<kDppQuadXor1>(__float_as_uint(v)));
  v = G > 1 ? w : v;
  w = v + __uint_as_float(dpp32<kDppQuadXor2>(__float_as_uint(v)));
  v = G > 2 ? w : v;
  w = v + __uint_as_float(dpp32<kDppRowHalfMirror>(__float_as_uint(v)));
  v = G > 4 ? w : v;
  w = v + __uint_as_float(dpp32<kDppRowMirror>(__float_as_uint(v)));
  v = G > 8 ? w : v;
  if (G > 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = G > 32 ? __uint_as_float(t[0]) + __uint_as_float(t[1]) : v;
  }
  return v;
}

// n / d for n < 2^20 and d's magic = ceil(2^31 / d) where n * d < 2^31
__device__ __forceinline__ int quotient(int n, uint32_t magic) { return (int)(((uint64_t)(uint32_t)n * magic) >> 31); }

// cos and sin of position * inv_freq, each within 1.4 * 2^-24 and the angle's own error, 2^-51 of it. The angle is
// formed in turns and reduced to an eighth of a turn either side of a quarter's multiple, both in 64 bits; the rest, below
// 0.8, is rounded once, and there the Taylor series of both are exact to 2^-28 with the terms taken. fp32 would lose the angle of
// far positions (2^18 * 1.0: off by 2^-6), and tables would have to be read for every token.
__device__ __forceinline__ float2 turn_of(int position, float inv_freq) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  double t = (double)position * ((double)inv_freq * kTurn);
  t -= rint(t);
  const double quarter = rint(4.0 * t);  // -2 .. 2
  const float x = (float)(6.28318530717958647693 * fma(-0.25, quarter, t)), y = x * x;
  float s = fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(y, s, 1.0f / 120.0f);
  s = fmaf(y, s, -1.0f / 6.0f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = fmaf(y, c, -1.0f / 720.0f);
  c = fmaf(y, c, 1.0f / 24.0f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.0f);
  const int q = (int)quarter;
  float2 r = q & 1 ? make_float2(-s, c) : make_float2(c, s);
  if (q & 2) r = make_float2(-r.x, -r.y);
  return r;
}

// The slots (a, b) turned by their (cos, sin), by minus the angle with BACK. Without a sine (position 0, or a slot that
// does not turn) neither value sees the other, so that it is not spoilt by a neighbour that is not finite.
template <bool BACK, int RUN>
__device__ __forceinline__ void turn(float (&a)[RUN], float (&b)[RUN], const float2 (&cs)[RUN]) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    const bool turns = cs[j].y != 0.f;
    const float pa = turns ? (BACK ? b[j] : -b[j]) * cs[j].y : 0.f, pb = turns ? (BACK ? -a[j] : a[j]) * cs[j].y : 0.f;
    a[j] = fmaf(a[j], cs[j].x, pa), b[j] = fmaf(b[j], cs[j].x, pb);
  }
}

// the angles of a group of slots, in the widest reads that its place allows
template <int RUN>
__device__ __forceinline__ void load_turns(const float2* p, float2 (&cs)[RUN]) {
  if constexpr (RUN % 2 == 0) {
#pragma unroll
    for (int j = 0; j < RUN; j += 2) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + j);  // whole groups: 16-byte aligned
      cs[j] = make_float2(v[0], v[1]), cs[j + 1] = make_float2(v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < RUN; ++j) cs[j] = p[j];
  }
}

// The (cos, sin) of tokens t0 .. t0 + n - 1, every slot, once per work-group and not per head: [token][D / 2]
__device__ __forceinline__ void fill_turns(const HeadsArgs& a, int64_t t0, int n, float2* s_turn) {
  const int S = a.D / 2;
  for (int e = threadIdx.x; e < n * S; e += kThreads) {
    const int t = quotient(e, a.slot_magic), s = e - t * S;
    float2 r = make_float2(1.0f, 0.0f);
    if (2 * s < a.R) {
      const int axis = a.axis ? a.axis[s] : 0;
      if (axis < a.axes) r = turn_of(a.pos[axis * a.pos_stride + t0 + t], a.inv_freq[s]);
    }
    s_turn[e] = r;
  }
}

// 1 / sqrt(mean + eps) of a row whose squares sum to ss, D values, to the last bit of the device's reciprocal
// root. Squares leave fp32's range long before the values do, as in the norm of whole rows: such a row is
// summed a second time, scaled by a power of two. scaled(k) multiplies the row's values by k
// and returns the same sum of them times k; afterwards the values are those of the row times `left`,
// and the result belongs to them. Every lane of the wave comes here.
struct Inverse {
  float r, left;
};
template <typename F>
__device__ __forceinline__ Inverse inverse_rms(float ss, float inv_D, float D, float eps, F scaled) {
  // a square rounded below fp32's normal range is off by at most 2^-150: beside a mean of 2^-100, or an
  // eps of it, that is nothing
  const float least = eps < 0x1p-100f ? 0x1p-100f * D : 0.f;
  Inverse i{__builtin_amdgcn_rsqf(fmaf(ss, inv_D, eps)), 1.0f};
  const bool fine = ss >= least && ss < __builtin_inff();
  if (__builtin_expect(__any(!fine), 0)) {
    // 2^-80 as 2^-40 now and 2^-40 in the result (2^100 as 2^34 and 2^66), so that neither leaves the normal
    // range before the normed value does
    const bool large = !(ss < __builtin_inff());
    const float k = fine ? 1.0f : large ? 0x1p-40f : 0x1p34f, rest = fine ? 1.0f : large ? 0x1p-40f : 0x1p66f;
    const float s2 = scaled(k, rest);
    i.left = k;
    // eps times (k rest)^2 in this order: the square alone may leave the range
    i.r = __builtin_amdgcn_rsqf(fmaf(s2, inv_D, eps * k * rest * k * rest)) * rest;
  }
  return i;
}

}  // namespace heads_dev
}  // namespace moe
