// value_dev.h - device helpers of the operators beside the experts
// (internal): runs of 8 values of the supported types to and from fp32.
//
// Rows may start at any multiple of the value size, so the 16-byte accesses
// here go through memcpy: gfx950 runs with unaligned access enabled, and the
// compiler emits one global_load/store_dwordx4 whatever the alignment.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_offload.h"

namespace moe {
namespace value_dev {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <int TYPE>
constexpr int value_size() {
  return TYPE == MOE_F32 ? 4 : TYPE == MOE_Q8_32 ? 1 : 2;
}

__device__ __forceinline__ float half_to_float(uint16_t b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return (float)h;
}
__device__ __forceinline__ uint16_t float_to_half(float v) {
  const _Float16 h = (_Float16)v;
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}
__device__ __forceinline__ uint16_t float_to_bf16(float v) {
  const __bf16 h = (__bf16)v;
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}
__device__ __forceinline__ float bf16_to_float(uint32_t b) { return __uint_as_float(b << 16); }

template <int TYPE>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (TYPE == MOE_F32) {
    return static_cast<const float*>(p)[i];
  } else {
    const uint16_t b = static_cast<const uint16_t*>(p)[i];
    return TYPE == MOE_F16 ? half_to_float(b) : bf16_to_float(b);
  }
}
template <int TYPE>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (TYPE == MOE_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = TYPE == MOE_F16 ? float_to_half(v) : float_to_bf16(v);
}

// the bits of 8 values from value i on (all inside the row)
template <int TYPE>
struct Raw8 {
  u32x4_t a, b;  // b: the second half of fp32 values
};
template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> load8(const void* p, int64_t i) {
  Raw8<TYPE> r;
  const char* q = static_cast<const char*>(p) + i * value_size<TYPE>();
  __builtin_memcpy(&r.a, q, 16);
  if constexpr (TYPE == MOE_F32) __builtin_memcpy(&r.b, q + 16, 16);
  return r;
}
template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw8<TYPE>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == MOE_F32) {
      v[i] = __uint_as_float(r.a[i]);
      v[4 + i] = __uint_as_float(r.b[i]);
    } else if constexpr (TYPE == MOE_F16) {
      v[2 * i] = half_to_float((uint16_t)r.a[i]);
      v[2 * i + 1] = half_to_float((uint16_t)(r.a[i] >> 16));
    } else {
      v[2 * i] = __uint_as_float(r.a[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
    }
  }
}
// PAST: past the caches, for outputs that they cannot hold anyway
template <int TYPE, bool PAST = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  typedef uint32_t loose_t __attribute__((ext_vector_type(4), aligned(2)));
  char* q = static_cast<char*>(p) + i * value_size<TYPE>();
  u32x4_t a, b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (TYPE == MOE_F32) {
      a[j] = __float_as_uint(v[j]);
      b[j] = __float_as_uint(v[4 + j]);
    } else {
      const uint32_t lo = TYPE == MOE_F16 ? float_to_half(v[2 * j]) : float_to_bf16(v[2 * j]);
      const uint32_t hi = TYPE == MOE_F16 ? float_to_half(v[2 * j + 1]) : float_to_bf16(v[2 * j + 1]);
      a[j] = lo | hi << 16;
    }
  }
  if constexpr (PAST) {
    __builtin_nontemporal_store(loose_t(a), reinterpret_cast<loose_t*>(q));
    if constexpr (TYPE == MOE_F32) __builtin_nontemporal_store(loose_t(b), reinterpret_cast<loose_t*>(q + 16));
    return;
  }
  __builtin_memcpy(q, &a, 16);
  if constexpr (TYPE == MOE_F32) __builtin_memcpy(q + 16, &b, 16);
}

// values i .. i + 7 of a row of n; those past it read as 0 and are not stored
template <int TYPE>
__device__ __forceinline__ void load8_tail(const void* p, int64_t i, int64_t n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = i + j < n ? load1<TYPE>(p, i + j) : 0.f;
}
template <int TYPE>
__device__ __forceinline__ void store8_tail(void* p, int64_t i, int64_t n, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) store1<TYPE>(p, i + j, v[j]);
}

}  // namespace value_dev
}  // namespace moe
