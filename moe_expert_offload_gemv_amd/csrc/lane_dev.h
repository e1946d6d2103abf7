// lane_dev.h - device helpers of the 4-bit matrix-core kernels (internal):
// weights and scales moved between the lanes of a wave, and a fused bit operation.
//
// A wave is seen as four lane groups of 16 columns, as the 16 x 16 x 32 products
// take their operands.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace lane_dev {

// (x & m) | c in one v_bitop3 (truth table of S0 & S1 | S2)
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(x, m, c, 0xEA);
}

// (lane group g, dword d) -> (lane group d, dword g) within each 16-lane
// column: afterwards dword i of lane group c is the old dword c of group i.
// V: four 32-bit members x, y, z, w
template <typename V>
__device__ __forceinline__ void transpose4(V& v) {
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v.x = c[0], v.y = c[1], v.z = d[0], v.w = d[1];
}

// Each lane group's value of x in every lane of its 16-lane column: out[g]
// holds group g's. Two swap rounds: [x0 x1 x2 x3] -> [x0 x1 x0 x1] and
// [x2 x3 x2 x3] -> [x0 x0 x0 x0], [x1 ...], [x2 ...], [x3 ...].
__device__ __forceinline__ void broadcast4(uint32_t x, uint32_t (&out)[4]) {
  const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  out[0] = lo[0], out[1] = lo[1], out[2] = hi[0], out[3] = hi[1];
}

}  // namespace lane_dev
}  // namespace moe
