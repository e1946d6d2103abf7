// balance.hip - the router's load over a batch of tokens, its balance and z
// losses and their gradient (moe_router_balance, moe_router_balance_grad).
//
//   balance_rows_kernel    logits once: softmax, lse and the top-k set of every
//                          token; per work-group sums of p and counts per expert
//   balance_finish_kernel  the work-groups' sums, counts, loads and losses
//   balance_grad_kernel    logits once more: dlogits
//
// A token's row is shared by G lanes (16, or a wave: lanes_of), so
// its maximum, sums and top-k are a few DPP steps, and a wave works on 64 / G
// rows at once. A lane holds NE logits of its row, always of the same experts:
// the sums over tokens stay in its registers (p and count per expert) until
// the work-group has seen its last row. All sums run in a fixed order.
//
// Only the k-th largest logit is needed, not the order of the picks: an
// expert counts if its logit is larger, or equal and one of the lowest ids
// that fill the set.
//
// Measured (kernels alone): 32768 x 512 fp32, 8 picks: rows 23-26 us for 67 MB (bound by
// instructions, 1150 for four rows of a wave: 16 us of them, two waves a SIMD), finishing 5.5, gradient 27.5 for
// 134 MB = 4.9 TB/s, the rate of a copy. 12288 x 256 bf16: 10.7 (3 of them instructions: 768 units of
// 16 rows leave half of the 512 work-groups idle in their second round), 5 and 7.5 us; 999 x 60
// fp16: 3.9, 5 and 3.2 us, each a launch and a few dependent trips to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"
#include "route_dev.h"
#include "value_dev.h"

namespace moe {
namespace {

using namespace value_dev;

constexpr int kBalanceBlocks = 512;  // work-groups that sum rows, two per CU
constexpr int kFinishExperts = 32;   // experts per finishing work-group
constexpr int kWaveRows = 2048;      // rows up to which each has a wave
constexpr int kMaxExperts = 4096;
constexpr float kMinusInf = -__builtin_inff();

// workspace: ticket, per work-group tokens and z sums, the finishing
// work-groups' loss terms, then the sums of p and counts [blocks][E]
constexpr int64_t kOffTokens = 256;
constexpr int64_t kOffZ = kOffTokens + 4 * kBalanceBlocks;
constexpr int64_t kOffTerms = kOffZ + 4 * kBalanceBlocks;
constexpr int64_t kOffSums = kOffTerms + 4 * (kMaxExperts / kFinishExperts);

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 64) return route_dev::wave_max_u32(v);
  v = max(v, route_dev::dpp32<route_dev::kDppQuadXor1>(v));
  v = max(v, route_dev::dpp32<route_dev::kDppQuadXor2>(v));
  v = max(v, route_dev::dpp32<route_dev::kDppRowHalfMirror>(v));
  return max(v, route_dev::dpp32<route_dev::kDppRowMirror>(v));
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(route_dev::dpp32<CTRL>(__float_as_uint(v)));
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G == 64) return route_dev::wave_sum(v);
  v = dpp_add<route_dev::kDppQuadXor1>(v);
  v = dpp_add<route_dev::kDppQuadXor2>(v);
  v = dpp_add<route_dev::kDppRowHalfMirror>(v);
  return dpp_add<route_dev::kDppRowMirror>(v);
}
template <int G>
__device__ __forceinline__ int group_sum_int(int v) {
  v += (int)route_dev::dpp32<route_dev::kDppQuadXor1>((uint32_t)v);
  v += (int)route_dev::dpp32<route_dev::kDppQuadXor2>((uint32_t)v);
  v += (int)route_dev::dpp32<route_dev::kDppRowHalfMirror>((uint32_t)v);
  v += (int)route_dev::dpp32<route_dev::kDppRowMirror>((uint32_t)v);
  if constexpr (G == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}
// sum over the rows' lanes that hold the same experts
template <int G, typename V>
__device__ __forceinline__ V sum_rows(V v) {
  if constexpr (G == 16) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// The same for 4 values at once, each lane row left with one of them: row g
// with the sum of v[g] (v_permlane32_swap exchanges the upper half of the first
// operand with the lower half of the second, v_permlane16_swap the odd rows of
// the first with the even rows of the second).
template <typename V>
__device__ __forceinline__ V sum_rows4(const V* v) {
  V h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v[i]),
                                                    __builtin_bit_cast(uint32_t, v[i + 2]), false, false);
    h[i] = __builtin_bit_cast(V, (uint32_t)s[0]) + __builtin_bit_cast(V, (uint32_t)s[1]);
  }
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, h[0]),
                                                  __builtin_bit_cast(uint32_t, h[1]), false, false);
  return __builtin_bit_cast(V, (uint32_t)s[0]) + __builtin_bit_cast(V, (uint32_t)s[1]);
}

// largest of a row's logits, NaNs passed over (-inf if there is none)
template <int G, int NE>
__device__ __forceinline__ float row_max(const float (&z)[NE]) {
  float mx = kMinusInf;
#pragma unroll
  for (int j = 0; j < NE; ++j) mx = fmaxf(mx, z[j]);
  return route_dev::order_logit(group_max<G>(route_dev::order_bits(mx)));
}

// expert of a lane's j-th logit: runs of 4 experts per lane
template <int G>
__device__ __forceinline__ int expert_of(int j, int gl) {
  return (j >> 2) * 4 * G + gl * 4 + (j & 3);
}

// The 4 values of a lane's run are read as one word whatever E is, without a
// branch that would hold up the loads behind it: a run that passes the last
// expert begins at E - 4 instead, and its first `skip` values, which are another
// run's (or before expert 0, for E < 4), are left out.
struct Run {
  int at, skip;
  __device__ __forceinline__ bool has(int i) const { return i >= skip; }
};
template <int G>
__device__ __forceinline__ Run run_of(int j, int gl, int E) {
  const int i = expert_of<G>(j & ~3, gl), at = min(i, E - 4);
  return {at, i - at};
}
// the shares of MOE_BALANCE_SHAPE are filled by more than half, all but the
// smallest: these of a lane's values are experts without a look
template <int G, int NE>
constexpr bool surely(int j) {
  return NE > 4 && j < NE / 2;
}
template <int TYPE>
struct Raw4 {
  uint32_t w[TYPE == MOE_F32 ? 4 : 2];
};
template <int TYPE, int NE>
__device__ __forceinline__ Raw4<TYPE> load_run(const char* p, Run r, int E) {
  Raw4<TYPE> v;
  if (NE == 4 && E < 4) {
#pragma unroll
    for (uint32_t& w : v.w) w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = max(r.at + i, 0);
      if constexpr (TYPE == MOE_F32)
        v.w[i] = reinterpret_cast<const uint32_t*>(p)[e];
      else
        v.w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (i & 1));
    }
    return v;
  }
  __builtin_memcpy(v.w, p + (int64_t)r.at * value_size<TYPE>(), sizeof v.w);
  return v;
}
template <int TYPE>
__device__ __forceinline__ void unpack4(const Raw4<TYPE>& r, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (TYPE == MOE_F32)
      v[j] = __uint_as_float(r.w[j]);
    else if constexpr (TYPE == MOE_F16)
      v[j] = half_to_float((uint16_t)(r.w[j >> 1] >> (16 * (j & 1))));
    else
      v[j] = bf16_to_float((r.w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
  }
}
template <int TYPE>
__device__ __forceinline__ void store_run(char* p, Run r, const float* v) {
  if (r.skip == 0) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == MOE_F32)
        w[j] = __float_as_uint(v[j]);
      else if (j < 2)
        w[j] = TYPE == MOE_F16 ? (float_to_half(v[2 * j]) | (uint32_t)float_to_half(v[2 * j + 1]) << 16)
                               : (float_to_bf16(v[2 * j]) | (uint32_t)float_to_bf16(v[2 * j + 1]) << 16);
    }
    __builtin_memcpy(p + (int64_t)r.at * value_size<TYPE>(), w, 4 * value_size<TYPE>());
  } else {
#pragma unroll
    for (int j = 1; j < 4; ++j)
      if (r.has(j)) store1<TYPE>(p, r.at + j, v[j]);
  }
}
// d added to what the run holds, or in its place
template <int TYPE, int NE>
__device__ __forceinline__ void put_run(char* p, Run r, int E, bool accumulate, float* d) {
  if (accumulate) {
    float old[4];
    unpack4<TYPE>(load_run<TYPE, NE>(p, r, E), old);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += old[i];
  }
  store_run<TYPE>(p, r, d);
}

// the 8 largest order bits of the row that are not above `below`, each lane's
// eight at a time, then the lanes' lists (sorting networks of route_dev.h)
template <int G, int NE, bool ALL>
__device__ __forceinline__ void top8(const uint32_t (&b)[NE], uint32_t below, uint32_t (&t)[8]) {
  auto at = [&](int j) { return ALL || b[j] <= below ? b[j] : 0u; };
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = j < NE ? at(j < NE ? j : 0) : 0u;
  route_dev::sort8_desc(t);
#pragma unroll
  for (int o = 8; o < NE; o += 8) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = at(o + j);
    route_dev::sort8_desc(u);
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = max(t[j], u[7 - j]);
    route_dev::clean8_desc(t);
  }
  route_dev::merge8_dpp<route_dev::kDppQuadXor1>(t);
  route_dev::merge8_dpp<route_dev::kDppQuadXor2>(t);
  route_dev::merge8_dpp<route_dev::kDppRowHalfMirror>(t);
  route_dev::merge8_dpp<route_dev::kDppRowMirror>(t);
  if constexpr (G == 64) {
    route_dev::merge8_swap<16>(t);
    route_dev::merge8_swap<32>(t);
  }
}
// t[i] of a descending list, as the least of the first: chosen by index, the list
// would be moved to LDS
__device__ __forceinline__ uint32_t pick(const uint32_t (&t)[8], int i) {
  uint32_t m = t[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) m = min(m, j <= i ? t[j] : ~0u);
  return m;
}
// The k-th largest of the row's order bits, and how many are larger. k <= 8: one
// pass of top8. k > 8: passes of 8 below what the passes before have passed over,
// equal logits together, until the k-th is among them (1967 x 305, 10 picks: 22 us for forward
// and gradient, 29 with the bits found one by one; 12288 x 128, 16 picks: 17 and 21.5).
template <int G, int NE, bool TOP8>
__device__ __forceinline__ uint32_t kth_bits(const uint32_t (&b)[NE], int k, int& above) {
  uint32_t t[8], m;
  above = 0;
  if constexpr (TOP8) {
    top8<G, NE, true>(b, 0, t);
    m = pick(t, k - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) above += t[i] > m ? 1 : 0;
    return m;
  } else {
    // a row keeps its place while others of the wave go on; at most ceil(k / 8)
    // passes, for each but the last leaves 8 logits or more behind
    uint32_t below = ~0u;
    int left = k;  // > 0: the k-th is the left-th of those not above `below`
    m = 0;
    do {
      top8<G, NE, false>(b, below, t);
      const uint32_t v = pick(t, min(left, 8) - 1);
      int n = 0;  // of those not above `below`: equal to v or larger
#pragma unroll
      for (int j = 0; j < NE; ++j) n += b[j] >= v && b[j] <= below ? 1 : 0;
      n = group_sum_int<G>(n);
      m = left > 0 ? v : m;
      left -= left > 0 ? n : 0;
      below = v - 1;  // v > 0: fewer than k logits are above it
    } while (__ballot(left > 0));
    int n = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) n += b[j] > m ? 1 : 0;
    above = group_sum_int<G>(n);
    return m;
  }
}

// Two waves a SIMD hide each other's latencies (one: 30 us for 32768 x 512 fp32);
// 64 experts a lane do not fit in that many registers.
template <int ZT, int G, int NE, bool TOP8>
__global__ __launch_bounds__(256, NE <= 32 ? 2 : 1) void balance_rows_kernel(BalanceArgs a) {
  __shared__ float s_p[NE * G];
  __shared__ int s_c[NE * G];
  __shared__ float s_z[4];
  __shared__ int s_n[4];
  constexpr int R = 64 / G;  // rows of a wave at a time
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gl = lane & (G - 1), g = lane / G;
  const int E = a.E, k = a.k;
  float p[NE];
  int c[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) p[j] = 0.f, c[j] = 0;
  float z2 = 0.f;
  int n = 0;
  // a row's logits are on their way while the row before is worked on; for a
  // token left out (or past the last) row 0 is read and counts as -inf
  const int64_t stride = (int64_t)gridDim.x * 4 * R;
  Raw4<ZT> raw[NE / 4];
  bool in;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    in = row < a.T && (!a.valid || a.valid[row]);
    const char* zr = static_cast<const char*>(a.logits) + (in ? row : 0) * a.z_stride * value_size<ZT>();
#pragma unroll
    for (int j = 0; j < NE; j += 4) raw[j / 4] = load_run<ZT, NE>(zr, run_of<G>(j, gl, E), E);
  };
  int64_t row0 = ((int64_t)blockIdx.x * 4 + wave) * R;
  if (row0 < a.T) fetch(row0 + g);  // without tokens there is no row 0 either
  for (; row0 < a.T; row0 += stride) {
    const int64_t row = row0 + g;
    float e[NE];
    uint32_t b[NE];
#pragma unroll
    for (int j = 0; j < NE; j += 4) unpack4<ZT>(raw[j / 4], e + j);
    const bool used = in;
    fetch(row + stride);
    if (__ballot(!used)) {
#pragma unroll
      for (int j = 0; j < NE; ++j) e[j] = used ? e[j] : kMinusInf;
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const bool yes = surely<G, NE>(j) || run_of<G>(j, gl, E).has(j & 3);
      e[j] = yes ? e[j] : kMinusInf;
      b[j] = yes ? route_dev::order_bits(e[j]) : 0u;
    }
    const float mx = row_max<G, NE>(e);
    const float base = mx == kMinusInf ? 0.f : mx;  // a row of -inf alone: every exp is 0
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      e[j] = __expf(e[j] - base);
      sum += e[j];
    }
    sum = group_sum<G>(sum);
    const float lse = base + logf(sum);  // -inf for a row of -inf
    const bool counted = used && lse != kMinusInf;
    if (gl == 0 && row < a.T) a.lse[row] = used ? lse : kMinusInf;
    const float inv = counted ? 1.0f / sum : 0.f;
    z2 = counted ? fmaf(lse, lse, z2) : z2;
    n += counted ? 1 : 0;
    if (ZT == MOE_F32 && __ballot(lse != lse)) {
      // the NaN whose bits are all ones (no 16-bit one has them in fp32) has the order bits of no
      // expert: one more makes it the lowest of the row's logits instead
      int gt = gl;
      asm volatile("" : "+v"(gt));  // as below
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (run_of<G>(j, gt, E).has(j & 3)) b[j] = max(b[j], 1u);
    }
    int above;
    const uint32_t m = kth_bits<G, NE, TOP8>(b, k, above);
    // in the set: bits above floor, all ones for a row that does not count
    const uint32_t floor = counted ? m - 1 : ~0u;
    int chosen = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      p[j] = fmaf(e[j], inv, p[j]);
      chosen += b[j] > floor ? 1 : 0;
    }
    if (__ballot(group_sum_int<G>(chosen) > k) == 0) {
#pragma unroll
      for (int j = 0; j < NE; ++j) c[j] += b[j] > floor ? 1 : 0;
    } else {
      // more equal logits than places: the lowest ids of them, one by one
      int left = k - above, last = -1;
      // its compares stay in here: kept from row to row they would take all scalar registers
      int gt = gl;
      asm volatile("" : "+v"(gt));
      while (__ballot(left > 0)) {
        int id = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
          const int ex = run_of<G>(j, gt, E).at + (j & 3);
          if (b[j] == m && ex > last) id = min(id, ex);
        }
        id = 0x7FFFFFFF - (int)group_max<G>((uint32_t)(0x7FFFFFFF - id));
        if (left > 0) last = id;
        --left;
      }
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const bool yes = b[j] > m || (b[j] == m && run_of<G>(j, gt, E).at + (j & 3) <= last);
        c[j] += counted && yes ? 1 : 0;
      }
    }
  }
  // the wave's rows, then the waves in turn
  z2 = sum_rows<G>(z2);
  n = sum_rows<G>(n);
  if (lane == 0) s_z[wave] = z2, s_n[wave] = n;
  if constexpr (G == 16) {
#pragma unroll
    for (int j = 0; j < NE; j += 4) p[j / 4] = sum_rows4(p + j), c[j / 4] = sum_rows4(c + j);
  }
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int j = 0; j < (G == 16 ? NE / 4 : NE); ++j) {
        const Run r = run_of<G>(G == 16 ? 4 * j : j, gl, E);
        const int i = G == 16 ? g : j & 3, ex = r.at + i;
        if (!r.has(i)) continue;
        s_p[ex] = w ? s_p[ex] + p[j] : p[j];
        s_c[ex] = w ? s_c[ex] + c[j] : c[j];
      }
    }
    __syncthreads();
  }
  uint8_t* ws = a.ws;
  float* sums = reinterpret_cast<float*>(ws + kOffSums) + (int64_t)blockIdx.x * 2 * E;
  for (int ex = threadIdx.x; ex < E; ex += 256) {
    sums[ex] = s_p[ex];
    sums[E + ex] = __int_as_float(s_c[ex]);
  }
  if (threadIdx.x == 0) {
    reinterpret_cast<int*>(ws + kOffTokens)[blockIdx.x] = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
    reinterpret_cast<float*>(ws + kOffZ)[blockIdx.x] = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
    if (blockIdx.x == 0) *reinterpret_cast<uint32_t*>(ws) = 0;  // the finishing kernel's ticket
  }
}

// Work-group b sums experts 32 b .. 32 b + 31 over the partial sums, 32 slices of
// them side by side and a slice's loads at once; the last one to finish adds the
// groups' loss terms in order.
constexpr int kSlices = 32, kPerSlice = kBalanceBlocks / kSlices;
__global__ __launch_bounds__(kFinishExperts * kSlices) void balance_finish_kernel(BalanceArgs a, int blocks) {
  __shared__ float s_p[kSlices][kFinishExperts];
  __shared__ int s_c[kSlices][kFinishExperts];
  __shared__ float s_z[kSlices / 2];
  __shared__ int s_n[kSlices / 2], s_last;
  const int t = threadIdx.x, E = a.E;
  static_assert(kBalanceBlocks <= kFinishExperts * kSlices, "a thread per partial sum");
  int n = t < blocks ? reinterpret_cast<const int*>(a.ws + kOffTokens)[t] : 0;
  float z2 = t < blocks ? reinterpret_cast<const float*>(a.ws + kOffZ)[t] : 0.f;
  const int ex = blockIdx.x * kFinishExperts + (t & 31), slice = t >> 5;
  const float* sums = reinterpret_cast<const float*>(a.ws + kOffSums) + min(ex, E - 1);
  float vp[kPerSlice], vc[kPerSlice];
#pragma unroll
  for (int i = 0; i < kPerSlice; ++i) {
    const int b = min(slice + kSlices * i, blocks - 1);  // past the last: it again, not added
    vp[i] = sums[(int64_t)b * 2 * E];
    vc[i] = sums[(int64_t)b * 2 * E + E];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  z2 = route_dev::wave_sum(z2);
  if ((t & 63) == 0) s_n[t >> 6] = n, s_z[t >> 6] = z2;
  float p = 0.f;
  int c = 0;
#pragma unroll
  for (int i = 0; i < kPerSlice; ++i) {
    const bool yes = slice + kSlices * i < blocks;
    p += yes ? vp[i] : 0.f;
    c += yes ? __float_as_int(vc[i]) : 0;
  }
  s_p[slice][t & 31] = p;
  s_c[slice][t & 31] = c;
  __syncthreads();
  if (t >= 64) return;
  n = 0, z2 = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices / 2; ++i) n += s_n[i], z2 += s_z[i];
  const float each = n > 0 ? 1.0f / (float)n : 0.f;
  float* terms = reinterpret_cast<float*>(a.ws + kOffTerms);
  float term = 0.f;
  if (t < kFinishExperts && ex < E) {
    p = 0.f, c = 0;
#pragma unroll
    for (int s = 0; s < kSlices; ++s) p += s_p[s][t], c += s_c[s][t];
    const float load = n > 0 ? (float)((double)E * c / ((double)a.k * n)) : 0.f;
    a.load[ex] = load;
    a.counts[ex] = a.accumulate ? a.counts[ex] + c : c;
    term = load * (p * each);
  }
  term = route_dev::wave_sum(term);
  if (t == 0) {
    __hip_atomic_store(&terms[blockIdx.x], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the term is visible to whoever sees this work-group's ticket
    const uint32_t ticket = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.ws), 1u, __ATOMIC_ACQ_REL,
                                                   __HIP_MEMORY_SCOPE_AGENT);
    s_last = ticket == gridDim.x - 1;
  }
  if (!__builtin_amdgcn_readfirstlane(s_last)) return;  // one wave: written above by its lane 0
  float bal = 0.f;
  for (int b = t; b < (int)gridDim.x; b += 64)
    bal += __hip_atomic_load(&terms[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  bal = a.balance * route_dev::wave_sum(bal);
  const float zt = a.z != 0.f ? a.z * (z2 * each) : 0.f;  // lse^2 may overflow where no z loss is asked for
  if (t == 0) a.stats[0] = bal + zt, a.stats[1] = bal, a.stats[2] = zt, a.stats[3] = (float)n;
}

template <int ZT, int G, int NE>
__global__ __launch_bounds__(256) void balance_grad_kernel(BalanceGradArgs a) {
  constexpr int R = 64 / G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gl = lane & (G - 1), g = lane / G;
  const int E = a.E;
  float load[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const Run r = run_of<G>(j, gl, E);
    const float v = a.load[max(r.at + (j & 3), 0)];
    load[j] = r.has(j & 3) ? v : 0.f;
  }
  const float n = a.stats[3];
  const float gain = n > 0.f ? (a.dloss ? *a.dloss : 1.0f) / n : 0.f;
  for (int64_t row0 = ((int64_t)blockIdx.x * 4 + wave) * R; row0 < a.T; row0 += (int64_t)gridDim.x * 4 * R) {
    const int64_t row = row0 + g;
    const bool in = row < a.T;
    const char* zr = static_cast<const char*>(a.logits) + (in ? row : 0) * a.z_stride * value_size<ZT>();
    float p[NE];
#pragma unroll
    for (int j = 0; j < NE; j += 4) unpack4<ZT>(load_run<ZT, NE>(zr, run_of<G>(j, gl, E), E), p + j);
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (!surely<G, NE>(j)) p[j] = run_of<G>(j, gl, E).has(j & 3) ? p[j] : kMinusInf;
    const float lse = in ? a.lse[row] : kMinusInf;
    const bool counted = lse != kMinusInf;
    // the softmax again as in the forward pass, not exp(z - lse): beside a
    // large maximum the rounding of lse would scale the whole row
    const float mx = row_max<G, NE>(p);
    const float base = mx == kMinusInf ? 0.f : mx;
    float sum = 0.f, inner = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      p[j] = __expf(p[j] - base);
      sum += p[j];
      inner = fmaf(p[j], load[j], inner);
    }
    sum = group_sum<G>(sum);
    const float inv = counted ? 1.0f / sum : 0.f;
    inner = group_sum<G>(inner) * inv;
    const float scale = counted ? gain * inv : 0.f;
    const float rest = counted ? 2.0f * a.z * lse : 0.f;
    const bool write = in && (counted || !a.accumulate);
    if (write) {
      char* dr = static_cast<char*>(a.dlogits) + row * a.d_stride * (a.d_type == MOE_F32 ? 4 : 2);
#pragma unroll
      for (int j = 0; j < NE; j += 4) {
        const Run r = run_of<G>(j, gl, E);
        if (!surely<G, NE>(j) && r.skip >= 4) continue;
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = counted ? scale * p[j + i] * fmaf(a.balance, load[j + i] - inner, rest) : 0.f;
        if (a.d_type == MOE_F32) put_run<MOE_F32, NE>(dr, r, E, a.accumulate, d);
        else if (a.d_type == MOE_F16) put_run<MOE_F16, NE>(dr, r, E, a.accumulate, d);
        else put_run<MOE_BF16, NE>(dr, r, E, a.accumulate, d);
      }
    }
  }
}

int balance_blocks(int64_t T, int rows_at_once) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kBalanceBlocks, (T + rows_at_once - 1) / rows_at_once));
}

template <int ZT, int G, int NE>
hipError_t launch_rows(const BalanceArgs& a, hipStream_t s) {
  const int blocks = balance_blocks(a.T, 4 * 64 / G);
  const Launch l{s};
  hipError_t e = a.k <= 8 ? launch(balance_rows_kernel<ZT, G, NE, true>, dim3(blocks), dim3(256), l, a)
                          : launch(balance_rows_kernel<ZT, G, NE, false>, dim3(blocks), dim3(256), l, a);
  if (e != hipSuccess) return e;
  return launch(balance_finish_kernel, dim3((a.E + kFinishExperts - 1) / kFinishExperts),
                dim3(kFinishExperts * kSlices), l, a, blocks);
}
template <int ZT, int G, int NE>
hipError_t launch_grad(const BalanceGradArgs& a, hipStream_t s) {
  // eight work-groups of 4 waves per CU at most: the loads stay in registers over many rows
  const int64_t want = (a.T + 4 * 64 / G - 1) / (4 * 64 / G);
  return launch(balance_grad_kernel<ZT, G, NE>, dim3((unsigned)std::min<int64_t>(want, 2048)), dim3(256), Launch{s}, a);
}

// Lanes of a row. Few rows are latency alone: a wave each, with a quarter of the
// values per lane (forward and gradient, bf16: 91 x 512, 10 picks, 15.4 us against 22.7 with
// 16 lanes; 2048 x 512, 18.5 against 22.3; 2048 x 256, 8 picks, 14.1 against 14.9; up to 128
// experts 16 lanes are as quick or quicker: 2048 x 128, 12.6 against 13.5).
int lanes_of(int64_t T, int E) { return E > 512 || (E > 128 && T <= kWaveRows) ? 64 : 16; }

// f<ZT, G, NE>: the smallest lane share that holds E experts
#define MOE_BALANCE_SHAPE(f, ZT, a, s)                 \
  (a.E <= 512 && lanes_of(a.T, a.E) == 64              \
       ? (a.E <= 256 ? f<ZT, 64, 4>(a, s)              \
                     : f<ZT, 64, 8>(a, s))             \
   : a.E <= 64   ? f<ZT, 16, 4>(a, s)                  \
   : a.E <= 128  ? f<ZT, 16, 8>(a, s)                  \
   : a.E <= 256  ? f<ZT, 16, 16>(a, s)                 \
   : a.E <= 512  ? f<ZT, 16, 32>(a, s)                 \
   : a.E <= 1024 ? f<ZT, 64, 16>(a, s)                 \
   : a.E <= 2048 ? f<ZT, 64, 32>(a, s)                 \
                 : f<ZT, 64, 64>(a, s))

}  // namespace

// enough for fewer tokens too: up to kWaveRows of them may take more work-groups
int64_t balance_workspace_bytes(int64_t T, int32_t E) {
  const int64_t wave = std::min<int64_t>(T, kWaveRows);
  const int blocks = std::max(balance_blocks(T, 4 * 64 / lanes_of(T, E)), balance_blocks(wave, 4 * 64 / lanes_of(wave, E)));
  return (kOffSums + (int64_t)blocks * 2 * E * 4 + 255) / 256 * 256;
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (a.z_type == MOE_F32) return MOE_BALANCE_SHAPE(launch_rows, MOE_F32, a, s);
  if (a.z_type == MOE_F16) return MOE_BALANCE_SHAPE(launch_rows, MOE_F16, a, s);
  return MOE_BALANCE_SHAPE(launch_rows, MOE_BF16, a, s);
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.z_type == MOE_F32) return MOE_BALANCE_SHAPE(launch_grad, MOE_F32, a, s);
  if (a.z_type == MOE_F16) return MOE_BALANCE_SHAPE(launch_grad, MOE_F16, a, s);
  return MOE_BALANCE_SHAPE(launch_grad, MOE_BF16, a, s);
}

}  // namespace moe
