// balance.hip - the router's load over a batch of tokens, its balance and z
// losses and their gradient (moe_router_balance, moe_router_balance_grad).
//
//   balance_rows_kernel    logits once: softmax, lse and the top-k set of every
//                          token; per work-group sums of p and counts per expert
//   balance_finish_kernel  the work-groups' sums, counts, loads and losses
//   balance_grad_kernel    logits once more: dlogits
//
// A token's row is shared by G lanes (16 up to 512 experts, else a wave), so
// its maximum, sums and top-k are a few DPP steps, and a wave works on 64 / G
// rows at once. A lane holds NE logits of its row, always of the same experts:
// the sums over tokens stay in its registers (p and count per expert) until
// the work-group has seen its last row. All sums run in a fixed order.
//
// Only the k-th largest logit is needed, not the order of the picks: an
// expert counts if its logit is larger, or equal and one of the lowest ids
// that fill the set.
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

// 4 values of a row of n from value i on; past it: -inf
template <int TYPE>
__device__ __forceinline__ void load4(const char* p, int i, int n, float* v) {
  if (i + 4 <= n) {
    uint32_t w[4];
    __builtin_memcpy(w, p + (int64_t)i * value_size<TYPE>(), 4 * value_size<TYPE>());
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == MOE_F32)
        v[j] = __uint_as_float(w[j]);
      else if constexpr (TYPE == MOE_F16)
        v[j] = half_to_float((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
      else
        v[j] = bf16_to_float((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? load1<TYPE>(p, i + j) : kMinusInf;
  }
}
template <int TYPE>
__device__ __forceinline__ void store4(char* p, int i, int n, const float* v) {
  if (i + 4 <= n) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == MOE_F32)
        w[j] = __float_as_uint(v[j]);
      else if (j < 2)
        w[j] = TYPE == MOE_F16 ? (float_to_half(v[2 * j]) | (uint32_t)float_to_half(v[2 * j + 1]) << 16)
                               : (float_to_bf16(v[2 * j]) | (uint32_t)float_to_bf16(v[2 * j + 1]) << 16);
    }
    __builtin_memcpy(p + (int64_t)i * value_size<TYPE>(), w, 4 * value_size<TYPE>());
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) store1<TYPE>(p, i + j, v[j]);
  }
}

// order bits of a lane's logit (0: past the last expert)
template <int G>
__device__ __forceinline__ uint32_t bits_of(float z, int j, int gl, int E) {
  return expert_of<G>(j, gl) < E ? route_dev::order_bits(z) : 0u;
}

// order bits of the k-th largest logit of the row. k <= 8: each lane sorts
// its logits eight at a time and keeps its 8 largest, then the lanes of the row
// merge their lists (sorting networks of route_dev.h): 236 instructions for
// four rows of 256 experts. k > 8: the bits are found from the top one down by
// counting the logits not below each candidate.
template <int G, int NE, bool TOP8>
__device__ __forceinline__ uint32_t kth_bits(const float (&z)[NE], int gl, int E, int k) {
  if constexpr (TOP8) {
    uint32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = j < NE ? bits_of<G>(z[j], j, gl, E) : 0u;
    route_dev::sort8_desc(t);
#pragma unroll
    for (int b = 8; b < NE; b += 8) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = bits_of<G>(z[b + j], b + j, gl, E);
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
    uint32_t m = t[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = i < k ? t[i] : m;
    return m;
  } else {
    uint32_t m = 0;
    for (int b = 31; b >= 0; --b) {
      const uint32_t c = m | (1u << b);
      int n = 0;
#pragma unroll
      for (int j = 0; j < NE; ++j) n += bits_of<G>(z[j], j, gl, E) >= c ? 1 : 0;
      if (group_sum_int<G>(n) >= k) m = c;
    }
    return m;
  }
}

template <int ZT, int G, int NE, bool TOP8>
__global__ __launch_bounds__(256) void balance_rows_kernel(BalanceArgs a) {
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
  for (int64_t row0 = ((int64_t)blockIdx.x * 4 + wave) * R; row0 < a.T; row0 += (int64_t)gridDim.x * 4 * R) {
    const int64_t row = row0 + g;
    const bool in = row < a.T && (!a.valid || a.valid[row]);
    float z[NE];
    const char* zr = static_cast<const char*>(a.logits) + (row < a.T ? row : 0) * a.z_stride * value_size<ZT>();
#pragma unroll
    for (int j = 0; j < NE; j += 4) load4<ZT>(zr, expert_of<G>(j, gl), E, z + j);
    const float mx = row_max<G, NE>(z);
    const float base = mx == kMinusInf ? 0.f : mx;  // a row of -inf alone: every exp is 0
    float e[NE], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      e[j] = __expf(z[j] - base);
      sum += e[j];
    }
    sum = group_sum<G>(sum);
    const float lse = in ? base + logf(sum) : kMinusInf;
    const bool counted = in && lse != kMinusInf;
    if (gl == 0 && row < a.T) a.lse[row] = lse;
    const float inv = counted ? 1.0f / sum : 0.f;
    z2 = counted ? fmaf(lse, lse, z2) : z2;
    n += counted ? 1 : 0;
    const uint32_t m = kth_bits<G, NE, TOP8>(z, gl, E, k);
    int above = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const uint32_t b = bits_of<G>(z[j], j, gl, E);
      above += b > m ? 1 : 0;
      equal += b == m ? 1 : 0;
    }
    above = group_sum_int<G>(above);
    equal = group_sum_int<G>(equal);
    int last = E;  // equal ones up to this id are in the set
    if (__ballot(above + equal > k)) {
      // more equal logits than places: the lowest ids, one by one
      int left = k - above;
      last = -1;
      while (__ballot(left > 0)) {
        int id = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
          const int ex = expert_of<G>(j, gl);
          if (bits_of<G>(z[j], j, gl, E) == m && ex > last) id = min(id, ex);
        }
        id = 0x7FFFFFFF - (int)group_max<G>((uint32_t)(0x7FFFFFFF - id));
        if (left > 0) last = id;
        --left;
      }
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const uint32_t b = bits_of<G>(z[j], j, gl, E);
      const bool chosen = b > m || (b == m && expert_of<G>(j, gl) <= last);
      c[j] += counted && chosen ? 1 : 0;
      p[j] = counted ? fmaf(e[j], inv, p[j]) : p[j];
    }
  }
  // the wave's rows, then the waves in turn
  z2 = sum_rows<G>(z2);
  n = sum_rows<G>(n);
  if (lane == 0) s_z[wave] = z2, s_n[wave] = n;
  for (int w = 0; w < 4; ++w) {
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (w == 0) p[j] = sum_rows<G>(p[j]), c[j] = sum_rows<G>(c[j]);
      if (wave == w && g == 0) {
        const int ex = expert_of<G>(j, gl);
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

// Work-group b sums experts 32 b .. 32 b + 31 over the partial sums; the last
// one to finish adds the groups' loss terms in order.
__global__ __launch_bounds__(256) void balance_finish_kernel(BalanceArgs a, int blocks) {
  __shared__ float s_p[8][kFinishExperts];
  __shared__ int s_c[8][kFinishExperts];
  __shared__ float s_z[4];
  __shared__ int s_n[4], s_last;
  const int t = threadIdx.x, E = a.E;
  int n = 0;
  float z2 = 0.f;
  for (int b = t; b < blocks; b += 256) {
    n += reinterpret_cast<const int*>(a.ws + kOffTokens)[b];
    z2 += reinterpret_cast<const float*>(a.ws + kOffZ)[b];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  z2 = route_dev::wave_sum(z2);
  if ((t & 63) == 0) s_n[t >> 6] = n, s_z[t >> 6] = z2;
  const int ex = blockIdx.x * kFinishExperts + (t & 31), slice = t >> 5;
  float p = 0.f;
  int c = 0;
  if (ex < E) {
    const float* sums = reinterpret_cast<const float*>(a.ws + kOffSums) + ex;
    for (int b = slice; b < blocks; b += 8) {
      p += sums[(int64_t)b * 2 * E];
      c += __float_as_int(sums[(int64_t)b * 2 * E + E]);
    }
  }
  s_p[slice][t & 31] = p;
  s_c[slice][t & 31] = c;
  __syncthreads();
  n = (s_n[0] + s_n[1]) + (s_n[2] + s_n[3]);
  z2 = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
  const float each = n > 0 ? 1.0f / (float)n : 0.f;
  float* terms = reinterpret_cast<float*>(a.ws + kOffTerms);
  if (t < 64) {
    float term = 0.f;
    if (t < kFinishExperts && ex < E) {
      p = 0.f, c = 0;
#pragma unroll
      for (int s = 0; s < 8; ++s) p += s_p[s][t], c += s_c[s][t];
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
  }
  __syncthreads();
  if (!s_last || t >= 64) return;
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
    const int ex = expert_of<G>(j, gl);
    load[j] = ex < E ? a.load[ex] : 0.f;
  }
  const float n = a.stats[3];
  const float gain = n > 0.f ? (a.dloss ? *a.dloss : 1.0f) / n : 0.f;
  for (int64_t row0 = ((int64_t)blockIdx.x * 4 + wave) * R; row0 < a.T; row0 += (int64_t)gridDim.x * 4 * R) {
    const int64_t row = row0 + g;
    const bool in = row < a.T;
    const char* zr = static_cast<const char*>(a.logits) + (in ? row : 0) * a.z_stride * value_size<ZT>();
    float p[NE];
#pragma unroll
    for (int j = 0; j < NE; j += 4) load4<ZT>(zr, expert_of<G>(j, gl), E, p + j);
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
        const int ex = expert_of<G>(j, gl);
        if (ex >= E) continue;
        float d[4], old[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = counted ? scale * p[j + i] * fmaf(a.balance, load[j + i] - inner, rest) : 0.f;
        if (a.accumulate) {
          if (a.d_type == MOE_F32) load4<MOE_F32>(dr, ex, E, old);
          else if (a.d_type == MOE_F16) load4<MOE_F16>(dr, ex, E, old);
          else load4<MOE_BF16>(dr, ex, E, old);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] += old[i];
        }
        if (a.d_type == MOE_F32) store4<MOE_F32>(dr, ex, E, d);
        else if (a.d_type == MOE_F16) store4<MOE_F16>(dr, ex, E, d);
        else store4<MOE_BF16>(dr, ex, E, d);
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
  return launch(balance_finish_kernel, dim3((a.E + kFinishExperts - 1) / kFinishExperts), dim3(256), l, a, blocks);
}
template <int ZT, int G, int NE>
hipError_t launch_grad(const BalanceGradArgs& a, hipStream_t s) {
  // eight work-groups of 4 waves per CU at most: the loads stay in registers over many rows
  const int64_t want = (a.T + 4 * 64 / G - 1) / (4 * 64 / G);
  return launch(balance_grad_kernel<ZT, G, NE>, dim3((unsigned)std::min<int64_t>(want, 2048)), dim3(256), Launch{s}, a);
}

// f<ZT, G, NE>: the smallest lane share that holds E experts
#define MOE_BALANCE_SHAPE(f, ZT, a, s)                 \
  (a.E <= 64     ? f<ZT, 16, 4>(a, s)                  \
   : a.E <= 128  ? f<ZT, 16, 8>(a, s)                  \
   : a.E <= 256  ? f<ZT, 16, 16>(a, s)                 \
   : a.E <= 512  ? f<ZT, 16, 32>(a, s)                 \
   : a.E <= 1024 ? f<ZT, 64, 16>(a, s)                 \
   : a.E <= 2048 ? f<ZT, 64, 32>(a, s)                 \
                 : f<ZT, 64, 64>(a, s))

}  // namespace

int64_t balance_workspace_bytes(int64_t T, int32_t E) {
  const int blocks = balance_blocks(T, E <= 512 ? 16 : 4);
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
