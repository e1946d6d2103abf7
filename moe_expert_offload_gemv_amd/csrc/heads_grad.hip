// heads_grad.hip - gradient of the norm and rotation of heads
// (moe_qk_norm_rope_grad).
//
// With xh = x / sqrt(mean(x^2) + eps), g' the output's gradient turned back and u = g' * weight:
//   dx = (u - xh * mean(u * xh)) / sqrt(mean(x^2) + eps)        dweight = sum over rows of g' * xh
//
// Bound by traffic: x and the gradient are read once, dx is written once; nothing of the
// forward pass is kept but its input. Rows lie as in the forward kernel. A work-group goes through
// its share of the rows and keeps its sum of dweight in registers, then in the workspace;
// heads_dweight_kernel adds the work-groups' shares in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "heads_dev.h"
#include "kernels.h"

namespace moe {
namespace {

using namespace heads_dev;

constexpr int kGradRows = 2;       // rows per row group, loaded at once
constexpr int kGradBlocks = 1024;  // work-groups: four a CU

template <int XT, int GT, int RUN, int NG, bool PAIRS>
__global__ __launch_bounds__(kThreads) void heads_grad_kernel(HeadsArgs a) {
  constexpr int U = kGradRows;
  extern __shared__ __attribute__((aligned(16))) float2 s_turn[];
  const bool is_k = (int)blockIdx.x >= a.q.blocks;
  const HeadsPart p = is_k ? a.k : a.q;
  const int G = a.lanes, l = threadIdx.x & (G - 1), mine = threadIdx.x >> a.lanes_log;
  const int at_once = kThreads >> a.lanes_log, S = a.D / 2;
  const int64_t block = (int)blockIdx.x - (is_k ? a.q.blocks : 0);
  Place place[NG];
  float wa[NG][RUN], wb[NG][RUN], sum_a[NG][RUN], sum_b[NG][RUN];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    place[g] = place_of<RUN, PAIRS>(l + G * g, a.D, a.R);
    RawRun<MOE_F32, RUN> w[2];
    if (p.weight) {
      w[0] = load_run<MOE_F32, RUN>(reinterpret_cast<const char*>(p.weight + place[g].a));
      w[1] = load_run<MOE_F32, RUN>(reinterpret_cast<const char*>(p.weight + place[g].b));
    } else {
#pragma unroll
      for (int j = 0; j < RUN; ++j) w[0].v[j] = w[1].v[j] = __float_as_uint(1.0f);
    }
    unpack_slots<MOE_F32, PAIRS, RUN>(w, wa[g], wb[g]);
#pragma unroll
    for (int j = 0; j < RUN; ++j) sum_a[g][j] = sum_b[g][j] = 0.f;
  }
  for (int64_t chunk = block;; chunk += p.blocks) {
    const int64_t r0 = chunk * p.rows;
    if (r0 >= a.T * p.H) break;
    const int64_t t0 = r0 / p.H;
    const int h0 = (int)(r0 - t0 * p.H), n = (int)std::min<int64_t>(p.rows, a.T * p.H - r0);
    RawRun<XT, RUN> raw[U][NG][2];
    RawRun<GT, RUN> grad[U][NG][2];
    int token[U];
    int64_t out[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * at_once >= n) break;
      const int i = h0 + min(u * at_once + mine, n - 1);  // past the last row: it again, not counted
      token[u] = quotient(i, p.magic);
      const int h = i - token[u] * p.H;
      const int64_t t = t0 + token[u];
      const char* x = static_cast<const char*>(p.x) + (t * p.x_stride + h * p.x_head) * value_size<XT>();
      const char* gr = static_cast<const char*>(p.g) + (t * p.g_stride + h * p.g_head) * value_size<GT>();
      out[u] = t * p.out_stride + h * p.out_head;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (a.norm) {
          raw[u][g][0] = load_run<XT, RUN>(x + place[g].a * value_size<XT>());
          raw[u][g][1] = load_run<XT, RUN>(x + place[g].b * value_size<XT>());
        }
        grad[u][g][0] = load_run<GT, RUN>(gr + place[g].a * value_size<GT>());
        grad[u][g][1] = load_run<GT, RUN>(gr + place[g].b * value_size<GT>());
      }
    }
    if (a.R) {
      __syncthreads();  // every wave is done with the rows before
      fill_turns(a, t0, quotient(h0 + n - 1, p.magic) + 1, s_turn);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * at_once >= n) break;
      const bool in = u * at_once + mine < n;
      float ga[NG][RUN], gb[NG][RUN];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float ya[RUN], yb[RUN];
        unpack_slots<GT, PAIRS, RUN>(grad[u][g], ya, yb);
        const float2* angles = s_turn + token[u] * S + (place[g].in ? RUN * (l + G * g) : 0);
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
          const float2 cs = a.R ? angles[j] : make_float2(1.0f, 0.0f);
          turn(ya[j], yb[j], make_float2(cs.x, -cs.y), ga[g][j], gb[g][j]);
          ga[g][j] = place[g].in ? ga[g][j] : 0.f;
          gb[g][j] = place[g].in ? gb[g][j] : 0.f;
        }
      }
      if (a.norm) {
        float va[NG][RUN], vb[NG][RUN], ss = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          unpack_slots<XT, PAIRS, RUN>(raw[u][g], va[g], vb[g]);
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            va[g][j] = place[g].in ? va[g][j] : 0.f;
            vb[g][j] = place[g].in ? vb[g][j] : 0.f;
            ss = fmaf(va[g][j], va[g][j], ss);
            ss = fmaf(vb[g][j], vb[g][j], ss);
          }
        }
        const Inverse inv = inverse_rms(lanes_sum(ss, G), (float)a.D, a.eps, [&](float k) {
          float s2 = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
              const float x = va[g][j] * k, y = vb[g][j] * k;
              s2 = fmaf(x, x, s2);
              s2 = fmaf(y, y, s2);
            }
          return lanes_sum(s2, G);
        });
        float dot = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            va[g][j] = va[g][j] * inv.half * inv.r;
            vb[g][j] = vb[g][j] * inv.half * inv.r;
            sum_a[g][j] = in ? fmaf(ga[g][j], va[g][j], sum_a[g][j]) : sum_a[g][j];
            sum_b[g][j] = in ? fmaf(gb[g][j], vb[g][j], sum_b[g][j]) : sum_b[g][j];
            ga[g][j] *= wa[g][j];
            gb[g][j] *= wb[g][j];
            dot = fmaf(ga[g][j], va[g][j], dot);
            dot = fmaf(gb[g][j], vb[g][j], dot);
          }
        const float mean = lanes_sum(dot, G) / (float)a.D;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            ga[g][j] = fmaf(-mean, va[g][j], ga[g][j]) * inv.r * inv.half;
            gb[g][j] = fmaf(-mean, vb[g][j], gb[g][j]) * inv.r * inv.half;
          }
      }
      if (!in) continue;
      char* row = static_cast<char*>(p.out) + out[u] * (a.out_type == MOE_F32 ? 4 : 2);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (place[g].in) store_slots<PAIRS, RUN>(a.out_type, row, place[g], ga[g], gb[g]);
    }
  }
  if (!p.dweight) return;
  // the row groups' sums, in their order
  float* s_sum = reinterpret_cast<float*>(s_turn);  // [at_once][D]
  __syncthreads();
#pragma unroll
  for (int g = 0; g < NG; ++g)
    if (place[g].in) store_slots<PAIRS, RUN>(MOE_F32, reinterpret_cast<char*>(s_sum + mine * a.D), place[g], sum_a[g], sum_b[g]);
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float v = 0.f;
    for (int i = 0; i < at_once; ++i) v += s_sum[i * a.D + d];
    p.sums[block * a.D + d] = v;
  }
}

// Values 32 b .. of the weights of queries (the first work-groups) or keys: 32 slices of the shares side by side
constexpr int kSlices = 32;
__global__ __launch_bounds__(32 * kSlices) void heads_dweight_kernel(HeadsArgs a) {
  __shared__ float s_sum[kSlices][32];
  const int per = (a.D + 31) / 32;
  const bool is_k = !a.q.dweight || (int)blockIdx.x >= per;
  const HeadsPart p = is_k ? a.k : a.q;
  const int d = ((int)blockIdx.x - (is_k && a.q.dweight ? per : 0)) * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (d < a.D)
    for (int b = slice; b < p.blocks; b += kSlices) v += p.sums[(int64_t)b * a.D + d];
  s_sum[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (threadIdx.x >= 32 || d >= a.D) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) v += s_sum[i][threadIdx.x];
  p.dweight[d] = a.accumulate ? p.dweight[d] + v : v;
}

template <int XT, int RUN, int NG, bool PAIRS>
hipError_t launch_grad_types(const HeadsArgs& a, const Launch& l, dim3 grid) {
  if (a.g_type == MOE_F32) return launch(heads_grad_kernel<XT, MOE_F32, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
  if (a.g_type == MOE_F16) return launch(heads_grad_kernel<XT, MOE_F16, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
  return launch(heads_grad_kernel<XT, MOE_BF16, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
}
template <int XT, bool PAIRS>
hipError_t launch_grad_run(const HeadsArgs& a, int run, const Launch& l, dim3 grid) {
  switch (run) {
    case 8: return launch_grad_types<XT, 8, 1, PAIRS>(a, l, grid);
    case 4: return launch_grad_types<XT, 4, 1, PAIRS>(a, l, grid);
    case 2: return launch_grad_types<XT, 2, 2, PAIRS>(a, l, grid);
    default: return launch_grad_types<XT, 1, 4, PAIRS>(a, l, grid);
  }
}
template <int XT>
hipError_t launch_grad(const HeadsArgs& a, int run, const Launch& l, dim3 grid) {
  return a.pairs ? launch_grad_run<XT, true>(a, run, l, grid) : launch_grad_run<XT, false>(a, run, l, grid);
}

// work-groups of queries and of keys at most, by their share of the heads
int most_blocks(int H, int others) {
  return H ? std::max(1, (int)((int64_t)kGradBlocks * H / (H + others))) : 0;
}

}  // namespace

int64_t heads_grad_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
  const int64_t blocks = std::min<int64_t>(T * Hq, most_blocks(Hq, Hk)) + std::min<int64_t>(T * Hk, most_blocks(Hk, Hq));
  return (blocks * D * 4 + 255) / 256 * 256;
}

hipError_t launch_heads_grad(HeadsArgs a, uint8_t* ws, hipStream_t s) {
  const HeadsShape shape = heads_shape(a.D, a.R, a.pairs);
  a.lanes_log = shape.lanes_log, a.lanes = 1 << shape.lanes_log;
  a.slot_magic = (uint32_t)(((1ll << 31) + a.D / 2 - 1) / (a.D / 2));
  const int Hq = a.q.H, Hk = a.k.H;
  if (Hq) heads_split(a.q, a, kGradRows, most_blocks(Hq, Hk));
  if (Hk) heads_split(a.k, a, kGradRows, most_blocks(Hk, Hq));
  a.q.sums = reinterpret_cast<float*>(ws);
  a.k.sums = a.q.sums + (int64_t)a.q.blocks * a.D;
  const int per = (a.D + 31) / 32, groups = (a.q.dweight ? per : 0) + (a.k.dweight ? per : 0);
  const uint32_t sums = groups ? (uint32_t)(kThreads >> a.lanes_log) * a.D * 4 : 0;
  const Launch l{s, nullptr, nullptr, std::max(heads_lds(a), sums)};
  const dim3 grid((unsigned)(a.q.blocks + a.k.blocks));
  hipError_t e = !grid.x               ? hipSuccess  // no tokens: the weights' gradients are 0
                 : a.x_type == MOE_F32 ? launch_grad<MOE_F32>(a, shape.run, l, grid)
                 : a.x_type == MOE_F16 ? launch_grad<MOE_F16>(a, shape.run, l, grid)
                                       : launch_grad<MOE_BF16>(a, shape.run, l, grid);
  if (e != hipSuccess || !groups) return e;
  return launch(heads_dweight_kernel, dim3(groups), dim3(32 * kSlices), Launch{s}, a);
}

}  // namespace moe
