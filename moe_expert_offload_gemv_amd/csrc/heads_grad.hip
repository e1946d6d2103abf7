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
//
// Measured: 4096 x 36 heads of 128 bf16, 113 MB, 28.8 us = 3.9 TB/s, and 3.9 for the shares; 4096 x 32 of 128 fp32, 201 MB,
// 46 together, 42 = 4.8 TB/s without the shares. The streams are the same; a lane of 16-bit heads has 32 bytes on their way,
// one of fp32 64, and 16 waves a CU are too few for the former.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "heads_dev.h"
#include "kernels.h"

namespace moe {
namespace {

using namespace heads_dev;

constexpr int kGradSteps = 64;      // rows per row group whose angles are formed together
constexpr int kGradBlocks = 1024;  // work-groups: four a CU

// what a lane has of a row: its values as loaded, and where they belong
template <int XT, int GT, int RUN, int NG>
struct GradRow {
  RawRun<XT, RUN> x[NG][2];
  RawRun<GT, RUN> g[NG][2];
  int64_t out;
  int token;
};

// USUAL: a norm and a rotation, dx of x's type, and heads that fill their lanes (64, 128, ...)
template <int XT, int GT, int RUN, int NG, bool PAIRS, bool USUAL>
__global__ __launch_bounds__(kThreads) void heads_grad_kernel(HeadsArgs a) {
  using Row = GradRow<XT, GT, RUN, NG>;
  extern __shared__ __attribute__((aligned(16))) float2 s_turn[];
  const bool is_k = (int)blockIdx.x >= a.q.blocks;
  const HeadsPart p = is_k ? a.k : a.q;
  const int G = a.lanes, l = threadIdx.x & (G - 1), mine = threadIdx.x >> a.lanes_log;
  const int at_once = kThreads >> a.lanes_log, S = a.D / 2;
  const float inv_D = 1.0f / (float)a.D;
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
  const int64_t all = a.T * p.H;
  for (int64_t chunk = block;; chunk += p.blocks) {
    const int64_t r0 = chunk * p.rows;
    if (r0 >= all) break;
    const int64_t t0 = r0 / p.H;
    const int h0 = (int)(r0 - t0 * p.H), n = (int)std::min<int64_t>(p.rows, all - r0);
    // a row group's row of step u; past the last row: it again, not counted
    auto fetch = [&](int u, Row& to) __attribute__((always_inline)) {
      const int i = h0 + min(u * at_once + mine, n - 1);
      to.token = quotient(i, p.magic);
      const int h = i - to.token * p.H;
      const int64_t t = t0 + to.token;
      const char* x = static_cast<const char*>(p.x) + (t * p.x_stride + h * p.x_head) * value_size<XT>();
      const char* gr = static_cast<const char*>(p.g) + (t * p.g_stride + h * p.g_head) * value_size<GT>();
      to.out = t * p.out_stride + h * p.out_head;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (USUAL || a.norm) {
          to.x[g][0] = load_run<XT, RUN>(x + place[g].a * value_size<XT>());
          to.x[g][1] = load_run<XT, RUN>(x + place[g].b * value_size<XT>());
        }
        to.g[g][0] = load_run<GT, RUN>(gr + place[g].a * value_size<GT>());
        to.g[g][1] = load_run<GT, RUN>(gr + place[g].b * value_size<GT>());
      }
    };
    const int steps = (n + at_once - 1) / at_once;
    Row next;
    fetch(0, next);
    if (USUAL || a.R) {
      __syncthreads();  // every wave is done with the rows before
      fill_turns(a, t0, quotient(h0 + n - 1, p.magic) + 1, s_turn);
      __syncthreads();
    }
    // ALL: every row group has a row
    auto step = [&](auto ALL, int u, Row& now) __attribute__((always_inline)) {
      const bool in = decltype(ALL)::value || u * at_once + mine < n;
      float ga[NG][RUN], gb[NG][RUN];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        unpack_slots<GT, PAIRS, RUN>(now.g[g], ga[g], gb[g]);
        if (USUAL || a.R) {
          float2 angles[RUN];
          load_turns<RUN>(s_turn + now.token * S + (USUAL || place[g].in ? RUN * (l + G * g) : 0), angles);
          turn<true, RUN>(ga[g], gb[g], angles);
        }
      }
      if (USUAL || a.norm) {
        float va[NG][RUN], vb[NG][RUN], ss = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          unpack_slots<XT, PAIRS, RUN>(now.x[g], va[g], vb[g]);
          float part = 0.f;
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            part = fmaf(va[g][j], va[g][j], part);
            part = fmaf(vb[g][j], vb[g][j], part);
          }
          ss += USUAL || place[g].in ? part : 0.f;
        }
        const Inverse inv = inverse_rms(lanes_sum(ss, G), inv_D, (float)a.D, a.eps, [&](float k, float rest) {
          float s2 = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
              va[g][j] *= k, vb[g][j] *= k;
              const float x = USUAL || place[g].in ? va[g][j] * rest : 0.f, y = USUAL || place[g].in ? vb[g][j] * rest : 0.f;
              s2 = fmaf(x, x, s2);
              s2 = fmaf(y, y, s2);
            }
          return lanes_sum(s2, G);
        });
        float dot = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float part = 0.f;
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            va[g][j] *= inv.r;
            vb[g][j] *= inv.r;
            sum_a[g][j] = in ? fmaf(ga[g][j], va[g][j], sum_a[g][j]) : sum_a[g][j];
            sum_b[g][j] = in ? fmaf(gb[g][j], vb[g][j], sum_b[g][j]) : sum_b[g][j];
            ga[g][j] *= wa[g][j];
            gb[g][j] *= wb[g][j];
            part = fmaf(ga[g][j], va[g][j], part);
            part = fmaf(gb[g][j], vb[g][j], part);
          }
          dot += USUAL || place[g].in ? part : 0.f;
        }
        const float mean = lanes_sum(dot, G) * inv_D;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < RUN; ++j) {
            ga[g][j] = fmaf(-mean, va[g][j], ga[g][j]) * inv.r;
            gb[g][j] = fmaf(-mean, vb[g][j], gb[g][j]) * inv.r;
          }
        if (inv.left != 1.0f) {
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < RUN; ++j) ga[g][j] *= inv.left, gb[g][j] *= inv.left;
        }
      }
      const int64_t out = now.out;
      fetch(u + 1, now);
      if (!in) return;
      if constexpr (USUAL) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
          store_slots_as<XT, PAIRS, RUN>(static_cast<char*>(p.out) + out * value_size<XT>(), place[g], ga[g], gb[g]);
        return;
      }
      char* row = static_cast<char*>(p.out) + out * (a.out_type == MOE_F32 ? 4 : 2);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (place[g].in) store_slots<PAIRS, RUN>(a.out_type, row, place[g], ga[g], gb[g]);
    };
    // Whole steps of the usual case store without a condition: then the next step's loads can be waited for with
    // these stores still on their way (the first step stands before the loop so that its loads, too, are
    // followed by stores wherever they are waited for). Worth little beside four other work-groups: 4096 x 32 heads of
    // 128 fp32 47.7 us with the condition, 46.3 so.
    const int whole = n / at_once;
    if (whole) {
      step(std::true_type{}, 0, next);
#pragma unroll 1
      for (int u = 1; u < whole; ++u) step(std::true_type{}, u, next);
    }
    if (whole < steps) step(std::false_type{}, whole, next);
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
  constexpr int kAtOnce = 8;  // loads; past the last share: it again, not added
  for (int b0 = slice; b0 < p.blocks; b0 += kAtOnce * kSlices) {
    float part[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) part[i] = p.sums[(int64_t)min(b0 + i * kSlices, p.blocks - 1) * a.D + min(d, a.D - 1)];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) v += b0 + i * kSlices < p.blocks ? part[i] : 0.f;
  }
  s_sum[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (threadIdx.x >= 32 || d >= a.D) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) v += s_sum[i][threadIdx.x];
  p.dweight[d] = a.accumulate ? p.dweight[d] + v : v;
}

template <int XT, int RUN, int NG, bool PAIRS, bool USUAL>
hipError_t launch_grad_types(const HeadsArgs& a, const Launch& l, dim3 grid) {
  if (a.g_type == MOE_F32) return launch(heads_grad_kernel<XT, MOE_F32, RUN, NG, PAIRS, USUAL>, grid, dim3(kThreads), l, a);
  if (a.g_type == MOE_F16) return launch(heads_grad_kernel<XT, MOE_F16, RUN, NG, PAIRS, USUAL>, grid, dim3(kThreads), l, a);
  return launch(heads_grad_kernel<XT, MOE_BF16, RUN, NG, PAIRS, USUAL>, grid, dim3(kThreads), l, a);
}
template <int XT, bool PAIRS>
hipError_t launch_grad_run(const HeadsArgs& a, int run, const Launch& l, dim3 grid) {
  const bool usual = a.norm && a.R && a.out_type == a.x_type && (run << a.lanes_log) * 2 == a.D;
  switch (run) {
    case 6: return usual ? launch_grad_types<XT, 6, 1, PAIRS, true>(a, l, grid) : launch_grad_types<XT, 6, 1, PAIRS, false>(a, l, grid);
    case 5: return usual ? launch_grad_types<XT, 5, 1, PAIRS, true>(a, l, grid) : launch_grad_types<XT, 5, 1, PAIRS, false>(a, l, grid);
    case 4: return usual ? launch_grad_types<XT, 4, 1, PAIRS, true>(a, l, grid) : launch_grad_types<XT, 4, 1, PAIRS, false>(a, l, grid);
    case 2: return launch_grad_types<XT, 2, 2, PAIRS, false>(a, l, grid);
    default: return launch_grad_types<XT, 1, 4, PAIRS, false>(a, l, grid);
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
  const HeadsShape shape = heads_shape(a.D, a.R, a.pairs, true);
  a.lanes_log = shape.lanes_log, a.lanes = 1 << shape.lanes_log;
  a.slot_magic = (uint32_t)(((1ll << 31) + a.D / 2 - 1) / (a.D / 2));
  const int Hq = a.q.H, Hk = a.k.H;
  if (Hq) heads_split(a.q, a, most_blocks(Hq, Hk), kGradSteps, most_blocks(Hq, Hk));
  if (Hk) heads_split(a.k, a, most_blocks(Hk, Hq), kGradSteps, most_blocks(Hk, Hq));
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
