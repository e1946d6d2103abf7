// heads.hip - RMS norm of each query and key head and the rotation by its
// position, in one pass (moe_qk_norm_rope): the step between the query/key/value
// product and attention.
//
//   v = x * weight / sqrt(mean(x^2) + eps)          over the head's D values
//   (a, b) -> (a cos - b sin, b cos + a sin)        for each of the R / 2 pairs
//
// Bound by traffic: every value is read and written once. A row is a head of a token,
// in the registers of G lanes (heads_dev.h); a work-group takes up to 4 rows per row
// group, all loads before the first use, and forms the angles of its tokens once in LDS
// meanwhile. Queries and keys are two ranges of work-groups of one launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "heads_dev.h"
#include "kernels.h"

namespace moe {
namespace {

using namespace heads_dev;

template <int XT, int RUN, int NG, bool PAIRS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a) {
  constexpr int U = kHeadRows;
  extern __shared__ __attribute__((aligned(16))) float2 s_turn[];
  const bool is_k = (int)blockIdx.x >= a.q.blocks;
  const HeadsPart p = is_k ? a.k : a.q;
  const int G = a.lanes, l = threadIdx.x & (G - 1), mine = threadIdx.x >> a.lanes_log;
  const int at_once = kThreads >> a.lanes_log, S = a.D / 2;
  Place place[NG];
  float wa[NG][RUN], wb[NG][RUN];
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
  }
  for (int64_t chunk = (int)blockIdx.x - (is_k ? a.q.blocks : 0);; chunk += p.blocks) {
    const int64_t r0 = chunk * p.rows;
    if (r0 >= a.T * p.H) break;
    const int64_t t0 = r0 / p.H;
    const int h0 = (int)(r0 - t0 * p.H), n = (int)std::min<int64_t>(p.rows, a.T * p.H - r0);
    RawRun<XT, RUN> raw[U][NG][2];
    int token[U];
    int64_t out[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * at_once >= n) break;
      const int i = h0 + min(u * at_once + mine, n - 1);  // past the last row: it again, never stored
      token[u] = quotient(i, p.magic);
      const int h = i - token[u] * p.H;
      const char* x = static_cast<const char*>(p.x) + ((t0 + token[u]) * p.x_stride + h * p.x_head) * value_size<XT>();
      out[u] = (t0 + token[u]) * p.out_stride + h * p.out_head;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        raw[u][g][0] = load_run<XT, RUN>(x + place[g].a * value_size<XT>());
        raw[u][g][1] = load_run<XT, RUN>(x + place[g].b * value_size<XT>());
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
      Inverse inv{1.0f, 1.0f};
      if (a.norm)
        inv = inverse_rms(lanes_sum(ss, G), (float)a.D, a.eps, [&](float k) {
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
      if (u * at_once + mine >= n) continue;
      char* row = static_cast<char*>(p.out) + out[u] * (a.out_type == MOE_F32 ? 4 : 2);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!place[g].in) continue;
        const float2* angles = s_turn + token[u] * S + RUN * (l + G * g);
        float ya[RUN], yb[RUN];
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
          const float x = va[g][j] * inv.half * inv.r * wa[g][j], y = vb[g][j] * inv.half * inv.r * wb[g][j];
          turn(x, y, a.R ? angles[j] : make_float2(1.0f, 0.0f), ya[j], yb[j]);
        }
        store_slots<PAIRS, RUN>(a.out_type, row, place[g], ya, yb);
      }
    }
  }
}

template <int RUN, int NG, bool PAIRS>
hipError_t launch_types(const HeadsArgs& a, const Launch& l, dim3 grid) {
  if (a.x_type == MOE_F32) return launch(heads_kernel<MOE_F32, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
  if (a.x_type == MOE_F16) return launch(heads_kernel<MOE_F16, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
  return launch(heads_kernel<MOE_BF16, RUN, NG, PAIRS>, grid, dim3(kThreads), l, a);
}
template <bool PAIRS>
hipError_t launch_run(const HeadsArgs& a, int run, const Launch& l, dim3 grid) {
  switch (run) {
    case 8: return launch_types<8, 1, PAIRS>(a, l, grid);
    case 4: return launch_types<4, 1, PAIRS>(a, l, grid);
    case 2: return launch_types<2, 2, PAIRS>(a, l, grid);
    default: return launch_types<1, 4, PAIRS>(a, l, grid);
  }
}

}  // namespace

HeadsShape heads_shape(int D, int R, bool pairs) {
  HeadsShape s;
  // a run lies on one side of every boundary: that of the values that turn, and the middle of either side
  for (s.run = 8; s.run > 1; s.run /= 2)
    if (pairs ? D % (2 * s.run) == 0 : R / 2 % s.run == 0 && (D - R) / 2 % s.run == 0) break;
  const int groups = D / 2 / s.run, per_lane = s.run >= 4 ? 1 : s.run == 2 ? 2 : 4;
  for (s.lanes_log = 0; (per_lane << s.lanes_log) < groups; ++s.lanes_log) {
  }
  return s;
}

// Rows of a work-group: as many as its loads in flight hold, fewer while that leaves CUs without one,
// and no more than the LDS has angles for (32 KB: five work-groups a CU).
void heads_split(HeadsPart& p, const HeadsArgs& a, int max_rows, int64_t max_blocks) {
  const int at_once = kThreads >> a.lanes_log;
  const int64_t rows = a.T * p.H, want = (rows + 512 * at_once - 1) / (512 * at_once);
  p.rows = at_once * (int)std::max<int64_t>(1, std::min<int64_t>(want, max_rows));
  if (a.R) {
    const int tokens = 32768 / (a.D / 2 * 8);
    p.rows = std::min(p.rows, p.H == 1 ? tokens : (tokens - 2) * p.H);
  }
  p.magic = (uint32_t)(((1ll << 31) + p.H - 1) / std::max(p.H, 1));
  p.blocks = (int)std::min<int64_t>((rows + p.rows - 1) / p.rows, max_blocks);
}
uint32_t heads_lds(const HeadsArgs& a) {
  if (!a.R) return 0;
  int tokens = 0;
  for (const HeadsPart* p : {&a.q, &a.k})
    if (p->H) tokens = std::max(tokens, p->H == 1 ? p->rows : (p->rows + p->H - 2) / p->H + 1);
  return (uint32_t)tokens * (a.D / 2) * 8;
}

hipError_t launch_heads(HeadsArgs a, hipStream_t s) {
  const HeadsShape shape = heads_shape(a.D, a.R, a.pairs);
  a.lanes_log = shape.lanes_log, a.lanes = 1 << shape.lanes_log;
  a.slot_magic = (uint32_t)(((1ll << 31) + a.D / 2 - 1) / (a.D / 2));
  // rows beyond the grid are taken in turn by the same work-groups
  for (HeadsPart* p : {&a.q, &a.k})
    if (p->H) heads_split(*p, a, kHeadRows, 1 << 20);
  const Launch l{s, nullptr, nullptr, heads_lds(a)};
  const dim3 grid((unsigned)(a.q.blocks + a.k.blocks));
  return a.pairs ? launch_run<true>(a, shape.run, l, grid) : launch_run<false>(a, shape.run, l, grid);
}

}  // namespace moe
