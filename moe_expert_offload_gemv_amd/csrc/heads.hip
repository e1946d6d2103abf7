// heads.hip - RMS norm of each query and key head and the rotation by its
// position, in one pass (moe_qk_norm_rope): the step between the query/key/value
// product and attention.
//
//   v = x * weight / sqrt(mean(x^2) + eps)          over the head's D values
//   (a, b) -> (a cos - b sin, b cos + a sin)        for each of the R / 2 pairs
//
// Bound by traffic: every value is read and written once. A row is a head of a token,
// in the registers of G lanes (heads_dev.h); a work-group takes up to 8 rows per row
// group, the next one's loads on their way behind each, and forms the angles of all their tokens
// once in LDS beforehand. Queries and keys are two ranges of work-groups of one launch.
//
// Measured (as nodes of a graph): 4096 x 36 heads of 128 bf16, 75 MB, 14.6-15 us = 5.1 TB/s, a copy's rate
// (2 rows a group and no loads ahead 16.7, 4 rows at once 18.4); 12287 x 16 heads of 80 fp16, three axes, 63 MB,
// 17.3 = 3.6 TB/s (10 of 16 lanes have values, and 2.3e5 instructions a SIMD are 15 of it); one token,
// 18 heads of 128 fp32, 3.2: a launch, two trips to memory and the angles between.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "heads_dev.h"
#include "kernels.h"

namespace moe {
namespace {

using namespace heads_dev;

constexpr int kHeadSteps = 8;   // rows per row group whose angles are formed together
constexpr int kHeadAim = 1536;  // work-groups of queries, and of keys

// what a lane has of a row: its values as loaded, and where they go
template <int XT, int RUN, int NG>
struct HeadRow {
  RawRun<XT, RUN> x[NG][2];
  int64_t out;
  int token;
};

template <int XT, int RUN, int NG, bool PAIRS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a) {
  using Row = HeadRow<XT, RUN, NG>;
  extern __shared__ __attribute__((aligned(16))) float2 s_turn[];
  const bool is_k = (int)blockIdx.x >= a.q.blocks;
  const HeadsPart p = is_k ? a.k : a.q;
  const int G = a.lanes, l = threadIdx.x & (G - 1), mine = threadIdx.x >> a.lanes_log;
  const int at_once = kThreads >> a.lanes_log, S = a.D / 2;
  const float inv_D = 1.0f / (float)a.D;
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
    // a row group's row of step u; past the last row: it again, never stored
    auto fetch = [&](int u, Row& to) __attribute__((always_inline)) {
      const int i = h0 + min(u * at_once + mine, n - 1);
      to.token = quotient(i, p.magic);
      const int h = i - to.token * p.H;
      const int64_t t = t0 + to.token;
      const char* x = static_cast<const char*>(p.x) + (t * p.x_stride + h * p.x_head) * value_size<XT>();
      to.out = t * p.out_stride + h * p.out_head;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        to.x[g][0] = load_run<XT, RUN>(x + place[g].a * value_size<XT>());
        to.x[g][1] = load_run<XT, RUN>(x + place[g].b * value_size<XT>());
      }
    };
    const int steps = (n + at_once - 1) / at_once;
    Row next;
    fetch(0, next);
    if (a.R) {
      __syncthreads();  // every wave is done with the rows before
      fill_turns(a, t0, quotient(h0 + n - 1, p.magic) + 1, s_turn);
      __syncthreads();
    }
    auto step = [&](int u, Row& now) __attribute__((always_inline)) {
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
        ss += place[g].in ? part : 0.f;
      }
      float r = 1.0f;
      if (a.norm)
        r = inverse_rms(lanes_sum(ss, G), inv_D, (float)a.D, a.eps, [&](float k, float rest) {
              float s2 = 0.f;
#pragma unroll
              for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int j = 0; j < RUN; ++j) {
                  va[g][j] *= k, vb[g][j] *= k;
                  const float x = place[g].in ? va[g][j] * rest : 0.f, y = place[g].in ? vb[g][j] * rest : 0.f;
                  s2 = fmaf(x, x, s2);
                  s2 = fmaf(y, y, s2);
                }
              return lanes_sum(s2, G);
            }).r;
      const int token = now.token;
      char* row = static_cast<char*>(p.out) + now.out * (a.out_type == MOE_F32 ? 4 : 2);
      if (u + 1 < steps) fetch(u + 1, now);
      if (u * at_once + mine >= n) return;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!place[g].in) continue;
#pragma unroll
        for (int j = 0; j < RUN; ++j) va[g][j] = va[g][j] * r * wa[g][j], vb[g][j] = vb[g][j] * r * wb[g][j];
        if (a.R) {
          float2 angles[RUN];
          load_turns<RUN>(s_turn + token * S + RUN * (l + G * g), angles);
          turn<false, RUN>(va[g], vb[g], angles);
        }
        store_slots<PAIRS, RUN>(a.out_type, row, place[g], va[g], vb[g]);
      }
    };
#pragma unroll 1
    for (int u = 0; u < steps; ++u) step(u, next);
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
    case 6: return launch_types<6, 1, PAIRS>(a, l, grid);
    case 4: return launch_types<4, 1, PAIRS>(a, l, grid);
    case 2: return launch_types<2, 2, PAIRS>(a, l, grid);
    default: return launch_types<1, 4, PAIRS>(a, l, grid);
  }
}

}  // namespace

// The slots of a run and the lanes of a head. A run lies on one side of every boundary: that of the values that
// turn, and the middle of either side. Of the runs that do, the one that leaves the fewest lanes without
// values, 4 before others (us: 12287 x 10 heads of 192 bf16, 6 slots 24.5, 4 slots 27.3; gradient of 4096 x 32 heads of 72
// and 80, 6 and 5 slots 17.4 and 19.5, 4 slots 23.3 and 23.2; forward, 5 slots of 80 are slower than 4, 21.5 and 19.7;
// 8 slots, half as many lanes and twice the registers, lose at 4096 x 36 of 128: 17.7 and 16.7, gradient 41.5 and 34.4).
HeadsShape heads_shape(int D, int R, bool pairs, bool grad) {
  HeadsShape best{1, 0};
  int most = 0;
  for (int run : {4, 6, 5, 2, 1}) {
    if (run == 5 && !grad) continue;
    if (pairs ? D % (2 * run) : R / 2 % run || (D - R) / 2 % run) continue;
    const int groups = D / 2 / run, per_lane = run >= 4 ? 1 : run == 2 ? 2 : 4;
    if (run < 4 && most) break;  // narrower accesses only where nothing else fits
    int log = 0;
    while ((per_lane << log) < groups) ++log;
    const int filled = 64 * groups / (per_lane << log);
    if (log <= 6 && filled > most) best = HeadsShape{run, log}, most = filled;
  }
  return best;
}

// Rows of a work-group and work-groups: as many of these as are aimed at, up to max_rows rows per row group each and no
// more rows than the LDS has angles for (32 KB: five work-groups a CU). Beyond max_blocks they take rows in turn,
// all of them about as often.
void heads_split(HeadsPart& p, const HeadsArgs& a, int64_t aim, int max_rows, int64_t max_blocks) {
  const int at_once = kThreads >> a.lanes_log;
  const int64_t rows = a.T * p.H, want = (rows + aim * at_once - 1) / (aim * at_once);
  p.rows = at_once * (int)std::max<int64_t>(1, std::min<int64_t>(want, max_rows));
  if (a.R) {
    const int tokens = 32768 / (a.D / 2 * 8);
    p.rows = std::min(p.rows, p.H == 1 ? tokens : (tokens - 2) * p.H);
  }
  p.magic = (uint32_t)(((1ll << 31) + p.H - 1) / std::max(p.H, 1));
  const int64_t chunks = (rows + p.rows - 1) / p.rows, turns = (chunks + max_blocks - 1) / max_blocks;
  p.blocks = turns ? (int)((chunks + turns - 1) / turns) : 0;
}
uint32_t heads_lds(const HeadsArgs& a) {
  if (!a.R) return 0;
  int tokens = 0;
  for (const HeadsPart* p : {&a.q, &a.k})
    if (p->H) tokens = std::max(tokens, p->H == 1 ? p->rows : (p->rows + p->H - 2) / p->H + 1);
  return (uint32_t)tokens * (a.D / 2) * 8;
}

hipError_t launch_heads(HeadsArgs a, hipStream_t s) {
  const HeadsShape shape = heads_shape(a.D, a.R, a.pairs, false);
  a.lanes_log = shape.lanes_log, a.lanes = 1 << shape.lanes_log;
  a.slot_magic = (uint32_t)(((1ll << 31) + a.D / 2 - 1) / (a.D / 2));
  // rows beyond the grid are taken in turn by the same work-groups
  for (HeadsPart* p : {&a.q, &a.k})
    if (p->H) heads_split(*p, a, kHeadAim, kHeadSteps, 1 << 20);
  const Launch l{s, nullptr, nullptr, heads_lds(a)};
  const dim3 grid((unsigned)(a.q.blocks + a.k.blocks));
  return a.pairs ? launch_run<true>(a, shape.run, l, grid) : launch_run<false>(a, shape.run, l, grid);
}

}  // namespace moe
