// decode.hip - gfx950 GEMV kernels of the decode path of one MoE layer.
//
//   gemv_route_gateup_kernel
//                         with logits given (E <= 512): wave 0 of every
//                         work-group routes the token (top-k, slot-table
//                         lookup) while waves 1-3 stage the activations
//                         in LDS, then all waves run the gate/up GEMV
//                         below; one wave per pick applies the
//                         lookup's side effects (stamp, pick record, count)
//                         and publishes the pick for the down GEMV. This
//                         saves the routing launch and the dependent read of
//                         its output on the decode critical path.
//                         A cold pick p < capture_picks that the cache step
//                         will admit (its previous miss lies inside the
//                         window, from the last-miss clocks the step began
//                         with) also writes the bytes it reads over PCIe into
//                         the layer's capture block p (the down GEMV adds the
//                         down matrix) and names it in the layer's capture
//                         directory, so its promotion is an HBM-to-HBM copy
//                         instead of a second PCIe transfer.
//   gemv_gateup_kernel    h = silu(W_gate x) * (W_up x) per pick, picks routed
//                         by route.hip; hot picks stream from HBM while cold
//                         picks stream over PCIe in the same launch.
//   gemv_down_combine_kernel
//                         y_pick = W_down h, then the weighted sum over the
//                         picks of a token in pick order (+ the old y with
//                         MOE_ACCUMULATE).
//   Timing mode splits both into a hot-only and a cold-only launch
//   (gemv_down_pick_kernel writes the hot picks' y_pick for the combine), so
//   each is measured against its own bound: HBM or PCIe.
//
// What is computed follows the pointer-table GEMV of the
// "a6000-custom-kernels" README (diagram of the moe_cache_gemv kernel and the
// paragraph under it): each routed expert is found through a table, hot ones
// in a VRAM pool, cold ones in pinned host RAM read zero-copy, cold reads
// logged for a later promotion pass, use-stamps kept for eviction. The fused
// gate/up GEMV follows the narrow-batch mat-vec of the mx-llama.cpp FEATURES
// page (gate and up lanes fused, one mat-vec per expert assignment).
//
// GEMV mapping (MI355X, wave64): a weight row is a run of 16-byte nibble
// blocks; LPR consecutive lanes share a row and each lane owns BPL blocks of
// it, so one wave-wide 128-bit load covers 64 consecutive blocks (1 KiB) and
// the activation slice a lane needs stays in its registers for every row the
// wave visits. Per block the lane forms sum_j q_j x_j with q in 0..15 (byte
// to float conversions of masked nibbles), then adds d * (that - 8 sum_j x_j),
// which is sum_j d (q_j - 8) x_j in fp32.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemv_dev.h"
#include "kernels.h"
#include "route_dev.h"

namespace moe {

using namespace gemv_dev;

// ---------------------------------------------------------------------------
// routing + lookup + gate/up GEMV + SwiGLU; grid = (row chunks of F, picks of a
// token, tokens).
// Wave 0 of each work-group routes the token and looks the pick up (once per
// work-group, not per wave: 2048 waves repeating the top-k and the loads of
// the logits and the table row contended for each CU's scalar unit and
// memory pipeline) while waves 1-3 stage the token's activations in LDS;
// the pick, its slot and the capture decision reach the other waves through
// LDS.
// r.policy = 1: wave 0 of work-group x = 0 of each pick applies the pick's
// side effects (the same as route_kernel's); 0: none (a second launch of the
// same step, in the timing split).
template <int LPR, int BPL, int NIT, int MODE>
__global__ __launch_bounds__(256) void gemv_route_gateup_kernel(GemvArgs a, RouteArgs r) {
  constexpr int NJ = kFusedRouteMaxExperts / 64;
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS_WG = 4 * NIT * RPW;
  constexpr int KB = LPR * BPL;  // blocks per row: H / 32
  // the activations, float4 c of block b at 8 b + (c ^ (b & 7)): the
  // staging writes (8 lanes per block) and the slice reads (one block per
  // lane) both hit distinct banks
  __shared__ float4 s_x[KB * 8 + 1];  // + a spare entry
  __shared__ int32_t s_pick[3];  // expert, slot (-1: cold), capture (1) or not
  // the arguments the routing needs, fetched at entry in one scalar round
  // trip (fetched where first used, the later ones would each add a
  // dependent round trip ahead of the routing loads)
  const float* logits = r.logits;
  const int32_t* tbl = r.tbl;
  const uint32_t* last_miss = r.last_miss;
  const Ctrl* ctrl = r.ctrl;
  asm volatile("" ::"s"(logits), "s"(tbl), "s"(last_miss), "s"(ctrl), "s"(r.E), "s"(a.k), "s"(r.capture_picks),
               "s"(r.policy), "s"(r.S), "s"(r.window), "s"(r.admit_misses), "s"(r.pub_seq), "s"(r.pub_value),
               "s"(a.out), "s"(a.x));
  // grid (row chunks, pick, token): no division for the pick index
  const int t = blockIdx.z, pick = blockIdx.y, p = t * a.k + pick;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lb = lane % LPR, rg = lane / LPR;
  const int E = r.E;
  const bool may_capture = p < r.capture_picks;

  if (wave != 0) {
    // waves 1-3 stage the activations; wave 0 goes straight to the routing
    // (behind these loads and their LDS writes its routing loads would wait
    // out a memory round trip first)
    // (every load issued, index clamped, before the first LDS write, so the
    // loads overlap)
    const float4* src = reinterpret_cast<const float4*>(a.x + (int64_t)t * a.H);
    constexpr int NQ = (KB * 8 + 191) / 192;
    float4 xq[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int q = threadIdx.x - 64 + 192 * i;
      xq[i] = src[q < KB * 8 ? q : KB * 8 - 1];
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {  // lanes past the end write the spare entry
      const int q = threadIdx.x - 64 + 192 * i, b = q >> 3, c = q & 7;
      s_x[q < KB * 8 ? b * 8 + (c ^ (b & 7)) : KB * 8] = xq[i];
    }
  }
  // wave 0 of work-group x = 0 applies the side effects and needs every
  // pick's logit for the weight; the others route up to their own pick
  const bool policy_wave = r.policy && blockIdx.x == 0 && wave == 0;
  if (wave == 0) {
    float z[NJ];
    int32_t tb[NJ];
    uint32_t lm[NJ];
    // the loads are issued without per-lane branches (index clamped into
    // the layer's experts, the value dropped afterwards), so none waits
    // behind one; the last-miss row exists only when picks may be captured
    // (a work-group-uniform condition)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + 64 * j, ec = e < E ? e : E - 1;
      z[j] = logits[(int64_t)t * E + ec];
      tb[j] = tbl[ec];
      lm[j] = 0u;
    }
    if (may_capture) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int e = lane + 64 * j;
        lm[j] = last_miss[e < E ? e : E - 1];
      }
    }
    // the step's clock, loaded behind the routing loads and needed only
    // once the pick is known
    const uint32_t clk = ctrl->clock + (uint32_t)t;
    static_assert(NJ == 8, "the fused routing holds 8 experts per lane");
    // order bits, 0 past the layer's experts (the mask is all ones where
    // lane + 64 j < E); the table and last-miss values past E are never
    // read, as every pick is an expert of the layer
    uint32_t v[NJ];
    const int past = lane - E;
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = route_dev::order_bits(z[j]) & (uint32_t)((past + 64 * j) >> 31);
    // lane i < k ends with pick i's order bits (the weight needs them all)
    uint32_t my_bits = 0;
    int e;
    if (a.k <= 8) {
      uint32_t top[8];
      route_dev::wave_top8(v, top);
      uint32_t bits;
      e = route_dev::top8_expert(v, top, pick, E, bits);
#pragma unroll
      for (int i = 0; i < 8; ++i) my_bits = lane == i ? top[i] : my_bits;
    } else {
      route_dev::WaveTopK<NJ> tk;
      tk.init_bits(v);
      int my_e;
      route_dev::wave_topk_rounds(tk, E, policy_wave ? a.k : pick + 1, lane, my_e, my_bits);
      e = __builtin_amdgcn_readlane(my_e, pick);
    }
    int slot_l = -1;
    uint32_t lm_l = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      slot_l = j == (e >> 6) ? tb[j] : slot_l;
      lm_l = j == (e >> 6) ? lm[j] : lm_l;
    }
    const int slot = __builtin_amdgcn_readlane(slot_l, e & 63);
    const uint32_t prev = (uint32_t)__builtin_amdgcn_readlane((int)lm_l, e & 63);
    // the cache step admits a cold pick on its first miss, or on a repeat
    // inside the window (a repeat earlier in this same step is not seen here)
    const bool hot = slot >= 0;
    const bool capture = !hot && may_capture && r.S > 0 &&
                         (r.admit_misses == 1 || (prev != 0 && clk - prev < (uint32_t)r.window));
    if (lane == 0) s_pick[0] = e, s_pick[1] = slot, s_pick[2] = capture ? 1 : 0;
    if (policy_wave) {
      const float wl = route_dev::wave_pick_weight(my_bits, a.k, lane);
      const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), pick));
      if (lane == 0) {
        uint64_t rec = ((uint64_t)clk << 32) | ((uint64_t)r.layer << 12) | (uint64_t)e;
        if (hot) {
          rec |= kRecordHit;
          atomicMax(&r.stamps[slot], clk);
        }
        r.records[p] = rec;
        atomicAdd(&r.counts[e], 1u);
        r.ids[p] = e;
        r.w[p] = w;
        r.addr[p] = hot ? r.pool + (int64_t)slot * r.expert_bytes : r.host + (int64_t)e * r.expert_bytes;
        r.kind[p] = hot ? kHot : (capture ? (uint8_t)(kCold | kCaptured) : kCold);
        // the directory entry names what block p will hold after this forward
        if (capture) r.cap_dir[p] = ((uint64_t)clk << 32) | (uint64_t)e;
        if (r.ids_user) r.ids_user[p] = e;
        if (r.w_user) r.w_user[p] = w;
        if (p == 0) atomicMax(&r.ctrl->step_tokens, (uint32_t)r.T);
      }
    }
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(s_pick[0]);
  const int slot = __builtin_amdgcn_readfirstlane(s_pick[1]);
  const bool capture = __builtin_amdgcn_readfirstlane(s_pick[2]) != 0;
  const bool hot = slot >= 0;
  const uint8_t* base = hot ? r.pool + (int64_t)slot * r.expert_bytes : r.host + (int64_t)e * r.expert_bytes;

  if (r.pub_seq && blockIdx.x == gridDim.x - 1) {
    // the host threads compute the cold picks: the last work-group of each
    // pick only hands the pick over (so no GEMV wave waits on host writes).
    // System-scope stores write through the caches to host memory; once they
    // are acknowledged the flag follows them. No cache-wide write-back (a
    // system-scope release would write back all of L2).
    if (wave == 0) {
      if (pick == 0) {
        const uint64_t* src = reinterpret_cast<const uint64_t*>(a.x + (int64_t)t * a.H);
        uint64_t* dst = reinterpret_cast<uint64_t*>(r.pub_x + (int64_t)t * a.H);
        for (int i = lane; i < a.H / 2; i += 64)
          __hip_atomic_store(dst + i, src[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      }
      if (lane == 0) {  // the routing weight stays here: the host answers unweighted outputs
        __hip_atomic_store(&r.pub_e[p], e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        __hip_atomic_store(&r.pub_kind[p], hot ? 0 : 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      if (lane == 0) __hip_atomic_store(&r.pub_seq[p], r.pub_value, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
    }
    return;
  }
  if (!wanted<MODE>(hot ? kHot : kCold)) return;

  const int row0 = blockIdx.x * ROWS_WG + wave * NIT * RPW + rg;
  RowTile<LPR, BPL, NIT> g, u;
  load_gateup(g, u, base, a.lay, row0, a.F, lb, !hot);
  // the lane's activation slice from LDS (blocks lb + LPR j), with the
  // per-block sums of the -8 offset, added in the order load_slice uses
  float xs[BPL][32], sx[BPL];
#pragma unroll
  for (int j = 0; j < BPL; ++j) {
    const int b = lb + LPR * j;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 q = s_x[b * 8 + (c ^ (b & 7))];
      xs[j][4 * c + 0] = q.x, xs[j][4 * c + 1] = q.y, xs[j][4 * c + 2] = q.z, xs[j][4 * c + 3] = q.w;
      s += (q.x + q.y) + (q.z + q.w);
    }
    sx[j] = s;
  }
  gateup_store<LPR, BPL, NIT>(g, u, xs, sx, row0, lb, a.F, a.out + (int64_t)p * a.F);
  // after the arithmetic, so the loads are consumed as they arrive
  if (capture) {
    uint8_t* cap = a.capture + (int64_t)p * a.lay.bytes;
    g.store(reinterpret_cast<uint4*>(cap + a.lay.gate_nib), reinterpret_cast<uint16_t*>(cap + a.lay.gate_scl), row0,
            a.F, lb);
    u.store(reinterpret_cast<uint4*>(cap + a.lay.up_nib), reinterpret_cast<uint16_t*>(cap + a.lay.up_scl), row0, a.F,
            lb);
  }
}

// ---------------------------------------------------------------------------
// gate/up GEMV + SwiGLU for the picks tagged `want`. grid = (row chunks of F,
// picks); 4 waves per group, each NIT row groups of 64/LPR rows.
template <int LPR, int BPL, int NIT, int MODE>
__global__ __launch_bounds__(256) void gemv_gateup_kernel(GemvArgs a) {
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS_WG = 4 * NIT * RPW;
  const int p = blockIdx.y;
  if (!wanted<MODE>(a.kind[p])) return;
  const int t = p / a.k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lb = lane % LPR, rg = lane / LPR;
  const uint8_t* base = a.addr[p];
  const bool cold = (a.kind[p] & kCold) != 0;
  const int row0 = blockIdx.x * ROWS_WG + wave * NIT * RPW + rg;
  RowTile<LPR, BPL, NIT> g, u;
  load_gateup(g, u, base, a.lay, row0, a.F, lb, cold);
  float xs[BPL][32], sx[BPL];
  load_slice<LPR, BPL>(a.x + (int64_t)t * a.H, lb, xs, sx);
  gateup_store<LPR, BPL, NIT>(g, u, xs, sx, row0, lb, a.F, a.out + (int64_t)p * a.F);
}


// ---------------------------------------------------------------------------
// down GEMV of the hot picks: y_pick[p] = W_down h[p]. grid = (row chunks of
// H, picks).
template <int LPR, int BPL, int NIT, int MODE>
__global__ __launch_bounds__(256) void gemv_down_pick_kernel(GemvArgs a) {
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS_WG = 4 * NIT * RPW;
  const int p = blockIdx.y;
  // the arguments in one scalar fetch at entry, then the pick's tag and
  // expert address in one round trip (the address fetched after the tag
  // test would be a second one ahead of the weight loads)
  asm volatile("" ::"s"(a.kind), "s"(a.addr), "s"(a.x), "s"(a.ypick), "s"(a.H), "s"(a.F), "s"(a.lay.down_nib),
               "s"(a.lay.down_scl));
  const int kd = a.kind[p];
  const uint8_t* base = a.addr[p];
  asm volatile("" ::"v"(kd), "s"(base));
  if (!wanted<MODE>((uint8_t)kd)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lb = lane % LPR, rg = lane / LPR;
  const int row0 = blockIdx.x * ROWS_WG + wave * NIT * RPW + rg;
  // the pick's h row in LDS, once per work-group (with LPR < 64 every row
  // group of a wave would load it again), the work-group sharing the copy,
  // its loads issued before the weight loads
  using V = SwizVec<LPR, BPL, 256>;
  __shared__ float4 hsh[V::KV];
  V hv;
  hv.load(a.x + (int64_t)p * a.F, threadIdx.x);
  RowTile<LPR, BPL, NIT> d;
  d.load(reinterpret_cast<const uint4*>(base + a.lay.down_nib),
         reinterpret_cast<const uint16_t*>(base + a.lay.down_scl), row0, a.H, lb);
  hv.store(hsh, threadIdx.x);
  __syncthreads();
  float hs[BPL][32], sh[BPL];
  V::slice(hsh, lb, hs, sh);
  down_store<LPR, BPL, NIT>(d, hs, sh, row0, lb, a.H, a.ypick + (int64_t)p * a.H);
}

// ---------------------------------------------------------------------------
// down GEMV of the cold picks + weighted combine of every pick. grid = (row
// chunks of H, tokens); the kCombineWaves waves take picks wave, wave +
// kCombineWaves, ... of the token over the same rows (at top-8 one pick per
// wave, every pick's loads in flight at once); hot picks come from y_pick.
// Sum in pick order.
constexpr int kCombineWaves = 8;

// One pick's down rows for gemv_down_combine_kernel, into part[i].
// Hot picks (PACE false) stage the h row through registers, its loads issued
// before the weight loads, so each row's arithmetic waits for that row only.
// Cold picks pace their zero-copy reads with explicit waits, next to which the
// compiler kept a register-staged row in scratch memory; they are bound by
// PCIe anyway and stage h by the LDS-DMA copy, issued after their weights.
template <int LPR, int BPL, int NIT, bool PACE, bool STAGE>
__device__ __forceinline__ void down_pick_rows(const GemvArgs& a, int64_t p, int i, int row0, int lane,
                                               float4* hsh, float (*part)[NIT * (64 / LPR)]) {
  constexpr int RPW = 64 / LPR;
  using V = SwizVec<LPR, BPL>;
  using D = SharedVec<LPR, BPL>;
  const int lb = lane % LPR, rg = lane / LPR;
  const uint8_t* base = a.addr[p];
  V hv;
  if (STAGE && !PACE) hv.load(a.x + p * a.F, lane);
  RowTile<LPR, BPL, NIT> d;
  d.load(reinterpret_cast<const uint4*>(base + a.lay.down_nib),
         reinterpret_cast<const uint16_t*>(base + a.lay.down_scl), row0 + rg, a.H, lb, PACE);
  float hs[BPL][32], sh[BPL];
  if (STAGE && !PACE) {
    hv.store(hsh, lane);
    V::slice(hsh, lb, hs, sh);
  } else if (STAGE) {
    D::issue(a.x + p * a.F, hsh, 0, 1, lane);
    D::wait_wave();
    D::slice(hsh, lb, hs, sh);
  } else {
    load_slice<LPR, BPL>(a.x + p * a.F, lb, hs, sh);
  }
  float pv[1][4], sv[1];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    pv[0][it] = d.partial(it, hs, sh);
    __builtin_amdgcn_sched_barrier(0);
  }
  reduce4_rows<LPR, 1>(pv, sv);
  if (lb < NIT) part[i][lb * RPW + rg] = sv[0];
  if ((a.kind[p] & kCaptured) && p < a.capture_picks) {  // after the arithmetic, as in the gate/up GEMV
    uint8_t* cap = a.capture + p * a.lay.bytes;
    d.store(reinterpret_cast<uint4*>(cap + a.lay.down_nib), reinterpret_cast<uint16_t*>(cap + a.lay.down_scl),
            row0 + rg, a.H, lb);
  }
}

template <int LPR, int BPL, int NIT, int MODE>
__global__ __launch_bounds__(64 * kCombineWaves) void gemv_down_combine_kernel(GemvArgs a) {
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS = NIT * RPW;
  __shared__ float part[32][ROWS];
  // each wave stages its pick's h row in LDS once (with LPR < 64 every row
  // group would load it again), while the 8 copies fit in 64 KiB
  using V = SwizVec<LPR, BPL>;
  constexpr bool kStage = V::KV <= 512;
  __shared__ float4 hsh[kStage ? kCombineWaves : 1][kStage ? V::KV : 1];
  // the arguments in one scalar fetch at entry (fetched where first used,
  // a second batch would be a dependent round trip ahead of the picks' tags
  // and addresses)
  asm volatile("" ::"s"(a.kind), "s"(a.addr), "s"(a.x), "s"(a.k), "s"(a.H), "s"(a.F), "s"(a.lay.down_nib),
               "s"(a.lay.down_scl), "s"(a.capture), "s"(a.capture_picks), "s"(a.ypick), "s"(a.w), "s"(a.out));
  const int t = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row0 = blockIdx.x * ROWS;
  for (int i = wave; i < a.k; i += kCombineWaves) {
    const int64_t p = (int64_t)t * a.k + i;
    if (!wanted<MODE>(a.kind[p])) continue;
    if (a.kind[p] & kCold)
      down_pick_rows<LPR, BPL, NIT, true, kStage>(a, p, i, row0, lane, hsh[kStage ? wave : 0], part);
    else
      down_pick_rows<LPR, BPL, NIT, false, kStage>(a, p, i, row0, lane, hsh[kStage ? wave : 0], part);
  }
  __syncthreads();
  for (int rr = threadIdx.x; rr < ROWS; rr += 64 * kCombineWaves) {
    const int r = row0 + rr;
    if (r >= a.H) continue;
    float acc = 0.f;
    for (int i = 0; i < a.k; ++i) {
      const int64_t p = (int64_t)t * a.k + i;
      const float v = wanted<MODE>(a.kind[p]) ? part[i][rr] : a.ypick[p * a.H + r];
      acc = fmaf(a.w[p], v, acc);
    }
    float* yp = a.out + (int64_t)t * a.H + r;
    *yp = a.accumulate ? *yp + acc : acc;
  }
}

// ---------------------------------------------------------------------------
// Grouped decode (batches of kGroupedMinTokens tokens or more).
//
// group_picks_kernel: one work-group counts the picks per expert in LDS,
// scans the counts, lists the experts with picks, cold experts first (their
// reads cross PCIe and take longest), then the largest groups (ties: lower
// expert), so the longest work-groups start first, and
// places every pick in its expert's range of `order` (the order inside a
// range is not fixed; every pick is computed on its own, so results do not
// depend on it).
__global__ __launch_bounds__(256) void group_picks_kernel(GroupArgs a) {
  __shared__ int32_t cnt[4096], fill[4096];
  __shared__ uint8_t hot[4096];
  __shared__ int32_t wsum[4], gwsum[4];
  __shared__ int4 lst[kMaxGroupsSorted];
  __shared__ __attribute__((aligned(16))) uint32_t keys[kMaxGroupsSorted + 4];
  const int tid = threadIdx.x;
  for (int e = tid; e < a.E; e += 256) cnt[e] = 0, hot[e] = a.tbl[e] >= 0;  // the table read overlaps the count
  __syncthreads();
  for (int p = tid; p < a.P; p += 256) atomicAdd(&cnt[a.ids[p]], 1);
  __syncthreads();
  // thread tid scans experts [tid * per, (tid + 1) * per)
  const int per = (a.E + 255) / 256, e0 = tid * per, e1 = min(a.E, e0 + per);
  int s = 0, gs = 0;
  for (int e = e0; e < e1; ++e) s += cnt[e], gs += cnt[e] > 0;
  // exclusive prefix sums of s and gs over the 256 threads: a shuffle scan
  // in each wave, then the wave totals (a serial scan by one thread was
  // 256 dependent LDS round trips, most of the kernel's time)
  int incl = s, gincl = gs;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o, 64), gv = __shfl_up(gincl, o, 64);
    if ((tid & 63) >= o) incl += v, gincl += gv;
  }
  if ((tid & 63) == 63) wsum[tid >> 6] = incl, gwsum[tid >> 6] = gincl;
  __syncthreads();
  int pos = incl - s, gi = gincl - gs, ng = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < (tid >> 6)) pos += wsum[w], gi += gwsum[w];
    ng += gwsum[w];
  }
  if (tid == 0) *a.n_groups = ng;
  const bool ranked = ng <= kMaxGroupsSorted;
  for (int e = e0; e < e1; ++e) {
    const int c = cnt[e];
    fill[e] = pos;
    if (c > 0) {
      if (ranked) {
        // sort key, smaller first: cold before hot, then more picks, then a lower expert (unique)
        keys[gi] = ((uint32_t)hot[e] << 31) | ((uint32_t)(8191 - min(c, 8191)) << 12) | (uint32_t)e;
        lst[gi] = make_int4(e, pos, c, 0);
      } else {
        a.groups[gi] = make_int4(e, pos, c, 0);  // too many to rank: expert order
      }
      ++gi;
    }
    pos += c;
  }
  if (ranked && tid < 4) keys[ng + tid] = 0xffffffffu;  // padding: ranks below no key
  __syncthreads();
  if (ranked) {
    // rank = keys below this group's: four keys per LDS read, the reads unrolled
    const uint4* k4 = reinterpret_cast<const uint4*>(keys);
    for (int g = tid; g < ng; g += 256) {
      const uint32_t me = keys[g];
      int rank = 0;
#pragma unroll 4
      for (int h = 0; h < (ng + 3) / 4; ++h) {
        const uint4 o = k4[h];
        rank += (o.x < me) + (o.y < me) + (o.z < me) + (o.w < me);
      }
      a.groups[rank] = lst[g];
    }
  }
  for (int p = tid; p < a.P; p += 256) a.order[atomicAdd(&fill[a.ids[p]], 1)] = p;
}

// Picks whose rows fit the work-group's LDS budget (64 KiB) at once, 1..16.
template <int LPR, int BPL>
constexpr int chunk_picks() {
  constexpr int n = 65536 / (16 * SharedVec<LPR, BPL>::KV);
  return n < 1 ? 1 : (n > 16 ? 16 : n);
}

// gate/up of one expert group: grid = (row chunks of F, up to P groups);
// the weight rows are loaded once and dotted with the activations of every
// pick of the group. The picks' rows pass through LDS, a chunk of them at a
// time (usually the whole group): one wait per chunk.
template <int LPR, int BPL, int NIT>
__global__ __launch_bounds__(256) void grouped_gateup_kernel(GemvArgs a, GroupArgs gr) {
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS_WG = 4 * NIT * RPW;
  using V = SharedVec<LPR, BPL>;
  constexpr int NB = chunk_picks<LPR, BPL>();
  __shared__ float4 xsh[NB][V::KV];
  if ((int)blockIdx.y >= *gr.n_groups) return;
  const int4 grp = gr.groups[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lb = lane % LPR, rg = lane / LPR;
  const int p0 = gr.order[grp.y];
  const uint8_t* base = a.addr[p0];
  const bool cold = (a.kind[p0] & kCold) != 0;
  const int row0 = blockIdx.x * ROWS_WG + wave * NIT * RPW + rg;
  RowTile<LPR, BPL, NIT> g, u;
  load_gateup(g, u, base, a.lay, row0, a.F, lb, cold);
#pragma unroll 1
  for (int c0 = 0; c0 < grp.z; c0 += NB) {
    const int nc = grp.z - c0 < NB ? grp.z - c0 : NB;
    for (int b = 0; b < nc; ++b) V::issue(a.x + (int64_t)(gr.order[grp.y + c0 + b] / a.k) * a.H, xsh[b], wave, 4, lane);
    V::wait();  // the chunk's rows (and, the first time, the weights) are in
    // one pick at a time: the weights stay in registers (packed)
#pragma unroll 1
    for (int b = 0; b < nc; ++b) {
      const int p = gr.order[grp.y + c0 + b];
      g.keep_packed();
      u.keep_packed();
      float xs[BPL][32], sx[BPL];
      V::slice(xsh[b], lb, xs, sx);
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        const float gv = row_reduce<LPR>(g.partial(it, xs, sx));
        const float uv = row_reduce<LPR>(u.partial(it, xs, sx));
        const int r = row0 + it * RPW;
        if (lb == 0 && r < a.F) a.out[(int64_t)p * a.F + r] = silu(gv) * uv;
      }
    }
    if (c0 + NB < grp.z) __syncthreads();  // everyone is done with the chunk before it is overwritten
  }
}

// down of one expert group: ypick[p] = W_down h[p] for every pick p of the
// group; grid = (row chunks of H, up to P groups); h rows through LDS as above.
template <int LPR, int BPL, int NIT>
__global__ __launch_bounds__(256) void grouped_down_kernel(GemvArgs a, GroupArgs gr) {
  constexpr int RPW = 64 / LPR;
  constexpr int ROWS_WG = 4 * NIT * RPW;
  using V = SharedVec<LPR, BPL>;
  constexpr int NB = chunk_picks<LPR, BPL>();
  __shared__ float4 hsh[NB][V::KV];
  if ((int)blockIdx.y >= *gr.n_groups) return;
  const int4 grp = gr.groups[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lb = lane % LPR, rg = lane / LPR;
  const int p0 = gr.order[grp.y];
  const uint8_t* base = a.addr[p0];
  const bool cold = (a.kind[p0] & kCold) != 0;
  const int row0 = blockIdx.x * ROWS_WG + wave * NIT * RPW + rg;
  RowTile<LPR, BPL, NIT> d;
  d.load(reinterpret_cast<const uint4*>(base + a.lay.down_nib),
         reinterpret_cast<const uint16_t*>(base + a.lay.down_scl), row0, a.H, lb, cold);
#pragma unroll 1
  for (int c0 = 0; c0 < grp.z; c0 += NB) {
    const int nc = grp.z - c0 < NB ? grp.z - c0 : NB;
    for (int b = 0; b < nc; ++b) V::issue(a.x + (int64_t)gr.order[grp.y + c0 + b] * a.F, hsh[b], wave, 4, lane);
    V::wait();
#pragma unroll 1
    for (int b = 0; b < nc; ++b) {
      const int p = gr.order[grp.y + c0 + b];
      d.keep_packed();
      float hs[BPL][32], sh[BPL];
      V::slice(hsh[b], lb, hs, sh);
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        const float v = row_reduce<LPR>(d.partial(it, hs, sh));
        const int r = row0 + it * RPW;
        if (lb == 0 && r < a.H) a.ypick[(int64_t)p * a.H + r] = v;
      }
    }
    if (c0 + NB < grp.z) __syncthreads();
  }
}

// y[t] (=|+=) sum over the picks of token t in pick order of w * ypick;
// grid = (chunks of 256 of H, tokens).
__global__ __launch_bounds__(256) void combine_picks_kernel(GemvArgs a) {
  const int t = blockIdx.y;
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= a.H) return;
  float acc = 0.f;
  for (int i = 0; i < a.k; ++i) {
    const int64_t p = (int64_t)t * a.k + i;
    acc = fmaf(a.w[p], a.ypick[p * a.H + r], acc);
  }
  float* yp = a.out + (int64_t)t * a.H + r;
  *yp = a.accumulate ? *yp + acc : acc;
}

// ---------------------------------------------------------------------------
// combine with the cold picks computed by the host threads. grid = (row
// chunks of 256 of H, tokens). A token with a cold pick waits (bounded) for
// the host's answer, polled by thread 0 of each group (a few groups: many
// pollers of one host line slow the host threads' memory); the sum runs in
// pick order like gemv_down_combine_kernel's. System-scope loads read host
// memory past the caches; no acquire (that would invalidate the caches on
// every poll).
__global__ __launch_bounds__(256) void host_combine_kernel(HostCombineArgs a) {
  __shared__ int answered;
  const int t = blockIdx.y;
  if (threadIdx.x == 0) {
    bool cold = false;
    for (int i = 0; i < a.k; ++i) cold |= (a.kind[(int64_t)t * a.k + i] & kCold) != 0;
    bool ok = true;
    if (cold) {
      uint32_t n = 0;
      uint64_t d = 0;
      for (; n < a.max_polls; ++n) {
        d = __hip_atomic_load(a.done, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        if ((int32_t)((uint32_t)d - a.seq) >= 0) break;
        __builtin_amdgcn_s_sleep(2);
      }
      ok = n < a.max_polls && (d >> 32) == 0;
      if (!ok) atomicOr(&a.ctrl->host_fault, 1u);
    }
    answered = ok;
  }
  __syncthreads();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= a.H) return;
  float acc = 0.f;
  for (int i = 0; i < a.k; ++i) {
    const int64_t p = (int64_t)t * a.k + i;
    float v;
    if (a.kind[p] & kCold)
      v = answered ? __hip_atomic_load(a.y_cold + p * a.H + r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM) : 0.f;
    else
      v = a.ypick[p * a.H + r];
    acc = fmaf(a.w[p], v, acc);
  }
  float* yp = a.y + (int64_t)t * a.H + r;
  *yp = a.accumulate ? *yp + acc : acc;
}

// ---------------------------------------------------------------------------
// launchers

hipError_t launch_host_combine(const HostCombineArgs& a, const Launch& l) {
  if (a.T < 1 || a.k < 1 || a.H < 1 || !a.done || !a.y_cold || !a.ctrl) return hipErrorInvalidValue;
  return launch(host_combine_kernel, dim3((a.H + 255) / 256, a.T), dim3(256), l, a);
}


bool gemv_shape(int kb, GemvShape* out) {
  if (kb <= 0) return false;
  int lpr = 1;
  while (lpr < 64 && (kb % (lpr * 2)) == 0) lpr *= 2;
  const int bpl = kb / lpr;
  if (lpr < 8 || bpl > 4) return false;
  out->lpr = lpr;
  out->bpl = bpl;
  return true;
}

namespace {
constexpr int kNitGateUp = 4;
constexpr int kNitDown = 4;
constexpr int kNitCombine = 4;

template <int LPR, int BPL>
hipError_t gateup_t(const GemvArgs& a, const Launch& l, int mode) {
  constexpr int ROWS_WG = 4 * kNitGateUp * (64 / LPR);
  const dim3 grid((a.F + ROWS_WG - 1) / ROWS_WG, a.T * a.k);
  if (mode == kOnlyHot) return launch(gemv_gateup_kernel<LPR, BPL, kNitGateUp, kOnlyHot>, grid, dim3(256), l, a);
  if (mode == kOnlyCold) return launch(gemv_gateup_kernel<LPR, BPL, kNitGateUp, kOnlyCold>, grid, dim3(256), l, a);
  return launch(gemv_gateup_kernel<LPR, BPL, kNitGateUp, kAll>, grid, dim3(256), l, a);
}
template <int LPR, int BPL>
hipError_t route_gateup_t(const GemvArgs& a, const RouteArgs& r, const Launch& l, int mode) {
  constexpr int ROWS_WG = 4 * kNitGateUp * (64 / LPR);
  // one more work-group per pick hands the pick to the host threads
  const dim3 grid((a.F + ROWS_WG - 1) / ROWS_WG + (r.pub_seq ? 1 : 0), a.k, a.T);
  if (mode == kOnlyHot)
    return launch(gemv_route_gateup_kernel<LPR, BPL, kNitGateUp, kOnlyHot>, grid, dim3(256), l, a, r);
  if (mode == kOnlyCold)
    return launch(gemv_route_gateup_kernel<LPR, BPL, kNitGateUp, kOnlyCold>, grid, dim3(256), l, a, r);
  return launch(gemv_route_gateup_kernel<LPR, BPL, kNitGateUp, kAll>, grid, dim3(256), l, a, r);
}
template <int LPR, int BPL>
hipError_t down_pick_t(const GemvArgs& a, const Launch& l, int mode) {
  constexpr int ROWS_WG = 4 * kNitDown * (64 / LPR);
  const dim3 grid((a.H + ROWS_WG - 1) / ROWS_WG, a.T * a.k);
  if (mode != kOnlyHot) return hipErrorInvalidValue;
  return launch(gemv_down_pick_kernel<LPR, BPL, kNitDown, kOnlyHot>, grid, dim3(256), l, a);
}
template <int LPR, int BPL>
hipError_t down_combine_t(const GemvArgs& a, const Launch& l, int mode) {
  constexpr int ROWS = kNitCombine * (64 / LPR);
  const dim3 grid((a.H + ROWS - 1) / ROWS, a.T);
  if (mode == kOnlyCold)
    return launch(gemv_down_combine_kernel<LPR, BPL, kNitCombine, kOnlyCold>, grid, dim3(64 * kCombineWaves), l, a);
  if (mode != kAll) return hipErrorInvalidValue;
  return launch(gemv_down_combine_kernel<LPR, BPL, kNitCombine, kAll>, grid, dim3(64 * kCombineWaves), l, a);
}

// grouped kernels: as many rows per wave as the per-pick GEMVs (measured at
// 60 layers, batch 32: 707 tokens/s, against 676 with half as many)
constexpr int kNitGrouped = 4;
template <int LPR, int BPL>
hipError_t grouped_gateup_t(const GemvArgs& a, const GroupArgs& g, const Launch& l, int) {
  constexpr int ROWS_WG = 4 * kNitGrouped * (64 / LPR);
  return launch(grouped_gateup_kernel<LPR, BPL, kNitGrouped>, dim3((a.F + ROWS_WG - 1) / ROWS_WG, g.P), dim3(256), l,
                a, g);
}
template <int LPR, int BPL>
hipError_t grouped_down_t(const GemvArgs& a, const GroupArgs& g, const Launch& l, int) {
  constexpr int ROWS_WG = 4 * kNitGrouped * (64 / LPR);
  return launch(grouped_down_kernel<LPR, BPL, kNitGrouped>, dim3((a.H + ROWS_WG - 1) / ROWS_WG, g.P), dim3(256), l,
                a, g);
}

#define MOE_DISPATCH_GEMV(FN, KB, ARGS, L, MODE, ...)         \
  do {                                                        \
    GemvShape sh;                                             \
    if (!gemv_shape((KB), &sh)) return hipErrorInvalidValue;  \
    switch (sh.lpr * 8 + sh.bpl) {                            \
      case 8 * 8 + 1: return FN<8, 1>(ARGS, ##__VA_ARGS__, L, MODE);         \
      case 8 * 8 + 2: return FN<8, 2>(ARGS, ##__VA_ARGS__, L, MODE);         \
      case 8 * 8 + 3: return FN<8, 3>(ARGS, ##__VA_ARGS__, L, MODE);         \
      case 8 * 8 + 4: return FN<8, 4>(ARGS, ##__VA_ARGS__, L, MODE);         \
      case 16 * 8 + 1: return FN<16, 1>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 16 * 8 + 2: return FN<16, 2>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 16 * 8 + 3: return FN<16, 3>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 16 * 8 + 4: return FN<16, 4>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 32 * 8 + 1: return FN<32, 1>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 32 * 8 + 2: return FN<32, 2>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 32 * 8 + 3: return FN<32, 3>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 32 * 8 + 4: return FN<32, 4>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 64 * 8 + 1: return FN<64, 1>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 64 * 8 + 2: return FN<64, 2>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 64 * 8 + 3: return FN<64, 3>(ARGS, ##__VA_ARGS__, L, MODE);       \
      case 64 * 8 + 4: return FN<64, 4>(ARGS, ##__VA_ARGS__, L, MODE);       \
      default: return hipErrorInvalidValue;                   \
    }                                                         \
  } while (0)
}  // namespace

hipError_t launch_gemv_gateup(const GemvArgs& a, const Launch& l, int mode) {
  MOE_DISPATCH_GEMV(gateup_t, a.H / 32, a, l, mode);
}
hipError_t launch_gemv_route_gateup(const GemvArgs& a, const RouteArgs& r, const Launch& l, int mode) {
  if (!r.logits || r.E < 1 || r.E > kFusedRouteMaxExperts || a.k < 1 || a.k > 32 || a.k > r.E || a.T < 1 ||
      a.T > 65535)
    return hipErrorInvalidValue;
  MOE_DISPATCH_GEMV(route_gateup_t, a.H / 32, a, l, mode, r);
}
hipError_t launch_group_picks(const GroupArgs& a, hipStream_t s) {
  if (a.P < 1 || a.E < 1 || a.E > 4096) return hipErrorInvalidValue;
  return launch(group_picks_kernel, dim3(1), dim3(256), Launch{s}, a);
}
hipError_t launch_grouped_gateup(const GemvArgs& a, const GroupArgs& g, const Launch& l) {
  if (g.P < 1) return hipErrorInvalidValue;
  MOE_DISPATCH_GEMV(grouped_gateup_t, a.H / 32, a, l, 0, g);
}
hipError_t launch_grouped_down(const GemvArgs& a, const GroupArgs& g, const Launch& l) {
  if (g.P < 1) return hipErrorInvalidValue;
  MOE_DISPATCH_GEMV(grouped_down_t, a.F / 32, a, l, 0, g);
}
hipError_t launch_combine_picks(const GemvArgs& a, const Launch& l) {
  if (a.T < 1 || a.k < 1 || a.H < 1) return hipErrorInvalidValue;
  return launch(combine_picks_kernel, dim3((a.H + 255) / 256, a.T), dim3(256), l, a);
}
hipError_t launch_gemv_down_pick(const GemvArgs& a, const Launch& l, int mode) {
  MOE_DISPATCH_GEMV(down_pick_t, a.F / 32, a, l, mode);
}
hipError_t launch_gemv_down_combine(const GemvArgs& a, const Launch& l, int mode) {
  if (a.k > 32) return hipErrorInvalidValue;
  MOE_DISPATCH_GEMV(down_combine_t, a.F / 32, a, l, mode);
}

}  // namespace moe
