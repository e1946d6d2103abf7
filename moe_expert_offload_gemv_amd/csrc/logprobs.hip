// logprobs.hip - what a row of an output head's logits says: the log probability
// of a given token, the entropy, the most likely tokens (moe_token_logprobs), and the
// gradient of the first two to the logits (moe_token_logprobs_grad).
//
//   logprob_rows_kernel    a row, or a slice of it, once: maximum, sum of e^(z - max), sum of
//                          e^(z - max) (z - max), and the top_n largest of it
//   logprob_finish_kernel  the slices of a row put together (few rows: they are cut into slices)
//   logprob_grad_kernel    logits once more: dlogits
//
// Bound by traffic, one read of the logits: a thread keeps a running maximum and both sums
// over 16 values at a time, the next 16 on their way, in powers of two; 11 issue slots a value of which the
// power takes four, so that 16-bit logits are nearly as long in the vector unit as on their way. Rows are cut
// into slices, if they are long and few, while all of them fit on the chip at once.
//
// The top_n largest come out of the same read. A thread also notes the largest of its values in LDS.
// The top_n-th largest of the threads' maxima is a bound that top_n values reach at least (taken in
// each wave, and the best wave's); the few runs whose largest reaches it are read again, from
// cache, and what reaches it in them, about two or three times top_n values, is ranked by counting; more, where values
// lie close together or far from zero, are cut to a few by their bits first. Equal
// values: a token's rank counts equal ones of lower id, so ties go to the lower id whatever
// the order in which the values were found.
//
// Measured (as nodes of a graph): 4096 x 65537 bf16, 537 MB, 122 us = 4.4 TB/s, with its gradient, 1074 MB more, 311 = 5.2
// TB/s; 4096 x 32000 fp32 93 = 5.6 TB/s; 301 x 131072 bf16 with 8 alternatives 27.7 (floor 15: finding them takes 5, the
// finishing launch 5); 4096 x 8000 bf16 18.6, with 20 alternatives 39.7 (to find them is four times the work of the
// sums there: a bound, a second look and ranks for 8000 values); 1 x 65537 fp32 with 20, 12.5: two launches of a few dependent
// trips to memory and LDS each, 5.5 without alternatives; around 1000 instead of 0, 2000 x 8000 fp32 with 20 takes 67 and
// 32 x 32000 62, for the bound's 16 bits then tell little apart.
// Measured and not kept: the search by one wave of the work-group (1 x 65537 with 20: 18); an atomic for all hits of
// a thread at once (4096 x 8000: 55 against 45, the compiler's scan over the lanes); loads past the caches (4096 x 32000
// fp32 97 against 91).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"
#include "route_dev.h"
#include "value_dev.h"

namespace moe {
namespace {

using namespace value_dev;

constexpr float kLog2e = 1.44269504089f;
constexpr float kLowest = -3.4028234664e38f, kMinusInf = -__builtin_inff();
// powers below this are 0 in fp32; a finite floor keeps 0 * (z - max) a zero where z is -inf
constexpr float kFloor = -200.0f;
constexpr int kULog = 1, kU = 1 << kULog;  // runs of 8 values of a thread, loaded at once
constexpr int kNotes = 8;          // noted maxima of a thread
constexpr int kSliceStep = 2048;   // slices are whole multiples
constexpr int kMaxSlices = 64;
constexpr int kSliceTarget = 1024; // rows times slices at most: four work-groups a CU, all of them at once
constexpr int kWaveRow = 2048;     // rows up to this long have one wave
// Rows up to this long are not cut: a work-group a row in one launch, against a work-group a slice, a second launch to join
// them and, with alternatives, a second search. Few rows leave CUs idle, so the more rows there are the longer they may be.
// With alternatives the limit could lie higher and without them lower; it is one, so that what else is said of a row has
// the same bits with and without them. us cut and uncut, without alternatives bf16, fp32, with 8 bf16, fp32:
//     1 row    24000   5.7  5.5   5.6  5.4  10.5  9.5  10.4  9.4
//              40000   5.7  6.6   5.4  6.5  10.3 10.7  10.2 10.3
//    32 rows   32000   6.4  6.4   6.4  6.4  11.6 10.9  11.6 10.6
//              65537   6.7  8.8   7.0  8.8  12.6 13.5  12.6 13.0
//    64        40000   6.9  7.0   7.8  8.0  13.1 11.4  13.8 11.6
//              80000   8.7 10.8  10.5 13.3  15.1 15.5  16.5 15.8
//   128        65537  10.6 10.6  12.6 11.9  17.2 14.9  19.1 15.1
//             131072  12.4 15.4  16.4 18.8  18.9 19.8  22.5 20.9
//   200        80000  12.4 12.9  16.4 14.6  19.3 16.6  23.1 17.8
//             262144  28.2 41.9  48.0 59.4  35.0 45.7  54.1 61.1
//   301       131072  19.4 21.8  37.5 32.9  27.4 27.6  43.5 36.3
//             262144  40.1 52.0  72.1 73.3  47.3 55.1  79.6 69.5
// From one and a half rows a CU on they are not cut at any length:
//   400       262144  51.7 54.6  98.7 78.9  59.4 61.4   107 84.1
//   512       262144  60.1 54.9   109 98.9  69.8 59.7   115  106
constexpr int kWholeRow = 32768, kWholeRowMore = 300;  // and more for each row
constexpr int kMostCut = 384;                          // rows of which no length is cut

// Maximum, sum of 2^((x - max) c) and of the same times (x - max) c. The sums of a row are held in 64 bits: beside a
// confident word, which is 1, the others are far below 2^-24 each, and their mass is what its log probability says. In 32
// bits the thread that holds that word would drop its share of them, an error that grows with the row. Runs of 16 values
// are summed in 32 bits first, so that 64 bits cost some ten instructions for 16 values; such a run is off by
// a few roundings of itself at most.
struct Sums {
  float m;
  double s, u;
};
// the sums of `a` referred to the maximum m >= a.m, and others of that maximum added
__device__ __forceinline__ void refer(Sums& a, float m, float c, float s = 0.f, float u = 0.f) {
  const float d = fmaxf((a.m - m) * c, kFloor);
  const double f = __builtin_amdgcn_exp2f(d);
  a.u = fma(f, fma(a.s, (double)d, a.u), (double)u);
  a.s = fma(f, a.s, (double)s);
  a.m = m;
}
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = route_dev::dpp32<CTRL>((uint32_t)b), hi = route_dev::dpp32<CTRL>((uint32_t)(b >> 32));
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Both sums of the lanes, in every lane: even lanes go on with one of them and odd ones with the other
__device__ __forceinline__ void wave_sums(Sums& t) {
  using namespace route_dev;
  constexpr int kRowRor4 = 0x124, kRowRor8 = 0x128;  // rotations within 16 lanes
  const bool odd = threadIdx.x & 1;
  double v = (odd ? t.u : t.s) + dpp64<kDppQuadXor1>(odd ? t.s : t.u);
  v += dpp64<kDppQuadXor2>(v);
  v += dpp64<kRowRor4>(v);
  v += dpp64<kRowRor8>(v);
  t.s = (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
  t.u = (lane_value(v, 1) + lane_value(v, 17)) + (lane_value(v, 33) + lane_value(v, 49));
}

__device__ __forceinline__ uint32_t key_of(float v) { return route_dev::order_bits(v); }

// 8 logits from logit i of a row on (below 2^22 of them): a 32-bit offset from the row's address
template <int ZT>
__device__ __forceinline__ Raw8<ZT> load_run(const char* row, int i) {
  return load8<ZT>(row + (uint32_t)i * (uint32_t)value_size<ZT>(), 0);
}
// The logits i .. i + 7 of those before `end`, in one load: where fewer are left, the last 8, with -inf
// in the place of those before i. v[j] is logit base + j; returns base.
template <int ZT>
__device__ __forceinline__ int load_logits(const char* row, int i, int end, float (&v)[8]) {
  if (end < 8) {  // the same for the work-group
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < end ? load1<ZT>(row, i + j) : kMinusInf;
    return i;
  }
  const int base = min(i, end - 8), skip = i - base;
  unpack8<ZT>(load_run<ZT>(row, base), v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j >= skip ? v[j] : kMinusInf;
  return base;
}

// what a row's sums say of it
struct RowResult {
  float m, log_sum;
  bool none, bad;  // every logit -inf; a NaN, or a logit of +inf
};
__device__ __forceinline__ RowResult row_result(const Sums& t, float most, float scale) {
  RowResult r;
  const float z = t.m * scale;
  r.bad = !(t.s == t.s) || z == __builtin_inff();
  r.none = !r.bad && (most == kMinusInf || z == kMinusInf);
  r.m = t.m;
  // the logarithm of both halves of the sum: 1 and a little must not become 1
  const float hi = (float)t.s;
  r.log_sum = fmaf((float)(t.s - hi), __builtin_amdgcn_rcpf(hi), logf(hi));
  return r;
}
constexpr uint32_t kNan = 0x7FC00000u;

// A row's outputs, by one thread: in 64 bits, for the gradient's p are e^(z - lse), and a
// rounding of lse would scale them all. lse is handed on in two floats.
template <int ZT>
__device__ __forceinline__ void put_row(const LogprobArgs& a, int64_t row, const Sums& t, const RowResult& r) {
  const double log_sum = log(t.s), scale = a.scale, lse = t.m * scale + log_sum;
  const float nan = __uint_as_float(kNan);
  if (a.logp) {
    const int64_t y = a.targets[row];
    float v = 0.f;
    if (y >= 0 && y < a.V) {
      const float x = load1<ZT>(static_cast<const char*>(a.logits) + row * a.z_stride * value_size<ZT>(), y);
      v = r.bad ? nan : r.none ? kMinusInf : (float)(((double)x - t.m) * scale - log_sum);
    }
    a.logp[row] = v;
  }
  if (a.entropy) {
    const float h = (float)(log_sum - t.u / t.s * 0.69314718055994530942);
    a.entropy[row] = r.bad ? nan : r.none ? 0.f : fmaxf(h, 0.f);
  }
  if (a.lse) {
    const float hi = r.bad ? nan : r.none ? kMinusInf : (float)lse;
    a.lse[2 * row] = hi;
    a.lse[2 * row + 1] = r.bad || r.none ? 0.f : (float)(lse - hi);
  }
}
// log probability of a row's value above -inf. By way of halves: the difference of two logits may pass fp32's range
// where scale times it does not.
__device__ __forceinline__ float row_logp(const RowResult& r, float x, float scale) {
  return fmaf(0.5f * x - 0.5f * r.m, 2.0f * scale, -r.log_sum);
}

// Ranks `count` candidates (value, id) and hands each with its rank to f; every thread of the
// work-group comes here. The order of the candidates has no part in the ranks. Four lanes share a
// candidate and compare it with every fourth, four at a time (the array holds whole sixteens).
struct Candidate {
  uint32_t key;
  int id;
};
template <int THREADS, typename F>
__device__ __forceinline__ void rank_candidates(const Candidate* s_c, int count, F f) {
  const int whole_waves = (4 * count + 63) & ~63;
#pragma unroll 1
  for (int e = threadIdx.x; e < whole_waves; e += THREADS) {
    const int i = e >> 2;
    const Candidate me = s_c[min(i, count - 1)];
    uint32_t rank = 0;
#pragma unroll 1
    for (int j0 = e & 3; j0 < count; j0 += 16) {
      Candidate o[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = s_c[j0 + 4 * r];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        rank += j0 + 4 * r < count && (o[r].key > me.key || (o[r].key == me.key && o[r].id < me.id));
    }
    rank += route_dev::dpp32<route_dev::kDppQuadXor1>(rank);
    rank += route_dev::dpp32<route_dev::kDppQuadXor2>(rank);
    if ((e & 3) == 0 && i < count) f(me, (int)rank);
  }
}

// A key that at least n of the wave's lanes reach: the largest such one but for its last 16 bits
__device__ __forceinline__ uint32_t nth_of_lanes(uint32_t key, int n) {
  uint32_t bound = 0;
#pragma unroll 1
  for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1)
    if (__popcll(__ballot(key >= (bound | bit))) >= n) bound |= bit;
  return bound;
}

__device__ __forceinline__ float quad_max(float v) {
  using namespace route_dev;
  v = fmaxf(v, __uint_as_float(dpp32<kDppQuadXor1>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(dpp32<kDppQuadXor2>(__float_as_uint(v))));
}
__device__ __forceinline__ float wave_max(float v) {
  using namespace route_dev;
  v = quad_max(v);
  v = fmaxf(v, __uint_as_float(dpp32<kDppRowHalfMirror>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp32<kDppRowMirror>(__float_as_uint(v))));
  const int u = __float_as_int(v);
  const float a = __int_as_float(__builtin_amdgcn_readlane(u, 0)), b = __int_as_float(__builtin_amdgcn_readlane(u, 16));
  const float c = __int_as_float(__builtin_amdgcn_readlane(u, 32)), d = __int_as_float(__builtin_amdgcn_readlane(u, 48));
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// The top_n best of `count` candidates, ranked. Counting takes their number squared: more than a few are
// first cut to a few that have the best among them (64 x 131072 with 32 alternatives, slices of 8192: 21.5 us
// and 15.4).
constexpr int kFew = 64;
struct Few {
  Candidate c[kFew];
  int n;
};
// The least candidate of such a few, by key, then by the higher id: bits of the key until those that reach it are few,
// and where equal keys are too many for that, bits of the id. PER candidates lie in a lane; every wave finds it for itself.
template <int PER>
__device__ __forceinline__ Candidate least_of_few(const Candidate* s_c, int count, int top_n) {
  const int lane = threadIdx.x & 63;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = lane + 64 * i < count ? s_c[lane + 64 * i].key : 0u;
  Candidate least{0u, 0x7FFFFFFF};
  int reached = count;
#pragma unroll 1
  for (uint32_t bit = 1u << 31; bit && reached > kFew; bit >>= 1) {
    int many = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) many += __popcll(__ballot(key[i] >= (least.key | bit)));
    if (many >= top_n) least.key |= bit, reached = many;
  }
  if (reached <= kFew) return least;
  int id[PER], missing = top_n;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    missing -= __popcll(__ballot(key[i] > least.key));
    id[i] = key[i] == least.key ? s_c[lane + 64 * i].id : 0x7FFFFFFF;
  }
  least.id = (1 << 22) - 1;  // no id is above
#pragma unroll 1
  for (int bit = 1 << 21; bit; bit >>= 1) {
    int many = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) many += __popcll(__ballot(id[i] <= least.id - bit));
    if (many >= missing) least.id -= bit;
  }
  return least;
}
template <int THREADS, int MOST, typename F>
__device__ __forceinline__ void rank_top(const Candidate* s_c, int count, int top_n, Few& s_few, F f) {
  if (count > kFew) {
    const Candidate least = count <= 256 ? least_of_few<4>(s_c, count, top_n) : least_of_few<MOST / 64>(s_c, count, top_n);
    if (threadIdx.x == 0) s_few.n = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < count; i += THREADS) {
      const Candidate me = s_c[i];
      if (me.key > least.key || (me.key == least.key && me.id <= least.id)) s_few.c[atomicAdd(&s_few.n, 1)] = me;
    }
    __syncthreads();
    s_c = s_few.c, count = s_few.n;
  }
  rank_candidates<THREADS>(s_c, count, f);
}

// The top_n largest values above -inf of a slice, [begin, end) of a row, whose threads' maxima are `most` and
// whose noted maxima lie in s_note: into s_c, unordered, at most kCand of them; returns how many.
template <int THREADS>
struct Top {
  static constexpr int kCand = THREADS * 4 > 512 ? 1024 : 512;
  float note[kNotes][THREADS];
  uint16_t list[kNotes * THREADS];
  Candidate c[kCand];
  int n_list, n_c;
  Few few;
  uint32_t bound[THREADS / 64];
  int before[THREADS / 64 + 1];
};
template <int ZT, int THREADS>
__device__ int find_top(Top<THREADS>& s, const char* row, int begin, int end, float most, int top_n, int iters, int note_log) {
  constexpr int W = THREADS / 64;
  constexpr uint32_t kNothing = 0x007FFFFFu;  // key_of(-inf)
  const int tid = threadIdx.x, wave = tid >> 6;
  uint32_t bound = nth_of_lanes(key_of(most), top_n);
  if ((tid & 63) == 0) s.bound[wave] = bound;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) bound = max(bound, s.bound[w]);
  const int notes = (iters + (1 << note_log) - 1) >> note_log;
  constexpr int kIter = THREADS * 8 * kU;
  auto push = [&](uint32_t t, int i) __attribute__((always_inline)) {
    float v[8];
    const int first = load_logits<ZT>(row, i, end, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t k = key_of(v[j]);
      if (k < t) continue;
      const int at = atomicAdd(&s.n_c, 1);
      if (at < Top<THREADS>::kCand) s.c[at] = Candidate{k, first + j};
    }
  };
  // all values of keys >= t, as many as there is room for; returns how many there are
  auto gather = [&](uint32_t t) {
    __syncthreads();
    if (tid == 0) s.n_list = s.n_c = 0;
    __syncthreads();
    if (iters == 1) {
      // a thread's values are still in its CU's cache
      if (key_of(most) >= t) {
#pragma unroll 1
        for (int i = begin + tid * 8; i < end; i += THREADS * 8) push(t, i);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < notes; ++i)
        if (key_of(s.note[i][tid]) >= t) s.list[atomicAdd(&s.n_list, 1)] = (uint16_t)(i * THREADS + tid);
      __syncthreads();
      const int log = note_log + kULog, items = s.n_list << log;
#pragma unroll 1
      for (int e = tid; e < items; e += THREADS) {
        const int note = s.list[e >> log], r = e & ((1 << log) - 1), it = (note / THREADS << note_log) + r / kU;
        const int i = begin + it * kIter + ((r % kU) * THREADS + note % THREADS) * 8;
        if (i < end) push(t, i);
      }
    }
    __syncthreads();
    return s.n_c;
  };
  uint32_t t = max(bound, kNothing + 1);
  int count;
  bool above = false;  // without the values equal to the bound
  for (;;) {
    count = gather(t + above);
    if (count <= Top<THREADS>::kCand) break;
    // More than there is room for. Without the values equal to the bound (a mask's lowest value, say)?
    if (!above) {
      above = true;
      continue;
    }
    // still: a key that top_n of those that found room reach, but few, is a higher bound
    t = least_of_few<Top<THREADS>::kCand / 64>(s.c, Top<THREADS>::kCand, top_n).key;
    above = false;
  }
  if (!above) return count;
  // those above the bound, and of those equal to it the first ones, in order
  for (int it = 0; it < iters && count < top_n; ++it) {
    if (!__syncthreads_or(key_of(iters == 1 ? most : s.note[it >> note_log][tid]) >= t)) continue;
#pragma unroll 1
    for (int r = 0; r < kU && count < top_n; ++r) {
      const int i = begin + it * kIter + (r * THREADS + tid) * 8;
      float v[8];
      const int first = load_logits<ZT>(row, i, end, v);
      int mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += key_of(v[j]) == t;
      int upto = mine;  // over the lanes up to this one
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int other = __shfl_up(upto, o, 64);
        upto += (tid & 63) >= o ? other : 0;
      }
      __syncthreads();
      if ((tid & 63) == 63) s.before[wave] = upto;
      __syncthreads();
      int all = 0, at = count + upto - mine;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w < wave) at += s.before[w];
        all += s.before[w];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (key_of(v[j]) == t) {
          if (at < top_n) s.c[at] = Candidate{t, first + j};
          ++at;
        }
      count = min(count + all, top_n);
    }
  }
  __syncthreads();
  return count;
}

// One work-group per row or slice, in turn. TOP: the largest are asked for.
template <int ZT, int THREADS, bool TOP>
__global__ __launch_bounds__(THREADS, TOP ? 4 : ZT == MOE_F32 ? 6 : 8) void logprob_rows_kernel(LogprobArgs a) {
  constexpr int W = THREADS / 64;
  constexpr int kIter = THREADS * 8 * kU;
  __shared__ Top<TOP ? THREADS : 64> s_top;
  __shared__ Sums s_sum[W];
  __shared__ float s_most[W];
  const int tid = threadIdx.x;
  const float c = a.scale * kLog2e;
  for (int64_t item = blockIdx.x; item < a.T * a.slices; item += gridDim.x) {
    const int64_t row = item / a.slices;
    const int slice = (int)(item - row * a.slices);
    const char* z = static_cast<const char*>(a.logits) + row * a.z_stride * value_size<ZT>();
    const int begin = slice * (int)a.slice, end = min(begin + (int)a.slice, (int)a.V);
    const int iters = (end - begin + kIter - 1) / kIter;
    Sums t{kLowest, 0.0, 0.0};
    float most = kMinusInf, noted = kMinusInf;
    Raw8<ZT> raw[kU];
    auto fetch = [&](int at) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < kU; ++r) raw[r] = load_run<ZT>(z, at + r * THREADS * 8);
    };
    // maximum and sums of the first `runs` runs of v
    auto add = [&](const float (&v)[kU][8], int runs) __attribute__((always_inline)) {
      float m = kMinusInf;
#pragma unroll
      for (int r = 0; r < kU; ++r) {
        if (r >= runs) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, v[r][j]);
      }
      most = fmaxf(most, m);
      noted = fmaxf(noted, m);
      m = fmaxf(t.m, m);
      float s = 0.f, u = 0.f;
#pragma unroll
      for (int r = 0; r < kU; ++r) {
        if (r >= runs) break;
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = (v[r][j] - m) * c;
          e[j] = __builtin_amdgcn_exp2f(d);
          u = fmaf(e[j], fmaxf(d, kFloor), u);
        }
        s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      }
      refer(t, m, c, s, u);
    };
    auto note = [&](int it) __attribute__((always_inline)) {
      if constexpr (TOP)
        if (((it + 1) & ((1 << a.note_log) - 1)) == 0 || it + 1 == iters) {
          s_top.note[it >> a.note_log][tid] = noted;
          noted = kMinusInf;
        }
    };
    const int whole = (end - begin) / kIter;
    if (whole) fetch(begin + tid * 8);
    int it = 0;
#pragma unroll 1
    for (; it < whole; ++it) {
      float v[kU][8];
#pragma unroll
      for (int r = 0; r < kU; ++r) unpack8<ZT>(raw[r], v[r]);
      // the next values on their way, those of the last ones again behind them
      fetch(begin + min(it + 1, whole - 1) * kIter + tid * 8);
      add(v, kU);
      note(it);
    }
    if (it < iters) {
      float v[kU][8];
      const int at = begin + it * kIter;
#pragma unroll
      for (int r = 0; r < kU; ++r) load_logits<ZT>(z, at + (r * THREADS + tid) * 8, end, v[r]);
      add(v, (end - at + THREADS * 8 - 1) / (THREADS * 8));
      note(it);
    }
    // over the lanes, then the waves in their order
    refer(t, wave_max(t.m), c);
    wave_sums(t);
    float wave_most = wave_max(most);
    if constexpr (W > 1) {
      __syncthreads();  // the item before has been read
      if ((tid & 63) == 0) s_sum[tid >> 6] = t, s_most[tid >> 6] = wave_most;
      __syncthreads();
      static_assert(W == 4, "a lane of each quad per wave");
      t = s_sum[tid & 3], wave_most = s_most[tid & 3];
      refer(t, quad_max(t.m), c);
      wave_most = quad_max(wave_most);
      t.s += dpp64<route_dev::kDppQuadXor1>(t.s), t.u += dpp64<route_dev::kDppQuadXor1>(t.u);
      t.s += dpp64<route_dev::kDppQuadXor2>(t.s), t.u += dpp64<route_dev::kDppQuadXor2>(t.u);
    }
    const RowResult r = row_result(t, wave_most, a.scale);
    if (a.slices == 1) {
      if (tid == 0) put_row<ZT>(a, row, t, r);
    } else if (tid == 0) {
      a.sums[item] = LogprobSlice{t.s, t.u, t.m, wave_most};
    }
    if constexpr (TOP) {
      int* ids = a.slices == 1 ? a.top_ids + row * a.top_n : a.slice_ids + item * a.top_n;
      float* out = a.slices == 1 ? a.top_logp + row * a.top_n : a.slice_values + item * a.top_n;
      // the same for the whole work-group
      const bool none = r.bad || (a.slices == 1 && r.none);
      const int count = none ? 0 : find_top<ZT, THREADS>(s_top, z, begin, end, most, a.top_n, iters, a.note_log);
      rank_top<THREADS, Top<THREADS>::kCand>(s_top.c, count, a.top_n, s_top.few, [&](const Candidate& me, int rank) {
        if (rank >= a.top_n) return;
        const float x = route_dev::order_logit(me.key);
        ids[rank] = me.id;
        out[rank] = a.slices == 1 ? row_logp(r, x, a.scale) : x;
      });
      for (int i = count + tid; i < a.top_n; i += THREADS) ids[i] = -1, out[i] = r.bad ? __uint_as_float(kNan) : kMinusInf;
      __syncthreads();  // s_top is written again by the next item
    }
  }
}

// The slices of a row: their sums referred to the row's maximum, added in order; the best of their top_n.
constexpr int kFinish = 256;
template <int ZT>
__global__ __launch_bounds__(kFinish) void logprob_finish_kernel(LogprobArgs a) {
  constexpr int kCand = kMaxSlices * kMaxTop;
  __shared__ Candidate s_c[kCand];
  __shared__ Few s_few;
  __shared__ int s_n;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  const float c = a.scale * kLog2e;
  // every wave forms the row's sums: a lane per slice
  static_assert(kMaxSlices == 64, "a lane per slice");
  const LogprobSlice p = a.sums[row * a.slices + std::min(lane, a.slices - 1)];
  const bool in = lane < a.slices;
  Sums t{p.m, in ? p.s : 0.0, in ? p.u : 0.0};
  const float most = wave_max(p.most), m = wave_max(t.m);
  refer(t, m, c);
  wave_sums(t);
  const RowResult r = row_result(t, most, a.scale);
  if (tid == 0) put_row<ZT>(a, row, t, r);
  if (!a.top_n) return;
  if (tid == 0) s_n = 0;
  __syncthreads();
  // The slices' lists are in order: where top_n / deep slices, rounded up, have their deep-th value at a bound or
  // above it, top_n values reach it. The first depth at which half of the slices are enough, for the best of
  // few values would be a bound of none.
  const int64_t lists = row * a.slices * a.top_n;
  int deep = 1;
  while (deep < a.top_n && 2 * ((a.top_n + deep - 1) / deep) > a.slices) deep *= 2;
  deep = min(deep, a.top_n);
  const uint32_t mine = in ? key_of(a.slice_values[lists + lane * a.top_n + deep - 1]) : 0u;
  const int n = r.bad || r.none ? 0 : a.slices * a.top_n;
  constexpr int kMine = kCand / kFinish;
  float value[kMine];
  int id[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int e = tid + kFinish * i;
    if (kFinish * i < n) value[i] = a.slice_values[lists + min(e, n - 1)], id[i] = a.slice_ids[lists + min(e, n - 1)];
  }
  const uint32_t bound = nth_of_lanes(mine, (a.top_n + deep - 1) / deep);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (kFinish * i >= n) break;
    const uint32_t key = key_of(value[i]);
    if (tid + kFinish * i < n && id[i] >= 0 && key >= bound) s_c[atomicAdd(&s_n, 1)] = Candidate{key, id[i]};
  }
  __syncthreads();
  const int count = s_n;
  rank_top<kFinish, kCand>(s_c, count, a.top_n, s_few, [&](const Candidate& me, int rank) {
    if (rank >= a.top_n) return;
    a.top_ids[row * a.top_n + rank] = me.id;
    a.top_logp[row * a.top_n + rank] = row_logp(r, route_dev::order_logit(me.key), a.scale);
  });
  for (int i = count + tid; i < a.top_n; i += kFinish) {
    a.top_ids[row * a.top_n + i] = -1;
    a.top_logp[row * a.top_n + i] = r.bad ? __uint_as_float(kNan) : kMinusInf;
  }
}

// dz_j = scale (a (j == y) - p_j (a + b (log p_j + entropy))); 32 values of a thread at once, 13 issue slots each (23
// with the target compared at every value: 87 % of the vector unit's time)
template <int ZT, int DT, int THREADS>
__device__ __forceinline__ void grad_piece(const LogprobGradArgs& a, const char* z, char* out, int first, int y, float ga, float gb, float hi, float lo, float entropy, bool zero) {
  constexpr int kRuns = 4;
  const float scale = a.scale, sa = scale * ga, sb = scale * gb, base = fmaf(sb, entropy, sa);
  const int V = (int)a.V, at = first + threadIdx.x * 8;
  Raw8<ZT> raw[kRuns];
  if (!zero) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
      if (at + r * THREADS * 8 + 8 <= V) raw[r] = load_run<ZT>(z, at + r * THREADS * 8);
  }
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int i = at + r * THREADS * 8;
    if (i >= V) break;
    const bool tail = i + 8 > V;  // a row's last values: the last 8 instead would be written twice
    float v[8];
    if (zero) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    } else {
      if (tail)
        load8_tail<ZT>(z, i, V, v);
      else
        unpack8<ZT>(raw[r], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float lp = fmaf(v[j], scale, -hi) - lo, q = __builtin_amdgcn_exp2f(lp * kLog2e);
        v[j] = -q * fmaf(sb, fmaxf(lp, kFloor), base);
      }
      if ((uint32_t)(y - i) < 8u) {  // one thread of the row
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += y - i == j ? sa : 0.f;
      }
    }
    char* p = out + (uint32_t)i * (uint32_t)value_size<DT>();
    if (a.accumulate) {
      float old[8];
      if (tail)
        load8_tail<DT>(p, 0, V - i, old);
      else
        unpack8<DT>(load8<DT>(p, 0), old);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    if (tail)
      store8_tail<DT>(p, 0, V - i, v);
    else if (a.past)
      store8<DT, true>(p, 0, v);
    else
      store8<DT>(p, 0, v);
  }
}
template <int ZT, int THREADS>
__global__ __launch_bounds__(THREADS) void logprob_grad_kernel(LogprobGradArgs a, int pieces) {
  constexpr int kPiece = THREADS * 8 * 4;
  for (int64_t item = blockIdx.x; item < a.T * pieces; item += gridDim.x) {
    const int64_t row = item / pieces;
    const int first = (int)(item - row * pieces) * kPiece;
    int y = a.targets ? a.targets[row] : -1;
    if (y >= a.V) y = -1;
    const float ga = y >= 0 && a.dlogp ? a.dlogp[row] : 0.f, gb = a.dentropy ? a.dentropy[row] : 0.f;
    if (!a.dlogp || y < 0) y = -(1 << 30);  // far from every logit
    const float hi = a.lse[2 * row], lo = a.lse[2 * row + 1], entropy = a.dentropy ? a.entropy[row] : 0.f;
    // nothing is asked of the row, or it has no tokens: zeros, whatever its logits
    const bool zero = (ga == 0.f && gb == 0.f) || hi == kMinusInf;
    if (zero && a.accumulate) continue;
    const char* z = static_cast<const char*>(a.logits) + row * a.z_stride * value_size<ZT>();
    char* out = static_cast<char*>(a.dlogits) + row * a.d_stride * (a.d_type == MOE_F32 ? 4 : 2);
    if (a.d_type == MOE_F32)
      grad_piece<ZT, MOE_F32, THREADS>(a, z, out, first, y, ga, gb, hi, lo, entropy, zero);
    else if (a.d_type == MOE_F16)
      grad_piece<ZT, MOE_F16, THREADS>(a, z, out, first, y, ga, gb, hi, lo, entropy, zero);
    else
      grad_piece<ZT, MOE_BF16, THREADS>(a, z, out, first, y, ga, gb, hi, lo, entropy, zero);
  }
}

int slices_of(int64_t T, int64_t V) {
  if (T < 1 || T >= kMostCut || V <= kWholeRow + kWholeRowMore * T) return 1;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kSliceTarget / T, kMaxSlices));
  const int64_t slice = ((V + want - 1) / want + kSliceStep - 1) / kSliceStep * kSliceStep;
  return (int)((V + slice - 1) / slice);
}

int64_t slice_bytes(int top_n) { return (int64_t)sizeof(LogprobSlice) + 8 * (int64_t)top_n; }

template <int ZT, int THREADS>
hipError_t launch_rows(const LogprobArgs& a, dim3 grid, hipStream_t s) {
  return a.top_n ? launch(logprob_rows_kernel<ZT, THREADS, true>, grid, dim3(THREADS), Launch{s}, a)
                 : launch(logprob_rows_kernel<ZT, THREADS, false>, grid, dim3(THREADS), Launch{s}, a);
}
template <int ZT>
hipError_t launch_types(LogprobArgs a, hipStream_t s) {
  const int threads = a.V <= kWaveRow ? 64 : 256;
  a.slices = slices_of(a.T, a.V);
  a.slice = a.slices == 1 ? a.V : ((a.V + a.slices - 1) / a.slices + kSliceStep - 1) / kSliceStep * kSliceStep;
  const int64_t per_iter = (int64_t)threads * 8 * kU, iters = (a.slice + per_iter - 1) / per_iter;
  for (a.note_log = 0; iters > (int64_t)kNotes << a.note_log; ++a.note_log) {
  }
  if (a.slices > 1) {
    const int64_t items = a.T * a.slices;
    a.sums = reinterpret_cast<LogprobSlice*>(a.ws);
    a.slice_values = reinterpret_cast<float*>(a.sums + items);
    a.slice_ids = reinterpret_cast<int*>(a.slice_values + items * a.top_n);
  }
  // rows beyond the grid are taken in turn by the same work-groups
  const dim3 grid((unsigned)std::min<int64_t>(a.T * a.slices, 1 << 20));
  const hipError_t e = threads == 64 ? launch_rows<ZT, 64>(a, grid, s) : launch_rows<ZT, 256>(a, grid, s);
  if (e != hipSuccess || a.slices == 1) return e;
  return launch(logprob_finish_kernel<ZT>, dim3((unsigned)a.T), dim3(kFinish), Launch{s}, a);
}
template <int ZT>
hipError_t launch_grad_types(const LogprobGradArgs& a, hipStream_t s) {
  const int threads = a.V <= kWaveRow ? 64 : 256;
  const int64_t piece = (int64_t)threads * 8 * 4;
  const int pieces = (int)((a.V + piece - 1) / piece);
  const dim3 grid((unsigned)std::min<int64_t>(a.T * pieces, 1 << 22));
  return threads == 64 ? launch(logprob_grad_kernel<ZT, 64>, grid, dim3(64), Launch{s}, a, pieces)
                       : launch(logprob_grad_kernel<ZT, 256>, grid, dim3(256), Launch{s}, a, pieces);
}

}  // namespace

// Never less for more rows, though many rows are not cut: up to kSliceTarget slices in all
int64_t logprob_workspace_bytes(int64_t T, int64_t V, int top_n) {
  if (T < 1 || V <= kWholeRow + kWholeRowMore) return 0;
  return std::min<int64_t>(T * kMaxSlices, kSliceTarget) * slice_bytes(top_n);
}
int64_t logprob_workspace_used(int64_t T, int64_t V, int top_n) {
  const int slices = slices_of(T, V);
  return slices > 1 ? T * slices * slice_bytes(top_n) : 0;
}

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.z_type == MOE_F32) return launch_types<MOE_F32>(a, s);
  if (a.z_type == MOE_F16) return launch_types<MOE_F16>(a, s);
  return launch_types<MOE_BF16>(a, s);
}
hipError_t launch_logprobs_grad(LogprobGradArgs a, hipStream_t s) {
  // From 64 MB on past the caches, which would keep little of it and drop the logits for it (us, kept and past, forward and
  // gradient: 4096 x 65537 bf16 322 and 312, 4096 x 32000 164 and 131, 1000 x 32001 fp32 85 and 77). What is smaller
  // is read from them by the product that comes next.
  a.past = a.T * a.V * (a.d_type == MOE_F32 ? 4 : 2) >= 64ll << 20;
  if (a.z_type == MOE_F32) return launch_grad_types<MOE_F32>(a, s);
  if (a.z_type == MOE_F16) return launch_grad_types<MOE_F16>(a, s);
  return launch_grad_types<MOE_BF16>(a, s);
}

}  // namespace moe
