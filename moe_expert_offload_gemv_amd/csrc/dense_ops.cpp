// dense_ops.cpp - the entry points of the operators beside the experts:
// argument checks, then the launches of norm.hip, dense_q4.hip and balance.hip
// on the caller's stream. Nothing is kept between calls.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/moe_offload.h"
#include "kernels.h"
#include "runtime.h"

namespace {

constexpr int32_t kMaxTokens = 1 << 24;  // token counts stay exact in fp32, grids and offsets in range
constexpr int32_t kMaxOut = 1 << 22;

bool value_type(int32_t t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
int64_t value_size(int32_t t) { return t == MOE_F32 ? 4 : t == MOE_Q8_32 ? 1 : 2; }

// rows of n values from p with this stride: p present, aligned to its values,
// rows apart (at most 2^36: 2^24 rows of 4-byte values stay within 63 bits)
bool rows_ok(const void* p, int32_t type, int64_t n, int64_t stride) {
  return p && (uintptr_t)p % (uintptr_t)value_size(type) == 0 && stride >= n && stride <= (int64_t)1 << 36;
}
bool aligned(const void* p, uintptr_t to) { return (uintptr_t)p % to == 0; }

int device_ok(int32_t device, const char* what) {
  static std::atomic<int> count{-1};  // devices of the process, asked for once
  int n = count.load(std::memory_order_relaxed);
  if (n < 0) {
    if (hipGetDeviceCount(&n) != hipSuccess) {
      (void)hipGetLastError();
      n = 0;
    } else {
      count.store(n, std::memory_order_relaxed);
    }
  }
  if (device < 0 || device >= n) return moe_thread_fail(MOE_E_INVAL, "%s: no HIP device %d", what, device);
  return MOE_OK;
}

int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return MOE_OK;
  return moe_thread_fail(MOE_E_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
}

#define REFUSE(cond, ...) \
  do {                    \
    if (cond) return moe_thread_fail(MOE_E_INVAL, __VA_ARGS__); \
  } while (0)

}  // namespace

extern "C" int moe_add_rmsnorm(int32_t device, void* stream, int32_t n_tokens, int32_t hidden, int32_t x_type,
                               const void* x, int64_t x_stride, int32_t res_type, const void* residual,
                               int64_t res_stride, void* residual_out, int64_t res_out_stride, const float* weight,
                               float eps, int32_t out_type, void* out, int64_t out_stride, float* scales,
                               int64_t scales_stride) {
  const char* me = "moe_add_rmsnorm";
  REFUSE(n_tokens < 0 || n_tokens > kMaxTokens || hidden < 1 || hidden > 1 << 24,
         "%s: n_tokens %d or hidden %d out of range", me, n_tokens, hidden);
  REFUSE(!value_type(x_type) || !(value_type(out_type) || out_type == MOE_Q8_32), "%s: bad type of x or out", me);
  REFUSE(!(eps >= 0.f), "%s: eps %g", me, eps);
  REFUSE(out_type == MOE_Q8_32 && hidden % 32, "%s: 8-bit out needs hidden %d to be a multiple of 32", me, hidden);
  REFUSE((residual == nullptr) != (residual_out == nullptr), "%s: residual and residual_out go together", me);
  REFUSE(residual && !value_type(res_type), "%s: bad type of the residual", me);
  REFUSE((scales == nullptr) != (out_type != MOE_Q8_32) && n_tokens > 0, "%s: scales go with 8-bit out", me);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(x, x_type, hidden, x_stride), "%s: x null, unaligned or its stride below hidden", me);
    REFUSE(!rows_ok(out, out_type, hidden, out_stride), "%s: out null, unaligned or its stride below hidden",
           me);
    REFUSE(residual && (!rows_ok(residual, res_type, hidden, res_stride) ||
                        !rows_ok(residual_out, res_type, hidden, res_out_stride)),
           "%s: residual unaligned or its stride below hidden", me);
    REFUSE(residual && residual == residual_out && res_stride != res_out_stride,
           "%s: residual in place with two strides", me);
    REFUSE(out == x && (out_type != x_type || out_stride != x_stride), "%s: out in place of x with another type or stride",
           me);
    REFUSE(residual && (out == residual || out == residual_out || x == residual_out), "%s: outputs overlap", me);
    REFUSE(out_type == MOE_Q8_32 && !rows_ok(scales, MOE_F32, hidden / 32, scales_stride),
           "%s: scales unaligned or their stride below hidden / 32", me);
    REFUSE(!aligned(weight, 4), "%s: weight unaligned", me);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  moe::NormArgs a{};
  a.x = x, a.res = residual, a.res_out = residual_out, a.weight = weight, a.out = out, a.scales = scales;
  a.x_stride = x_stride, a.res_stride = res_stride, a.res_out_stride = res_out_stride, a.out_stride = out_stride;
  a.scales_stride = scales_stride;
  a.T = n_tokens, a.H = hidden;
  a.x_type = x_type, a.res_type = res_type, a.out_type = out_type, a.eps = eps;
  DeviceGuard g(device);
  return launched(moe::launch_add_rmsnorm(a, (hipStream_t)stream), me);
}

extern "C" int moe_q4_split(int32_t rows, int32_t k, const void* blocks, void* nibbles, void* scales) {
  REFUSE(rows < 0 || k < 32 || k % 32 || k > 1 << 20, "moe_q4_split: rows %d or k %d out of range", rows, k);
  REFUSE(rows > 0 && (!blocks || !nibbles || !scales), "moe_q4_split: null pointer");
  const uint8_t* s = static_cast<const uint8_t*>(blocks);
  uint8_t *nib = static_cast<uint8_t*>(nibbles), *scl = static_cast<uint8_t*>(scales);
  for (int64_t b = 0; b < (int64_t)rows * (k / 32); ++b) {
    std::memcpy(scl + 2 * b, s + 18 * b, 2);
    std::memcpy(nib + 16 * b, s + 18 * b + 2, 16);
  }
  return MOE_OK;
}

extern "C" int64_t moe_q4_workspace_bytes(int32_t n_tokens, int32_t n_out, int32_t k, int32_t x_type) {
  if (n_tokens < 0 || n_tokens > kMaxTokens || n_out < 1 || n_out > kMaxOut || k < 32 || k % 32 || k > 1 << 20 ||
      !(value_type(x_type) || x_type == MOE_Q8_32))
    return -1;
  return n_tokens ? moe::q4_workspace_bytes(n_tokens, n_out, k, x_type) : 0;
}

extern "C" int moe_q4_matmul(int32_t device, void* stream, int32_t n_tokens, int32_t n_out, int32_t k, int32_t x_type,
                             const void* x, int64_t x_stride, const float* x_scales, int64_t x_scales_stride,
                             const void* nibbles, const void* w_scales, int32_t y_type, void* y, int64_t y_stride,
                             void* workspace, int64_t workspace_bytes, uint32_t flags) {
  const char* me = "moe_q4_matmul";
  const int64_t need = moe_q4_workspace_bytes(n_tokens, n_out, k, x_type);
  REFUSE(need < 0, "%s: n_tokens %d, n_out %d, k %d or the type of x out of range", me, n_tokens, n_out, k);
  REFUSE(!value_type(y_type), "%s: bad type of y", me);
  REFUSE(flags & ~MOE_ACCUMULATE, "%s: unknown flags", me);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(x, x_type, k, x_stride), "%s: x null, unaligned or its stride below k", me);
    REFUSE(!rows_ok(y, y_type, n_out, y_stride), "%s: y null, unaligned or its stride below n_out", me);
    REFUSE((x_scales != nullptr) != (x_type == MOE_Q8_32), "%s: x_scales go with 8-bit x", me);
    REFUSE(x_scales && !rows_ok(x_scales, MOE_F32, k / 32, x_scales_stride),
           "%s: x_scales unaligned or their stride below k / 32", me);
    REFUSE(!nibbles || !w_scales || !aligned(nibbles, 16) || !aligned(w_scales, 16),
           "%s: weight planes null or not 16-byte aligned", me);
    REFUSE(x == y, "%s: y in place of x", me);
    REFUSE(need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need),
           "%s: workspace null, unaligned or below %lld bytes", me, (long long)need);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  moe::Q4Args a{};
  a.x = x, a.x_scales = x_scales, a.nibbles = nibbles, a.w_scales = static_cast<const uint16_t*>(w_scales), a.y = y;
  a.ws = static_cast<uint8_t*>(workspace);
  a.x_stride = x_stride, a.x_scales_stride = x_scales_stride, a.y_stride = y_stride;
  a.T = n_tokens, a.N = n_out, a.K = k;
  a.x_type = x_type, a.y_type = y_type, a.accumulate = (flags & MOE_ACCUMULATE) != 0;
  DeviceGuard g(device);
  return launched(moe::launch_q4_matmul(a, (hipStream_t)stream), me);
}

extern "C" int64_t moe_router_balance_workspace_bytes(int32_t n_tokens, int32_t n_experts) {
  if (n_tokens < 0 || n_tokens > kMaxTokens || n_experts < 1 || n_experts > 4096) return -1;
  return moe::balance_workspace_bytes(n_tokens, n_experts);
}

extern "C" int moe_router_balance(int32_t device, void* stream, int32_t n_tokens, int32_t n_experts, int32_t top_k,
                                  int32_t z_type, const void* logits, int64_t z_stride, const uint8_t* valid,
                                  float balance_coef, float z_coef, int32_t* counts, float* load, float* stats,
                                  float* lse, void* workspace, int64_t workspace_bytes, uint32_t flags) {
  const char* me = "moe_router_balance";
  const int64_t need = moe_router_balance_workspace_bytes(n_tokens, n_experts);
  REFUSE(need < 0 || top_k < 1 || top_k > 32 || top_k > n_experts, "%s: n_tokens %d, n_experts %d or top_k %d out of range",
         me, n_tokens, n_experts, top_k);
  REFUSE(!value_type(z_type), "%s: bad type of the logits", me);
  REFUSE(flags & ~MOE_ACCUMULATE, "%s: unknown flags", me);
  REFUSE(!counts || !load || !stats || !aligned(counts, 4) || !aligned(load, 4) || !aligned(stats, 4),
         "%s: counts, load or stats null or unaligned", me);
  REFUSE(n_tokens > 0 && !rows_ok(logits, z_type, n_experts, z_stride),
         "%s: logits null, unaligned or their stride below n_experts", me);
  REFUSE(n_tokens > 0 && (!lse || !aligned(lse, 4)), "%s: lse null or unaligned", me);
  REFUSE(!workspace || !aligned(workspace, 256) || workspace_bytes < need,
         "%s: workspace null, unaligned or below %lld bytes", me, (long long)need);
  if (int rc = device_ok(device, me)) return rc;
  moe::BalanceArgs a{};
  a.logits = logits, a.valid = valid, a.counts = counts, a.load = load, a.stats = stats, a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.z_stride = z_stride, a.T = n_tokens, a.E = n_experts, a.k = top_k, a.z_type = z_type;
  a.accumulate = (flags & MOE_ACCUMULATE) != 0;
  a.balance = balance_coef, a.z = z_coef;
  DeviceGuard g(device);
  return launched(moe::launch_balance(a, (hipStream_t)stream), me);
}

extern "C" int moe_router_balance_grad(int32_t device, void* stream, int32_t n_tokens, int32_t n_experts,
                                       int32_t z_type, const void* logits, int64_t z_stride, const float* load,
                                       const float* stats, const float* lse, const float* dloss, float balance_coef,
                                       float z_coef, int32_t d_type, void* dlogits, int64_t d_stride, uint32_t flags) {
  const char* me = "moe_router_balance_grad";
  REFUSE(n_tokens < 0 || n_tokens > kMaxTokens || n_experts < 1 || n_experts > 4096,
         "%s: n_tokens %d or n_experts %d out of range", me, n_tokens, n_experts);
  REFUSE(!value_type(z_type) || !value_type(d_type), "%s: bad type of the logits or dlogits", me);
  REFUSE(flags & ~MOE_ACCUMULATE, "%s: unknown flags", me);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(logits, z_type, n_experts, z_stride),
           "%s: logits null, unaligned or their stride below n_experts", me);
    REFUSE(!rows_ok(dlogits, d_type, n_experts, d_stride),
           "%s: dlogits null, unaligned or their stride below n_experts", me);
    REFUSE(!load || !stats || !lse || !aligned(load, 4) || !aligned(stats, 4) || !aligned(lse, 4) || !aligned(dloss, 4),
           "%s: load, stats or lse null or unaligned", me);
    REFUSE(dlogits == logits && (d_type != z_type || d_stride != z_stride || (flags & MOE_ACCUMULATE)),
           "%s: dlogits in place of the logits with another type or stride, or accumulating", me);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  moe::BalanceGradArgs a{};
  a.logits = logits, a.load = load, a.stats = stats, a.lse = lse, a.dloss = dloss, a.dlogits = dlogits;
  a.z_stride = z_stride, a.d_stride = d_stride, a.T = n_tokens;
  a.E = n_experts, a.z_type = z_type, a.d_type = d_type, a.accumulate = (flags & MOE_ACCUMULATE) != 0;
  a.balance = balance_coef, a.z = z_coef;
  DeviceGuard g(device);
  return launched(moe::launch_balance_grad(a, (hipStream_t)stream), me);
}
