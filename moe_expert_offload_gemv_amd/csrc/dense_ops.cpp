// dense_ops.cpp - the entry points of the operators beside the experts:
// argument checks, then the launches of norm.hip, dense_q4.hip, dense_q4_linear.hip,
// heads.hip, heads_grad.hip, logprobs.hip and balance.hip on the caller's stream. Nothing is kept between calls.
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
// heads [T][H][n] from p: aligned to their values, the heads of a token apart within its row, or the
// tokens of a head within the head's (strides at most 2^36 each: 2^24 tokens and 2^10 heads of 4-byte values
// stay within 63 bits)
bool heads_ok(const void* p, int32_t type, int64_t T, int64_t H, int64_t n, int64_t stride, int64_t head_stride) {
  const int64_t most = (int64_t)1 << 36;
  if (!p || (uintptr_t)p % (uintptr_t)value_size(type) || stride < n || head_stride < n || stride > most || head_stride > most)
    return false;
  return stride >= (H - 1) * head_stride + n || head_stride >= (T - 1) * stride + n;
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

extern "C" int moe_q4_linear(int32_t device, void* stream, int32_t n_tokens, int32_t n_out, int32_t k, int32_t x_type,
                             const void* x, int64_t x_stride, const float* x_scales, int64_t x_scales_stride,
                             const void* nibbles, const void* w_scales, const float* bias, int32_t act, int32_t mul_type,
                             const void* mul, int64_t mul_stride, int32_t res_type, const void* residual, int64_t res_stride,
                             int32_t y_type, void* y, int64_t y_stride, void* workspace, int64_t workspace_bytes) {
  const char* me = "moe_q4_linear";
  const int64_t need = moe_q4_workspace_bytes(n_tokens, n_out, k, x_type);
  REFUSE(need < 0, "%s: n_tokens %d, n_out %d, k %d or the type of x out of range", me, n_tokens, n_out, k);
  REFUSE(!value_type(y_type), "%s: bad type of y", me);
  REFUSE(act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH, "%s: unknown act %d", me, act);
  REFUSE((mul && !value_type(mul_type)) || (residual && !value_type(res_type)), "%s: bad type of mul or the residual", me);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(x, x_type, k, x_stride), "%s: x null, unaligned or its stride below k", me);
    REFUSE(!rows_ok(y, y_type, n_out, y_stride), "%s: y null, unaligned or its stride below n_out", me);
    REFUSE((x_scales != nullptr) != (x_type == MOE_Q8_32), "%s: x_scales go with 8-bit x", me);
    REFUSE(x_scales && !rows_ok(x_scales, MOE_F32, k / 32, x_scales_stride),
           "%s: x_scales unaligned or their stride below k / 32", me);
    REFUSE(!nibbles || !w_scales || !aligned(nibbles, 16) || !aligned(w_scales, 16),
           "%s: weight planes null or not 16-byte aligned", me);
    REFUSE(!aligned(bias, 4), "%s: bias unaligned", me);
    REFUSE(mul && !rows_ok(mul, mul_type, n_out, mul_stride), "%s: mul unaligned or its stride below n_out", me);
    REFUSE(residual && !rows_ok(residual, res_type, n_out, res_stride),
           "%s: residual unaligned or its stride below n_out", me);
    REFUSE(x == y, "%s: y in place of x", me);
    REFUSE((y == mul && (y_type != mul_type || y_stride != mul_stride)) ||
               (y == residual && (y_type != res_type || y_stride != res_stride)),
           "%s: y in place of mul or the residual with another type or stride", me);
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
  a.x_type = x_type, a.y_type = y_type;
  a.epi.bias = bias, a.epi.mul = mul, a.epi.res = residual, a.epi.mul_stride = mul_stride, a.epi.res_stride = res_stride;
  a.epi.mul_type = mul_type, a.epi.res_type = res_type, a.epi.act = act;
  DeviceGuard g(device);
  return launched(moe::launch_q4_linear(a, (hipStream_t)stream), me);
}

namespace {

// what the norm and rotation of heads and its gradient have alike
int heads_common(const char* me, int32_t n_tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t x_type,
                 const float* q_weight, const float* k_weight, float eps, int32_t rotary_dim, const float* inv_freq,
                 const int32_t* positions, int64_t pos_stride, int32_t n_axes, const uint8_t* pair_axis, uint32_t flags,
                 moe::HeadsArgs* a) {
  REFUSE(n_tokens < 0 || n_tokens > kMaxTokens || q_heads < 1 || q_heads > 1024 || k_heads < 0 || k_heads > 1024 ||
             head_dim < 2 || head_dim > 512 || head_dim % 2,
         "%s: n_tokens %d, q_heads %d, k_heads %d or head_dim %d out of range", me, n_tokens, q_heads, k_heads, head_dim);
  REFUSE(rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2, "%s: rotary_dim %d of head_dim %d", me, rotary_dim, head_dim);
  REFUSE(!(eps >= 0.f), "%s: eps %g", me, eps);
  REFUSE((flags & MOE_NO_NORM) && (q_weight || k_weight), "%s: weights without a norm", me);
  REFUSE((flags & MOE_NO_NORM) && rotary_dim == 0, "%s: neither norm nor rotation", me);
  REFUSE(rotary_dim == 0 && (inv_freq || positions || pair_axis), "%s: positions or inv_freq without rotary_dim", me);
  REFUSE(rotary_dim && (n_axes < 1 || n_axes > 8), "%s: n_axes %d", me, n_axes);
  REFUSE(rotary_dim && (!inv_freq || !aligned(inv_freq, 4)), "%s: inv_freq null or unaligned", me);
  // rows of positions are read alone: they may be one and the same
  REFUSE(rotary_dim && n_tokens > 0 && (!positions || !aligned(positions, 4)), "%s: positions null or unaligned", me);
  REFUSE(rotary_dim && n_axes > 1 && (pos_stride < 0 || pos_stride > (int64_t)1 << 36), "%s: stride of positions", me);
  REFUSE(!aligned(q_weight, 4) || (k_heads && !aligned(k_weight, 4)), "%s: weights unaligned", me);
  REFUSE(!value_type(x_type), "%s: bad type of q and k", me);
  a->q.weight = q_weight, a->k.weight = k_weight, a->q.H = q_heads, a->k.H = k_heads;
  a->inv_freq = inv_freq, a->pos = positions, a->axis = pair_axis, a->pos_stride = pos_stride;
  a->T = n_tokens, a->D = head_dim, a->R = rotary_dim, a->axes = n_axes, a->x_type = x_type;
  a->pairs = (flags & MOE_ROPE_PAIRS) != 0, a->norm = !(flags & MOE_NO_NORM), a->eps = eps;
  return MOE_OK;
}

}  // namespace

extern "C" int moe_qk_norm_rope(int32_t device, void* stream, int32_t n_tokens, int32_t q_heads, int32_t k_heads,
                                int32_t head_dim, int32_t x_type, const void* q, int64_t q_stride, int64_t q_head_stride,
                                const void* k, int64_t k_stride, int64_t k_head_stride, const float* q_weight,
                                const float* k_weight, float eps, int32_t rotary_dim, const float* inv_freq,
                                const int32_t* positions, int64_t pos_stride, int32_t n_axes, const uint8_t* pair_axis,
                                int32_t out_type, void* q_out, int64_t q_out_stride, int64_t q_out_head_stride, void* k_out,
                                int64_t k_out_stride, int64_t k_out_head_stride, uint32_t flags) {
  const char* me = "moe_qk_norm_rope";
  moe::HeadsArgs a{};
  REFUSE(flags & ~(MOE_ROPE_PAIRS | MOE_NO_NORM), "%s: unknown flags", me);
  if (int rc = heads_common(me, n_tokens, q_heads, k_heads, head_dim, x_type, q_weight, k_weight, eps, rotary_dim, inv_freq,
                            positions, pos_stride, n_axes, pair_axis, flags, &a))
    return rc;
  REFUSE(!value_type(out_type), "%s: bad type of the outputs", me);
  if (n_tokens > 0) {
    REFUSE(!heads_ok(q, x_type, n_tokens, q_heads, head_dim, q_stride, q_head_stride) ||
               !heads_ok(q_out, out_type, n_tokens, q_heads, head_dim, q_out_stride, q_out_head_stride),
           "%s: q or q_out null, unaligned or its strides let heads overlap", me);
    REFUSE(k_heads && (!heads_ok(k, x_type, n_tokens, k_heads, head_dim, k_stride, k_head_stride) ||
                       !heads_ok(k_out, out_type, n_tokens, k_heads, head_dim, k_out_stride, k_out_head_stride)),
           "%s: k or k_out null, unaligned or its strides let heads overlap", me);
    REFUSE((q_out == q && (out_type != x_type || q_out_stride != q_stride || q_out_head_stride != q_head_stride)) ||
               (k_heads && k_out == k &&
                (out_type != x_type || k_out_stride != k_stride || k_out_head_stride != k_head_stride)),
           "%s: in place with another type or strides", me);
    REFUSE(k_heads && (q_out == k_out || q_out == k || k_out == q), "%s: outputs overlap", me);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  a.q.x = q, a.q.x_stride = q_stride, a.q.x_head = q_head_stride;
  a.q.out = q_out, a.q.out_stride = q_out_stride, a.q.out_head = q_out_head_stride;
  a.k.x = k, a.k.x_stride = k_stride, a.k.x_head = k_head_stride;
  a.k.out = k_out, a.k.out_stride = k_out_stride, a.k.out_head = k_out_head_stride;
  a.out_type = out_type;
  DeviceGuard g(device);
  return launched(moe::launch_heads(a, (hipStream_t)stream), me);
}

extern "C" int64_t moe_qk_norm_rope_grad_workspace_bytes(int32_t n_tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  if (n_tokens < 0 || n_tokens > kMaxTokens || q_heads < 1 || q_heads > 1024 || k_heads < 0 || k_heads > 1024 || head_dim < 2 ||
      head_dim > 512 || head_dim % 2)
    return -1;
  return moe::heads_grad_workspace_bytes(n_tokens, q_heads, k_heads, head_dim);
}

extern "C" int moe_qk_norm_rope_grad(int32_t device, void* stream, int32_t n_tokens, int32_t q_heads, int32_t k_heads,
                                     int32_t head_dim, int32_t x_type, const void* q, int64_t q_stride, int64_t q_head_stride,
                                     const void* k, int64_t k_stride, int64_t k_head_stride, const float* q_weight,
                                     const float* k_weight, float eps, int32_t rotary_dim, const float* inv_freq,
                                     const int32_t* positions, int64_t pos_stride, int32_t n_axes, const uint8_t* pair_axis,
                                     int32_t g_type, const void* gq, int64_t gq_stride, int64_t gq_head_stride,
                                     const void* gk, int64_t gk_stride, int64_t gk_head_stride, int32_t d_type, void* dq,
                                     int64_t dq_stride, int64_t dq_head_stride, void* dk, int64_t dk_stride,
                                     int64_t dk_head_stride, float* dq_weight, float* dk_weight, void* workspace,
                                     int64_t workspace_bytes, uint32_t flags) {
  const char* me = "moe_qk_norm_rope_grad";
  moe::HeadsArgs a{};
  REFUSE(flags & ~(MOE_ROPE_PAIRS | MOE_NO_NORM | MOE_ACCUMULATE), "%s: unknown flags", me);
  if (int rc = heads_common(me, n_tokens, q_heads, k_heads, head_dim, x_type, q_weight, k_weight, eps, rotary_dim, inv_freq,
                            positions, pos_stride, n_axes, pair_axis, flags, &a))
    return rc;
  const bool norm = !(flags & MOE_NO_NORM);
  REFUSE(!value_type(g_type) || !value_type(d_type), "%s: bad type of the gradients", me);
  REFUSE(!norm && (dq_weight || dk_weight), "%s: gradients of weights without a norm", me);
  REFUSE(!k_heads && dk_weight, "%s: dk_weight without keys", me);
  REFUSE(!aligned(dq_weight, 4) || !aligned(dk_weight, 4), "%s: gradients of weights unaligned", me);
  REFUSE(dq_weight && dq_weight == dk_weight, "%s: outputs overlap", me);
  if (n_tokens > 0) {
    REFUSE((norm && !heads_ok(q, x_type, n_tokens, q_heads, head_dim, q_stride, q_head_stride)) ||
               !heads_ok(gq, g_type, n_tokens, q_heads, head_dim, gq_stride, gq_head_stride) ||
               !heads_ok(dq, d_type, n_tokens, q_heads, head_dim, dq_stride, dq_head_stride),
           "%s: q, gq or dq null, unaligned or its strides let heads overlap", me);
    REFUSE(k_heads && ((norm && !heads_ok(k, x_type, n_tokens, k_heads, head_dim, k_stride, k_head_stride)) ||
                       !heads_ok(gk, g_type, n_tokens, k_heads, head_dim, gk_stride, gk_head_stride) ||
                       !heads_ok(dk, d_type, n_tokens, k_heads, head_dim, dk_stride, dk_head_stride)),
           "%s: k, gk or dk null, unaligned or its strides let heads overlap", me);
    REFUSE((dq == gq && (d_type != g_type || dq_stride != gq_stride || dq_head_stride != gq_head_stride)) ||
               (norm && dq == q && (d_type != x_type || dq_stride != q_stride || dq_head_stride != q_head_stride)) ||
               (k_heads && dk == gk && (d_type != g_type || dk_stride != gk_stride || dk_head_stride != gk_head_stride)) ||
               (k_heads && norm && dk == k &&
                (d_type != x_type || dk_stride != k_stride || dk_head_stride != k_head_stride)),
           "%s: in place with another type or strides", me);
    REFUSE(k_heads && (dq == dk || dq == gk || dk == gq || (norm && (dq == k || dk == q))), "%s: outputs overlap", me);
    const int64_t need = dq_weight || dk_weight ? moe::heads_grad_workspace_bytes(n_tokens, q_heads, k_heads, head_dim) : 0;
    REFUSE(need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need),
           "%s: workspace null, unaligned or below %lld bytes", me, (long long)need);
  }
  if (int rc = device_ok(device, me)) return rc;
  a.q.x = q, a.q.x_stride = q_stride, a.q.x_head = q_head_stride;
  a.q.g = gq, a.q.g_stride = gq_stride, a.q.g_head = gq_head_stride;
  a.q.out = dq, a.q.out_stride = dq_stride, a.q.out_head = dq_head_stride, a.q.dweight = dq_weight;
  a.k.x = k, a.k.x_stride = k_stride, a.k.x_head = k_head_stride;
  a.k.g = gk, a.k.g_stride = gk_stride, a.k.g_head = gk_head_stride;
  a.k.out = dk, a.k.out_stride = dk_stride, a.k.out_head = dk_head_stride, a.k.dweight = dk_weight;
  a.g_type = g_type, a.out_type = d_type, a.accumulate = (flags & MOE_ACCUMULATE) != 0;
  DeviceGuard g(device);
  return launched(moe::launch_heads_grad(a, static_cast<uint8_t*>(workspace), (hipStream_t)stream), me);
}

extern "C" int64_t moe_token_logprobs_workspace_bytes(int32_t n_tokens, int32_t n_vocab, int32_t top_n) {
  if (n_tokens < 0 || n_tokens > kMaxTokens || n_vocab < 1 || n_vocab > kMaxOut || top_n < 0 || top_n > moe::kMaxTop ||
      top_n > n_vocab)
    return -1;
  return moe::logprob_workspace_bytes(n_tokens, n_vocab, top_n);
}

extern "C" int moe_token_logprobs(int32_t device, void* stream, int32_t n_tokens, int32_t n_vocab, int32_t z_type,
                                  const void* logits, int64_t z_stride, const int32_t* targets, float scale, float* logp,
                                  float* entropy, float* lse, int32_t top_n, int32_t* top_ids, float* top_logp,
                                  void* workspace, int64_t workspace_bytes) {
  const char* me = "moe_token_logprobs";
  REFUSE(moe_token_logprobs_workspace_bytes(n_tokens, n_vocab, top_n) < 0,
         "%s: n_tokens %d, n_vocab %d or top_n %d out of range", me, n_tokens, n_vocab, top_n);
  const int64_t need = moe::logprob_workspace_used(n_tokens, n_vocab, top_n);
  REFUSE(!value_type(z_type), "%s: bad type of the logits", me);
  REFUSE(!(scale >= 0x1p-64f && scale <= 0x1p64f), "%s: scale %g out of range", me, scale);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(logits, z_type, n_vocab, z_stride), "%s: logits null, unaligned or their stride below n_vocab", me);
    REFUSE((targets == nullptr) != (logp == nullptr), "%s: targets and logp go together", me);
    REFUSE((top_ids != nullptr) != (top_n > 0) || (top_logp != nullptr) != (top_n > 0), "%s: top_ids and top_logp go with top_n", me);
    REFUSE(!aligned(targets, 4) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_ids, 4) ||
               !aligned(top_logp, 4),
           "%s: targets or an output unaligned", me);
    REFUSE(!logp && !entropy && !lse && !top_n, "%s: nothing is asked for", me);
    REFUSE(need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need),
           "%s: workspace null, unaligned or below %lld bytes", me, (long long)need);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  moe::LogprobArgs a{};
  a.logits = logits, a.targets = targets, a.logp = logp, a.entropy = entropy, a.lse = lse;
  a.top_ids = top_ids, a.top_logp = top_logp, a.ws = static_cast<uint8_t*>(workspace);
  a.z_stride = z_stride, a.T = n_tokens, a.V = n_vocab, a.z_type = z_type, a.top_n = top_n, a.scale = scale;
  DeviceGuard g(device);
  return launched(moe::launch_logprobs(a, (hipStream_t)stream), me);
}

extern "C" int moe_token_logprobs_grad(int32_t device, void* stream, int32_t n_tokens, int32_t n_vocab, int32_t z_type,
                                       const void* logits, int64_t z_stride, const int32_t* targets, float scale,
                                       const float* lse, const float* entropy, const float* dlogp, const float* dentropy,
                                       int32_t d_type, void* dlogits, int64_t d_stride, uint32_t flags) {
  const char* me = "moe_token_logprobs_grad";
  REFUSE(n_tokens < 0 || n_tokens > kMaxTokens || n_vocab < 1 || n_vocab > kMaxOut, "%s: n_tokens %d or n_vocab %d out of range",
         me, n_tokens, n_vocab);
  REFUSE(!value_type(z_type) || !value_type(d_type), "%s: bad type of the logits or dlogits", me);
  REFUSE(!(scale >= 0x1p-64f && scale <= 0x1p64f), "%s: scale %g out of range", me, scale);
  REFUSE(flags & ~MOE_ACCUMULATE, "%s: unknown flags", me);
  if (n_tokens > 0) {
    REFUSE(!rows_ok(logits, z_type, n_vocab, z_stride), "%s: logits null, unaligned or their stride below n_vocab", me);
    REFUSE(!rows_ok(dlogits, d_type, n_vocab, d_stride), "%s: dlogits null, unaligned or their stride below n_vocab", me);
    REFUSE(!lse || !aligned(lse, 4), "%s: lse null or unaligned", me);
    REFUSE(!dlogp && !dentropy, "%s: neither dlogp nor dentropy", me);
    REFUSE((dlogp && !targets) || (dentropy && !entropy), "%s: dlogp needs targets, dentropy the entropy", me);
    REFUSE(!aligned(targets, 4) || !aligned(entropy, 4) || !aligned(dlogp, 4) || !aligned(dentropy, 4),
           "%s: targets, entropy, dlogp or dentropy unaligned", me);
    REFUSE(dlogits == logits && (d_type != z_type || d_stride != z_stride || (flags & MOE_ACCUMULATE)),
           "%s: dlogits in place of the logits with another type or stride, or accumulating", me);
  }
  if (int rc = device_ok(device, me)) return rc;
  if (n_tokens == 0) return MOE_OK;
  moe::LogprobGradArgs a{};
  a.logits = logits, a.targets = targets, a.lse = lse, a.entropy = entropy, a.dlogp = dlogp, a.dentropy = dentropy;
  a.dlogits = dlogits, a.z_stride = z_stride, a.d_stride = d_stride, a.T = n_tokens, a.V = n_vocab;
  a.z_type = z_type, a.d_type = d_type, a.accumulate = (flags & MOE_ACCUMULATE) != 0, a.scale = scale;
  DeviceGuard g(device);
  return launched(moe::launch_logprobs_grad(a, (hipStream_t)stream), me);
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
