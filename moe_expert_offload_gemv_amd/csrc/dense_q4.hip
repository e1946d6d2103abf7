// dense_q4.hip - the dense products with 4-bit weights without an epilogue (moe_q4_matmul),
// and the workspace of both kinds.
namespace moe {
namespace {
constexpr bool kEpilogue = false;
}
}  // namespace moe
#include "dense_q4_dev.h"

namespace moe {

int64_t q4_workspace_bytes(int64_t T, int64_t N, int64_t K, int32_t x_type) {
  const int WK = wide_split(T, N, K, x_type);
  if (!WK) return 0;
  const int terms = x_type == MOE_F32 ? terms_of<MOE_F32>() : 1, runs = x_type == MOE_Q8_32 ? runs_of<MOE_Q8_32>() : 1;
  return Operand::make(nullptr, std::min(T, kPassTokens), K, terms, runs, wide_side(WK)).bytes;
}

hipError_t launch_q4_matmul(const Q4Args& a, hipStream_t s) { return launch_q4(a, s); }

}  // namespace moe
