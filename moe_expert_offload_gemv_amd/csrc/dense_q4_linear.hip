// dense_q4_linear.hip - the dense products with 4-bit weights whose results pass through bias,
// activation, factor and residual before they are stored (moe_q4_linear).
namespace moe {
namespace {
constexpr bool kEpilogue = true;
}
}  // namespace moe
#include "dense_q4_dev.h"

namespace moe {

hipError_t launch_q4_linear(const Q4Args& a, hipStream_t s) { return launch_q4(a, s); }

}  // namespace moe
