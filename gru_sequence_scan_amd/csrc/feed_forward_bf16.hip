// The feed-forward's products in bf16.
#include "feed_forward_gemm.hpp"

namespace rnnk {
hipError_t launch_feed_bf16(int op, const FeedArgs& a, const FeedPlan& p, hipStream_t st) {
  return launch_feed_type<bf16>(op, a, p, st);
}
}  // namespace rnnk
