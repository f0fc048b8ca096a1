// The feed-forward's products in fp32.
#include "feed_forward_gemm.hpp"

namespace rnnk {
hipError_t launch_feed_f32(int op, const FeedArgs& a, const FeedPlan& p, hipStream_t st) {
  return launch_feed_type<float>(op, a, p, st);
}
}  // namespace rnnk
