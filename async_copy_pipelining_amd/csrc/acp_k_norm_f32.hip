// Group norm of f32 tensors.
#include "acp_norm_impl.hpp"

namespace acp {

hipError_t norm_launch_f32(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s) {
  return norm::run<float>(op, k, a, s);
}

}  // namespace acp
