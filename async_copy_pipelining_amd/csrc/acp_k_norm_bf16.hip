// Group norm of bf16 tensors.
#include "acp_norm_impl.hpp"

namespace acp {

hipError_t norm_launch_bf16(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s) {
  return norm::run<dev::bf16_t>(op, k, a, s);
}

}  // namespace acp
