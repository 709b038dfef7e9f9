// Group norm of f16 tensors.
#include "acp_norm_impl.hpp"

namespace acp {

hipError_t norm_launch_f16(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s) {
  return norm::run<_Float16>(op, k, a, s);
}

}  // namespace acp
