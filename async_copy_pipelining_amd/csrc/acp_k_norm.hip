// Group norm: the sums of columns, which are the same for every type, and the
// choice of the type.
#include "acp_dev_norm_bwd.hpp"

namespace acp {
namespace dev {

__global__ __launch_bounds__(kRowThreads) void norm_columns_kernel(const NormCore A) {
  sum_columns(A, blockIdx.x, 2u * static_cast<uint64_t>(A.c));
}

}  // namespace dev

uint32_t norm_column_grid(const NormArgs& a) { return a.dgamma || a.dbeta ? (2u * a.c + kColumns - 1u) / kColumns : 0u; }

hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s) {
  const uint32_t grid = norm_column_grid(a);
  if (grid == 0) return hipSuccess;
  NormCore core = a;
  void* args[] = {&core};
  return hipLaunchKernel(reinterpret_cast<const void*>(dev::norm_columns_kernel), dim3(grid), dim3(kRowThreads), args, 0, s);
}

hipError_t norm_launch(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return norm_launch_f16(op, k, a, s);
  if (k.dt == kRowBF16) return norm_launch_bf16(op, k, a, s);
  return norm_launch_f32(op, k, a, s);
}

}  // namespace acp
