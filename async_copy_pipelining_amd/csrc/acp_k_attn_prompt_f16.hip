// Attention of many rows over caches that are read as f16.
#include "acp_dev_attn_prompt.hpp"

namespace acp {

hipError_t attend_prompt_f16(int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dev::attend_prompt_for<_Float16>(cache, padded, a, s);
}

}  // namespace acp
