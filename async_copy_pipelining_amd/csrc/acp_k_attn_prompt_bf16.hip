// Attention of many rows over caches that are read as bf16.
#include "acp_dev_attn_prompt.hpp"

namespace acp {

hipError_t attend_prompt_bf16(int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dev::attend_prompt_for<dev::bf16_t>(cache, padded, a, s);
}

}  // namespace acp
