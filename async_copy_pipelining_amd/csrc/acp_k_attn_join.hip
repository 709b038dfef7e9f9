// Attention whose keys were split: the partial results of a row joined, in the
// order of the splits; and the choice of the type.
#include "acp_dev_attn.hpp"

namespace acp {
namespace dev {

// A wave has a row: output = sum w_j o_j / sum w_j l_j, w_j = 2^(m_j - max m).
template <class T, int M>
__global__ __launch_bounds__(kAttendThreads) void attend_join_kernel(const AttendArgs A) {
  const uint32_t id = wave_index(), lane = threadIdx.x & 63u;
  if (id >= A.tokens * A.heads.d) return;
  const uint32_t token = divide(id, A.heads), head = id - token * A.heads.d;
  const uint32_t seq = sequence_of(A.batch, token);
  if (seq >= A.batch.sequences) return;
  uint32_t slot = 0, start = token;
  const uint32_t kv = divide(head, A.group);
  if (A.batch.starts != nullptr) {
    if (A.batch.starts[seq] < 0 || static_cast<int32_t>(token) < A.batch.starts[seq]) return;
    start = static_cast<uint32_t>(A.batch.starts[seq]);
    slot = static_cast<uint32_t>(static_cast<uint64_t>(start) * A.group.d / M) + seq;
  } else {
    slot = seq * ((A.group.d + M - 1) / M);
  }
  const uint32_t row = (token - start) * A.group.d + (head - kv * A.group.d);
  Tile t;
  if (!t.find<M>(A, slot + row / M)) return;
  const uint32_t splits = t.splits(A);
  if (splits == 1u) return;  // written already
  const uint64_t rows = static_cast<uint64_t>(A.tokens) * A.heads.d;
  float m = -__builtin_inff();
  for (uint32_t j = lane; j < splits; j += 64u) m = __builtin_fmaxf(m, A.stat[2 * (j * rows + id)]);
  m = as_float(static_cast<uint32_t>(over_lanes(static_cast<int>(as_bits(m)), 6, [](int a, int b) {
    return static_cast<int>(as_bits(__builtin_fmaxf(as_float(static_cast<uint32_t>(a)), as_float(static_cast<uint32_t>(b)))));
  })));
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
#pragma unroll 4
  for (uint32_t j = 0; j < splits; ++j) {
    const uint64_t at = j * rows + id;
    const float w = exp2_of(A.stat[2 * at] - base);
    l = __builtin_fmaf(w, A.stat[2 * at + 1], l);
    const float* p = A.part + at * A.dim;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 64u * e < A.dim) o[e] = __builtin_fmaf(w, p[lane + 64u * e], o[e]);
  }
  char* y = head_row(A, A.out, token, head);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 64u * e < A.dim)
      put_value(y + (lane + 64u * e) * 2, l == 0.0f ? 0.0f : o[e] / l, static_cast<const T*>(nullptr));
}

}  // namespace dev

hipError_t attend_step_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dt == kRowF16 ? attend_step_f16(cache, padded, a, s) : attend_step_bf16(cache, padded, a, s);
}

hipError_t attend_prompt_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dt == kRowF16 ? attend_prompt_f16(cache, padded, a, s) : attend_prompt_bf16(cache, padded, a, s);
}

hipError_t attend_join_launch(int dt, int tile_rows, const AttendArgs& a, hipStream_t s) {
  using namespace dev;
  const bool few = tile_rows == kStepRows;
  const void* f = dt == kRowF16 ? (few ? reinterpret_cast<const void*>(attend_join_kernel<_Float16, kStepRows>)
                                       : reinterpret_cast<const void*>(attend_join_kernel<_Float16, kPromptRows>))
                                : (few ? reinterpret_cast<const void*>(attend_join_kernel<bf16_t, kStepRows>)
                                       : reinterpret_cast<const void*>(attend_join_kernel<bf16_t, kPromptRows>));
  constexpr uint32_t kWaves = kAttendThreads / 64;
  AttendArgs copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(f, dim3((a.tokens * a.heads.d + kWaves - 1) / kWaves), dim3(kAttendThreads), args, 0, s);
}

}  // namespace acp
