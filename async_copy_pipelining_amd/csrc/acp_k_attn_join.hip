// Attention whose keys were split: the partial results of a row joined, in the
// order of the splits; and the choice of the type.
#include "acp_dev_attn.hpp"

namespace acp {
namespace dev {

// output = sum w_j o_j / sum w_j l_j, w_j = 2^(m_j - max m).  A lane has four
// channels, `lanes` of them a row, and 2^shares_log2 such groups of lanes share a
// row's partial results, whose sums meet in LDS: a long context of few rows would
// wait for one after another.  Join of 32 tokens over up to 32768 positions: 6.7 us.
template <class T, int M>
__global__ __launch_bounds__(kAttendThreads) void attend_join_kernel(const AttendArgs A, int lanes_log2, int shares_log2,
                                                                     Div blocks) {
  __shared__ float sums[kAttendThreads][6];
  const uint32_t rows_each = kAttendThreads >> (lanes_log2 + shares_log2);
  const uint32_t item = divide(blockIdx.x, blocks), block = blockIdx.x - item * blocks.d;
  const uint32_t slot = divide(item, A.kv_heads), group = item - slot * A.kv_heads.d;
  Tile t;
  if (!t.find<M>(A, slot)) return;
  const uint32_t* record = A.joins + 2 * static_cast<uint64_t>(item);
  const uint32_t first = record[0], splits = record[1];
  if (splits < 2u) return;  // written already
  // starts that do not ascend give tiles without a record
  if (first >= A.shares || splits > A.shares - first) return;
  const uint32_t shares = 1u << shares_log2;
  const uint32_t c = (threadIdx.x & ((1u << lanes_log2) - 1u)) * 4u;
  const uint32_t share = threadIdx.x >> lanes_log2 & (shares - 1u);
  // row of the tile, and which of the group's heads
  const uint32_t index = block * rows_each + (threadIdx.x >> (lanes_log2 + shares_log2));
  const uint32_t side = index / M, row = t.first + index % M;
  const bool real = row < static_cast<uint32_t>(t.rows) && side >> A.side_log2 == 0u;
  uint32_t token, head;
  t.place(A, real ? row : t.first, (group << A.side_log2) + (real ? side : 0u), &token, &head);
  const uint32_t each = static_cast<uint32_t>(M) << A.side_log2;
  float m = -__builtin_inff(), l = 0.0f;
  af4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 4;
  if (real) {
    for (uint32_t j0 = share; j0 < splits; j0 += U * shares) {
      float mj[U], lj[U];
      af4 oj[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const uint32_t j = j0 + k * shares;
        mj[k] = -__builtin_inff();
        lj[k] = 0.0f;
        oj[k] = af4{0.0f, 0.0f, 0.0f, 0.0f};
        if (j < splits) {
          // the tile is the last of its first share's, and the first of the others'
          const uint64_t at = ((static_cast<uint64_t>(first + j) * A.kv_heads.d + group) * 2u + (j == 0u)) * each + index;
          mj[k] = A.stat[2 * at];
          lj[k] = A.stat[2 * at + 1];
          if (c < A.dim) oj[k] = *reinterpret_cast<const af4*>(A.part + at * A.dim + c);
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < U; ++k) top = __builtin_fmaxf(top, mj[k]);
      const float base = top == -__builtin_inff() ? 0.0f : top;
      const float keep = exp2_of(m - base);
      o *= keep;
      l *= keep;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float w = exp2_of(mj[k] - base);
        l = __builtin_fmaf(w, lj[k], l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(w, oj[k][e], o[e]);
      }
      m = top;
    }
  }
  if (shares > 1u) {
    float* mine = sums[threadIdx.x];
    mine[0] = m;
    mine[1] = l;
#pragma unroll
    for (int e = 0; e < 4; ++e) mine[2 + e] = o[e];
    __syncthreads();
    if (share != 0u) return;
    const uint32_t step = 1u << lanes_log2;
    float top = m;
    for (uint32_t k = 1; k < shares; ++k) top = __builtin_fmaxf(top, sums[threadIdx.x + k * step][0]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
    l = 0.0f;
    o = af4{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t k = 0; k < shares; ++k) {
      const float* s = sums[threadIdx.x + k * step];
      const float w = exp2_of(s[0] - base);
      l = __builtin_fmaf(w, s[1], l);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(w, s[2 + e], o[e]);
    }
  }
  if (!real || c >= A.dim) return;
  char* y = head_row(A, A.out, token, head) + c * 2;
  float f[8] = {};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = l == 0.0f ? 0.0f : o[e] / l;
  const rw4 w = narrow(f, static_cast<const T*>(nullptr));
  *reinterpret_cast<rw2_any*>(y) = rw2{w[0], w[1]};
}

}  // namespace dev

hipError_t attend_step_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dt == kRowF16 ? attend_step_f16(cache, padded, a, s) : attend_step_bf16(cache, padded, a, s);
}

hipError_t attend_prompt_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s) {
  return dt == kRowF16 ? attend_prompt_f16(cache, padded, a, s) : attend_prompt_bf16(cache, padded, a, s);
}

hipError_t attend_join_launch(int dt, int tile_rows, const AttendArgs& a, const JoinShape& k, hipStream_t s) {
  using namespace dev;
  const void* f = nullptr;
#define ACP_JOIN(M)                                                                          \
  if (tile_rows == M)                                                                        \
  f = dt == kRowF16 ? reinterpret_cast<const void*>(attend_join_kernel<_Float16, M>)         \
                    : reinterpret_cast<const void*>(attend_join_kernel<bf16_t, M>)
  ACP_JOIN(kStepRows);
  ACP_JOIN(128);
  ACP_JOIN(256);
#undef ACP_JOIN
  if (f == nullptr) return hipErrorInvalidValue;
  AttendArgs copy = a;
  JoinShape shape = k;
  void* args[] = {&copy, &shape.lanes_log2, &shape.shares_log2, &shape.blocks};
  return hipLaunchKernel(f, dim3(a.kv_heads.d * a.slots.d * k.blocks.d), dim3(kAttendThreads), args, 0, s);
}

}  // namespace acp
