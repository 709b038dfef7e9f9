// Rotary positions and head norms, forward: y = R(position) (x * rstd * w).
//
// Each element is read and written once; the angles of a unit are formed once
// for all heads of a token, so large calls are bound by HBM: [16384, 32 + 8, 128]
// bfloat16 turned in 58 us (5.7 TB/s), normed and turned in 60.  Small ones are
// bound by the chain from a position over its frequencies to the angles: 4.1 us
// for 16 tokens.
#include "acp_dev_heads.hpp"

namespace acp {
namespace dev {

// Passes in flight of queries, which mostly have several times the heads, and of keys.
constexpr int kPassesQ = 4, kPassesK = 2;

// The passes [from, to) of one side of a wave's tokens, the first U of them loaded.
template <class T, bool PAIRS, bool WHOLE, bool NORM, int U>
__device__ __forceinline__ void side_forward(const HeadsCore& A, const HeadSide& S, Passes<T, PAIRS, WHOLE, U>& in,
                                             const HeadPlace& at, const Unit<T, PAIRS>& u, const Waves<kChunk<T>>& w,
                                             uint32_t from, uint32_t to) {
  constexpr int V = kChunk<T>;
  if (from >= to) return;
  const bool real = at.token < A.tokens;
  const uint32_t token = real ? at.token : 0u;
  const char* x = token_row(A, S.x, token);
  char* y = token_row(A, S.y, token);
  float wa[V], wb[V];
  if constexpr (NORM) load_weight<T, PAIRS, WHOLE>(S.weight, u, wa, wb);
  for (uint32_t p = from; p < to; p += U) {
    if (p != from) in.load(A, x, S.x.s[2], u, real ? S.heads : 0u, at.slot, p, to);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (p + k >= to) break;
      const uint32_t head = in.head(A, p + k, at.slot);
      const bool there = real && head < S.heads;
      float a[V], b[V];
      in.piece[k].values(u, there, a, b);
      if constexpr (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], sum));
        const float r = head_rstd(sum_lanes(sum, A.lanes_log2), static_cast<float>(A.dim), A.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[i] = a[i] * r * wa[i];
          b[i] = b[i] * r * wb[i];
        }
      }
      turn<PAIRS>(a, b, w, u.turned);
      in.piece[k].store(!NORM && A.keep, y + head * S.y.s[2], u, there, a, b);
    }
  }
}

template <class T, bool PAIRS, bool WHOLE, bool NORM>
__global__ __launch_bounds__(kHeadThreads) void heads_forward_kernel(const HeadsForward A) {
  const uint32_t wave = wave_index();
  if (wave >= A.groups * A.parts.d) return;
  const HeadPlace at(A, wave);
  const Unit<T, PAIRS> u(A, at.unit);
  const bool real = at.token < A.tokens;
  const uint32_t token = real ? at.token : 0u;
  // the wave's passes of queries and keys, which follow one another
  const HeadSide &Q = A.side[0], &K = A.side[1];
  const uint32_t first = at.pass, last = first + A.per_wave;
  const uint32_t q_to = last < Q.passes ? last : Q.passes;
  const uint32_t k_from = first > Q.passes ? first - Q.passes : 0u, k_last = last > Q.passes ? last - Q.passes : 0u;
  const uint32_t k_to = k_last < K.passes ? k_last : K.passes;
  Passes<T, PAIRS, WHOLE, kPassesQ> q;
  Passes<T, PAIRS, WHOLE, kPassesK> k;
  q.load(A, token_row(A, Q.x, token), Q.x.s[2], u, real ? Q.heads : 0u, at.slot, first, q_to);
  k.load(A, token_row(A, K.x, token), K.x.s[2], u, real ? K.heads : 0u, at.slot, k_from, k_to);
  Waves<kChunk<T>> w;
  if (A.rotated) {
    int32_t position = 0;
    if (real)
      position = A.positions ? A.positions[at.token]
                             : static_cast<int32_t>(at.token - divide(at.token, A.span) * A.span.d);
    w.template at<WHOLE>(A, u, position);
  }
  side_forward<T, PAIRS, WHOLE, NORM>(A, Q, q, at, u, w, first, q_to);
  side_forward<T, PAIRS, WHOLE, NORM>(A, K, k, at, u, w, k_from, k_to);
}

}  // namespace dev

namespace {

template <class T, bool NORM>
const void* forward_kernel(const HeadsShape& k) {
  using namespace dev;
  const void* f = k.pairs ? (k.whole ? reinterpret_cast<const void*>(heads_forward_kernel<T, true, true, NORM>)
                                     : reinterpret_cast<const void*>(heads_forward_kernel<T, true, false, NORM>))
                          : (k.whole ? reinterpret_cast<const void*>(heads_forward_kernel<T, false, true, NORM>)
                                     : reinterpret_cast<const void*>(heads_forward_kernel<T, false, false, NORM>));
  return f;
}

template <bool NORM>
hipError_t forward_launch(const HeadsShape& k, const HeadsForward& a, hipStream_t s) {
  const void* f = k.dt == kRowF16    ? forward_kernel<_Float16, NORM>(k)
                  : k.dt == kRowBF16 ? forward_kernel<dev::bf16_t, NORM>(k)
                                     : forward_kernel<float, NORM>(k);
  constexpr uint32_t kWaves = kHeadThreads / 64;
  HeadsForward copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(f, dim3((a.groups * a.parts.d + kWaves - 1) / kWaves), dim3(kHeadThreads), args, 0, s);
}

}  // namespace

hipError_t rotate_launch(const HeadsShape& k, const HeadsForward& a, hipStream_t s) {
  return forward_launch<false>(k, a, s);
}
hipError_t head_norm_launch(const HeadsShape& k, const HeadsForward& a, hipStream_t s) {
  return forward_launch<true>(k, a, s);
}

}  // namespace acp
