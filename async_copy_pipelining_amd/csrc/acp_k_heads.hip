// Rotary positions and head norms, forward: y = R(position) (x * rstd * w).
//
// Each element is read and written once; the angles of a unit are formed once
// for all heads of a token, so large calls are bound by HBM.
#include "acp_dev_heads.hpp"

namespace acp {
namespace dev {

constexpr int kPassesInFlight = 4;

// The passes [from, to) of one side of a wave's tokens.
template <class T, bool PAIRS, bool WHOLE, bool NORM>
__device__ __forceinline__ void side_forward(const HeadsCore& A, const HeadSide& S, const HeadPlace& at,
                                             const Unit<T, PAIRS>& u, const Waves<kChunk<T>>& w, uint32_t from,
                                             uint32_t to) {
  constexpr int V = kChunk<T>, U = kPassesInFlight;
  const bool real = at.token < A.tokens;
  const uint32_t token = real ? at.token : 0u;
  const char* x = token_row(A, S.x, token);
  char* y = token_row(A, S.y, token);
  float wa[V], wb[V];
  if constexpr (NORM) load_weight<T, PAIRS, WHOLE>(S.weight, u, wa, wb);
  for (uint32_t p = from; p < to; p += U) {
    Piece<T, PAIRS, WHOLE> piece[U];
    uint32_t head[U];
    bool there[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      head[k] = ((p + k) << A.heads_log2) + at.slot;
      there[k] = real && p + k < to && head[k] < S.heads;
      piece[k].load(x + head[k] * S.x.s[2], u, there[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (p + k >= to) break;
      float a[V], b[V];
      piece[k].values(u, there[k], a, b);
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
      piece[k].store(y + head[k] * S.y.s[2], u, there[k], a, b);
    }
  }
}

template <class T, bool PAIRS, bool WHOLE, bool NORM>
__global__ __launch_bounds__(kHeadThreads) void heads_forward_kernel(const HeadsForward A) {
  const uint32_t wave = wave_index();
  if (wave >= A.groups * A.parts.d) return;
  const HeadPlace at(A, wave);
  const Unit<T, PAIRS> u(A, at.unit);
  Waves<kChunk<T>> w;
  if (A.rotated) {
    int32_t position = 0;
    if (at.token < A.tokens)
      position = A.positions ? A.positions[at.token]
                             : static_cast<int32_t>(at.token - divide(at.token, A.span) * A.span.d);
    w.template at<WHOLE>(A, u.first, u.turned, position);
  }
  uint32_t from = at.pass, to = from + A.per_wave;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const HeadSide& S = A.side[k];
    const uint32_t end = to < S.passes ? to : S.passes;
    if (from < end) side_forward<T, PAIRS, WHOLE, NORM>(A, S, at, u, w, from, end);
    from = from > S.passes ? from - S.passes : 0u;
    to = to > S.passes ? to - S.passes : 0u;
  }
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
