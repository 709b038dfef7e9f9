// Head norms, backward.  With g = R^T dy, a = g w and rstd from x again:
//   dx = rstd (a - x rstd^2 mean(a x)),   dw = sum over tokens and heads of g x rstd
//
// x and dy are read once and dx is written once.  A lane has the same unit of
// every row, so it adds up its own channels of dw in registers; a workgroup
// leaves one row of partial sums, which a second kernel adds in a fixed order.
// [16384, 32 + 8, 128] bfloat16: 101 us, 5.0 TB/s (4.3 of it the second kernel).
// Loads before the angles, as in the forward pass, take registers that cost more
// (106 us).
#include "acp_dev_heads.hpp"

namespace acp {
namespace dev {

constexpr int kPassesInFlight = 2;

template <class T, bool PAIRS, bool WHOLE>
__device__ __forceinline__ void side_backward(const HeadsCore& A, const HeadGradSide& S, const HeadPlace& at,
                                              const Unit<T, PAIRS>& u, const Waves<kChunk<T>>& w, uint32_t from,
                                              uint32_t to, float (&da)[kChunk<T>], float (&db)[kChunk<T>]) {
  constexpr int V = kChunk<T>, U = kPassesInFlight;
  const bool real = at.token < A.tokens;
  const uint32_t token = real ? at.token : 0u;
  const char* x = token_row(A, S.x, token);
  const char* dy = token_row(A, S.dy, token);
  char* dx = token_row(A, S.dx, token);
  float wa[V], wb[V];
  load_weight<T, PAIRS, WHOLE>(S.weight, u, wa, wb);
  const float dim = static_cast<float>(A.dim);
  for (uint32_t p = from; p < to; p += U) {
    Piece<T, PAIRS, WHOLE> px[U], pg[U];
    uint32_t head[U];
    bool there[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      head[k] = ((p + k) << A.heads_log2) + at.slot;
      there[k] = real && p + k < to && head[k] < S.heads;
      px[k].load(x + head[k] * S.x.s[2], u, there[k]);
      pg[k].load(dy + head[k] * S.dy.s[2], u, there[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (p + k >= to) break;
      float a[V], b[V], ga[V], gb[V];
      px[k].values(u, there[k], a, b);
      pg[k].values(u, there[k], ga, gb);
      turn<PAIRS>(ga, gb, w, u.turned);
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], sum));
        dot = __builtin_fmaf(ga[i] * wa[i], a[i], __builtin_fmaf(gb[i] * wb[i], b[i], dot));
      }
      const float r = head_rstd(sum_lanes(sum, A.lanes_log2), dim, A.eps);
      const float m = sum_lanes(dot, A.lanes_log2) / dim * r * r;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (there[k]) {
          da[i] = __builtin_fmaf(ga[i], a[i] * r, da[i]);
          db[i] = __builtin_fmaf(gb[i], b[i] * r, db[i]);
        }
        a[i] = r * __builtin_fmaf(-a[i], m, ga[i] * wa[i]);
        b[i] = r * __builtin_fmaf(-b[i], m, gb[i] * wb[i]);
      }
      Piece<T, PAIRS, WHOLE>::store(false, dx + head[k] * S.dx.s[2], u, there[k], a, b);
    }
  }
}

template <class T, bool PAIRS, bool WHOLE>
__global__ __launch_bounds__(kHeadThreads) void heads_backward_kernel(const HeadsBackward A) {
  constexpr int V = kChunk<T>;
  constexpr uint32_t kWaves = kHeadThreads / 64;
  extern __shared__ float sums[];  // [wave][side][dim]
  float da[2][V], db[2][V];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) da[k][i] = db[k][i] = 0.0f;
  const uint32_t items = A.groups * A.parts.d, step = gridDim.x * kWaves;
  for (uint32_t wave = wave_index(); wave < items; wave += step) {
    const HeadPlace at(A, wave);
    const Unit<T, PAIRS> u(A, at.unit);
    Waves<V> w;
    if (A.rotated) {
      int32_t position = 0;
      if (at.token < A.tokens)
        position = A.positions ? A.positions[at.token]
                               : static_cast<int32_t>(at.token - divide(at.token, A.span) * A.span.d);
      w.template at<WHOLE>(A, u, position);
    }
    uint32_t from = at.pass, to = from + A.per_wave;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const HeadGradSide& S = A.side[k];
      const uint32_t end = to < S.passes ? to : S.passes;
      if (from < end) side_backward<T, PAIRS, WHOLE>(A, S, at, u, w, from, end, da[k], db[k]);
      from = from > S.passes ? from - S.passes : 0u;
      to = to > S.passes ? to - S.passes : 0u;
    }
  }
  if (A.side[0].part == nullptr && A.side[1].part == nullptr) return;
  // lanes of one unit, then the waves
  const uint32_t lane = threadIdx.x & 63u, row_lanes = 1u << A.lanes_log2;
  const Unit<T, PAIRS> u(A, lane & (row_lanes - 1u));
  float* mine = sums + (threadIdx.x >> 6) * 2u * A.dim;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      for (uint32_t d = row_lanes; d < 64u; d <<= 1) {
        da[k][i] += __shfl_xor(da[k][i], static_cast<int>(d));
        db[k][i] += __shfl_xor(db[k][i], static_cast<int>(d));
      }
      if (lane < row_lanes) {
        if (i < u.n[0]) mine[k * A.dim + u.at[0] + i] = da[k][i];
        if (i < u.n[1]) mine[k * A.dim + u.at[1] + i] = db[k][i];
      }
    }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < 2u * A.dim; c += kHeadThreads) {
    float* part = A.side[c >= A.dim].part;
    if (part == nullptr) continue;
    float v = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kWaves; ++k) v += sums[k * 2u * A.dim + c];
    part[static_cast<uint64_t>(blockIdx.x) * A.part_pitch + (c >= A.dim ? c - A.dim : c)] = v;
  }
}

// kHeadColumns columns of the parts: a lane adds every sixteenth row of one.
__global__ __launch_bounds__(kHeadThreads) void head_columns_kernel(const HeadColumns A) {
  constexpr uint32_t kRows = kHeadThreads / kHeadColumns;
  __shared__ float sums[kRows][kHeadColumns];
  const uint32_t col = threadIdx.x % kHeadColumns, row = threadIdx.x / kHeadColumns;
  const uint32_t c = blockIdx.x * kHeadColumns + col;
  const uint32_t side = c >= A.dim;
  float* out = c < 2u * A.dim ? A.out[side] : nullptr;
  float v = 0.0f;
  if (out != nullptr) {
#pragma unroll 8
    for (uint32_t r = row; r < A.rows; r += kRows) v += A.part[static_cast<uint64_t>(r) * A.pitch + c];
  }
  sums[row][col] = v;
  __syncthreads();
  if (row == 0 && out != nullptr) {
    v = 0.0f;
    for (uint32_t r = 0; r < kRows; ++r) v += sums[r][col];
    out[side ? c - A.dim : c] = v;
  }
}

}  // namespace dev

namespace {

template <class T>
const void* backward_kernel(const HeadsShape& k) {
  using namespace dev;
  return k.pairs ? (k.whole ? reinterpret_cast<const void*>(heads_backward_kernel<T, true, true>)
                            : reinterpret_cast<const void*>(heads_backward_kernel<T, true, false>))
                 : (k.whole ? reinterpret_cast<const void*>(heads_backward_kernel<T, false, true>)
                            : reinterpret_cast<const void*>(heads_backward_kernel<T, false, false>));
}

}  // namespace

hipError_t head_norm_backward_launch(const HeadsShape& k, const HeadsBackward& a, uint32_t workgroups, hipStream_t s) {
  const void* f = k.dt == kRowF16    ? backward_kernel<_Float16>(k)
                  : k.dt == kRowBF16 ? backward_kernel<dev::bf16_t>(k)
                                     : backward_kernel<float>(k);
  HeadsBackward copy = a;
  void* args[] = {&copy};
  const uint32_t lds = (kHeadThreads / 64) * 2u * a.dim * 4u;
  return hipLaunchKernel(f, dim3(workgroups), dim3(kHeadThreads), args, lds, s);
}

hipError_t head_columns_launch(const HeadColumns& a, hipStream_t s) {
  HeadColumns copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(dev::head_columns_kernel),
                         dim3((2u * a.dim + kHeadColumns - 1) / kHeadColumns), dim3(kHeadThreads), args, 0, s);
}

}  // namespace acp
