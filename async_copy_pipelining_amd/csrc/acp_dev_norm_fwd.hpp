// Group norm with an activation: forward kernels.
#pragma once

#include "acp_dev_norm.hpp"

namespace acp {
namespace dev {

// Writes the 8-bit form of a chunk of x in the pass that normalises it.
template <class T, int KIND, int PK>
struct Saver {
  static constexpr int V = kChunk<T>;
  static constexpr bool LINEAR = KIND != kNormAny;
  Walk<LINEAR> codes, scales;

  __device__ __forceinline__ Saver(const NormForwardSaved& A, const Spot& w)
      : codes(walk_codes<V, LINEAR>(A, A.codes, w)), scales(walk_scales<LINEAR>(A, A.scales, w)) {}
  // all lanes of a scale block come here together; n: channels to write
  __device__ __forceinline__ void save(const NormCore& A, const Spot& w, uint32_t k, int n, const float (&x)[V]) const {
    const float s = block_scale(PK - 1, block_amax(x, A.lb_log2));
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = x[e];
    const Codes<V> c = encode<T>(PK - 1, v, s);
    store_codes<V, KIND == kNormAny>(codes.at(A, k), n, c);
    if (n > 0) {
      if ((w.cl & ((1u << A.lb_log2) - 1u)) == 0) *reinterpret_cast<float*>(scales.at(A, k)) = s;
    }
  }
};

template <class T, int KIND>
struct Saver<T, KIND, 0> {
  __device__ __forceinline__ Saver(const NormForward&, const Spot&) {}
};

template <int PK>
using ForwardArgs = std::conditional_t<PK != 0, NormForwardSaved, NormForward>;

// ---------------------------------------------------------------- per row

// One row a sample: rows are samples, and a group lies in 2^group_lanes_log2
// lanes of a wave, so mean and variance are two trains of cross-lane moves on
// values that stay in registers, with no LDS and no barrier.  Each chunk's
// place takes the one U steps on as soon as it is used.  Bound by HBM:
// [16384, 4096] bfloat16 in heads of 64 channels 48.9 us, 5.7 TB/s; [32, 2048]
// float16 3.7 us, where the launch is all of it (medians of 30 traced calls).
template <class T, int PK, int ACT>
__global__ __launch_bounds__(kRowThreads) void norm_row_kernel(const ForwardArgs<PK> A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  const Spot w(A, blockIdx.x, V);
  const Walk<true> px = walk<T, true>(A, A.x, w), py = walk<T, true>(A, A.y, w);
  rw4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, false, false>(px.at(A, u), w.channels(A, u), A.c >= V);
  const Saver<T, kNormWhole, PK> saver(A, w);
  const Params<V> p(A, w.c, w.valid);
  const float inv = 1.0f / static_cast<float>(A.per_group);
  const bool lead = (w.cl & ((1u << A.group_lanes_log2) - 1u)) == 0;
  const uint32_t g = divide(w.c, A.per);
  if (w.rl >= A.row_lanes) return;
  for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((k0 + u) * w.step >= w.rows) break;
      const int n = w.channels(A, k0 + u);
      float x[V];
      widen(raw[u], x, static_cast<const T*>(nullptr));
      raw[u] = load_chunk<T, false, false>(px.at(A, k0 + U + u), w.channels(A, k0 + U + u), A.c >= V);
      if constexpr (PK != 0) saver.save(A, w, k0 + u, n, x);
      // 1 / channels is a power of two here: each term divided by it keeps its
      // bits, and no sum of finite values is past float32
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) sum = __builtin_fmaf(x[e], inv, sum);
      const float m = sum_lanes(sum, A.group_lanes_log2);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[e] -= m;
        sq = __builtin_fmaf(x[e], x[e], sq);
      }
      sq = sum_lanes(sq, A.group_lanes_log2);
      // squares past float32: NaN, as join_lanes has it, not a root of zero
      const float rstd = rsqrt_any(__builtin_fmaf(sq - sq == 0.0f ? sq : as_float(0x7FC00000u), inv, A.eps));
      if (n > 0 && lead) {
        const uint64_t at = static_cast<uint64_t>(w.r0 + w.rl + (k0 + u) * w.step) * A.groups + g;
        if (A.mean) A.mean[at] = m;
        if (A.rstd) A.rstd[at] = rstd;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] * rstd, p.gamma[e], p.beta[e]);
      act_values<ACT, V>(x);
      store_chunk<T, false>(py.at(A, k0 + u), n, narrow(x, static_cast<const T*>(nullptr)));
    }
  }
}

// ---------------------------------------------------------------- slab

// All rows of a sample for a block of whole groups: a lane holds up to
// kSlabRows chunks, so x is read once.  A workgroup's loads, its join and its
// stores follow one another; the other workgroups of the CU fill the gaps.
// [128, 500, 1024] float16, 32 groups: 53 us without an activation (4.9 TB/s
// in row segments of 128 bytes), 65 us with gelu (68 us traced, in which the
// vector units issue 68 % of the time and 16 waves a CU wait 45 % of theirs), 78
// to 90 us traced with silu and an i8 form saved (330 MB, 3.7 to 4.2 TB/s; 94 to
// 120 us with 16 chunks in each of 512 lanes).
template <class T, int KIND, int PK, int ACT>
__global__ __launch_bounds__(kSlabThreads) void norm_slab_kernel(const ForwardArgs<PK> A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = kSlabRows;
  extern __shared__ float2 sh[];
  const Spot w(A, near_group(blockIdx.x, gridDim.x), V);
  const Walk<LINEAR> px = walk<T, LINEAR>(A, A.x, w);
  rw4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * A.row_lanes < w.rows) raw[u] = load_chunk<T, false, TAIL>(px.at(A, u), w.channels(A, u), A.c >= V);
  LaneStats<V, WHOLE> st;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * A.row_lanes >= w.rows) break;
    float x[V];
    place_tail<T, TAIL>(&raw[u], w.channels(A, u), A.c >= V);
    widen(raw[u], x, static_cast<const T*>(nullptr));
    if (u == 0) st.first(x);
    if (w.channels(A, u) > 0) st.add(x);
  }
  const RunRows rr(A, w.rows, w.step);
  st.put(sh, w.valid > 0 ? static_cast<float>(rr.of(w.rl)) : 0.0f);
  __syncthreads();
  const BlockGroups b(A, w.blk, A.lanes.d * V);
  const int lg = join_log2(b.g1 - b.g0 + 1, blockDim.x);
  float2* stats = sh + blockDim.x * (WHOLE ? 1 : V);
  const float total = static_cast<float>(A.rows) * static_cast<float>(A.per_group);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += blockDim.x >> lg) {
    const float2 v = join_lanes<V, WHOLE>(A, sh, b, w.blk, g, rr, lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0) {
      const float rstd = rsqrt_any(v.y / total + A.eps);
      stats[g - b.g0] = make_float2(v.x, rstd);
      const uint64_t at = static_cast<uint64_t>(w.n) * A.groups + g;
      if (A.mean) A.mean[at] = v.x;
      if (A.rstd) A.rstd[at] = rstd;
    }
  }
  const Params<V> p(A, w.c, w.valid);
  __syncthreads();
  if (w.rl >= A.row_lanes) return;
  float mu[WHOLE ? 1 : V], scale[V];
  if constexpr (WHOLE) {
    const float2 v = w.valid > 0 ? stats[divide(w.c, A.per) - b.g0] : make_float2(0.0f, 0.0f);
    mu[0] = v.x;
#pragma unroll
    for (int e = 0; e < V; ++e) scale[e] = p.gamma[e] * v.y;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 v = e < w.valid ? stats[divide(w.c + e, A.per) - b.g0] : make_float2(0.0f, 0.0f);
      mu[e] = v.x;
      scale[e] = p.gamma[e] * v.y;
    }
  }
  const Walk<LINEAR> py = walk<T, LINEAR>(A, A.y, w);
  const Saver<T, KIND, PK> saver(A, w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * A.row_lanes >= w.rows) break;
    const int n = w.channels(A, u);
    float x[V];
    widen(raw[u], x, static_cast<const T*>(nullptr));
    if constexpr (PK != 0) saver.save(A, w, u, n, x);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] - mu[WHOLE ? 0 : e], scale[e], p.beta[e]);
    act_values<ACT, V>(x);
    store_chunk<T, TAIL>(py.at(A, u), n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// ---------------------------------------------------------------- by parts

// Statistics of a run of rows: (mean, sum of squared deviations) of every
// group's piece in this channel block, into part[n][g][run][piece].  The
// loads keep the data in the caches for the second pass.  [4, 64, 64, 320]
// bfloat16, groups of 10 channels: 6.4 us (median of 30 traced calls) for 10.5
// MB, of which about 2.5 us pass before a kernel's first loads arrive.
template <class T, int KIND>
__global__ __launch_bounds__(kRowThreads) void norm_stats_kernel(const NormStats A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = 2 * kRowUnroll;
  __shared__ float2 sh[kRowThreads * (WHOLE ? 1 : V)];
  const Spot w(A, blockIdx.x, V);
  const Walk<LINEAR> px = walk<T, LINEAR>(A, A.x, w);
  LaneStats<V, WHOLE> st;
  if (w.valid > 0) {
    for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
      rw4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, true, TAIL>(px.at(A, k0 + u), w.channels(A, k0 + u), A.c >= V);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[V];
        place_tail<T, TAIL>(&raw[u], w.channels(A, k0 + u), A.c >= V);
        widen(raw[u], x, static_cast<const T*>(nullptr));
        if (k0 == 0 && u == 0) st.first(x);
        if (w.channels(A, k0 + u) > 0) st.add(x);
      }
    }
  }
  const RunRows rr(A, w.rows, w.step);
  st.put(sh, w.valid > 0 ? static_cast<float>(rr.of(w.rl)) : 0.0f);
  __syncthreads();
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, kRowThreads);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += kRowThreads >> lg) {
    const float2 v = join_lanes<V, WHOLE>(A, sh, b, w.blk, g, rr, lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0)
      reinterpret_cast<float2*>(A.part)[((static_cast<uint64_t>(w.n) * A.groups + g) * A.runs.d + w.run) * A.pieces +
                                        (w.blk - g * A.per_group / width)] = v;
  }
}

// mean and rstd of group g of sample n from its parts, in all of the 2^lg
// lanes that share the group.
__device__ __forceinline__ float2 join_parts(const NormCore& A, uint32_t n, uint32_t g, uint32_t width, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const float2* part = reinterpret_cast<const float2*>(A.part) +
                       (static_cast<uint64_t>(n) * A.groups + g) * A.parts * A.pieces;
  const float m0 = part[0].x;
  // rows of run i: `all` full rounds of the deal, and what it has of the last
  const uint32_t round = A.parts * A.row_lanes, all = A.rows / round, rest = A.rows - all * round;
  auto rows_of = [&](uint32_t i) {
    const uint32_t from = i * A.row_lanes, more = rest > from ? rest - from : 0u;
    return static_cast<float>(all * A.row_lanes + (more < A.row_lanes ? more : A.row_lanes));
  };
  float a1 = 0.0f, a2 = 0.0f;
  if (A.pieces == 1) {
    constexpr int U = 8;  // parts in flight
    const float ch = static_cast<float>(A.per_group);
    for (uint32_t e = lane; e < A.parts; e += U << lg) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = part[e + (u << lg) < A.parts ? e + (u << lg) : e];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = e + (u << lg);
        const float cnt = i >= A.parts ? 0.0f : rows_of(i) * ch;
        const float d = v[u].x - m0;
        a1 = __builtin_fmaf(cnt, d, a1);
        a2 += __builtin_fmaf(cnt * d, d, i >= A.parts ? 0.0f : v[u].y);
      }
    }
  } else {
    const uint32_t b0 = g * A.per_group / width;
    for (uint32_t e = lane; e < A.parts * A.pieces; e += 1u << lg) {
      const uint32_t run = e / A.pieces, piece = e - run * A.pieces;
      const uint32_t ch = piece_channels(A, g, b0 + piece, width);
      if (ch == 0) continue;
      const float cnt = rows_of(run) * static_cast<float>(ch);
      const float2 v = part[e];
      const float d = v.x - m0;
      a1 = __builtin_fmaf(cnt, d, a1);
      a2 += __builtin_fmaf(cnt * d, d, v.y);
    }
  }
  a1 = sum_lanes(a1, lg);
  a2 = sum_lanes(a2, lg);
  const float total = static_cast<float>(A.rows) * static_cast<float>(A.per_group);
  const float m = a1 / total;
  const float var = __builtin_fmaxf(0.0f, __builtin_fmaf(-a1, m, a2)) / total;
  // as in join_lanes: what is not finite stays a NaN
  return make_float2(m0 + m, rsqrt_any((a2 - a2 == 0.0f ? var : as_float(0x7FC00000u)) + A.eps));
}

// y, and where asked mean, rstd and the 8-bit form of x.  The first chunks
// are on their way while the parts are joined, by every workgroup for its own
// groups, which saves a launch of about 2.5 us.  [4, 64, 64, 320] bfloat16
// with silu: 8.9 us (median of 30 traced calls); x passes the L2s once more.
template <class T, int KIND, int PK, int ACT>
__global__ __launch_bounds__(kRowThreads) void norm_apply_kernel(const ForwardArgs<PK> A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 sh[];
  const Spot w(A, blockIdx.x, V);
  const Walk<LINEAR> px = walk<T, LINEAR>(A, A.x, w), py = walk<T, LINEAR>(A, A.y, w);
  const Saver<T, KIND, PK> saver(A, w);
  rw4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, false, TAIL>(px.at(A, u), w.channels(A, u), A.c >= V);
  const Params<V> p(A, w.c, w.valid);
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, kRowThreads);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += kRowThreads >> lg) {
    const float2 v = join_parts(A, w.n, g, width, lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0) {
      sh[g - b.g0] = v;
      if (w.run == 0 && g * A.per_group >= b.lo) {
        const uint64_t at = static_cast<uint64_t>(w.n) * A.groups + g;
        if (A.mean) A.mean[at] = v.x;
        if (A.rstd) A.rstd[at] = v.y;
      }
    }
  }
  __syncthreads();
  if (w.rl >= A.row_lanes) return;
  float mu[V], scale[V], rstd0 = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (WHOLE && e > 0) {
      mu[e] = mu[0];
      scale[e] = p.gamma[e] * rstd0;
      continue;
    }
    const float2 v = e < w.valid ? sh[divide(w.c + e, A.per) - b.g0] : make_float2(0.0f, 0.0f);
    mu[e] = v.x;
    scale[e] = p.gamma[e] * v.y;
    if (e == 0) rstd0 = v.y;
  }
  for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((k0 + u) * w.step >= w.rows) break;
      const int n = w.channels(A, k0 + u);
      float x[V];
      place_tail<T, TAIL>(&raw[u], n, A.c >= V);
      widen(raw[u], x, static_cast<const T*>(nullptr));
      raw[u] = load_chunk<T, false, TAIL>(px.at(A, k0 + U + u), w.channels(A, k0 + U + u), A.c >= V);
      if constexpr (PK != 0) saver.save(A, w, k0 + u, n, x);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] - mu[e], scale[e], p.beta[e]);
      act_values<ACT, V>(x);
      store_chunk<T, TAIL>(py.at(A, k0 + u), n, narrow(x, static_cast<const T*>(nullptr)));
    }
  }
}

}  // namespace dev
}  // namespace acp
