// Group norm with an activation, forward.
#include "acp_dev_norm.hpp"

namespace acp {
namespace dev {

// Writes the 8-bit form of a chunk of x in the pass that normalises it.
// TAIL: a row may end inside a chunk.
template <class T, bool LINEAR, bool TAIL>
struct Saver {
  static constexpr int V = kChunk<T>;
  Walk<LINEAR> codes, scales;

  __device__ __forceinline__ Saver(const NormArgs& A, const Spot& w)
      : codes(walk_codes<V, LINEAR>(A, w)), scales(walk_scales<LINEAR>(A, w)) {}
  // all lanes of a scale block come here together; n: channels to write
  __device__ __forceinline__ void save(const NormArgs& A, const Spot& w, uint32_t k, int n, const float (&x)[V]) const {
    const float s = block_scale(A.format, block_amax(x, A.lb_log2));
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = x[e];
    const Codes<V> c = encode<T>(A.format, v, s);
    store_codes<V, TAIL>(codes.at(A, k), n, c);
    if (n > 0) {
      if ((w.cl & ((1u << A.lb_log2) - 1u)) == 0) *reinterpret_cast<float*>(scales.at(A, k)) = s;
    }
  }
};

// ---------------------------------------------------------------- per row

// One row a sample: rows are samples, and a group lies in 2^group_lanes_log2
// lanes of a wave.
template <class T, bool SAVE>
__global__ __launch_bounds__(kRowThreads) void norm_row_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  const Spot w(A, blockIdx.x, V);
  const Walk<true> px = walk<T, true>(A, A.x, w), py = walk<T, true>(A, A.y, w);
  const Saver<T, true, false> saver(A, w);
  const Params<V> p(A, w.c, w.valid);
  const float inv = 1.0f / static_cast<float>(A.per_group);
  const bool lead = (w.cl & ((1u << A.group_lanes_log2) - 1u)) == 0;
  const uint32_t g = w.c / A.per_group;
  if (w.rl >= A.row_lanes) return;
  for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
    rw4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, false, false>(px.at(A, k0 + u), w.channels(A, k0 + u));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((k0 + u) * A.row_lanes >= w.rows) break;
      const int n = w.channels(A, k0 + u);
      float x[V];
      widen(raw[u], x, static_cast<const T*>(nullptr));
      if constexpr (SAVE) saver.save(A, w, k0 + u, n, x);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) sum += x[e];
      const float m = sum_lanes(sum, A.group_lanes_log2) * inv;
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[e] -= m;
        sq = __builtin_fmaf(x[e], x[e], sq);
      }
      const float rstd = rsqrt_any(__builtin_fmaf(sum_lanes(sq, A.group_lanes_log2), inv, A.eps));
      if (n > 0 && lead) {
        const uint64_t at = static_cast<uint64_t>(w.r0 + w.rl + (k0 + u) * A.row_lanes) * A.groups + g;
        if (A.mean) A.mean[at] = m;
        if (A.rstd) A.rstd[at] = rstd;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] * rstd, p.gamma[e], p.beta[e]);
      act_values(A.act, x);
      store_chunk<T, false>(py.at(A, k0 + u), n, narrow(x, static_cast<const T*>(nullptr)));
    }
  }
}

// ---------------------------------------------------------------- slab

// All rows of a sample for a block of whole groups: a lane holds up to
// kSlabRows chunks, so x is read once.
template <class T, bool WHOLE, bool SAVE>
__global__ __launch_bounds__(kSlabThreads) void norm_slab_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kSlabRows;
  extern __shared__ float2 sh[];
  const Spot w(A, near_group(blockIdx.x, gridDim.x), V);
  const Walk<true> px = walk<T, true>(A, A.x, w);
  rw4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * A.row_lanes < w.rows) raw[u] = load_chunk<T, false, !WHOLE>(px.at(A, u), w.channels(A, u));
  LaneStats<V, WHOLE> st;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * A.row_lanes >= w.rows) break;
    float x[V];
    widen(raw[u], x, static_cast<const T*>(nullptr));
    if (u == 0) st.first(x);
    if (w.channels(A, u) > 0) st.add(x);
  }
  st.put(sh, static_cast<float>(lane_rows(A, w.rows, w.rl)));
  __syncthreads();
  const BlockGroups b(A, w.blk, A.lanes.d * V);
  const int lg = join_log2(b.g1 - b.g0 + 1, blockDim.x);
  float2* stats = sh + blockDim.x * (WHOLE ? 1 : V);
  const float total = static_cast<float>(A.rows) * static_cast<float>(A.per_group);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += blockDim.x >> lg) {
    const float2 v = join_lanes<V, WHOLE>(A, sh, b, w.blk, g, w.rows, lg);
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
    const float2 v = w.valid > 0 ? stats[w.c / A.per_group - b.g0] : make_float2(0.0f, 0.0f);
    mu[0] = v.x;
#pragma unroll
    for (int e = 0; e < V; ++e) scale[e] = p.gamma[e] * v.y;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 v = e < w.valid ? stats[(w.c + e) / A.per_group - b.g0] : make_float2(0.0f, 0.0f);
      mu[e] = v.x;
      scale[e] = p.gamma[e] * v.y;
    }
  }
  const Walk<true> py = walk<T, true>(A, A.y, w);
  const Saver<T, true, !WHOLE> saver(A, w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u * A.row_lanes >= w.rows) break;
    const int n = w.channels(A, u);
    float x[V];
    widen(raw[u], x, static_cast<const T*>(nullptr));
    if constexpr (SAVE) saver.save(A, w, u, n, x);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] - mu[WHOLE ? 0 : e], scale[e], p.beta[e]);
    act_values(A.act, x);
    store_chunk<T, !WHOLE>(py.at(A, u), n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// ---------------------------------------------------------------- by parts

// Statistics of a run of rows: (mean, sum of squared deviations) of every
// group's piece in this channel block, into part[n][g][run][piece].  The
// loads keep the data in the caches for the second pass.
template <class T, bool WHOLE, bool LINEAR>
__global__ __launch_bounds__(kRowThreads) void norm_stats_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = 2 * kRowUnroll;
  __shared__ float2 sh[kRowThreads * (WHOLE ? 1 : V)];
  const Spot w(A, blockIdx.x, V);
  const Walk<LINEAR> px = walk<T, LINEAR>(A, A.x, w);
  LaneStats<V, WHOLE> st;
  if (w.valid > 0) {
    for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
      rw4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, true, !WHOLE>(px.at(A, k0 + u), w.channels(A, k0 + u));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[V];
        widen(raw[u], x, static_cast<const T*>(nullptr));
        if (k0 == 0 && u == 0) st.first(x);
        if (w.channels(A, k0 + u) > 0) st.add(x);
      }
    }
  }
  st.put(sh, static_cast<float>(lane_rows(A, w.rows, w.rl)));
  __syncthreads();
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, kRowThreads);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += kRowThreads >> lg) {
    const float2 v = join_lanes<V, WHOLE>(A, sh, b, w.blk, g, w.rows, lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0)
      reinterpret_cast<float2*>(A.part)[((static_cast<uint64_t>(w.n) * A.groups + g) * A.runs.d + w.run) * A.pieces +
                                        (w.blk - g * A.per_group / width)] = v;
  }
}

// mean and rstd of group g of sample n from its parts, in all of the 2^lg
// lanes that share the group.
__device__ __forceinline__ float2 join_parts(const NormArgs& A, uint32_t n, uint32_t g, uint32_t width, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const float2* part = reinterpret_cast<const float2*>(A.part) +
                       (static_cast<uint64_t>(n) * A.groups + g) * A.parts * A.pieces;
  const float m0 = part[0].x;
  const float last = static_cast<float>(A.rows - (A.parts - 1) * A.part_rows);
  const float full = static_cast<float>(A.part_rows);
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
        const float cnt = i >= A.parts ? 0.0f : (i + 1 == A.parts ? last : full) * ch;
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
      const float cnt = (run + 1 == A.parts ? last : full) * static_cast<float>(ch);
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
// are on their way while the parts are joined.
template <class T, bool WHOLE, bool SAVE, bool LINEAR>
__global__ __launch_bounds__(kRowThreads) void norm_apply_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 sh[];
  const Spot w(A, blockIdx.x, V);
  const Walk<LINEAR> px = walk<T, LINEAR>(A, A.x, w), py = walk<T, LINEAR>(A, A.y, w);
  const Saver<T, LINEAR, !WHOLE> saver(A, w);
  rw4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load_chunk<T, false, !WHOLE>(px.at(A, u), w.channels(A, u));
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
    const float2 v = e < w.valid ? sh[(w.c + e) / A.per_group - b.g0] : make_float2(0.0f, 0.0f);
    mu[e] = v.x;
    scale[e] = p.gamma[e] * v.y;
    if (e == 0) rstd0 = v.y;
  }
  for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((k0 + u) * A.row_lanes >= w.rows) break;
      const int n = w.channels(A, k0 + u);
      float x[V];
      widen(raw[u], x, static_cast<const T*>(nullptr));
      if constexpr (SAVE) saver.save(A, w, k0 + u, n, x);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] - mu[e], scale[e], p.beta[e]);
      act_values(A.act, x);
      // the chunk U steps on takes this one's place before its store is issued
      raw[u] = load_chunk<T, false, !WHOLE>(px.at(A, k0 + U + u), w.channels(A, k0 + U + u));
      store_chunk<T, !WHOLE>(py.at(A, k0 + u), n, narrow(x, static_cast<const T*>(nullptr)));
    }
  }
}

}  // namespace dev

namespace {

template <class K>
hipError_t launch_norm(K kernel, const NormArgs& a, uint32_t threads, uint32_t lds, hipStream_t s) {
  void* args[] = {const_cast<NormArgs*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(a.main_grid), dim3(threads), args, lds, s);
}

// groups that one channel block may touch
uint32_t block_groups(const NormArgs& a, int v) {
  const uint32_t g = (a.lanes.d * static_cast<uint32_t>(v) - 1) / a.per_group + 2;
  return g < a.groups ? g : a.groups;
}

template <class T>
hipError_t row_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  return k.packed ? launch_norm(dev::norm_row_kernel<T, true>, a, kRowThreads, 0, s)
                  : launch_norm(dev::norm_row_kernel<T, false>, a, kRowThreads, 0, s);
}

template <class T, bool WHOLE>
hipError_t slab_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  constexpr int V = dev::kChunk<T>;
  const uint32_t lds = (k.threads * (WHOLE ? 1 : V) + block_groups(a, V)) * 8u;
  return k.packed ? launch_norm(dev::norm_slab_kernel<T, WHOLE, true>, a, k.threads, lds, s)
                  : launch_norm(dev::norm_slab_kernel<T, WHOLE, false>, a, k.threads, lds, s);
}

template <class T, bool WHOLE>
hipError_t stats_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  return k.linear ? launch_norm(dev::norm_stats_kernel<T, WHOLE, true>, a, kRowThreads, 0, s)
                  : launch_norm(dev::norm_stats_kernel<T, WHOLE, false>, a, kRowThreads, 0, s);
}

template <class T, bool WHOLE>
hipError_t apply_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  const uint32_t lds = block_groups(a, dev::kChunk<T>) * 8u;
  if (k.linear)
    return k.packed ? launch_norm(dev::norm_apply_kernel<T, WHOLE, true, true>, a, kRowThreads, lds, s)
                    : launch_norm(dev::norm_apply_kernel<T, WHOLE, false, true>, a, kRowThreads, lds, s);
  return k.packed ? launch_norm(dev::norm_apply_kernel<T, WHOLE, true, false>, a, kRowThreads, lds, s)
                  : launch_norm(dev::norm_apply_kernel<T, WHOLE, false, false>, a, kRowThreads, lds, s);
}

}  // namespace

hipError_t norm_row_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return row_t<_Float16>(k, a, s);
  if (k.dt == kRowBF16) return row_t<dev::bf16_t>(k, a, s);
  return row_t<float>(k, a, s);
}

hipError_t norm_slab_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return k.whole ? slab_t<_Float16, true>(k, a, s) : slab_t<_Float16, false>(k, a, s);
  if (k.dt == kRowBF16) return k.whole ? slab_t<dev::bf16_t, true>(k, a, s) : slab_t<dev::bf16_t, false>(k, a, s);
  return k.whole ? slab_t<float, true>(k, a, s) : slab_t<float, false>(k, a, s);
}

hipError_t norm_stats_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return k.whole ? stats_t<_Float16, true>(k, a, s) : stats_t<_Float16, false>(k, a, s);
  if (k.dt == kRowBF16) return k.whole ? stats_t<dev::bf16_t, true>(k, a, s) : stats_t<dev::bf16_t, false>(k, a, s);
  return k.whole ? stats_t<float, true>(k, a, s) : stats_t<float, false>(k, a, s);
}

hipError_t norm_apply_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return k.whole ? apply_t<_Float16, true>(k, a, s) : apply_t<_Float16, false>(k, a, s);
  if (k.dt == kRowBF16) return k.whole ? apply_t<dev::bf16_t, true>(k, a, s) : apply_t<dev::bf16_t, false>(k, a, s);
  return k.whole ? apply_t<float, true>(k, a, s) : apply_t<float, false>(k, a, s);
}

}  // namespace acp
