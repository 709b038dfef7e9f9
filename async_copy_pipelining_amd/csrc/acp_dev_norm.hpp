// Group norm with an activation over channels-last rows: what its forward and
// backward kernels share.
//
// x[n, r, c], groups of `per_group` neighbouring channels, M = rows * per_group:
//   mu = sum x / M,  rstd = (sum (x - mu)^2 / M + eps)^-1/2
//   z = (x - mu) rstd,  u = z gamma[c] + beta[c],  y = act(u)
//   a = dy act'(u),  dbeta[c] = sum a,  dgamma[c] = sum a z
//   dx = rstd (gamma a - sum(gamma a) / M - z sum(gamma a z) / M)
//
// A workgroup covers a block of channels (`lanes` chunks of 16 bytes) and
// `row_lanes` rows at a time, so that a lane keeps its channels: parameters
// and per-channel sums stay in its registers.
//
// Three forms, each bound by the bytes it moves; the host takes the first
// that holds:
// * per row (one row a sample, a group's chunks a power of two of lanes): the
//   group sums are cross-lane moves within a wave;
// * slab (all rows of a sample, for a block of whole groups, fit a
//   workgroup's registers): x, and dy, are read once;
// * by parts: one kernel leaves partial sums of runs of rows in the
//   workspace, the next one joins them and makes the second pass.
// All sums have a fixed order, so results are the same from run to run.
// Kernels are built for one activation and one 8-bit form each: a wave's code
// has to come into the instruction cache, and for small tensors that is most
// of its time.
//
// Statistics: a lane sums d = x - k and d^2 where k is a value that it meets
// itself.  With k a member of the set, the sum of squares is at most about n
// times the sum of squared deviations, so the subtraction that removes the
// mean loses at most a factor n of the lane's few rows, whatever the data's
// offset or outliers.  Lanes and parts are joined the same way, each as
// (mean, sum of squared deviations) about the first one's mean.  Per row the
// group's sum is taken whole and the squares about its mean: that sum rounds at
// the size of the mean, a few 2^-24 of it (a second mean of what is left took 3
// to 6 % more time for float32).
#pragma once

#include <type_traits>

#include "acp_dev_rows.hpp"

namespace acp {
namespace dev {

// Where a lane of a workgroup works.
struct Spot {
  uint32_t n, run, blk;
  uint32_t cl, rl;   // chunk lane and row lane
  uint32_t c;        // first channel
  int valid;         // channels of the chunk; 0 for a lane without one
  // Steps of row_lanes rows are dealt out to the runs in turn, so that all
  // workgroups together read consecutive rows: row lane rl of the run has the
  // rows r0 + rl + k step, those below r0 + rows.
  uint32_t r0, rows, step;

  __device__ __forceinline__ Spot(const NormCore& A, uint32_t wg, int v) {
    const uint32_t q = divide(wg, A.runs);
    run = wg - q * A.runs.d;
    n = divide(q, A.blocks);
    blk = q - n * A.blocks.d;
    rl = divide(threadIdx.x, A.lanes);
    cl = threadIdx.x - rl * A.lanes.d;
    c = (blk * A.lanes.d + cl) * v;
    valid = 0;
    if (rl < A.row_lanes && c < A.c) valid = A.c - c < static_cast<uint32_t>(v) ? static_cast<int>(A.c - c) : v;
    r0 = run * A.row_lanes;
    step = A.runs.d * A.row_lanes;
    rows = A.rows > r0 ? A.rows - r0 : 0u;
  }
  // channels of row step k: none past the tensor's rows
  __device__ __forceinline__ int channels(const NormCore& A, uint32_t k) const {
    return rl + k * step < rows ? valid : 0;
  }
};

// The lane's chunk of one tensor, row step by row step.  LINEAR: a uniform
// address that moves by a uniform step, and a 32-bit lane offset.
template <bool LINEAR>
struct Walk {
  const RowTensor* t;
  char* base;
  uint32_t off;        // LINEAR
  int64_t step;
  uint32_t n, row;     // else: sample and the lane's first row
  uint32_t col;        // ... and bytes into the row

  __device__ __forceinline__ Walk(const NormCore& A, const RowTensor& rt, const Spot& w, uint32_t block_bytes,
                                  uint32_t lane_bytes)
      : t(&rt) {
    if constexpr (LINEAR) {
      base = rt.p + w.n * rt.s[0] + w.r0 * rt.s[2] + block_bytes;
      off = w.rl * static_cast<uint32_t>(rt.s[2]) + lane_bytes;
      step = w.step * rt.s[2];
    } else {
      step = w.step;
      n = w.n;
      row = w.r0 + w.rl;
      col = block_bytes + lane_bytes;
    }
  }
  __device__ __forceinline__ char* at(const NormCore& A, uint32_t k) const {
    if constexpr (LINEAR) {
      return base + k * step + off;
    } else {
      const uint32_t r = row + k * static_cast<uint32_t>(step), a = divide(r, A.row2);
      return t->p + n * t->s[0] + a * t->s[1] + (r - a * A.row2.d) * t->s[2] + col;
    }
  }
};

template <class T, bool LINEAR>
__device__ __forceinline__ Walk<LINEAR> walk(const NormCore& A, const RowTensor& t, const Spot& w) {
  return Walk<LINEAR>(A, t, w, w.blk * A.lanes.d * 16u, w.cl * 16u);
}
// the saved form's codes (V bytes a chunk) and scales (one for 2^lb_log2 chunks)
template <int V, bool LINEAR>
__device__ __forceinline__ Walk<LINEAR> walk_codes(const NormCore& A, const RowTensor& t, const Spot& w) {
  return Walk<LINEAR>(A, t, w, w.blk * A.lanes.d * V, w.cl * V);
}
template <bool LINEAR>
__device__ __forceinline__ Walk<LINEAR> walk_scales(const NormCore& A, const RowTensor& t, const Spot& w) {
  // a channel block that starts inside a scale block: both terms are of the whole row
  const uint32_t first = w.blk * A.lanes.d;
  return Walk<LINEAR>(A, t, w, (first >> A.lb_log2) * 4u,
                      (((first + w.cl) >> A.lb_log2) - (first >> A.lb_log2)) * 4u);
}

// Consecutive workgroups share cache lines at their edges: they run on one
// XCD, b -> (b % 8) * (g / 8) + b / 8.
__device__ __forceinline__ uint32_t near_group(uint32_t b, uint32_t g) {
  const uint32_t per = g >> 3;
  return b < per * 8u ? (b & 7u) * per + (b >> 3) : b;
}

// Lanes that share the sums of one group when `threads` lanes join `groups`
// of them: a power of two up to 64.
__device__ __forceinline__ int join_log2(uint32_t groups, uint32_t threads) {
  int k = 6;
  while (k > 0 && (groups << k) > threads) --k;
  return k;
}

// The groups that a channel block touches.
struct BlockGroups {
  uint32_t lo, hi, g0, g1;  // channels [lo, hi), groups g0..g1
  __device__ __forceinline__ BlockGroups(const NormCore& A, uint32_t blk, uint32_t width) {
    lo = blk * width;
    hi = lo + width < A.c ? lo + width : A.c;
    g0 = divide(lo, A.per);
    g1 = divide(hi - 1, A.per);
  }
};

// Channels of group g that lie in channel block blk.
__device__ __forceinline__ uint32_t piece_channels(const NormCore& A, uint32_t g, uint32_t blk, uint32_t width) {
  const uint32_t lo = g * A.per_group > blk * width ? g * A.per_group : blk * width;
  uint32_t hi = (g + 1) * A.per_group < (blk + 1) * width ? (g + 1) * A.per_group : (blk + 1) * width;
  hi = hi < A.c ? hi : A.c;
  return hi > lo ? hi - lo : 0u;
}

// 1 / sqrt(v) by the hardware's reciprocal root (1 ulp), which takes no
// denormal: those are scaled up first.
__device__ __forceinline__ float rsqrt_any(float v) {
  const bool tiny = v < 0x1p-96f;
  return __builtin_amdgcn_rsqf(tiny ? v * 0x1p96f : v) * (tiny ? 0x1p48f : 1.0f);
}

// A lane's statistics of the rows it meets.  WHOLE (its channels are of one
// group): one mean for all of them; else one a channel.
template <int V, bool WHOLE>
struct LaneStats {
  static constexpr int K = WHOLE ? 1 : V;
  float k0[K], s1[V], s2[V];
  bool any = false;

  __device__ __forceinline__ LaneStats() {
#pragma unroll
    for (int e = 0; e < V; ++e) s1[e] = s2[e] = 0.0f;
#pragma unroll
    for (int e = 0; e < K; ++e) k0[e] = 0.0f;
  }
  __device__ __forceinline__ void first(const float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < K; ++e) k0[e] = x[e];
  }
  __device__ __forceinline__ void add(const float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // WHOLE: two chains of sums are enough to hide an addition's latency
      const int s = WHOLE ? e & 1 : e;
      const float d = x[e] - k0[WHOLE ? 0 : e];
      s1[s] += d;
      s2[s] = __builtin_fmaf(d, d, s2[s]);
    }
  }
  // (mean, sum of squared deviations) of what n rows gave, into sh[lane * K + e]
  __device__ __forceinline__ void put(float2* sh, float n) {
    if constexpr (WHOLE) {
      const float a = s1[0] + s1[1], q = s2[0] + s2[1];
      const float m = n > 0.0f ? a / (n * V) : 0.0f;
      sh[threadIdx.x] = make_float2(k0[0] + m, __builtin_fmaxf(0.0f, __builtin_fmaf(-a, m, q)));
    } else {
      const float inv = n > 0.0f ? 1.0f / n : 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float m = s1[e] * inv;
        sh[threadIdx.x * V + e] =
            make_float2(k0[e] + m, __builtin_fmaxf(0.0f, __builtin_fmaf(-s1[e], m, s2[e])));
      }
    }
  }
};

// Rows that each row lane of a run has: `all`, and one more below `more`.
struct RunRows {
  uint32_t all, more;
  __device__ __forceinline__ RunRows(const NormCore& A, uint32_t rows, uint32_t step) {
    all = rows / step;
    more = rows - all * step;
    more = more < A.row_lanes ? more : A.row_lanes;
  }
  __device__ __forceinline__ uint32_t of(uint32_t rl) const { return all + (rl < more ? 1u : 0u); }
  __device__ __forceinline__ uint32_t total(const NormCore& A) const { return all * A.row_lanes + more; }
  __device__ __forceinline__ uint32_t lanes(const NormCore& A) const { return all ? A.row_lanes : more; }
};

// Joins the lanes' statistics of group g's piece in this channel block: its
// mean and squared deviations, in all 2^lg lanes that share the group.
template <int V, bool WHOLE>
__device__ __forceinline__ float2 join_lanes(const NormCore& A, const float2* sh, const BlockGroups& b, uint32_t blk,
                                             uint32_t g, const RunRows& rr, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const uint32_t width = A.lanes.d * V;
  const uint32_t p0 = g * A.per_group > b.lo ? g * A.per_group : b.lo;
  const uint32_t ch = piece_channels(A, g, blk, width);
  const uint32_t cols = WHOLE ? ch / V : ch;               // entries of a row lane
  const uint32_t first = WHOLE ? (p0 - b.lo) / V : p0 - b.lo;
  const uint32_t stride = WHOLE ? A.lanes.d : width;
  const uint32_t used = rr.lanes(A);
  const float m0 = sh[first].x;
  float a1 = 0.0f, a2 = 0.0f;
  uint32_t row = lane / cols, col = lane - row * cols;
  const uint32_t drow = (1u << lg) / cols, dcol = (1u << lg) - drow * cols;
  while (row < used) {
    const float2 v = sh[row * stride + first + col];
    const float n = static_cast<float>(rr.of(row) * (WHOLE ? V : 1));
    const float d = v.x - m0;
    a1 = __builtin_fmaf(n, d, a1);
    a2 += __builtin_fmaf(n * d, d, v.y);
    row += drow;
    col += dcol;
    if (col >= cols) {
      col -= cols;
      ++row;
    }
  }
  a1 = sum_lanes(a1, lg);
  a2 = sum_lanes(a2, lg);
  const float m = a1 / (static_cast<float>(rr.total(A)) * static_cast<float>(ch));
  const float q = __builtin_fmaxf(0.0f, __builtin_fmaf(-a1, m, a2));
  // the maximum drops a NaN: a piece with a NaN or an infinity, or whose
  // squared deviations overflow, keeps a NaN
  return make_float2(m0 + m, a2 - a2 == 0.0f ? q : as_float(0x7FC00000u));
}

// What a lane keeps of its channels.
template <int V>
struct Params {
  float gamma[V], beta[V];

  __device__ __forceinline__ Params(const NormCore& A, uint32_t c, int valid) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      gamma[e] = 1.0f;
      beta[e] = 0.0f;
    }
    if (A.gamma) load(A.gamma + c, valid, gamma);
    if (A.beta) load(A.beta + c, valid, beta);
  }
  __device__ static __forceinline__ void load(const float* p, int valid, float (&out)[V]) {
    if (valid == V) {
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const rw4 r = reinterpret_cast<const rw4_any*>(p)[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b = r[e];
          out[4 * k + e] = as_float(b);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < valid) out[e] = p[e];
    }
  }
};

}  // namespace dev
}  // namespace acp
