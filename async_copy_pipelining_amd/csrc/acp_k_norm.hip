// Group norm with an activation over channels-last rows, forward and backward.
//
// x[n, r, c], groups of `per_group` neighbouring channels, M = rows * per_group:
//   mu = sum x / M,  rstd = (sum (x - mu)^2 / M + eps)^-1/2
//   u = (x - mu) rstd gamma[c] + beta[c],  y = act(u)
//   z = (x - mu) rstd,  a = dy act'(u)
//   dbeta[c] = sum a,  dgamma[c] = sum a z
//   dx = rstd (gamma a - sum(gamma a) / M - z sum(gamma a z) / M)
//
// A workgroup covers a block of channels (`lanes` chunks of 16 bytes) and
// `row_lanes` rows at a time, so that a lane keeps its channels: parameters
// and per-channel sums stay in its registers.
//
// Two forms:
// * per row (one row a sample, a group's chunks a power of two of lanes): the
//   group sums are cross-lane moves in one wave; one pass over the data;
// * by parts: one kernel leaves partial sums of runs of rows in the workspace,
//   the next one joins them and makes the second pass.  All sums have a fixed
//   order, so results are the same from run to run.
//
// Statistics: a lane sums d = x - k and d^2 where k is the first value that
// it meets in that channel.  With k a member of the set, the sum of squares
// is at most about n times the sum of squared deviations, so the subtraction
// that removes the mean loses at most a factor n of the lane's few rows,
// whatever the data's offset or outliers.  Lanes, waves and runs are joined
// the same way, each as (mean, sum of squared deviations) about the first
// part's mean.
#include "acp_dev_rows.hpp"

namespace acp {
namespace dev {

// Where a lane of a workgroup works.
struct Spot {
  uint32_t n, chunk, blk;
  uint32_t cl, rl;   // chunk lane and row lane
  uint32_t c;        // first channel
  int valid;         // channels of the chunk
  uint32_t r0, r1;   // rows of the run

  __device__ __forceinline__ Spot(const NormArgs& A, uint32_t wg, int v) {
    const uint32_t q = wg / A.chunks;
    chunk = wg - q * A.chunks;
    n = q / A.blocks;
    blk = q - n * A.blocks;
    rl = divide(threadIdx.x, A.lanes);
    cl = threadIdx.x - rl * A.lanes.d;
    c = (blk * A.lanes.d + cl) * v;
    valid = 0;
    if (rl < A.row_lanes && c < A.c) valid = A.c - c < static_cast<uint32_t>(v) ? static_cast<int>(A.c - c) : v;
    r0 = chunk * A.rpc;
    r1 = A.rows - r0 < A.rpc ? A.rows : r0 + A.rpc;
  }
};

__device__ __forceinline__ char* row_at(const NormArgs& A, const RowTensor& t, uint32_t n, uint32_t r) {
  const uint32_t a = divide(r, A.row2);
  return t.p + n * t.s[0] + a * t.s[1] + (r - a * A.row2.d) * t.s[2];
}

__device__ __forceinline__ float sum_lanes(float v, int log2n) {
  for (int k = 0; k < log2n; ++k) v += __shfl_xor(v, 1 << k);
  return v;
}

// Channels of group g that lie in channel block blk.
__device__ __forceinline__ uint32_t piece_channels(const NormArgs& A, uint32_t g, uint32_t blk, uint32_t width) {
  const uint32_t lo = g * A.per_group > blk * width ? g * A.per_group : blk * width;
  uint32_t hi = (g + 1) * A.per_group < (blk + 1) * width ? (g + 1) * A.per_group : (blk + 1) * width;
  hi = hi < A.c ? hi : A.c;
  return hi > lo ? hi - lo : 0u;
}

// Lanes that share the sums of one group when a workgroup joins `groups` of
// them: a power of two up to 64, with groups * lanes about the workgroup.
__device__ __forceinline__ int join_log2(uint32_t groups) {
  int k = 6;
  while (k > 0 && (groups << k) > kRowThreads) --k;
  return k;
}

// ---------------------------------------------------------------- forward, by parts

// Statistics of a run of rows: (mean, sum of squared deviations) of every
// group's piece in this channel block, into part[n][g][chunk][piece].
// WHOLE: a chunk's channels are of one group.
template <class T, bool WHOLE>
__global__ __launch_bounds__(kRowThreads) void norm_stats_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  __shared__ float2 sh[kRowThreads * (WHOLE ? 1 : V)];
  const Spot w(A, blockIdx.x, V);
  const uint32_t width = A.lanes.d * V;
  float k0[V], s1[V], s2[V];
#pragma unroll
  for (int e = 0; e < V; ++e) k0[e] = s1[e] = s2[e] = 0.0f;
  if (w.valid > 0 && w.r0 + w.rl < w.r1) {
    widen(load_chunk<T>(row_at(A, A.x, w.n, w.r0 + w.rl) + static_cast<int64_t>(w.c) * sizeof(T), w.valid), k0,
          static_cast<const T*>(nullptr));
    for (uint32_t r = w.r0 + w.rl; r < w.r1; r += U * A.row_lanes) {
      rw4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t ru = r + u * A.row_lanes;
        raw[u] = load_chunk<T>(row_at(A, A.x, w.n, ru < w.r1 ? ru : r) + static_cast<int64_t>(w.c) * sizeof(T), w.valid);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + u * A.row_lanes >= w.r1) break;
        float x[V];
        widen(raw[u], x, static_cast<const T*>(nullptr));
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = x[e] - k0[e];
          s1[e] += d;
          s2[e] = __builtin_fmaf(d, d, s2[e]);
        }
      }
    }
  }
  // this lane's rows, and each channel's mean and squared deviations
  const uint32_t rows = w.r1 - w.r0;
  const float nt = rows > w.rl ? static_cast<float>((rows - w.rl - 1) / A.row_lanes + 1) : 0.0f;
  const float inv = nt > 0.0f ? 1.0f / nt : 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float m = s1[e] * inv;
    s2[e] = __builtin_fmaxf(0.0f, __builtin_fmaf(-s1[e], m, s2[e]));
    k0[e] += m;
  }
  if constexpr (WHOLE) {
    float d1 = 0.0f, d2 = 0.0f, q = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = k0[e] - k0[0];
      d1 += d;
      d2 = __builtin_fmaf(d, d, d2);
      q += s2[e];
    }
    const float m = d1 * (1.0f / V);
    sh[threadIdx.x] = make_float2(k0[0] + m, q + nt * __builtin_fmaxf(0.0f, __builtin_fmaf(-d1, m, d2)));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) sh[threadIdx.x * V + e] = make_float2(k0[e], s2[e]);
  }
  __syncthreads();
  // entry e of group g: row lane e / cols, and of that the piece's column
  // e % cols (a chunk of V channels, or one channel)
  const uint32_t lo = w.blk * width;
  const uint32_t hi = lo + width < A.c ? lo + width : A.c;
  const uint32_t g0 = lo / A.per_group, g1 = (hi - 1) / A.per_group;
  const int lg = join_log2(g1 - g0 + 1);
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const uint32_t used = rows < A.row_lanes ? rows : A.row_lanes;
  for (uint32_t g = g0 + (threadIdx.x >> lg); g <= g1; g += kRowThreads >> lg) {
    const uint32_t p0 = g * A.per_group > lo ? g * A.per_group : lo;
    const uint32_t ch = piece_channels(A, g, w.blk, width);
    const uint32_t cols = WHOLE ? ch / V : ch;
    const uint32_t first = WHOLE ? (p0 - lo) / V : p0 - lo;
    const float m0 = sh[first].x;
    float a1 = 0.0f, a2 = 0.0f;
    for (uint32_t e = lane; e < cols * used; e += 1u << lg) {
      const uint32_t row = e / cols, col = e - row * cols;
      const float2 v = sh[(WHOLE ? row * A.lanes.d : row * A.lanes.d * V) + first + col];
      const float n = static_cast<float>(((rows - row - 1) / A.row_lanes + 1) * (WHOLE ? V : 1));
      const float d = v.x - m0;
      a1 = __builtin_fmaf(n, d, a1);
      a2 += __builtin_fmaf(n * d, d, v.y);
    }
    a1 = sum_lanes(a1, lg);
    a2 = sum_lanes(a2, lg);
    if (lane == 0) {
      const float total = static_cast<float>(rows) * static_cast<float>(ch);
      const float m = a1 / total;
      float2* out = reinterpret_cast<float2*>(A.part);
      const uint64_t at = ((static_cast<uint64_t>(w.n) * A.groups + g) * A.chunks + w.chunk) * A.pieces +
                          (w.blk - g * A.per_group / width);
      out[at] = make_float2(m0 + m, __builtin_fmaxf(0.0f, __builtin_fmaf(-a1, m, a2)));
    }
  }
}

// mean and rstd of group g of sample n from its parts; all lanes of the
// 2^lg that share the group get them.
__device__ __forceinline__ float2 join_parts(const NormArgs& A, uint32_t n, uint32_t g, uint32_t width, uint32_t lane,
                                             int lg) {
  const float2* part = reinterpret_cast<const float2*>(A.part) +
                       (static_cast<uint64_t>(n) * A.groups + g) * A.chunks * A.pieces;
  const uint32_t b0 = g * A.per_group / width;
  const float m0 = part[0].x;
  float a1 = 0.0f, a2 = 0.0f;
  for (uint32_t e = lane; e < A.chunks * A.pieces; e += 1u << lg) {
    const uint32_t chunk = e / A.pieces, piece = e - chunk * A.pieces;
    const uint32_t ch = piece_channels(A, g, b0 + piece, width);
    if (ch == 0) continue;
    const uint32_t r0 = chunk * A.rpc;
    const float cnt = static_cast<float>(A.rows - r0 < A.rpc ? A.rows - r0 : A.rpc) * static_cast<float>(ch);
    const float2 v = part[e];
    const float d = v.x - m0;
    a1 = __builtin_fmaf(cnt, d, a1);
    a2 += __builtin_fmaf(cnt * d, d, v.y);
  }
  a1 = sum_lanes(a1, lg);
  a2 = sum_lanes(a2, lg);
  const float total = static_cast<float>(A.rows) * static_cast<float>(A.per_group);
  const float m = a1 / total;
  const float var = __builtin_fmaxf(0.0f, __builtin_fmaf(-a1, m, a2)) / total;
  // the maximum drops a NaN: a group with a NaN or an infinity, or whose
  // squared deviations overflow, keeps a NaN
  const float keep = a2 - a2 == 0.0f ? var : as_float(0x7FC00000u);
  return make_float2(m0 + m, 1.0f / sqrtf(keep + A.eps));
}

// ---------------------------------------------------------------- forward, second pass

// y, and where asked mean, rstd and the 8-bit form of x.
template <class T, bool PER_ROW, bool SAVE>
__global__ __launch_bounds__(kRowThreads) void norm_apply_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 stats[];  // by parts: mean and rstd of the block's groups
  const Spot w(A, blockIdx.x, V);
  float mu[V], scale[V], shift[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const bool in = e < w.valid;
    scale[e] = in && A.gamma ? A.gamma[w.c + e] : 1.0f;
    shift[e] = in && A.beta ? A.beta[w.c + e] : 0.0f;
  }
  if constexpr (!PER_ROW) {
    const uint32_t width = A.lanes.d * V;
    const uint32_t lo = w.blk * width;
    const uint32_t hi = lo + width < A.c ? lo + width : A.c;
    const uint32_t g0 = lo / A.per_group, g1 = (hi - 1) / A.per_group;
    const int lg = join_log2(g1 - g0 + 1);
    const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
    for (uint32_t g = g0 + (threadIdx.x >> lg); g <= g1; g += kRowThreads >> lg) {
      const float2 v = join_parts(A, w.n, g, width, lane, lg);
      if (lane == 0) {
        stats[g - g0] = v;
        if (w.chunk == 0 && g * A.per_group >= lo) {
          if (A.mean) A.mean[static_cast<uint64_t>(w.n) * A.groups + g] = v.x;
          if (A.rstd) A.rstd[static_cast<uint64_t>(w.n) * A.groups + g] = v.y;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 v = e < w.valid ? stats[(w.c + e) / A.per_group - g0] : make_float2(0.0f, 0.0f);
      mu[e] = v.x;
      scale[e] *= v.y;
    }
  }
  if (w.rl >= A.row_lanes) return;
  for (uint32_t rb = w.r0; rb < w.r1; rb += U * A.row_lanes) {
    rw4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = rb + u * A.row_lanes + w.rl;
      raw[u] = load_chunk<T>(row_at(A, A.x, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), r < w.r1 ? w.valid : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (rb + u * A.row_lanes >= w.r1) break;
      const uint32_t r = rb + u * A.row_lanes + w.rl;
      const bool live = r < w.r1 && w.valid > 0;
      float x[V];
      widen(raw[u], x, static_cast<const T*>(nullptr));
      if constexpr (SAVE) {
        const float s = block_scale(A.format, block_amax(x, A.lb_log2));
        float kept[V];
#pragma unroll
        for (int e = 0; e < V; ++e) kept[e] = x[e];
        const Codes<V> codes = encode<T>(A.format, kept, s);
        if (live) {
          store_codes<V>(row_at(A, A.px.codes, w.n, r) + w.c, w.valid, codes);
          if ((w.cl & ((1u << A.lb_log2) - 1u)) == 0) {
            const uint32_t per = (A.c + (V << A.lb_log2) - 1u) / (V << A.lb_log2);  // scale blocks of a row
            A.px.scales[(static_cast<uint64_t>(w.n) * A.rows + r) * per + ((w.c / V) >> A.lb_log2)] = s;
          }
        }
      }
      if constexpr (PER_ROW) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) sum += x[e];
        const float inv = 1.0f / static_cast<float>(A.per_group);
        const float m = sum_lanes(sum, A.group_lanes_log2) * inv;
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[e] -= m;
          sq = __builtin_fmaf(x[e], x[e], sq);
        }
        const float rstd = 1.0f / sqrtf(sum_lanes(sq, A.group_lanes_log2) * inv + A.eps);
        if (live && (w.cl & ((1u << A.group_lanes_log2) - 1u)) == 0) {
          const uint64_t at = static_cast<uint64_t>(r) * A.groups + w.c / A.per_group;
          if (A.mean) A.mean[at] = m;
          if (A.rstd) A.rstd[at] = rstd;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] * rstd, scale[e], shift[e]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf(x[e] - mu[e], scale[e], shift[e]);
      }
      act_values(A.act, x);
      if (live)
        store_chunk_n<T>(row_at(A, A.y, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), w.valid,
                         narrow(x, static_cast<const T*>(nullptr)));
    }
  }
}

// ---------------------------------------------------------------- backward

// What a lane keeps of its channels in a backward pass.
template <int V>
struct Channels {
  float mu[V], rstd[V], gamma[V], beta[V];

  __device__ __forceinline__ void params(const NormArgs& A, uint32_t c, int valid) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      gamma[e] = e < valid && A.gamma ? A.gamma[c + e] : 1.0f;
      beta[e] = e < valid && A.beta ? A.beta[c + e] : 0.0f;
    }
  }
  __device__ __forceinline__ void stats(const NormArgs& A, uint32_t n, uint32_t c, int valid) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint64_t at = static_cast<uint64_t>(n) * A.groups + (c + e) / A.per_group;
      mu[e] = e < valid ? A.mean[at] : 0.0f;
      rstd[e] = e < valid ? A.rstd[at] : 0.0f;
    }
  }
};

// x of a chunk of row r: the tensor's own values, or those of its 8-bit form.
template <class T, bool PACKED>
struct Source {
  static constexpr int V = kChunk<T>;
  rw4 raw;
  Codes<V> codes;
  float s;

  __device__ __forceinline__ void load(const NormArgs& A, const Spot& w, uint32_t r, int n) {
    if constexpr (PACKED) {
      const uint32_t per = (A.c + (V << A.lb_log2) - 1u) / (V << A.lb_log2);
      codes = load_codes<V>(row_at(A, A.px.codes, w.n, r) + w.c, n);
      s = n > 0 ? A.px.scales[(static_cast<uint64_t>(w.n) * A.rows + r) * per + ((w.c / V) >> A.lb_log2)] : 0.0f;
    } else {
      raw = load_chunk<T>(row_at(A, A.x, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), n);
    }
  }
  __device__ __forceinline__ void get(const NormArgs& A, float (&x)[V]) const {
    if constexpr (PACKED) decode(A.format, codes, s, x);
    else widen(raw, x, static_cast<const T*>(nullptr));
  }
};

// z and a = dy act'(u) of a chunk, from x and dy in their places.
template <int V>
__device__ __forceinline__ void z_and_a(const NormArgs& A, const Channels<V>& ch, float (&x)[V], float (&dy)[V]) {
  float u[V], value[V], slope[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    x[e] = (x[e] - ch.mu[e]) * ch.rstd[e];
    u[e] = __builtin_fmaf(x[e], ch.gamma[e], ch.beta[e]);
  }
  act_pairs(A.act, u, value, slope);
#pragma unroll
  for (int e = 0; e < V; ++e) dy[e] *= slope[e];
}

// Adds the row lanes' per-channel sums and writes them: out[0][c] and out[1][c].
template <int V>
__device__ __forceinline__ void write_sums(const NormArgs& A, const Spot& w, float2* sh, float* out,
                                           const float (&sa)[V], const float (&sz)[V]) {
  // entry (row lane, channel of the block), in V rounds of one channel a
  // lane so that the shared memory holds one float2 a lane
#pragma unroll
  for (int e = 0; e < V; ++e) {
    __syncthreads();
    sh[threadIdx.x] = make_float2(sa[e], sz[e]);
    __syncthreads();
    if (w.rl == 0 && e < w.valid) {
      float a = 0.0f, z = 0.0f;
      for (uint32_t r = 0; r < A.row_lanes; ++r) {
        const float2 v = sh[r * A.lanes.d + w.cl];
        a += v.x;
        z += v.y;
      }
      out[w.c + e] = a;
      out[A.c + w.c + e] = z;
    }
  }
}

// sum a and sum a z over a run of rows, for each channel: part[n][chunk][2][c].
template <class T, bool PACKED>
__global__ __launch_bounds__(kRowThreads) void norm_sums_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  __shared__ float2 sh[kRowThreads];
  const Spot w(A, blockIdx.x, V);
  Channels<V> ch;
  ch.params(A, w.c, w.valid);
  ch.stats(A, w.n, w.c, w.valid);
  float sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if (w.valid > 0) {
    for (uint32_t rb = w.r0 + w.rl; rb < w.r1; rb += U * A.row_lanes) {
      Source<T, PACKED> src[U];
      rw4 rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t r = rb + u * A.row_lanes;
        const int n = r < w.r1 ? w.valid : 0;
        src[u].load(A, w, r, n);
        rd[u] = load_chunk<T>(row_at(A, A.dy, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (rb + u * A.row_lanes >= w.r1) break;
        float x[V], a[V];
        src[u].get(A, x);
        widen(rd[u], a, static_cast<const T*>(nullptr));
        z_and_a(A, ch, x, a);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sa[e] += a[e];
          sz[e] = __builtin_fmaf(a[e], x[e], sz[e]);
        }
      }
    }
  }
  write_sums(A, w, sh, A.part + (static_cast<uint64_t>(w.n) * A.chunks + w.chunk) * 2u * A.c, sa, sz);
}

// Joins a sample's runs: its per-channel sums replace those of its first run,
// and coef[n][g] = (sum gamma a, sum gamma a z) / M.  A workgroup takes whole
// groups: as many as 256 channels hold, at least one.
__global__ __launch_bounds__(kRowThreads) void norm_coef_kernel(const NormArgs A) {
  __shared__ float2 sh[kRowThreads];
  const uint32_t gpw = A.per_group < kRowThreads ? kRowThreads / A.per_group : 1u;
  const uint32_t sets = (A.groups + gpw - 1) / gpw;
  const uint32_t n = blockIdx.x / sets;
  const uint32_t g0 = (blockIdx.x - n * sets) * gpw;
  const uint32_t gn = A.groups - g0 < gpw ? A.groups - g0 : gpw;
  const uint32_t c0 = g0 * A.per_group, c1 = (g0 + gn) * A.per_group;
  float* part = A.part + static_cast<uint64_t>(n) * A.chunks * 2u * A.c;
  float sa = 0.0f, sz = 0.0f;
  for (uint32_t c = c0 + threadIdx.x; c < c1; c += kRowThreads) {
    float a = 0.0f, z = 0.0f;
    for (uint32_t k = 0; k < A.chunks; ++k) {
      a += part[static_cast<uint64_t>(k) * 2u * A.c + c];
      z += part[static_cast<uint64_t>(k) * 2u * A.c + A.c + c];
    }
    part[c] = a;
    part[A.c + c] = z;
    const float gamma = A.gamma ? A.gamma[c] : 1.0f;
    sa = __builtin_fmaf(gamma, a, sa);
    sz = __builtin_fmaf(gamma, z, sz);
  }
  sh[threadIdx.x] = make_float2(sa, sz);
  __syncthreads();
  // the entries of a group: its channels, or all lanes where it is the only one
  const uint32_t entries = gpw == 1 ? kRowThreads : A.per_group;
  const int lg = join_log2(gn);
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const float inv = 1.0f / (static_cast<float>(A.rows) * static_cast<float>(A.per_group));
  for (uint32_t g = threadIdx.x >> lg; g < gn; g += kRowThreads >> lg) {
    float a = 0.0f, z = 0.0f;
    for (uint32_t e = lane; e < entries; e += 1u << lg) {
      const float2 v = sh[g * entries + e];
      a += v.x;
      z += v.y;
    }
    a = sum_lanes(a, lg);
    z = sum_lanes(z, lg);
    if (lane == 0)
      reinterpret_cast<float2*>(A.coef)[static_cast<uint64_t>(n) * A.groups + g0 + g] = make_float2(a * inv, z * inv);
  }
}

// dbeta and dgamma: column sums of col_rows rows of partial sums, `step`
// floats apart.  A workgroup takes 32 of the 2 c columns, 8 lanes each.
__device__ __forceinline__ void sum_columns(const NormArgs& A, uint32_t wg, uint64_t step) {
  __shared__ float sh[kRowThreads];
  const uint32_t col = wg * 32u + (threadIdx.x & 31u), sub = threadIdx.x >> 5;
  float s = 0.0f;
  if (col < 2u * A.c)
    for (uint32_t r = sub; r < A.col_rows; r += 8u) s += A.part[r * step + col];
  sh[threadIdx.x] = s;
  __syncthreads();
  if (sub == 0 && col < 2u * A.c) {
    for (uint32_t k = 1; k < 8u; ++k) s += sh[k * 32u + threadIdx.x];
    float* out = col < A.c ? A.dbeta : A.dgamma;
    if (out) out[col < A.c ? col : col - A.c] = s;
  }
}

__global__ __launch_bounds__(kRowThreads) void norm_columns_kernel(const NormArgs A) {
  sum_columns(A, blockIdx.x, 2u * static_cast<uint64_t>(A.c));
}

// dx.  By parts, the workgroups past main_grid add up dgamma and dbeta.  Per
// row, the group sums are taken here, and the per-channel sums of this
// workgroup's rows go to part[workgroup][2][c].
template <class T, bool PER_ROW, bool PACKED>
__global__ __launch_bounds__(kRowThreads) void norm_dx_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll / 2;
  __shared__ float2 sh[PER_ROW ? kRowThreads : 1];
  if constexpr (!PER_ROW) {
    if (blockIdx.x >= A.main_grid) {
      sum_columns(A, blockIdx.x - A.main_grid, static_cast<uint64_t>(A.chunks) * 2u * A.c);
      return;
    }
  }
  const Spot w(A, blockIdx.x, V);
  Channels<V> ch;
  ch.params(A, w.c, w.valid);
  float c1[V], c2[V], sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if constexpr (!PER_ROW) {
    ch.stats(A, w.n, w.c, w.valid);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 v = e < w.valid ? reinterpret_cast<const float2*>(
                                         A.coef)[static_cast<uint64_t>(w.n) * A.groups + (w.c + e) / A.per_group]
                                   : make_float2(0.0f, 0.0f);
      c1[e] = v.x;
      c2[e] = v.y;
    }
  }
  if (w.rl < A.row_lanes) {
    for (uint32_t rb = w.r0; rb < w.r1; rb += U * A.row_lanes) {
      Source<T, PACKED> src[U];
      rw4 rd[U];
      float2 st[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t r = rb + u * A.row_lanes + w.rl;
        const int n = r < w.r1 ? w.valid : 0;
        src[u].load(A, w, r, n);
        rd[u] = load_chunk<T>(row_at(A, A.dy, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), n);
        if constexpr (PER_ROW) {
          const uint64_t at = static_cast<uint64_t>(r) * A.groups + w.c / A.per_group;
          st[u] = n > 0 ? make_float2(A.mean[at], A.rstd[at]) : make_float2(0.0f, 0.0f);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (rb + u * A.row_lanes >= w.r1) break;
        const uint32_t r = rb + u * A.row_lanes + w.rl;
        const bool live = r < w.r1 && w.valid > 0;
        float x[V], a[V];
        src[u].get(A, x);
        widen(rd[u], a, static_cast<const T*>(nullptr));
        if constexpr (PER_ROW) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ch.mu[e] = st[u].x;
            ch.rstd[e] = st[u].y;
          }
        }
        z_and_a(A, ch, x, a);
        if constexpr (PER_ROW) {
          float ga = 0.0f, gz = 0.0f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sa[e] += a[e];
            sz[e] = __builtin_fmaf(a[e], x[e], sz[e]);
            a[e] *= ch.gamma[e];
            ga += a[e];
            gz = __builtin_fmaf(a[e], x[e], gz);
          }
          const float inv = 1.0f / static_cast<float>(A.per_group);
          ga = sum_lanes(ga, A.group_lanes_log2) * inv;
          gz = sum_lanes(gz, A.group_lanes_log2) * inv;
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] = st[u].y * (a[e] - ga - x[e] * gz);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] = ch.rstd[e] * (a[e] * ch.gamma[e] - c1[e] - x[e] * c2[e]);
        }
        if (live)
          store_chunk_n<T>(row_at(A, A.dx, w.n, r) + static_cast<int64_t>(w.c) * sizeof(T), w.valid,
                           narrow(a, static_cast<const T*>(nullptr)));
      }
    }
  }
  if constexpr (PER_ROW) write_sums(A, w, sh, A.part + static_cast<uint64_t>(w.chunk) * 2u * A.c, sa, sz);
}

}  // namespace dev

namespace {

template <class K>
hipError_t launch_norm(K kernel, const NormArgs& a, uint32_t grid, uint32_t lds, hipStream_t s) {
  void* args[] = {const_cast<NormArgs*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kRowThreads), args, lds, s);
}

uint32_t main_grid(const NormArgs& a) { return a.samples * a.blocks * a.chunks; }

// groups that one channel block may touch
uint32_t block_groups(const NormArgs& a, int v) {
  const uint32_t width = a.lanes.d * static_cast<uint32_t>(v);
  const uint32_t g = (width - 1) / a.per_group + 2;
  return g < a.groups ? g : a.groups;
}

template <class T>
hipError_t stats_t(const NormArgs& a, hipStream_t s) {
  return a.per_group % dev::kChunk<T> == 0 ? launch_norm(dev::norm_stats_kernel<T, true>, a, main_grid(a), 0, s)
                                           : launch_norm(dev::norm_stats_kernel<T, false>, a, main_grid(a), 0, s);
}

template <class T>
hipError_t apply_t(bool per_row, bool save, const NormArgs& a, hipStream_t s) {
  const uint32_t lds = per_row ? 0u : block_groups(a, dev::kChunk<T>) * 8u;
  if (per_row)
    return save ? launch_norm(dev::norm_apply_kernel<T, true, true>, a, main_grid(a), lds, s)
                : launch_norm(dev::norm_apply_kernel<T, true, false>, a, main_grid(a), lds, s);
  return save ? launch_norm(dev::norm_apply_kernel<T, false, true>, a, main_grid(a), lds, s)
              : launch_norm(dev::norm_apply_kernel<T, false, false>, a, main_grid(a), lds, s);
}

template <class T>
hipError_t sums_t(bool packed, const NormArgs& a, hipStream_t s) {
  return packed ? launch_norm(dev::norm_sums_kernel<T, true>, a, main_grid(a), 0, s)
                : launch_norm(dev::norm_sums_kernel<T, false>, a, main_grid(a), 0, s);
}

uint32_t column_grid(const NormArgs& a) { return a.dgamma || a.dbeta ? (2u * a.c + 31u) / 32u : 0u; }

template <class T>
hipError_t dx_t(bool per_row, bool packed, const NormArgs& a, hipStream_t s) {
  const uint32_t grid = per_row ? a.main_grid : a.main_grid + column_grid(a);
  if (per_row)
    return packed ? launch_norm(dev::norm_dx_kernel<T, true, true>, a, grid, 0, s)
                  : launch_norm(dev::norm_dx_kernel<T, true, false>, a, grid, 0, s);
  return packed ? launch_norm(dev::norm_dx_kernel<T, false, true>, a, grid, 0, s)
                : launch_norm(dev::norm_dx_kernel<T, false, false>, a, grid, 0, s);
}

}  // namespace

hipError_t norm_stats_launch(int dt, const NormArgs& a, hipStream_t s) {
  if (dt == kRowF16) return stats_t<_Float16>(a, s);
  if (dt == kRowBF16) return stats_t<dev::bf16_t>(a, s);
  return stats_t<float>(a, s);
}

hipError_t norm_apply_launch(int dt, bool per_row, bool save, const NormArgs& a, hipStream_t s) {
  if (dt == kRowF16) return apply_t<_Float16>(per_row, save, a, s);
  if (dt == kRowBF16) return apply_t<dev::bf16_t>(per_row, save, a, s);
  return apply_t<float>(per_row, save, a, s);
}

hipError_t norm_sums_launch(int dt, bool packed, const NormArgs& a, hipStream_t s) {
  if (dt == kRowF16) return sums_t<_Float16>(packed, a, s);
  if (dt == kRowBF16) return sums_t<dev::bf16_t>(packed, a, s);
  return sums_t<float>(packed, a, s);
}

hipError_t norm_coef_launch(const NormArgs& a, hipStream_t s) {
  const uint32_t gpw = a.per_group < kRowThreads ? kRowThreads / a.per_group : 1u;
  return launch_norm(dev::norm_coef_kernel, a, a.samples * ((a.groups + gpw - 1) / gpw), 0, s);
}

hipError_t norm_dx_launch(int dt, bool per_row, bool packed, const NormArgs& a, hipStream_t s) {
  NormArgs b = a;
  b.main_grid = main_grid(a);
  if (dt == kRowF16) return dx_t<_Float16>(per_row, packed, b, s);
  if (dt == kRowBF16) return dx_t<dev::bf16_t>(per_row, packed, b, s);
  return dx_t<float>(per_row, packed, b, s);
}

hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s) {
  const uint32_t grid = column_grid(a);
  if (grid == 0) return hipSuccess;
  return launch_norm(dev::norm_columns_kernel, a, grid, 0, s);
}

}  // namespace acp
