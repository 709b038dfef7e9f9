// Group norm with an activation, backward: from x or from its 8-bit form.
#include "acp_dev_norm.hpp"

namespace acp {
namespace dev {

// A chunk of x: the tensor's own values, or those of its 8-bit form.  TAIL: a
// row may end inside a chunk.
template <class T, bool PACKED, bool LINEAR, bool TAIL>
struct Source {
  static constexpr int V = kChunk<T>;
  struct Raw {
    rw4 raw;
    Codes<V> codes;
    float s;
  };
  Walk<LINEAR> x, scales;

  __device__ __forceinline__ Source(const NormArgs& A, const Spot& w)
      : x(PACKED ? walk_codes<V, LINEAR>(A, w) : walk<T, LINEAR>(A, A.x, w)), scales(walk_scales<LINEAR>(A, w)) {}
  template <bool KEEP>
  __device__ __forceinline__ void load(const NormArgs& A, uint32_t k, int n, Raw* r) const {
    if constexpr (PACKED) {
      r->codes = load_codes<V, KEEP, TAIL>(x.at(A, k), n);
      r->s = n > 0 ? *reinterpret_cast<const float*>(scales.at(A, k)) : 0.0f;
    } else {
      r->raw = load_chunk<T, KEEP, TAIL>(x.at(A, k), n);
    }
  }
  __device__ static __forceinline__ void get(const NormArgs& A, const Raw& r, float (&v)[V]) {
    if constexpr (PACKED) decode(A.format, r.codes, r.s, v);
    else widen(r.raw, v, static_cast<const T*>(nullptr));
  }
};

// Two values of each of a lane's channels: (mean, rstd), or the coefficients
// of dx.  WHOLE (the channels are of one group): one pair for all of them.
template <int V, bool WHOLE>
struct Pairs {
  static constexpr int K = WHOLE ? 1 : V;
  float p[K], q[K];

  __device__ __forceinline__ float first(int e) const { return p[WHOLE ? 0 : e]; }
  __device__ __forceinline__ float second(int e) const { return q[WHOLE ? 0 : e]; }
  // at(group) gives a pair
  template <class F>
  __device__ __forceinline__ void load(const NormArgs& A, uint32_t c, int valid, F at) {
#pragma unroll
    for (int e = 0; e < K; ++e) {
      const float2 v = e < valid ? at((c + e) / A.per_group) : make_float2(0.0f, 0.0f);
      p[e] = v.x;
      q[e] = v.y;
    }
  }
  __device__ __forceinline__ void load_stats(const NormArgs& A, uint32_t n, uint32_t c, int valid) {
    const uint64_t row = static_cast<uint64_t>(n) * A.groups;
    load(A, c, valid, [&](uint32_t g) { return make_float2(A.mean[row + g], A.rstd[row + g]); });
  }
};

// z in the place of x, and a = dy act'(u) in the place of dy
template <int V, bool WHOLE>
__device__ __forceinline__ void z_and_a(const NormArgs& A, const Pairs<V, WHOLE>& st, const Params<V>& p,
                                        float (&x)[V], float (&dy)[V]) {
  float u[V], value[V], slope[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    x[e] = (x[e] - st.first(e)) * st.second(e);
    u[e] = __builtin_fmaf(x[e], p.gamma[e], p.beta[e]);
  }
  act_pairs(A.act, u, value, slope);
#pragma unroll
  for (int e = 0; e < V; ++e) dy[e] *= slope[e];
}

// Adds the row lanes' per-channel sums: chan[channel of the block], for all
// threads to see.  In two steps, so that every thread has a share: it sums
// every P-th row lane of a channel, then the P parts are added.  sh holds
// blockDim.x * (V + 1) floats.
template <int V>
__device__ __forceinline__ void channel_sums(const NormArgs& A, float* sh, float* chan, const float (&s)[V]) {
  const uint32_t width = A.lanes.d * V, threads = blockDim.x;
  float* parts = sh + threads * V;
#pragma unroll
  for (int e = 0; e < V; ++e) sh[threadIdx.x * V + e] = s[e];
  __syncthreads();
  if (width * 2 <= threads) {
    const uint32_t P = threads / width;
    const uint32_t part = threadIdx.x / width, ch = threadIdx.x - part * width;
    float v = 0.0f;
    if (part < P)
      for (uint32_t r = part; r < A.row_lanes; r += P) v += sh[r * width + ch];
    parts[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < width) {
      v = 0.0f;
      for (uint32_t k = 0; k < P; ++k) v += parts[k * width + threadIdx.x];
      chan[threadIdx.x] = v;
    }
  } else {
    for (uint32_t ch = threadIdx.x; ch < width; ch += threads) {
      float v = 0.0f;
      for (uint32_t r = 0; r < A.row_lanes; ++r) v += sh[r * width + ch];
      chan[ch] = v;
    }
  }
  __syncthreads();
}

// Writes a channel block's sums: a[c], and z[c] a row of the tensor further.
__device__ __forceinline__ void write_channels(const NormArgs& A, const Spot& w, uint32_t width, float* out,
                                               const float* a, const float* z) {
  for (uint32_t ch = threadIdx.x; ch < width; ch += blockDim.x) {
    const uint32_t c = w.blk * width + ch;
    if (c < A.c) {
      out[c] = a[ch];
      out[A.c + c] = z[ch];
    }
  }
}

// dbeta and dgamma: column sums of col_rows rows of partial sums, `step`
// floats apart.  A workgroup takes 32 of the 2 c columns, 8 lanes each.
__device__ __forceinline__ void sum_columns(const NormArgs& A, uint32_t wg, uint64_t step) {
  __shared__ float sh[kRowThreads];
  const uint32_t col = wg * 32u + (threadIdx.x & 31u), sub = threadIdx.x >> 5;
  constexpr int U = 8;
  float s = 0.0f;
  if (col < 2u * A.c)
    for (uint32_t r = sub; r < A.col_rows; r += 8u * U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = r + 8u * u < A.col_rows ? A.part[(r + 8u * u) * step + col] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) s += v[u];
    }
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

// ---------------------------------------------------------------- per row

// One row a sample.  The group sums are taken here; the per-channel sums of
// this workgroup's rows go to part[run][2][c].
template <class T, bool PACKED>
__global__ __launch_bounds__(kRowThreads) void norm_row_backward_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll / 2;
  extern __shared__ float lds[];
  const Spot w(A, blockIdx.x, V);
  const Source<T, PACKED, true, false> src(A, w);
  const Walk<true> pd = walk<T, true>(A, A.dy, w), px = walk<T, true>(A, A.dx, w);
  const Params<V> p(A, w.c, w.valid);
  const float inv = 1.0f / static_cast<float>(A.per_group);
  const uint32_t g = w.c / A.per_group;
  float sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if (w.rl < A.row_lanes) {
    for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
      typename Source<T, PACKED, true, false>::Raw rx[U];
      rw4 rd[U];
      float2 stat[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int n = w.channels(A, k0 + u);
        src.template load<false>(A, k0 + u, n, &rx[u]);
        rd[u] = load_chunk<T, false, false>(pd.at(A, k0 + u), n);
        const uint64_t at = static_cast<uint64_t>(w.r0 + w.rl + (k0 + u) * A.row_lanes) * A.groups + g;
        stat[u] = n > 0 ? make_float2(A.mean[at], A.rstd[at]) : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((k0 + u) * A.row_lanes >= w.rows) break;
        const int n = w.channels(A, k0 + u);
        float x[V], a[V];
        src.get(A, rx[u], x);
        widen(rd[u], a, static_cast<const T*>(nullptr));
        Pairs<V, true> st;
        st.p[0] = stat[u].x;
        st.q[0] = stat[u].y;
        z_and_a(A, st, p, x, a);
        float ga = 0.0f, gz = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sa[e] += a[e];
          sz[e] = __builtin_fmaf(a[e], x[e], sz[e]);
          a[e] *= p.gamma[e];
          ga += a[e];
          gz = __builtin_fmaf(a[e], x[e], gz);
        }
        ga = sum_lanes(ga, A.group_lanes_log2) * inv;
        gz = sum_lanes(gz, A.group_lanes_log2) * inv;
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = stat[u].y * (a[e] - ga - x[e] * gz);
        store_chunk<T, false>(px.at(A, k0 + u), n, narrow(a, static_cast<const T*>(nullptr)));
      }
    }
  }
  if (!A.dgamma && !A.dbeta) return;
  const uint32_t width = A.lanes.d * V;
  float* ca = lds + blockDim.x * (V + 1);
  channel_sums<V>(A, lds, ca, sa);
  channel_sums<V>(A, lds, ca + width, sz);
  write_channels(A, w, width, A.part + static_cast<uint64_t>(w.run) * 2u * A.c, ca, ca + width);
}

// ---------------------------------------------------------------- slab

// All rows of a sample for a block of whole groups: a lane holds up to
// kSlabRowsBackward chunks, so dy and x are read once.  A workgroup walks
// samples run, run + runs, ... and leaves its per-channel sums in
// part[run][2][c].
template <class T, bool WHOLE, bool PACKED>
__global__ __launch_bounds__(kSlabThreadsBackward) void norm_slab_backward_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kSlabRowsBackward;
  extern __shared__ float lds[];
  Spot w(A, blockIdx.x, V);
  // the grid is (blocks, runs): neighbouring channel blocks of a sample run together
  const uint32_t q = near_group(blockIdx.x, gridDim.x);
  w.run = divide(q, A.blocks);
  w.blk = q - w.run * A.blocks.d;
  w.c = (w.blk * A.lanes.d + w.cl) * V;
  w.valid = 0;
  if (w.rl < A.row_lanes && w.c < A.c) w.valid = A.c - w.c < static_cast<uint32_t>(V) ? static_cast<int>(A.c - w.c) : V;
  w.r0 = 0;
  w.rows = A.rows;
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, blockDim.x);
  const Params<V> p(A, w.c, w.valid);
  const float inv = 1.0f / (static_cast<float>(A.rows) * static_cast<float>(A.per_group));
  float* ca = lds + blockDim.x * (V + 1);  // this sample's sums of a and of a z
  float* cz = ca + width;
  float* ta = cz + width;                  // those of all samples so far
  float* tz = ta + width;
  float2* coef = reinterpret_cast<float2*>(tz + width);
  for (uint32_t ch = threadIdx.x; ch < 2 * width; ch += blockDim.x) ta[ch] = 0.0f;
  for (w.n = w.run; w.n < A.samples; w.n += A.runs.d) {
    const Source<T, PACKED, true, !WHOLE> src(A, w);
    const Walk<true> pd = walk<T, true>(A, A.dy, w), px = walk<T, true>(A, A.dx, w);
    typename Source<T, PACKED, true, !WHOLE>::Raw rx[U];
    rw4 rd[U];
    float a[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes < w.rows) {
        const int n = w.channels(A, u);
        src.template load<false>(A, u, n, &rx[u]);
        rd[u] = load_chunk<T, false, !WHOLE>(pd.at(A, u), n);
      }
    }
    Pairs<V, WHOLE> st;
    st.load_stats(A, w.n, w.c, w.valid);
    float sa[V], sz[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes >= w.rows) break;
      float z[V];
      src.get(A, rx[u], z);
      widen(rd[u], a[u], static_cast<const T*>(nullptr));
      z_and_a(A, st, p, z, a[u]);
      if (w.channels(A, u) > 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sa[e] += a[u][e];
          sz[e] = __builtin_fmaf(a[u][e], z[e], sz[e]);
        }
      }
    }
    channel_sums<V>(A, lds, ca, sa);
    channel_sums<V>(A, lds, cz, sz);
    for (uint32_t ch = threadIdx.x; ch < width; ch += blockDim.x) {
      ta[ch] += ca[ch];
      tz[ch] += cz[ch];
    }
    for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += blockDim.x >> lg) {
      float va = 0.0f, vz = 0.0f;
      for (uint32_t ch = g * A.per_group - b.lo + (threadIdx.x & ((1u << lg) - 1u)); ch < (g + 1) * A.per_group - b.lo;
           ch += 1u << lg) {
        const float gamma = A.gamma ? A.gamma[b.lo + ch] : 1.0f;
        va = __builtin_fmaf(gamma, ca[ch], va);
        vz = __builtin_fmaf(gamma, cz[ch], vz);
      }
      va = sum_lanes(va, lg);
      vz = sum_lanes(vz, lg);
      if ((threadIdx.x & ((1u << lg) - 1u)) == 0) coef[g - b.g0] = make_float2(va * inv, vz * inv);
    }
    __syncthreads();
    Pairs<V, WHOLE> cf;
    cf.load(A, w.c, w.valid, [&](uint32_t g) { return coef[g - b.g0]; });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes >= w.rows) break;
      const int n = w.channels(A, u);
      float z[V], d[V];
      src.get(A, rx[u], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        z[e] = (z[e] - st.first(e)) * st.second(e);
        d[e] = st.second(e) * (a[u][e] * p.gamma[e] - cf.first(e) - z[e] * cf.second(e));
      }
      store_chunk<T, !WHOLE>(px.at(A, u), n, narrow(d, static_cast<const T*>(nullptr)));
    }
  }
  if (!A.dgamma && !A.dbeta) return;
  if (A.runs.d == 1) {  // one workgroup saw every sample
    for (uint32_t ch = threadIdx.x; ch < width && b.lo + ch < A.c; ch += blockDim.x) {
      if (A.dbeta) A.dbeta[b.lo + ch] = ta[ch];
      if (A.dgamma) A.dgamma[b.lo + ch] = tz[ch];
    }
  } else {
    write_channels(A, w, width, A.part + static_cast<uint64_t>(w.run) * 2u * A.c, ta, tz);
  }
}

// ---------------------------------------------------------------- by parts

// sum a and sum a z over a run of rows, for each channel: part[n][run][2][c].
// The loads keep the data in the caches for the second pass.
template <class T, bool WHOLE, bool PACKED, bool LINEAR>
__global__ __launch_bounds__(kRowThreads) void norm_sums_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float lds[];
  const Spot w(A, blockIdx.x, V);
  const Source<T, PACKED, LINEAR, !WHOLE> src(A, w);
  const Walk<LINEAR> pd = walk<T, LINEAR>(A, A.dy, w);
  const Params<V> p(A, w.c, w.valid);
  Pairs<V, WHOLE> st;
  st.load_stats(A, w.n, w.c, w.valid);
  float sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if (w.valid > 0) {
    for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
      typename Source<T, PACKED, LINEAR, !WHOLE>::Raw rx[U];
      rw4 rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int n = w.channels(A, k0 + u);
        src.template load<true>(A, k0 + u, n, &rx[u]);
        rd[u] = load_chunk<T, true, !WHOLE>(pd.at(A, k0 + u), n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((k0 + u) * A.row_lanes >= w.rows) break;
        float x[V], a[V];
        src.get(A, rx[u], x);
        widen(rd[u], a, static_cast<const T*>(nullptr));
        z_and_a(A, st, p, x, a);
        if (w.channels(A, k0 + u) > 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sa[e] += a[e];
            sz[e] = __builtin_fmaf(a[e], x[e], sz[e]);
          }
        }
      }
    }
  }
  const uint32_t width = A.lanes.d * V;
  float* ca = lds + blockDim.x * (V + 1);
  channel_sums<V>(A, lds, ca, sa);
  channel_sums<V>(A, lds, ca + width, sz);
  write_channels(A, w, width, A.part + (static_cast<uint64_t>(w.n) * A.runs.d + w.run) * 2u * A.c, ca, ca + width);
}

constexpr uint32_t kCoefThreads = 1024;

__host__ __device__ inline uint32_t coef_columns(uint32_t per_group) { return per_group <= 64 ? 64u : 256u; }
__host__ __device__ inline uint32_t coef_groups(uint32_t per_group) {
  const uint32_t cw = coef_columns(per_group);
  return per_group < cw ? cw / per_group : 1u;
}

// Joins a sample's parts: its per-channel sums replace those of its first
// part, and coef[n][g] = (sum gamma a, sum gamma a z) / M.  A workgroup takes
// whole groups, cw channels at a time, 1024 / cw lanes a channel.
__global__ __launch_bounds__(kCoefThreads) void norm_coef_kernel(const NormArgs A) {
  __shared__ float2 sh[kCoefThreads];
  const uint32_t cw = coef_columns(A.per_group), slots = kCoefThreads / cw, gpw = coef_groups(A.per_group);
  const uint32_t sets = (A.groups + gpw - 1) / gpw;
  const uint32_t n = blockIdx.x / sets;
  const uint32_t g0 = (blockIdx.x - n * sets) * gpw;
  const uint32_t gn = A.groups - g0 < gpw ? A.groups - g0 : gpw;
  const uint32_t c0 = g0 * A.per_group, c1 = (g0 + gn) * A.per_group;
  const uint32_t col = threadIdx.x & (cw - 1u), slot = threadIdx.x / cw;
  float* part = A.part + static_cast<uint64_t>(n) * A.parts * 2u * A.c;
  float sa = 0.0f, sz = 0.0f;  // of the first cw threads: gamma-weighted sums
  for (uint32_t base = c0; base < c1; base += cw) {
    const uint32_t c = base + col;
    float a = 0.0f, z = 0.0f;
    if (c < c1) {
      constexpr int U = 4;
      for (uint32_t k = slot; k < A.parts; k += U * slots) {
        float va[U], vz[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t i = k + u * slots;
          const float* q = part + static_cast<uint64_t>(i) * 2u * A.c + c;
          va[u] = i < A.parts ? q[0] : 0.0f;
          vz[u] = i < A.parts ? q[A.c] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          a += va[u];
          z += vz[u];
        }
      }
    }
    __syncthreads();
    sh[threadIdx.x] = make_float2(a, z);
    __syncthreads();
    if (slot == 0 && c < c1) {
      for (uint32_t k = 1; k < slots; ++k) {
        const float2 v = sh[k * cw + col];
        a += v.x;
        z += v.y;
      }
      part[c] = a;
      part[A.c + c] = z;
      const float gamma = A.gamma ? A.gamma[c] : 1.0f;
      sa = __builtin_fmaf(gamma, a, sa);
      sz = __builtin_fmaf(gamma, z, sz);
    }
  }
  __syncthreads();
  sh[threadIdx.x] = make_float2(sa, sz);
  __syncthreads();
  // the entries of a group: its channels, or all columns where it is the only one
  const uint32_t entries = gpw == 1 ? cw : A.per_group;
  const int lg = join_log2(gn, kCoefThreads);
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const float inv = 1.0f / (static_cast<float>(A.rows) * static_cast<float>(A.per_group));
  for (uint32_t g = threadIdx.x >> lg; g < gn; g += kCoefThreads >> lg) {
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

// dx; the workgroups past main_grid add up dgamma and dbeta.
template <class T, bool WHOLE, bool PACKED, bool LINEAR>
__global__ __launch_bounds__(kRowThreads) void norm_dx_kernel(const NormArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  if (blockIdx.x >= A.main_grid) {
    sum_columns(A, blockIdx.x - A.main_grid, static_cast<uint64_t>(A.parts) * 2u * A.c);
    return;
  }
  const Spot w(A, blockIdx.x, V);
  if (w.valid == 0) return;
  const Source<T, PACKED, LINEAR, !WHOLE> src(A, w);
  const Walk<LINEAR> pd = walk<T, LINEAR>(A, A.dy, w), px = walk<T, LINEAR>(A, A.dx, w);
  const Params<V> p(A, w.c, w.valid);
  Pairs<V, WHOLE> st, cf;
  st.load_stats(A, w.n, w.c, w.valid);
  cf.load(A, w.c, w.valid, [&](uint32_t g) {
    return reinterpret_cast<const float2*>(A.coef)[static_cast<uint64_t>(w.n) * A.groups + g];
  });
  for (uint32_t k0 = 0; k0 * A.row_lanes < w.rows; k0 += U) {
    typename Source<T, PACKED, LINEAR, !WHOLE>::Raw rx[U];
    rw4 rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = w.channels(A, k0 + u);
      src.template load<false>(A, k0 + u, n, &rx[u]);
      rd[u] = load_chunk<T, false, !WHOLE>(pd.at(A, k0 + u), n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = w.channels(A, k0 + u);
      if (n == 0) break;
      float x[V], a[V];
      src.get(A, rx[u], x);
      widen(rd[u], a, static_cast<const T*>(nullptr));
      z_and_a(A, st, p, x, a);
#pragma unroll
      for (int e = 0; e < V; ++e) a[e] = st.second(e) * (a[e] * p.gamma[e] - cf.first(e) - x[e] * cf.second(e));
      store_chunk<T, !WHOLE>(px.at(A, k0 + u), n, narrow(a, static_cast<const T*>(nullptr)));
    }
  }
}

}  // namespace dev

namespace {

template <class K>
hipError_t launch_norm(K kernel, const NormArgs& a, uint32_t grid, uint32_t threads, uint32_t lds, hipStream_t s) {
  void* args[] = {const_cast<NormArgs*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(threads), args, lds, s);
}

// LDS of channel_sums and `n` arrays of a block's channels
uint32_t sums_lds(const NormArgs& a, int v, uint32_t threads, uint32_t n) {
  return (threads * static_cast<uint32_t>(v + 1) + n * a.lanes.d * static_cast<uint32_t>(v)) * 4u;
}

template <class T>
hipError_t row_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  const uint32_t lds = sums_lds(a, dev::kChunk<T>, kRowThreads, 2);
  return k.packed ? launch_norm(dev::norm_row_backward_kernel<T, true>, a, a.main_grid, kRowThreads, lds, s)
                  : launch_norm(dev::norm_row_backward_kernel<T, false>, a, a.main_grid, kRowThreads, lds, s);
}

template <class T, bool WHOLE>
hipError_t slab_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  constexpr int V = dev::kChunk<T>;
  const uint32_t width = a.lanes.d * static_cast<uint32_t>(V);
  const uint32_t lds = sums_lds(a, V, k.threads, 4) + (width / a.per_group + 1) * 8u;
  return k.packed ? launch_norm(dev::norm_slab_backward_kernel<T, WHOLE, true>, a, a.main_grid, k.threads, lds, s)
                  : launch_norm(dev::norm_slab_backward_kernel<T, WHOLE, false>, a, a.main_grid, k.threads, lds, s);
}

template <class T, bool WHOLE, bool PACKED>
hipError_t sums_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  const uint32_t lds = sums_lds(a, dev::kChunk<T>, kRowThreads, 2);
  return k.linear ? launch_norm(dev::norm_sums_kernel<T, WHOLE, PACKED, true>, a, a.main_grid, kRowThreads, lds, s)
                  : launch_norm(dev::norm_sums_kernel<T, WHOLE, PACKED, false>, a, a.main_grid, kRowThreads, lds, s);
}

template <class T>
hipError_t sums_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.whole) return k.packed ? sums_t<T, true, true>(k, a, s) : sums_t<T, true, false>(k, a, s);
  return k.packed ? sums_t<T, false, true>(k, a, s) : sums_t<T, false, false>(k, a, s);
}

uint32_t column_grid(const NormArgs& a) { return a.dgamma || a.dbeta ? (2u * a.c + 31u) / 32u : 0u; }

template <class T, bool WHOLE, bool PACKED>
hipError_t dx_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  const uint32_t g = a.main_grid + column_grid(a);
  return k.linear ? launch_norm(dev::norm_dx_kernel<T, WHOLE, PACKED, true>, a, g, kRowThreads, 0, s)
                  : launch_norm(dev::norm_dx_kernel<T, WHOLE, PACKED, false>, a, g, kRowThreads, 0, s);
}

template <class T>
hipError_t dx_t(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.whole) return k.packed ? dx_t<T, true, true>(k, a, s) : dx_t<T, true, false>(k, a, s);
  return k.packed ? dx_t<T, false, true>(k, a, s) : dx_t<T, false, false>(k, a, s);
}

}  // namespace

hipError_t norm_row_backward_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return row_t<_Float16>(k, a, s);
  if (k.dt == kRowBF16) return row_t<dev::bf16_t>(k, a, s);
  return row_t<float>(k, a, s);
}

hipError_t norm_slab_backward_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return k.whole ? slab_t<_Float16, true>(k, a, s) : slab_t<_Float16, false>(k, a, s);
  if (k.dt == kRowBF16) return k.whole ? slab_t<dev::bf16_t, true>(k, a, s) : slab_t<dev::bf16_t, false>(k, a, s);
  return k.whole ? slab_t<float, true>(k, a, s) : slab_t<float, false>(k, a, s);
}

hipError_t norm_sums_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return sums_t<_Float16>(k, a, s);
  if (k.dt == kRowBF16) return sums_t<dev::bf16_t>(k, a, s);
  return sums_t<float>(k, a, s);
}

hipError_t norm_coef_launch(const NormArgs& a, hipStream_t s) {
  const uint32_t gpw = dev::coef_groups(a.per_group);
  return launch_norm(dev::norm_coef_kernel, a, a.samples * ((a.groups + gpw - 1) / gpw), dev::kCoefThreads, 0, s);
}

hipError_t norm_dx_launch(const NormShape& k, const NormArgs& a, hipStream_t s) {
  if (k.dt == kRowF16) return dx_t<_Float16>(k, a, s);
  if (k.dt == kRowBF16) return dx_t<dev::bf16_t>(k, a, s);
  return dx_t<float>(k, a, s);
}

hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s) {
  const uint32_t grid = column_grid(a);
  if (grid == 0) return hipSuccess;
  return launch_norm(dev::norm_columns_kernel, a, grid, kRowThreads, 0, s);
}

}  // namespace acp
