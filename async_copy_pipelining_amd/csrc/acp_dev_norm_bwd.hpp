// Group norm with an activation: backward kernels, from x or from its 8-bit
// form.
#pragma once

#include "acp_dev_norm.hpp"

namespace acp {
namespace dev {

// A chunk of x: the tensor's own values, or those of its 8-bit form.
template <class T, int KIND, int PK>
struct Source {
  static constexpr int V = kChunk<T>;
  static constexpr bool TAIL = KIND == kNormAny, LINEAR = !TAIL;
  struct Raw {
    Codes<V> codes;
    float s;
  };
  Walk<LINEAR> codes, scales;

  __device__ __forceinline__ Source(const NormBackwardSaved& A, const Spot& w)
      : codes(walk_codes<V, LINEAR>(A, A.codes, w)), scales(walk_scales<LINEAR>(A, A.scales, w)) {}
  template <bool KEEP>
  __device__ __forceinline__ void load(const NormCore& A, uint32_t k, int n, Raw* r) const {
    r->codes = load_codes<V, KEEP, TAIL>(codes.at(A, k), n, A.c >= V);
    r->s = n > 0 ? *reinterpret_cast<const float*>(scales.at(A, k)) : 0.0f;
  }
  __device__ static __forceinline__ void place(const NormCore& A, int n, Raw* r) {
    place_codes<V, TAIL>(&r->codes, n, A.c >= V);
  }
  // x - mu from a code and its scale, whose product the fma does not round
  template <class P>
  __device__ static __forceinline__ void centre(const Raw& r, const P& st, float (&v)[V]) {
    decode(PK - 1, r.codes, 1.0f, v);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = __builtin_fmaf(v[e], r.s, st.first(e));
  }
};

template <class T, int KIND>
struct Source<T, KIND, 0> {
  static constexpr int V = kChunk<T>;
  static constexpr bool TAIL = KIND == kNormAny, LINEAR = !TAIL;
  struct Raw {
    rw4 raw;
  };
  Walk<LINEAR> x;

  __device__ __forceinline__ Source(const NormBackward& A, const Spot& w) : x(walk<T, LINEAR>(A, A.x, w)) {}
  template <bool KEEP>
  __device__ __forceinline__ void load(const NormCore& A, uint32_t k, int n, Raw* r) const {
    r->raw = load_chunk<T, KEEP, TAIL>(x.at(A, k), n, A.c >= V);
  }
  __device__ static __forceinline__ void place(const NormCore& A, int n, Raw* r) {
    place_tail<T, TAIL>(&r->raw, n, A.c >= V);
  }
  template <class P>
  __device__ static __forceinline__ void centre(const Raw& r, const P& st, float (&v)[V]) {
    widen(r.raw, v, static_cast<const T*>(nullptr));
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += st.first(e);
  }
};

template <int PK>
using BackwardArgs = std::conditional_t<PK != 0, NormBackwardSaved, NormBackward>;

// Two values of each of a lane's channels: (-mean, rstd), or those of
// dx: (-rstd c1, -rstd c2) with c1 and c2 the group's two means.  WHOLE (the
// channels are of one group): one pair for all of them.
template <int V, bool WHOLE>
struct Pairs {
  static constexpr int K = WHOLE ? 1 : V;
  float p[K], q[K];

  __device__ __forceinline__ float first(int e) const { return p[WHOLE ? 0 : e]; }
  __device__ __forceinline__ float second(int e) const { return q[WHOLE ? 0 : e]; }
  // at(group) gives a pair
  template <class F>
  __device__ __forceinline__ void load(const NormCore& A, uint32_t c, int valid, F at) {
#pragma unroll
    for (int e = 0; e < K; ++e) {
      const float2 v = e < valid ? at(divide(c + e, A.per)) : make_float2(0.0f, 0.0f);
      p[e] = v.x;
      q[e] = v.y;
    }
  }
  // the second value times st's
  __device__ __forceinline__ void scale(const Pairs& st) {
#pragma unroll
    for (int e = 0; e < K; ++e) q[e] *= st.q[e];
  }
  __device__ __forceinline__ void load_stats(const NormCore& A, uint32_t n, uint32_t c, int valid) {
    const uint64_t row = static_cast<uint64_t>(n) * A.groups;
    load(A, c, valid, [&](uint32_t g) { return make_float2(-A.mean[row + g], A.rstd[row + g]); });
  }
};

// a = dy act'(z gamma + beta) in the place of dy.  Where the rows of a lane are
// of one sample, z is left as x - mu and rstd is in gamma, in the sums of a z once
// they are made, and in the coefficients of dx.
template <int ACT, int V>
__device__ __forceinline__ void times_slope(const Params<V>& p, const float (&z)[V], float (&dy)[V]) {
  if constexpr (ACT != kActNone) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float value, slope;
      act_both<ACT, kFine<V>>(__builtin_fmaf(z[e], p.gamma[e], p.beta[e]), &value, &slope);
      dy[e] *= slope;
    }
  }
}

template <int V, bool WHOLE>
__device__ __forceinline__ void scale_gamma(const Pairs<V, WHOLE>& st, Params<V>* p) {
#pragma unroll
  for (int e = 0; e < V; ++e) p->gamma[e] *= st.second(e);
}

// The same where nothing else needs gamma and beta: for silu they are scaled
// by -log2 e beforehand, so that t = -u log2 e is one fma and
//   silu' = s (1 + u (1 - s)) = s (1 + t (s - 1) ln 2),  s = 1 / (1 + 2^t)
// takes two more and a product.
template <int ACT, int V>
__device__ __forceinline__ void scale_params(Params<V>* p) {
  if constexpr (ACT == kActSilu) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      p->gamma[e] *= -1.44269504088896341f;
      p->beta[e] *= -1.44269504088896341f;
    }
  }
}
template <int ACT, int V>
__device__ __forceinline__ void times_slope_scaled(const Params<V>& p, const float (&z)[V], float (&dy)[V]) {
  if constexpr (ACT == kActSilu) {
    constexpr float kLn2 = 0.693147180559945309f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float t = __builtin_fmaf(z[e], p.gamma[e], p.beta[e]);
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
      const float m = __builtin_fmaf(s, kLn2, -kLn2);
      dy[e] *= s * __builtin_fmaf(t, m, 1.0f);
    }
  } else {
    times_slope<ACT>(p, z, dy);
  }
}

// Adds the row lanes' per-channel sums of a and of a z: chan[channel of the
// block], for all threads to see.  In two steps where a block is narrow, so
// that every thread has a share: it sums every P-th row lane of a channel,
// then the P parts are added.  sh holds blockDim.x * (V + 1) pairs.
template <int V>
__device__ __forceinline__ void channel_sums(const NormCore& A, float2* sh, float2* chan, const float (&sa)[V],
                                             const float (&sz)[V]) {
  const uint32_t width = A.lanes.d * V, threads = blockDim.x;
  float2* parts = sh + threads * V;
#pragma unroll
  for (int e = 0; e < V; ++e) sh[threadIdx.x * V + e] = make_float2(sa[e], sz[e]);
  __syncthreads();
  auto add = [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); };
  if (width * 2 <= threads) {
    const uint32_t P = threads / width;
    const uint32_t part = threadIdx.x / width, ch = threadIdx.x - part * width;
    float2 v = make_float2(0.0f, 0.0f);
    if (part < P)
      for (uint32_t r = part; r < A.row_lanes; r += P) v = add(v, sh[r * width + ch]);
    parts[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < width) {
      v = parts[threadIdx.x];
      for (uint32_t k = 1; k < P; ++k) v = add(v, parts[k * width + threadIdx.x]);
      chan[threadIdx.x] = v;
    }
  } else {
    for (uint32_t ch = threadIdx.x; ch < width; ch += threads) {
      float2 v = sh[ch];
      for (uint32_t r = 1; r < A.row_lanes; ++r) v = add(v, sh[r * width + ch]);
      chan[ch] = v;
    }
  }
  __syncthreads();
}

// gamma of the channel block, for the sums over a group
template <int V>
__device__ __forceinline__ void put_gamma(const Spot& w, const Params<V>& p, float* gl) {
  if (w.rl == 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) gl[w.cl * V + e] = p.gamma[e];
  }
}

// sum gamma a and sum gamma a z over the channels [p0, p1) of the block, in
// all of the 2^lg lanes that share them
__device__ __forceinline__ float2 weigh(const float2* chan, const float* gl, uint32_t p0, uint32_t p1, int lg) {
  float a = 0.0f, z = 0.0f;
  for (uint32_t ch = p0 + (threadIdx.x & ((1u << lg) - 1u)); ch < p1; ch += 1u << lg) {
    const float2 v = chan[ch];
    a = __builtin_fmaf(gl[ch], v.x, a);
    z = __builtin_fmaf(gl[ch], v.y, z);
  }
  return make_float2(sum_lanes(a, lg), sum_lanes(z, lg));
}

// Writes a channel block's sums: a[c], and z[c] a row of the tensor further.
__device__ __forceinline__ void write_channels(const NormCore& A, const Spot& w, uint32_t width, float* out,
                                               const float2* chan) {
  for (uint32_t ch = threadIdx.x; ch < width; ch += blockDim.x) {
    const uint32_t c = w.blk * width + ch;
    if (c < A.c) {
      out[c] = chan[ch].x;
      out[A.c + c] = chan[ch].y;
    }
  }
}

// dbeta and dgamma: column sums of col_rows rows of partial sums, `step`
// floats apart.  A workgroup takes kColumns of the 2 c columns, 16 lanes each, so
// that few rounds of loads follow one another: 4.6 us for 128 rows of 8192
// columns, mostly latency.
__device__ __forceinline__ void sum_columns(const NormCore& A, uint32_t wg, uint64_t step) {
  constexpr uint32_t S = kRowThreads / kColumns;
  __shared__ float sh[kRowThreads];
  const uint32_t col = wg * kColumns + threadIdx.x % kColumns, sub = threadIdx.x / kColumns;
  constexpr int U = 8;
  float s = 0.0f;
  if (col < 2u * A.c)
    for (uint32_t r = sub; r < A.col_rows; r += S * U) {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = r + S * u < A.col_rows ? A.part[(r + S * u) * step + col] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) s += v[u];
    }
  sh[threadIdx.x] = s;
  __syncthreads();
  if (sub == 0 && col < 2u * A.c) {
    for (uint32_t k = 1; k < S; ++k) s += sh[k * kColumns + threadIdx.x];
    float* out = col < A.c ? A.dbeta : A.dgamma;
    if (out) out[col < A.c ? col : col - A.c] = s;
  }
}

// ---------------------------------------------------------------- per row

// One row a sample.  The group sums are taken here; the per-channel sums of
// this workgroup's rows stay in registers until the end and go to
// part[run][2][c], which norm_columns_kernel adds up.  Bound by HBM: [8192,
// 4096] bfloat16 in heads of 64 channels 38.0 us (205 MB, 5.4 TB/s), and 4.6 us
// for the columns (medians of 30 traced calls).
template <class T, int PK, int ACT>
__global__ __launch_bounds__(kRowThreadsBackward) void norm_row_backward_kernel(const BackwardArgs<PK> A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 lds[];
  const Spot w(A, blockIdx.x, V);
  const Source<T, kNormWhole, PK> src(A, w);
  const Walk<true> pd = walk<T, true>(A, A.dy, w), px = walk<T, true>(A, A.dx, w);
  const float inv = 1.0f / static_cast<float>(A.per_group);
  const uint32_t g = divide(w.c, A.per);
  typename Source<T, kNormWhole, PK>::Raw rx[U];
  rw4 rd[U];
  float2 stat[U];
  auto load = [&](uint32_t k, int u) {
    const int n = w.channels(A, k);
    src.template load<false>(A, k, n, &rx[u]);
    rd[u] = load_chunk<T, false, false>(pd.at(A, k), n, A.c >= V);
    const uint64_t at = static_cast<uint64_t>(w.r0 + w.rl + k * w.step) * A.groups + g;
    stat[u] = n > 0 ? make_float2(A.mean[at], A.rstd[at]) : make_float2(0.0f, 0.0f);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u);
  const Params<V> p(A, w.c, w.valid);
  float sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if (w.rl < A.row_lanes) {
    for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((k0 + u) * w.step >= w.rows) break;
        const int n = w.channels(A, k0 + u);
        float x[V], a[V];
        Pairs<V, true> st;
        st.p[0] = -stat[u].x;
        st.q[0] = stat[u].y;
        src.centre(rx[u], st, x);
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] *= st.q[0];
        widen(rd[u], a, static_cast<const T*>(nullptr));
        load(k0 + U + u, u);
        times_slope<ACT>(p, x, a);
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
        for (int e = 0; e < V; ++e) a[e] = st.q[0] * __builtin_fmaf(-x[e], gz, a[e] - ga);
        store_chunk<T, false>(px.at(A, k0 + u), n, narrow(a, static_cast<const T*>(nullptr)));
      }
    }
  }
  if (!A.dgamma && !A.dbeta) return;
  float2* chan = lds + blockDim.x * (V + 1);
  channel_sums<V>(A, lds, chan, sa, sz);
  write_channels(A, w, A.lanes.d * V, A.part + static_cast<uint64_t>(w.run) * 2u * A.c, chan);
}

// ---------------------------------------------------------------- slab

// All rows of a sample for a block of whole groups: a lane holds up to
// kSlabRowsBackward chunks, so dy and x are read once.  A workgroup walks
// samples run, run + runs, ... and leaves its per-channel sums in
// part[run][2][c].  Small calls are bound by latency, where three barriers a
// sample cost less than a second pass ([2, 16, 16, 640] float16 from e4m3 11.1
// us, and 3.9 us for the columns, medians of 30 traced calls); [512, 256, 1024]
// float16 from x 211 us with silu (805 MB, 3.8 TB/s; the vector units issue 44 %
// of the time): a CU holds one workgroup of 512 lanes, so its loads
// and its stores take turns.  Eight chunks a lane with the slope computed
// twice took 200 us there, but 282 us for 192 on [4096, 64, 512] bfloat16 and
// 9.8 for 8.7 on [64, 32, 512].
template <class T, int KIND, int PK, int ACT>
__global__ __launch_bounds__(kSlabThreadsBackward) void norm_slab_backward_kernel(const BackwardArgs<PK> A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = kSlabRowsBackward;
  extern __shared__ float2 lds[];
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
  w.step = A.row_lanes;
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, blockDim.x);
  const Params<V> p(A, w.c, w.valid);
  const float inv = 1.0f / (static_cast<float>(A.rows) * static_cast<float>(A.per_group));
  float2* chan = lds + blockDim.x * (V + 1);  // this sample's sums of a and of a z
  float2* sums = chan + width;                // those of all samples so far
  float2* coef = sums + width;
  float* gl = reinterpret_cast<float*>(coef + (b.g1 - b.g0 + 1));
  for (uint32_t ch = threadIdx.x; ch < width; ch += blockDim.x) sums[ch] = make_float2(0.0f, 0.0f);
  put_gamma<V>(w, p, gl);
  for (w.n = w.run; w.n < A.samples; w.n += A.runs.d) {
    const Source<T, KIND, PK> src(A, w);
    const Walk<LINEAR> pd = walk<T, LINEAR>(A, A.dy, w), px = walk<T, LINEAR>(A, A.dx, w);
    typename Source<T, KIND, PK>::Raw rx[U];
    rw4 rd[U];
    float a[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes < w.rows) {
        const int n = w.channels(A, u);
        src.template load<false>(A, u, n, &rx[u]);
        rd[u] = load_chunk<T, false, TAIL>(pd.at(A, u), n, A.c >= V);
      }
    }
    Pairs<V, WHOLE> st;
    st.load_stats(A, w.n, w.c, w.valid);
    Params<V> ps = p;
    scale_gamma(st, &ps);
    float sa[V], sz[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes >= w.rows) break;
      float z[V];
      src.place(A, w.channels(A, u), &rx[u]);
      place_tail<T, TAIL>(&rd[u], w.channels(A, u), A.c >= V);
      src.centre(rx[u], st, z);
      widen(rd[u], a[u], static_cast<const T*>(nullptr));
      times_slope<ACT>(ps, z, a[u]);
      if (w.channels(A, u) > 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sa[e] += a[u][e];
          sz[e] = __builtin_fmaf(a[u][e], z[e], sz[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sz[e] *= st.second(e);
    channel_sums<V>(A, lds, chan, sa, sz);
    for (uint32_t ch = threadIdx.x; ch < width; ch += blockDim.x)
      sums[ch] = make_float2(sums[ch].x + chan[ch].x, sums[ch].y + chan[ch].y);
    for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += blockDim.x >> lg) {
      const float2 v = weigh(chan, gl, g * A.per_group - b.lo, (g + 1) * A.per_group - b.lo, lg);
      if ((threadIdx.x & ((1u << lg) - 1u)) == 0) {
        const float r = -inv * A.rstd[static_cast<uint64_t>(w.n) * A.groups + g];
        coef[g - b.g0] = make_float2(v.x * r, v.y * r);
      }
    }
    __syncthreads();
    Pairs<V, WHOLE> cf;
    cf.load(A, w.c, w.valid, [&](uint32_t g) { return coef[g - b.g0]; });
    cf.scale(st);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * A.row_lanes >= w.rows) break;
      const int n = w.channels(A, u);
      float z[V], d[V];
      src.centre(rx[u], st, z);
#pragma unroll
      for (int e = 0; e < V; ++e)
        d[e] = __builtin_fmaf(a[u][e], ps.gamma[e], __builtin_fmaf(z[e], cf.second(e), cf.first(e)));
      store_chunk<T, TAIL>(px.at(A, u), n, narrow(d, static_cast<const T*>(nullptr)));
    }
  }
  if (!A.dgamma && !A.dbeta) return;
  if (A.runs.d == 1) {  // one workgroup saw every sample
    for (uint32_t ch = threadIdx.x; ch < width && b.lo + ch < A.c; ch += blockDim.x) {
      if (A.dbeta) A.dbeta[b.lo + ch] = sums[ch].x;
      if (A.dgamma) A.dgamma[b.lo + ch] = sums[ch].y;
    }
  } else {
    write_channels(A, w, width, A.part + static_cast<uint64_t>(w.run) * 2u * A.c, sums);
  }
}

// ---------------------------------------------------------------- by parts

// Sums of a run of rows: for each channel sum a and sum a z, into
// part[n][run][2][c]; for each group's piece in this channel block sum gamma a
// and sum gamma a z, into coef[n][g][run][piece].  The loads keep the data in
// the caches for the second pass; each chunk's place takes the one U steps on
// as soon as it is used.  [128, 500, 1024] float16 from i8, silu: 45 to 54 us
// (197 MB, 3.6 to 4.4 TB/s; the vector units issue 67 % of the time, on decoding
// and the slope); [3, 37, 41, 352] float32, groups of 11 channels: 8.3 us (median
// of 30 traced calls).
template <class T, int KIND, int PK, int ACT>
__global__ __launch_bounds__(kRowThreads) void norm_sums_kernel(const BackwardArgs<PK> A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 lds[];
  const Spot w(A, blockIdx.x, V);
  const Source<T, KIND, PK> src(A, w);
  const Walk<LINEAR> pd = walk<T, LINEAR>(A, A.dy, w);
  typename Source<T, KIND, PK>::Raw rx[U];
  rw4 rd[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = w.channels(A, u);
    src.template load<true>(A, u, n, &rx[u]);
    rd[u] = load_chunk<T, true, TAIL>(pd.at(A, u), n, A.c >= V);
  }
  Params<V> p(A, w.c, w.valid);
  float2* chan = lds + blockDim.x * (V + 1);
  float* gl = reinterpret_cast<float*>(chan + A.lanes.d * V);
  put_gamma<V>(w, p, gl);
  Pairs<V, WHOLE> st;
  st.load_stats(A, w.n, w.c, w.valid);
  scale_gamma(st, &p);
  scale_params<ACT>(&p);
  float sa[V], sz[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sa[e] = sz[e] = 0.0f;
  if (w.valid > 0) {
    for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((k0 + u) * w.step >= w.rows) break;
        float z[V], a[V];
        src.place(A, w.channels(A, k0 + u), &rx[u]);
        place_tail<T, TAIL>(&rd[u], w.channels(A, k0 + u), A.c >= V);
        src.centre(rx[u], st, z);
        widen(rd[u], a, static_cast<const T*>(nullptr));
        const int next = w.channels(A, k0 + U + u);
        src.template load<true>(A, k0 + U + u, next, &rx[u]);
        rd[u] = load_chunk<T, true, TAIL>(pd.at(A, k0 + U + u), next, A.c >= V);
        times_slope_scaled<ACT>(p, z, a);
        if (w.channels(A, k0 + u) > 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sa[e] += a[e];
            sz[e] = __builtin_fmaf(a[e], z[e], sz[e]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) sz[e] *= st.second(e);
  const uint32_t width = A.lanes.d * V;
  channel_sums<V>(A, lds, chan, sa, sz);
  write_channels(A, w, width, A.part + (static_cast<uint64_t>(w.n) * A.runs.d + w.run) * 2u * A.c, chan);
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, kRowThreads);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += kRowThreads >> lg) {
    const uint32_t p0 = (g * A.per_group > b.lo ? g * A.per_group : b.lo) - b.lo;
    const float2 v = weigh(chan, gl, p0, p0 + piece_channels(A, g, w.blk, width), lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0)
      reinterpret_cast<float2*>(A.coef)[((static_cast<uint64_t>(w.n) * A.groups + g) * A.runs.d + w.run) * A.pieces +
                                        (w.blk - g * A.per_group / width)] = v;
  }
}

// (-rstd c1, -rstd c2) of group g of sample n from its parts, in all of the
// 2^lg lanes that share the group.
__device__ __forceinline__ float2 join_sums(const NormCore& A, uint32_t n, uint32_t g, uint32_t width, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1u);
  const uint64_t at = static_cast<uint64_t>(n) * A.groups + g;
  const float2* part = reinterpret_cast<const float2*>(A.coef) + at * A.parts * A.pieces;
  // channel blocks that the group reaches into; the others' places are unset
  const uint32_t reach = ((g + 1) * A.per_group - 1) / width - g * A.per_group / width + 1;
  float a = 0.0f, z = 0.0f;
  if (A.pieces == 1) {
    constexpr int U = 8;  // parts in flight
    for (uint32_t e = lane; e < A.parts; e += U << lg) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = e + (u << lg) < A.parts ? part[e + (u << lg)] : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        a += v[u].x;
        z += v[u].y;
      }
    }
  } else {
    for (uint32_t e = lane; e < A.parts * A.pieces; e += 1u << lg) {
      if (e % A.pieces >= reach) continue;
      a += part[e].x;
      z += part[e].y;
    }
  }
  const float r = -A.rstd[at] / (static_cast<float>(A.rows) * static_cast<float>(A.per_group));
  return make_float2(sum_lanes(a, lg) * r, sum_lanes(z, lg) * r);
}

// dx.  The first workgroups add up dgamma and dbeta.  The first chunks are on
// their way while the parts are joined.  Bound by HBM and VALU work alike:
// [128, 500, 1024] float16 from i8, silu 54 to 59 us (328 MB, 5.6 to 6.1 TB/s; the
// vector units issue 74 % of the time); [3, 37, 41, 352] float32 8.5 us.
template <class T, int KIND, int PK, int ACT>
__global__ __launch_bounds__(kRowThreads) void norm_dx_kernel(const BackwardArgs<PK> A) {
  constexpr bool WHOLE = KIND == kNormWhole, TAIL = KIND == kNormAny, LINEAR = !TAIL;
  constexpr int V = kChunk<T>, U = kRowUnroll;
  extern __shared__ float2 coef[];
  const uint32_t columns = gridDim.x - A.main_grid;
  if (blockIdx.x < columns) {
    sum_columns(A, blockIdx.x, 2u * static_cast<uint64_t>(A.c));
    return;
  }
  const Spot w(A, blockIdx.x - columns, V);
  const Source<T, KIND, PK> src(A, w);
  const Walk<LINEAR> pd = walk<T, LINEAR>(A, A.dy, w), px = walk<T, LINEAR>(A, A.dx, w);
  typename Source<T, KIND, PK>::Raw rx[U];
  rw4 rd[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = w.channels(A, u);
    src.template load<false>(A, u, n, &rx[u]);
    rd[u] = load_chunk<T, false, TAIL>(pd.at(A, u), n, A.c >= V);
  }
  Params<V> p(A, w.c, w.valid);
  Pairs<V, WHOLE> st, cf;
  st.load_stats(A, w.n, w.c, w.valid);
  const uint32_t width = A.lanes.d * V;
  const BlockGroups b(A, w.blk, width);
  const int lg = join_log2(b.g1 - b.g0 + 1, kRowThreads);
  for (uint32_t g = b.g0 + (threadIdx.x >> lg); g <= b.g1; g += kRowThreads >> lg) {
    const float2 v = join_sums(A, w.n, g, width, lg);
    if ((threadIdx.x & ((1u << lg) - 1u)) == 0) coef[g - b.g0] = v;
  }
  __syncthreads();
  if (w.valid == 0) return;
  cf.load(A, w.c, w.valid, [&](uint32_t g) { return coef[g - b.g0]; });
  cf.scale(st);
  scale_gamma(st, &p);
  float scale[V];
#pragma unroll
  for (int e = 0; e < V; ++e) scale[e] = p.gamma[e];
  scale_params<ACT>(&p);
  for (uint32_t k0 = 0; k0 * w.step < w.rows; k0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = w.channels(A, k0 + u);
      if (n == 0) return;
      float z[V], a[V];
      src.place(A, n, &rx[u]);
      place_tail<T, TAIL>(&rd[u], n, A.c >= V);
      src.centre(rx[u], st, z);
      widen(rd[u], a, static_cast<const T*>(nullptr));
      const int next = w.channels(A, k0 + U + u);
      src.template load<false>(A, k0 + U + u, next, &rx[u]);
      rd[u] = load_chunk<T, false, TAIL>(pd.at(A, k0 + U + u), next, A.c >= V);
      times_slope_scaled<ACT>(p, z, a);
#pragma unroll
      for (int e = 0; e < V; ++e)
        a[e] = __builtin_fmaf(a[e], scale[e], __builtin_fmaf(z[e], cf.second(e), cf.first(e)));
      store_chunk<T, TAIL>(px.at(A, k0 + u), n, narrow(a, static_cast<const T*>(nullptr)));
    }
  }
}

}  // namespace dev
}  // namespace acp
