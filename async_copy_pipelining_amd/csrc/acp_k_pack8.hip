// 8-bit checkpoints and the activations that write and read them: elementwise
// over 16-byte chunks of rows.  A block of 32..256 channels shares a scale;
// its 4..64 lanes are neighbours in one wave and find their largest |x| with
// cross-lane moves, so nothing goes through LDS.
#include "acp_dev_rows.hpp"

namespace acp {
namespace dev {

// One chunk of the launch: where its row lies and how many channels it holds.
struct Chunk {
  uint32_t i0, i1, i2;
  int64_t c;  // first channel
  int n;      // channels; none past the row's or the launch's end

  __device__ __forceinline__ Chunk(const RowsArgs& A, uint32_t i, int v) {
    const uint32_t row = divide(i, A.cpr);
    c = static_cast<int64_t>(i - row * A.cpr.d) * v;
    const uint32_t q = divide(row, A.n2);
    i2 = row - q * A.n2.d;
    i0 = divide(q, A.n1);
    i1 = q - i0 * A.n1.d;
    const int64_t left = A.c - c;
    n = i >= A.total || left <= 0 ? 0 : (left < v ? static_cast<int>(left) : v);
  }
  __device__ __forceinline__ char* at(const RowTensor& t, int esize) const {
    return t.p + i0 * t.s[0] + i1 * t.s[1] + i2 * t.s[2] + c * esize;
  }
};

template <class T, int V>
__device__ __forceinline__ void save_chunk(const RowsArgs& A, const Packed& p, const Chunk& k, uint32_t i,
                                           const float (&v)[V]) {
  float x[V];
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = v[e];
  const float s = block_scale(A.format, block_amax(x, A.lb_log2));
  const Codes<V> c = encode<T>(A.format, x, s);
  if (k.n > 0) {
    store_codes<V>(k.at(p.codes, 1), k.n, c);
    if ((i & ((1u << A.lb_log2) - 1u)) == 0) p.scales[i >> A.lb_log2] = s;
  }
}

template <int V>
__device__ __forceinline__ void saved_chunk(const RowsArgs& A, const Codes<V>& c, float s, float (&x)[V]) {
  decode(A.format, c, s, x);
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void pack8_kernel(const RowsArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  const uint32_t i0 = blockIdx.x * (kRowThreads * U) + threadIdx.x;
  rw4 r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * kRowThreads, V);
    r[u] = load_chunk<T>(k.at(A.x, sizeof(T)), k.n);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kRowThreads;
    const Chunk k(A, i, V);
    float x[V];
    widen(r[u], x, static_cast<const T*>(nullptr));
    save_chunk<T, V>(A, A.px, k, i, x);
  }
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void unpack8_kernel(const RowsArgs A) {
  constexpr int V = kChunk<T>, U = kRowUnroll;
  const uint32_t i0 = blockIdx.x * (kRowThreads * U) + threadIdx.x;
  Codes<V> c[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kRowThreads;
    const Chunk k(A, i, V);
    c[u] = load_codes<V>(k.at(A.px.codes, 1), k.n);
    s[u] = k.n > 0 ? A.px.scales[i >> A.lb_log2] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * kRowThreads, V);
    float x[V];
    saved_chunk<V>(A, c[u], s[u], x);
    if (k.n > 0) store_chunk_n<T>(k.at(A.y, sizeof(T)), k.n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// y = act(x) [* z], and x [and z] kept in 8 bits.
template <class T, bool GATED, bool SAVE>
__global__ __launch_bounds__(kRowThreads) void act_forward_kernel(const RowsArgs A) {
  constexpr int V = kChunk<T>, U = GATED ? kRowUnroll / 2 : kRowUnroll;
  const uint32_t i0 = blockIdx.x * (kRowThreads * U) + threadIdx.x;
  rw4 rx[U], rz[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * kRowThreads, V);
    rx[u] = load_chunk<T>(k.at(A.x, sizeof(T)), k.n);
    if constexpr (GATED) rz[u] = load_chunk<T>(k.at(A.z, sizeof(T)), k.n);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kRowThreads;
    const Chunk k(A, i, V);
    float x[V], z[V];
    widen(rx[u], x, static_cast<const T*>(nullptr));
    if constexpr (SAVE) save_chunk<T, V>(A, A.px, k, i, x);
    act_values(A.act, x);
    if constexpr (GATED) {
      widen(rz[u], z, static_cast<const T*>(nullptr));
      if constexpr (SAVE) save_chunk<T, V>(A, A.pz, k, i, z);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] *= z[e];
    }
    if (k.n > 0) store_chunk_n<T>(k.at(A.y, sizeof(T)), k.n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// dx = dy act'(x) [* z], dz = dy act(x), with x and z from their 8-bit forms.
template <class T, bool GATED>
__global__ __launch_bounds__(kRowThreads) void act_backward_kernel(const RowsArgs A) {
  constexpr int V = kChunk<T>, U = GATED ? kRowUnroll / 2 : kRowUnroll;
  const uint32_t i0 = blockIdx.x * (kRowThreads * U) + threadIdx.x;
  rw4 rd[U];
  Codes<V> cx[U], cz[U];
  float sx[U], sz[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * kRowThreads;
    const Chunk k(A, i, V);
    rd[u] = load_chunk<T>(k.at(A.dy, sizeof(T)), k.n);
    cx[u] = load_codes<V>(k.at(A.px.codes, 1), k.n);
    sx[u] = k.n > 0 ? A.px.scales[i >> A.lb_log2] : 0.0f;
    if constexpr (GATED) {
      cz[u] = load_codes<V>(k.at(A.pz.codes, 1), k.n);
      sz[u] = k.n > 0 ? A.pz.scales[i >> A.lb_log2] : 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * kRowThreads, V);
    float d[V], x[V], value[V], slope[V];
    widen(rd[u], d, static_cast<const T*>(nullptr));
    saved_chunk<V>(A, cx[u], sx[u], x);
    act_pairs(A.act, x, value, slope);
#pragma unroll
    for (int e = 0; e < V; ++e) slope[e] *= d[e];
    if constexpr (GATED) {
      float z[V];
      saved_chunk<V>(A, cz[u], sz[u], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        slope[e] *= z[e];
        value[e] *= d[e];
      }
      if (k.n > 0) store_chunk_n<T>(k.at(A.dz, sizeof(T)), k.n, narrow(value, static_cast<const T*>(nullptr)));
    }
    if (k.n > 0) store_chunk_n<T>(k.at(A.dx, sizeof(T)), k.n, narrow(slope, static_cast<const T*>(nullptr)));
  }
}

}  // namespace dev

namespace {

template <class K>
hipError_t launch_rows(K kernel, const RowsArgs& a, int unroll, hipStream_t s) {
  const uint32_t per = kRowThreads * static_cast<uint32_t>(unroll);
  const uint32_t grid = a.total / per + (a.total % per ? 1u : 0u);
  void* args[] = {const_cast<RowsArgs*>(&a)};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(kRowThreads), args, 0, s);
}

}  // namespace

hipError_t pack8_launch(int dt, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return launch_rows(dev::pack8_kernel<_Float16>, a, kRowUnroll, s);
  if (dt == kRowBF16) return launch_rows(dev::pack8_kernel<dev::bf16_t>, a, kRowUnroll, s);
  return launch_rows(dev::pack8_kernel<float>, a, kRowUnroll, s);
}

hipError_t unpack8_launch(int dt, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return launch_rows(dev::unpack8_kernel<_Float16>, a, kRowUnroll, s);
  if (dt == kRowBF16) return launch_rows(dev::unpack8_kernel<dev::bf16_t>, a, kRowUnroll, s);
  return launch_rows(dev::unpack8_kernel<float>, a, kRowUnroll, s);
}

template <class T>
static hipError_t act_forward_t(bool gated, bool save, const RowsArgs& a, hipStream_t s) {
  if (gated)
    return save ? launch_rows(dev::act_forward_kernel<T, true, true>, a, kRowUnroll / 2, s)
                : launch_rows(dev::act_forward_kernel<T, true, false>, a, kRowUnroll / 2, s);
  return save ? launch_rows(dev::act_forward_kernel<T, false, true>, a, kRowUnroll, s)
              : launch_rows(dev::act_forward_kernel<T, false, false>, a, kRowUnroll, s);
}

hipError_t act_forward_launch(int dt, bool gated, bool save, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return act_forward_t<_Float16>(gated, save, a, s);
  if (dt == kRowBF16) return act_forward_t<dev::bf16_t>(gated, save, a, s);
  return act_forward_t<float>(gated, save, a, s);
}

template <class T>
static hipError_t act_backward_t(bool gated, const RowsArgs& a, hipStream_t s) {
  return gated ? launch_rows(dev::act_backward_kernel<T, true>, a, kRowUnroll / 2, s)
               : launch_rows(dev::act_backward_kernel<T, false>, a, kRowUnroll, s);
}

hipError_t act_backward_launch(int dt, bool gated, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return act_backward_t<_Float16>(gated, a, s);
  if (dt == kRowBF16) return act_backward_t<dev::bf16_t>(gated, a, s);
  return act_backward_t<float>(gated, a, s);
}

}  // namespace acp
