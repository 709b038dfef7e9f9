// 8-bit checkpoints and the activations that write and read them: elementwise
// over 16-byte chunks of rows.  A block of 32..256 channels shares a scale;
// its 4..64 lanes are neighbours in one wave and find their largest |x| with
// cross-lane moves, so nothing goes through LDS.
//
// Each element is read and written once: large tensors are bound by HBM
// (a plain copy reaches 6.0 TB/s), small ones by the launch.  A chunk's
// address, scale and codes come from its index alone, so a lane has its one
// or two chunks in flight and no loop.  Least and median of 30 traced calls:
//   pack8     [262144, 256] bfloat16, rows 264 elements apart, i8: 36.8 and 37.5 us, 5.4 TB/s
//   unpack8   the same: 32.2 and 34.2 us, 5.9 TB/s (both in a row of calls 69.0 us, 5.9 TB/s)
//   act_forward   [8192, 5632] bfloat16, gated, both operands saved as i8: 65.1 and 73.8 us, 5.0 TB/s
//   act_backward  the same: 59.4 and 61.5 us, 6.0 TB/s (both in a row of calls 126 us, 5.9 TB/s)
//   pack8, unpack8 of [64, 1000] float32: 2.5 and 2.8, 2.6 and 2.8 us
#include "acp_dev_rows.hpp"

namespace acp {
namespace dev {

// One chunk of the launch: where its row lies and how many channels it holds.
struct Chunk {
  uint32_t i0, i1, i2;
  int64_t c;  // first channel
  int n;      // channels; none past the row's or the launch's end

  __device__ __forceinline__ Chunk(const RowsCore& A, uint32_t i, int v) {
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

template <class T, int V, bool TAIL>
__device__ __forceinline__ void save_chunk(const RowsCore& A, const Packed& p, const Chunk& k, uint32_t i,
                                           const float (&v)[V]) {
  float x[V];
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = v[e];
  const float s = block_scale(A.format, block_amax(x, A.lb_log2));
  const Codes<V> c = encode<T>(A.format, x, s);
  if (k.n > 0) {
    store_codes<V, TAIL>(k.at(p.codes, 1), k.n, c);
    if ((i & ((1u << A.lb_log2) - 1u)) == 0) p.scales[i >> A.lb_log2] = s;
  }
}

template <int V>
__device__ __forceinline__ void saved_chunk(const RowsCore& A, const Codes<V>& c, float s, float (&x)[V]) {
  decode(A.format, c, s, x);
}

template <class T, int U, bool TAIL>
__global__ __launch_bounds__(kRowThreads) void pack8_kernel(const RowsUse<1, 1> A) {
  constexpr int V = kChunk<T>;
  const uint32_t i0 = blockIdx.x * (blockDim.x * U) + threadIdx.x;
  rw4 r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * blockDim.x, V);
    r[u] = load_chunk<T, false, TAIL>(k.at(A.t[0], sizeof(T)), k.n, A.c >= V);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * blockDim.x;
    const Chunk k(A, i, V);
    float x[V];
    place_tail<T, TAIL>(&r[u], k.n, A.c >= V);
    widen(r[u], x, static_cast<const T*>(nullptr));
    save_chunk<T, V, TAIL>(A, A.p[0], k, i, x);
  }
}

template <class T, int U, bool TAIL>
__global__ __launch_bounds__(kRowThreads) void unpack8_kernel(const RowsUse<1, 1> A) {
  constexpr int V = kChunk<T>;
  const uint32_t i0 = blockIdx.x * (blockDim.x * U) + threadIdx.x;
  Codes<V> c[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * blockDim.x;
    const Chunk k(A, i, V);
    c[u] = load_codes<V, false, TAIL>(k.at(A.p[0].codes, 1), k.n, A.c >= V);
    s[u] = k.n > 0 ? A.p[0].scales[i >> A.lb_log2] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * blockDim.x, V);
    float x[V];
    place_codes<V, TAIL>(&c[u], k.n, A.c >= V);
    saved_chunk<V>(A, c[u], s[u], x);
    if (k.n > 0) store_chunk<T, TAIL>(k.at(A.t[0], sizeof(T)), k.n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// y = act(x) [* z], and x [and z] kept in 8 bits: the codes cost a third of
// the bytes that the activation itself moves, where a pass of their own would
// read the operands again.
template <class T, bool GATED, bool SAVE, int U, bool TAIL>
__global__ __launch_bounds__(kRowThreads) void act_forward_kernel(
    const RowsUse<GATED ? 3 : 2, SAVE ? (GATED ? 2 : 1) : 0> A) {
  constexpr int V = kChunk<T>;
  const uint32_t i0 = blockIdx.x * (blockDim.x * U) + threadIdx.x;
  rw4 rx[U], rz[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * blockDim.x, V);
    rx[u] = load_chunk<T, false, TAIL>(k.at(A.t[0], sizeof(T)), k.n, A.c >= V);
    if constexpr (GATED) rz[u] = load_chunk<T, false, TAIL>(k.at(A.t[2], sizeof(T)), k.n, A.c >= V);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * blockDim.x;
    const Chunk k(A, i, V);
    float x[V], z[V];
    place_tail<T, TAIL>(&rx[u], k.n, A.c >= V);
    widen(rx[u], x, static_cast<const T*>(nullptr));
    if constexpr (SAVE) save_chunk<T, V, TAIL>(A, A.p[0], k, i, x);
    act_values(A.act, x);
    if constexpr (GATED) {
      place_tail<T, TAIL>(&rz[u], k.n, A.c >= V);
      widen(rz[u], z, static_cast<const T*>(nullptr));
      if constexpr (SAVE) save_chunk<T, V, TAIL>(A, A.p[1], k, i, z);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] *= z[e];
    }
    if (k.n > 0) store_chunk<T, TAIL>(k.at(A.t[1], sizeof(T)), k.n, narrow(x, static_cast<const T*>(nullptr)));
  }
}

// dx = dy act'(x) [* z], dz = dy act(x), with x and z from their 8-bit forms.
// Value and slope share their exponential (silu) or tail (gelu).
template <class T, bool GATED, int U, bool TAIL>
__global__ __launch_bounds__(kRowThreads) void act_backward_kernel(const RowsUse<GATED ? 3 : 2, GATED ? 2 : 1> A) {
  constexpr int V = kChunk<T>;
  const uint32_t i0 = blockIdx.x * (blockDim.x * U) + threadIdx.x;
  rw4 rd[U];
  Codes<V> cx[U], cz[U];
  float sx[U], sz[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = i0 + u * blockDim.x;
    const Chunk k(A, i, V);
    rd[u] = load_chunk<T, false, TAIL>(k.at(A.t[0], sizeof(T)), k.n, A.c >= V);
    cx[u] = load_codes<V, false, TAIL>(k.at(A.p[0].codes, 1), k.n, A.c >= V);
    sx[u] = k.n > 0 ? A.p[0].scales[i >> A.lb_log2] : 0.0f;
    if constexpr (GATED) {
      cz[u] = load_codes<V, false, TAIL>(k.at(A.p[1].codes, 1), k.n, A.c >= V);
      sz[u] = k.n > 0 ? A.p[1].scales[i >> A.lb_log2] : 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Chunk k(A, i0 + u * blockDim.x, V);
    float d[V], x[V], value[V], slope[V];
    place_tail<T, TAIL>(&rd[u], k.n, A.c >= V);
    place_codes<V, TAIL>(&cx[u], k.n, A.c >= V);
    widen(rd[u], d, static_cast<const T*>(nullptr));
    saved_chunk<V>(A, cx[u], sx[u], x);
    act_pairs(A.act, x, value, slope);
#pragma unroll
    for (int e = 0; e < V; ++e) slope[e] *= d[e];
    if constexpr (GATED) {
      float z[V];
      place_codes<V, TAIL>(&cz[u], k.n, A.c >= V);
      saved_chunk<V>(A, cz[u], sz[u], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        slope[e] *= z[e];
        value[e] *= d[e];
      }
      if (k.n > 0) store_chunk<T, TAIL>(k.at(A.t[2], sizeof(T)), k.n, narrow(value, static_cast<const T*>(nullptr)));
    }
    if (k.n > 0) store_chunk<T, TAIL>(k.at(A.t[1], sizeof(T)), k.n, narrow(slope, static_cast<const T*>(nullptr)));
  }
}

}  // namespace dev

namespace {

template <int I>
using Int = std::integral_constant<int, I>;

// Up to this many chunks lanes take one each, so that a call spreads over the
// CUs and a wave's code is short enough to come in quickly; past it two, for
// more bytes in flight.  Both kernels of a pass together: [64, 1000] float32
// packed and unpacked 4.8 us with one chunk, 7.1 with four; [2048, 1000] 8.1
// and 8.5 with two; [16384, 1000] 36.7 and 33.3; [262144, 256] bfloat16 79 and
// 73 (74 with four); an activation of [1024, 1400] float16 8.3 and 9.8 (12.2
// with four).
constexpr uint32_t kOneChunk = 1u << 20;

// `kernel(one, tail)`: the kernel with one chunk a lane or two, for rows whose
// last chunk is cut short or not.
template <class T, class A, class F>
hipError_t launch_rows(const A& a, hipStream_t s, F kernel) {
  const bool one = a.total <= kOneChunk, tail = a.c % dev::kChunk<T> != 0;
  const uint32_t per = kRowThreads * (one ? 1u : 2u);
  const uint32_t grid = a.total / per + (a.total % per ? 1u : 0u);
  A u = a;
  void* args[] = {&u};
  auto pick = [&](auto t) { return one ? kernel(Int<1>(), t) : kernel(Int<2>(), t); };
  return hipLaunchKernel(reinterpret_cast<const void*>(tail ? pick(std::true_type()) : pick(std::false_type())),
                         dim3(grid), dim3(kRowThreads), args, 0, s);
}

// A kernel's arguments out of a call's.
template <int NT, int NP>
RowsUse<NT, NP> use(const RowsArgs& a, const RowTensor& t0, const RowTensor& t1, const RowTensor& t2) {
  RowsUse<NT, NP> u;
  static_cast<RowsCore&>(u) = a;
  u.t[0] = t0;
  if constexpr (NT > 1) u.t[1] = t1;
  if constexpr (NT > 2) u.t[2] = t2;
  if constexpr (NP > 0) u.p[0] = a.px;
  if constexpr (NP > 1) u.p[1] = a.pz;
  return u;
}

template <class T>
hipError_t pack8_t(const RowsArgs& a, hipStream_t s) {
  return launch_rows<T>(use<1, 1>(a, a.x, a.x, a.x), s,
                        [](auto u, auto tail) { return dev::pack8_kernel<T, u(), tail()>; });
}

template <class T>
hipError_t unpack8_t(const RowsArgs& a, hipStream_t s) {
  return launch_rows<T>(use<1, 1>(a, a.y, a.y, a.y), s,
                        [](auto u, auto tail) { return dev::unpack8_kernel<T, u(), tail()>; });
}

template <class T, bool GATED, bool SAVE>
hipError_t act_forward_t(const RowsArgs& a, hipStream_t s) {
  constexpr int NT = GATED ? 3 : 2, NP = SAVE ? (GATED ? 2 : 1) : 0;
  return launch_rows<T>(use<NT, NP>(a, a.x, a.y, a.z), s,
                        [](auto u, auto tail) { return dev::act_forward_kernel<T, GATED, SAVE, u(), tail()>; });
}

template <class T>
hipError_t act_forward_t(bool gated, bool save, const RowsArgs& a, hipStream_t s) {
  if (gated) return save ? act_forward_t<T, true, true>(a, s) : act_forward_t<T, true, false>(a, s);
  return save ? act_forward_t<T, false, true>(a, s) : act_forward_t<T, false, false>(a, s);
}

template <class T, bool GATED>
hipError_t act_backward_t(const RowsArgs& a, hipStream_t s) {
  constexpr int NT = GATED ? 3 : 2, NP = GATED ? 2 : 1;
  return launch_rows<T>(use<NT, NP>(a, a.dy, a.dx, a.dz), s,
                        [](auto u, auto tail) { return dev::act_backward_kernel<T, GATED, u(), tail()>; });
}

}  // namespace

hipError_t pack8_launch(int dt, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return pack8_t<_Float16>(a, s);
  if (dt == kRowBF16) return pack8_t<dev::bf16_t>(a, s);
  return pack8_t<float>(a, s);
}

hipError_t unpack8_launch(int dt, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return unpack8_t<_Float16>(a, s);
  if (dt == kRowBF16) return unpack8_t<dev::bf16_t>(a, s);
  return unpack8_t<float>(a, s);
}

hipError_t act_forward_launch(int dt, bool gated, bool save, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return act_forward_t<_Float16>(gated, save, a, s);
  if (dt == kRowBF16) return act_forward_t<dev::bf16_t>(gated, save, a, s);
  return act_forward_t<float>(gated, save, a, s);
}

hipError_t act_backward_launch(int dt, bool gated, const RowsArgs& a, hipStream_t s) {
  if (dt == kRowF16) return gated ? act_backward_t<_Float16, true>(a, s) : act_backward_t<_Float16, false>(a, s);
  if (dt == kRowBF16) return gated ? act_backward_t<dev::bf16_t, true>(a, s) : act_backward_t<dev::bf16_t, false>(a, s);
  return gated ? act_backward_t<float, true>(a, s) : act_backward_t<float, false>(a, s);
}

}  // namespace acp
