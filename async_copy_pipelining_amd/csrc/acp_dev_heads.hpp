// Device side of the head operators: a lane's unit of a row, the rotation.
#pragma once

#include "acp_dev_rows.hpp"
#include "acp_heads.hpp"

namespace acp {
namespace dev {

typedef double hd2 __attribute__((ext_vector_type(2)));
typedef hd2 hd2_any __attribute__((aligned(8)));
typedef float hf4 __attribute__((ext_vector_type(4)));
typedef hf4 hf4_any __attribute__((aligned(4)));

// A lane's two chunks of every row: first channel and channels of each.
// Turned units come first.  Halves: V channels of the first half and those
// they are paired with, half the turned channels further.  Pairs, and channels
// that are not turned, whose chunks have no need of each other: lanes that are
// neighbours have chunks that are, so that a load or store of the wave has whole
// runs of a row (2 V neighbours a lane, every other 16 bytes at a time: [20480 new
// tokens, 32 + 8 + 8 heads, 128] bfloat16 appended in 145 us, so in 110).
template <class T, bool PAIRS>
struct Unit {
  int at[2], n[2];
  bool turned;
  uint32_t first[2];  // its frequencies: V / 2 from each of these on

  __device__ __forceinline__ Unit(const HeadsCore& A, uint32_t u) {
    constexpr int V = kChunk<T>;
    const int half = static_cast<int>(A.rotated / 2), k = static_cast<int>(u < A.turn_units ? u : u - A.turn_units);
    turned = u < A.turn_units;
    if (!PAIRS && turned) {
      at[0] = k * V;
      at[1] = half + k * V;
      n[0] = n[1] = within(half - k * V);
      first[0] = u * V;
      first[1] = u * V + V / 2;
    } else {
      const int from = turned ? 0 : static_cast<int>(A.rotated), to = static_cast<int>(turned ? A.rotated : A.dim);
      const int further = static_cast<int>(turned ? A.turn_units : A.units - A.turn_units) * V;
      at[0] = from + k * V;
      at[1] = at[0] + further;
      n[0] = within(to - at[0]);
      n[1] = within(to - at[1]);
      first[0] = static_cast<uint32_t>(at[0]) / 2;
      first[1] = static_cast<uint32_t>(at[1]) / 2;
    }
    if (u >= A.units) n[0] = n[1] = 0;
  }
  static __device__ __forceinline__ int within(int n) {
    constexpr int V = kChunk<T>;
    return n < 0 ? 0 : n < V ? n : V;
  }
};

// cos and sin of a unit's angles.
//
// The angle's turns t = position * (frequency / 2 pi) are formed in 64 bits
// (positions go up to 2^31; 32 bits would leave 2^31 * 2^-24 turns of error),
// the nearest quarter q / 4 is taken off exactly, and the rest, at most an
// eighth of a turn, goes through the Taylor series of sine and cosine: terms
// up to x^9 and x^10 leave 2e-9 and 2e-10 at pi / 4.
template <int V>
struct Waves {
  float c[V], s[V];

  __device__ __forceinline__ void one(int i, double t, float scale, float sign) {
    const double q = __builtin_rint(4.0 * t);
    const float r = static_cast<float>(__builtin_fma(-0.25, q, t)) * 6.283185307179586f;
    const float z = r * r;
    float a = __builtin_fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
    a = __builtin_fmaf(z, a, 8.333333333333333e-3f);
    a = __builtin_fmaf(z, a, -0.16666666666666667f);
    a = __builtin_fmaf(z * r, a, r);  // sin r
    float b = __builtin_fmaf(z, -2.7557319223985888e-7f, 2.4801587301587302e-5f);
    b = __builtin_fmaf(z, b, -1.3888888888888889e-3f);
    b = __builtin_fmaf(z, b, 4.1666666666666664e-2f);
    b = __builtin_fmaf(z, b, -0.5f);
    b = __builtin_fmaf(z, b, 1.0f);   // cos r
    // a quarter turn more: (cos, sin) becomes (-sin, cos)
    const int k = static_cast<int>(static_cast<int64_t>(q)) & 3;
    const float ck = k & 1 ? a : b, sk = k & 1 ? b : a;
    c[i] = ((k + 1) & 2 ? -scale : scale) * ck;
    s[i] = (k & 2 ? -scale : scale) * sign * sk;
  }

  template <bool WHOLE, class U>
  __device__ __forceinline__ void at(const HeadsCore& A, const U& u, int32_t position) {
    constexpr double kTurn = 0.15915494309189533577;  // 1 / 2 pi
    double f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.0;
    auto index = [&](int i) { return u.first[i / (V / 2)] + i % (V / 2); };
    if (u.turned) {
      if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const hd2 w = *reinterpret_cast<const hd2_any*>(A.frequencies + index(i));
          f[i] = w[0];
          f[i + 1] = w[1];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (index(i) < A.rotated / 2) f[i] = A.frequencies[index(i)];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) one(i, static_cast<double>(position) * (f[i] * kTurn), A.turn_scale, A.sign);
  }
};

// The turned pairs of a unit; other channels stay as they are, whatever they hold.
template <bool PAIRS, int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const Waves<V>& w, bool turned) {
  if (!turned) return;
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float x = a[i], y = a[i + 1], u = b[i], v = b[i + 1];
      const float c = w.c[i / 2], s = w.s[i / 2], d = w.c[(V + i) / 2], t = w.s[(V + i) / 2];
      a[i] = x * c - y * s;
      a[i + 1] = y * c + x * s;
      b[i] = u * d - v * t;
      b[i + 1] = v * d + u * t;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * w.c[i] - y * w.s[i];
      b[i] = y * w.c[i] + x * w.s[i];
    }
  }
}

// A chunk of a row: one load but in rows of less than 16 bytes, which all waves
// that have none skip.
template <class T, bool TAIL>
__device__ __forceinline__ rw4 load_whole(const char* p, int n, bool room) {
  if constexpr (!TAIL) return load_chunk<T, false, false>(p, n, room);
  constexpr int V = kChunk<T>;
  rw4 w{0u, 0u, 0u, 0u};
  if (n >= V || (room && n > 0)) {
    w = __builtin_nontemporal_load(reinterpret_cast<const rw4_any*>(p - (n < V ? (V - n) * static_cast<int>(sizeof(T)) : 0)));
  } else if (n > 0) {
    w = load_chunk<T, false, true>(p, n, false);
  }
  return w;
}

// A chunk to a row.  Runs of lanes that fill whole lines of 128 bytes pass the L2s
// by ([16384, 32 + 8, 128] bfloat16, halves: 58 us, kept 62); of shorter ones two
// instructions fill a line, which only then is written (20480 tokens appended in
// pairs of half the channels: 105 us, not kept 110).  Norms, which have more to do
// for a row, lose more by the branch (60 us, 63).
template <class T, bool TAIL>
__device__ __forceinline__ void store_whole(char* p, int n, const rw4& r, bool keep) {
  constexpr int V = kChunk<T>;
  constexpr bool kBits = TAIL && sizeof(T) == 2;
  if (kBits && n < V) {
    // the bits of n: at most three stores
    uint32_t a = r[0], b = r[1];
    if (n & 4) {
      *reinterpret_cast<rw2_any*>(p) = rw2{a, b};
      p += 8;
      a = r[2];
      b = r[3];
    }
    if (n & 2) {
      *reinterpret_cast<rw1_any*>(p) = a;
      p += 4;
      a = b;
    }
    if (n & 1) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(a);
  } else if (!keep || n < V) {
    asm volatile("");  // keeps the branches apart: joined, the stores would lose their policy
    store_chunk<T, TAIL && !kBits>(p, n, r);
    asm volatile("");
  } else {
    *reinterpret_cast<rw4_any*>(p) = r;
  }
}
// V codes of a chunk, as many as n says.
template <int V, bool TAIL>
__device__ __forceinline__ void store_whole_codes(char* p, int n, const Codes<V>& c) {
  if (!TAIL || n >= V) {
    store_codes<V, false>(p, n, c);
    return;
  }
  uint32_t a = c.w[0];
  if constexpr (V == 8) {
    if (n & 4) {
      *reinterpret_cast<rw1_any*>(p) = a;
      p += 4;
      a = c.w[V / 4 - 1];
    }
  }
  if (n & 2) {
    typedef uint16_t any __attribute__((aligned(1)));
    *reinterpret_cast<any*>(p) = static_cast<uint16_t>(a);
    p += 2;
    a >>= 16;
  }
  if (n & 1) *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(a);
}

// A unit of a row.
template <class T, bool PAIRS, bool WHOLE>
struct Piece {
  static constexpr int V = kChunk<T>;
  rw4 raw[2];

  // a chunk of fewer channels in a row that has 16 bytes up to its end
  static __device__ __forceinline__ bool room(const Unit<T, PAIRS>& u, int k) { return u.at[k] + u.n[k] >= V; }

  __device__ __forceinline__ void load(const char* row, const Unit<T, PAIRS>& u, bool there) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      raw[k] = load_whole<T, !WHOLE>(row + u.at[k] * static_cast<int>(sizeof(T)), there ? u.n[k] : 0, room(u, k));
  }
  __device__ __forceinline__ void values(const Unit<T, PAIRS>& u, bool there, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) place_tail<T, !WHOLE>(&raw[k], there ? u.n[k] : 0, room(u, k));
    widen(raw[0], a, static_cast<const T*>(nullptr));
    widen(raw[1], b, static_cast<const T*>(nullptr));
  }
  static __device__ __forceinline__ void store(bool keep, char* row, const Unit<T, PAIRS>& u, bool there,
                                               const float (&a)[V], const float (&b)[V]) {
    store_whole<T, !WHOLE>(row + u.at[0] * static_cast<int>(sizeof(T)), there ? u.n[0] : 0,
                           narrow(a, static_cast<const T*>(nullptr)), keep);
    store_whole<T, !WHOLE>(row + u.at[1] * static_cast<int>(sizeof(T)), there ? u.n[1] : 0,
                           narrow(b, static_cast<const T*>(nullptr)), keep);
  }
};

// The lane's units of U passes over the heads.  A kernel loads the first ones of
// every tensor before it looks for positions and pages and forms angles: neither
// waits for the other.
template <class T, bool PAIRS, bool WHOLE, int U>
struct Passes {
  Piece<T, PAIRS, WHOLE> piece[U];

  static __device__ __forceinline__ uint32_t head(const HeadsCore& A, uint32_t pass, uint32_t slot) {
    return (pass << A.heads_log2) + slot;
  }
  __device__ __forceinline__ void load(const HeadsCore& A, const char* x, int64_t x_head, const Unit<T, PAIRS>& u,
                                       uint32_t heads, uint32_t slot, uint32_t from, uint32_t to) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t h = head(A, from + k, slot);
      piece[k].load(x + h * x_head, u, from + k < to && h < heads);
    }
  }
};

// The unit's channels of a weight.
template <class T, bool PAIRS, bool WHOLE>
__device__ __forceinline__ void load_weight(const float* w, const Unit<T, PAIRS>& u, float (&a)[kChunk<T>],
                                            float (&b)[kChunk<T>]) {
  constexpr int V = kChunk<T>;
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = b[i] = 1.0f;
  if (w == nullptr) return;
  if constexpr (WHOLE) {
    if (u.n[0] == 0) return;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const hf4 x = *reinterpret_cast<const hf4_any*>(w + u.at[0] + i);
      const hf4 y = *reinterpret_cast<const hf4_any*>(w + u.at[1] + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[i + k] = x[k];
        b[i + k] = y[k];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < u.n[0]) a[i] = w[u.at[0] + i];
      if (i < u.n[1]) b[i] = w[u.at[1] + i];
    }
  }
}

// Where a wave's lanes stand: its group of tokens, its passes, and each lane's
// token, head slot and unit.
struct HeadPlace {
  uint32_t group, pass;   // uniform
  uint32_t token, slot, unit;

  __device__ __forceinline__ HeadPlace(const HeadsCore& A, uint32_t wave) {
    const uint32_t lane = threadIdx.x & 63u;
    group = divide(wave, A.parts);
    pass = (wave - group * A.parts.d) * A.per_wave;
    const uint32_t row = lane >> A.lanes_log2;
    unit = lane & ((1u << A.lanes_log2) - 1u);
    slot = row & ((1u << A.heads_log2) - 1u);
    token = (group << (6 - A.lanes_log2 - A.heads_log2)) + (row >> A.heads_log2);
  }
};

__device__ __forceinline__ char* token_row(const HeadsCore& A, const HeadTensor& t, uint32_t token) {
  const uint32_t i = divide(token, A.n2);
  return t.p + i * t.s[0] + (token - i * A.n2.d) * t.s[1];
}

__device__ __forceinline__ uint32_t wave_index() {
  return blockIdx.x * (kHeadThreads / 64) + static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
}

// rstd of a head from its sum of squares: NaN where that is no number of
// float32 (its reciprocal root, zero, would make finite channels zero).
__device__ __forceinline__ float head_rstd(float sum, float dim, float eps) {
  const float v = sum / dim + eps;
  return v < __builtin_inff() ? __builtin_amdgcn_rsqf(v) : as_float(0x7FC00000u);
}

}  // namespace dev
}  // namespace acp
