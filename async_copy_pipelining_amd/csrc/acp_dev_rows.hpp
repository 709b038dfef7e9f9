// Device side of the row operators: chunk loads and stores, the activations,
// and the 8-bit forms.
#pragma once

#include <type_traits>

#include "acp_engine.hpp"
#include "acp_rows.hpp"

namespace acp {
namespace dev {

typedef unsigned rw4 __attribute__((ext_vector_type(4)));
typedef unsigned rw2 __attribute__((ext_vector_type(2)));
// the same at any byte address
typedef rw4 rw4_any __attribute__((aligned(1)));
typedef rw2 rw2_any __attribute__((aligned(1)));
typedef unsigned rw1_any __attribute__((aligned(1)));
typedef float rf2 __attribute__((ext_vector_type(2)));

struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ uint32_t divide(uint32_t n, const Div& d) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.mag) >> (31 + d.sh));
}

__device__ __forceinline__ float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// ---------------------------------------------------------------- across lanes

// f(v, w) with w from the other half of each 2^(STEP + 1) neighbouring lanes,
// where the lanes of a half hold one value already (steps are taken in
// order).  Within a row of 16 lanes these are DPP moves of the vector ALU
// (neighbour, pair, mirrored 8, mirrored 16), past it the row swaps; none
// waits for LDS as a general permute does.
template <int STEP, class F>
__device__ __forceinline__ int lane_step(int v, F f) {
  if constexpr (STEP == 0) return f(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true));
  if constexpr (STEP == 1) return f(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true));
  if constexpr (STEP == 2) return f(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));
  if constexpr (STEP == 3) return f(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));
  if constexpr (STEP == 4) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return f(static_cast<int>(p[0]), static_cast<int>(p[1]));
  }
  if constexpr (STEP == 5) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return f(static_cast<int>(p[0]), static_cast<int>(p[1]));
  }
  return v;
}

// f over the 2^n lanes that share a value to be made, n uniform; the lanes
// are aligned to 2^n and all of them get the result.
template <class F>
__device__ __forceinline__ int over_lanes(int v, int n, F f) {
  if (n > 0) v = lane_step<0>(v, f);
  if (n > 1) v = lane_step<1>(v, f);
  if (n > 2) v = lane_step<2>(v, f);
  if (n > 3) v = lane_step<3>(v, f);
  if (n > 4) v = lane_step<4>(v, f);
  if (n > 5) v = lane_step<5>(v, f);
  return v;
}

__device__ __forceinline__ float sum_lanes(float v, int n) {
  return as_float(static_cast<uint32_t>(over_lanes(static_cast<int>(as_bits(v)), n, [](int a, int b) {
    return static_cast<int>(as_bits(as_float(static_cast<uint32_t>(a)) + as_float(static_cast<uint32_t>(b))));
  })));
}

// ---------------------------------------------------------------- 16-byte chunks

template <class T>
constexpr int kChunk = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ void widen(const rw4& r, float (&f)[8], const _Float16*) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const uint32_t w = r[k];  // a scalar: a bit cast of the vector's element would read element 0
    const h2 h = __builtin_bit_cast(h2, w);
    f[2 * k] = static_cast<float>(h[0]);
    f[2 * k + 1] = static_cast<float>(h[1]);
  }
}
__device__ __forceinline__ void widen(const rw4& r, float (&f)[8], const bf16_t*) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = as_float(r[k] << 16);
    f[2 * k + 1] = as_float(r[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const rw4& r, float (&f)[4], const float*) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = as_float(r[k]);
}

// One rounding to nearest, ties to even, from the float32 result.
__device__ __forceinline__ rw4 narrow(const float (&f)[8], const _Float16*) {
  rw4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 h = {static_cast<_Float16>(f[2 * k]), static_cast<_Float16>(f[2 * k + 1])};
    r[k] = __builtin_bit_cast(uint32_t, h);
  }
  return r;
}
__device__ __forceinline__ rw4 narrow(const float (&f)[8], const bf16_t*) {
  rw4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 h = {static_cast<__bf16>(f[2 * k]), static_cast<__bf16>(f[2 * k + 1])};
    r[k] = __builtin_bit_cast(uint32_t, h);
  }
  return r;
}
__device__ __forceinline__ rw4 narrow(const float (&f)[4], const float*) {
  rw4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = as_bits(f[k]);
  return r;
}

// `n` channels at p (all of a chunk, or fewer at a row's end; none for n <= 0);
// channels past n read as zero.  KEEP: another kernel reads them again soon
// (the cached policy; else non-temporal).  Without TAIL n is all or none.
//
// The last chunk of a row that is cut short: in rows of at least a chunk
// (`room`) the 16 bytes that end with the row are loaded, and place_tail moves
// them down where they are used.  Loads of single channels would have to be
// put together, and so waited for, before the next chunk's load ([4, 69, 2988]
// bfloat16 backward 26 us with those).
template <class T, bool KEEP = false, bool TAIL = true>
__device__ __forceinline__ rw4 load_chunk(const char* p, int n, bool room) {
  constexpr int V = kChunk<T>;
  if (TAIL ? n >= V || (room && n > 0) : n > 0) {
    if constexpr (TAIL) p -= n < V ? (V - n) * static_cast<int>(sizeof(T)) : 0;
    if constexpr (KEEP) return *reinterpret_cast<const rw4_any*>(p);
    return __builtin_nontemporal_load(reinterpret_cast<const rw4_any*>(p));
  }
  if constexpr (!TAIL) return rw4{0u, 0u, 0u, 0u};
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < V - 1; ++k)
    if (k < n) {
      if constexpr (sizeof(T) == 2)
        w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[k]) << (16 * (k & 1));
      else
        w[k] = reinterpret_cast<const uint32_t*>(p)[k];
    }
  return rw4{w[0], w[1], w[2], w[3]};
}

template <class T, bool TAIL = true>
__device__ __forceinline__ void place_tail(rw4* r, int n, bool room) {
  constexpr int V = kChunk<T>;
  if (!TAIL || !room || n <= 0 || n >= V) return;
  const int gap = (V - n) * static_cast<int>(sizeof(T));  // bytes of the channels before
  uint32_t a = (*r)[0], b = (*r)[1], c = (*r)[2], d = (*r)[3];
  if (gap & 8) a = c, b = d, c = d = 0u;
  if (gap & 4) a = b, b = c, c = d, d = 0u;
  if (sizeof(T) == 2 && (gap & 2)) {
    a = a >> 16 | b << 16;
    b = b >> 16 | c << 16;
    c = c >> 16 | d << 16;
    d >>= 16;
  }
  *r = rw4{a, b, c, d};
}

template <class T, bool TAIL = true>
__device__ __forceinline__ void store_chunk(char* p, int n, const rw4& r) {
  constexpr int V = kChunk<T>;
  if (!TAIL || n >= V) {
    if (n > 0) __builtin_nontemporal_store(r, reinterpret_cast<rw4_any*>(p));
    return;
  }
#pragma unroll
  for (int k = 0; k < V - 1; ++k)
    if (k < n) {
      if constexpr (sizeof(T) == 2)
        reinterpret_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(r[k / 2] >> (16 * (k & 1)));
      else
        reinterpret_cast<uint32_t*>(p)[k] = r[k];
    }
}

// The codes of a chunk: V bytes in V / 4 words.
template <int V>
struct Codes {
  uint32_t w[V / 4];
};

// as load_chunk and place_tail
template <int V, bool KEEP = false, bool TAIL = true>
__device__ __forceinline__ Codes<V> load_codes(const char* p, int n, bool room) {
  Codes<V> c;
  if (TAIL ? n >= V || (room && n > 0) : n > 0) {
    if constexpr (TAIL) p -= n < V ? V - n : 0;
    if constexpr (V == 8) {
      const rw2_any* q = reinterpret_cast<const rw2_any*>(p);
      const rw2 r = KEEP ? *q : __builtin_nontemporal_load(q);
      c.w[0] = r[0];
      c.w[1] = r[1];
    } else {
      const rw1_any* q = reinterpret_cast<const rw1_any*>(p);
      c.w[0] = KEEP ? *q : __builtin_nontemporal_load(q);
    }
    return c;
  }
#pragma unroll
  for (int k = 0; k < V / 4; ++k) c.w[k] = 0u;
  if constexpr (!TAIL) return c;
#pragma unroll
  for (int k = 0; k < V - 1; ++k)
    if (k < n) c.w[k / 4] |= static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(p)[k]) << (8 * (k & 3));
  return c;
}

template <int V, bool TAIL = true>
__device__ __forceinline__ void place_codes(Codes<V>* c, int n, bool room) {
  if (!TAIL || !room || n <= 0 || n >= V) return;
  const int gap = (V - n) * 8;  // bits of the codes before
  if constexpr (V == 8) {
    const uint64_t v = (static_cast<uint64_t>(c->w[1]) << 32 | c->w[0]) >> gap;
    c->w[0] = static_cast<uint32_t>(v);
    c->w[1] = static_cast<uint32_t>(v >> 32);
  } else {
    c->w[0] >>= gap;
  }
}

template <int V, bool TAIL = true>
__device__ __forceinline__ void store_codes(char* p, int n, const Codes<V>& c) {
  if (!TAIL && n == 0) return;
  if (!TAIL || n >= V) {
    if constexpr (V == 8) {
      __builtin_nontemporal_store(rw2{c.w[0], c.w[1]}, reinterpret_cast<rw2_any*>(p));
    } else {
      __builtin_nontemporal_store(c.w[0], reinterpret_cast<rw1_any*>(p));
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < V - 1; ++k)
    if (k < n) reinterpret_cast<uint8_t*>(p)[k] = static_cast<uint8_t>(c.w[k / 4] >> (8 * (k & 3)));
}

// ---------------------------------------------------------------- 8-bit forms

// Scale of a block from the bits of its largest |x| (an unsigned maximum of
// the sign-less bits, which puts NaN above infinity above every number).
//   i8:   max(fl(amax / 127), 2^-126), at most the largest float32 whose
//         127-fold is finite
//   e4m3: the smallest power of two >= 2^-126 with amax <= 448 * scale
//   a NaN or an infinity in the block: NaN, so all of it unpacks to NaN
__device__ __forceinline__ float block_scale(int format, uint32_t amax) {
  if (amax >= 0x7F800000u) return as_float(0x7FC00000u);
  if (format == 0) {
    const float s = as_float(amax) / 127.0f;
    return __builtin_fminf(__builtin_fmaxf(s, 0x1p-126f), 0x1.020406p+121f);
  }
  // amax = m 2^k with 1 <= m < 2, and 448 = 1.75 * 2^8
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

// Codes of x in a block of scale s.
//
// i8: round-half-even of the exact quotient x / s.  t = x * (1/s) is within
// 127 * 2^-21 of it, so its rounding q can only be wrong where t lies within
// 2^-13 of a half; there the remainder x - q s decides, which one fma gives
// exactly (it is a multiple of half an ulp of s and at most about s / 2).
// Adding 1.5 * 2^23 rounds t and leaves the two's complement code in the low
// byte.
// e4m3: x / s is exact (s is a power of two); the conversion rounds to
// nearest even, and |x / s| <= 448 is the format's largest value.  Under the
// scale of T's own largest values, 256 s would be past them: those that would
// round to it take 240 s.
template <class T>
constexpr float kTopScale = std::is_same_v<T, _Float16> ? 0x1p8f : 0x1p120f;

template <class T, int V>
__device__ __forceinline__ Codes<V> encode(int format, float (&x)[V], float s) {
  Codes<V> c;
  if (format == 0) {
    constexpr float kRound = 12582912.0f;
    const float inv = __builtin_amdgcn_rcpf(s);
    float u[V], off = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float t = x[k] * inv;
      u[k] = t + kRound;
      off = __builtin_fmaxf(off, __builtin_fabsf(t - (u[k] - kRound)));
    }
    if (off > 0.4998f) {
      const float half = 0.5f * s;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float q = u[k] - kRound;
        const float r = __builtin_fmaf(-q, s, x[k]);
        const float a = __builtin_fabsf(r);
        if (a > half || (a == half && (as_bits(u[k]) & 1u))) u[k] += __builtin_copysignf(1.0f, r);
      }
    }
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const uint32_t lo = __builtin_amdgcn_perm(as_bits(u[4 * k + 1]), as_bits(u[4 * k]), 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(as_bits(u[4 * k + 3]), as_bits(u[4 * k + 2]), 0x04000C0Cu);
      c.w[k] = lo | hi;
    }
  } else {
    const float inv = as_float((254u << 23) - as_bits(s));
    if (s >= kTopScale<T>) {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = __builtin_fminf(__builtin_fmaxf(x[k], -240.0f * s), 240.0f * s);
    }
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k] * inv, x[4 * k + 1] * inv, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2] * inv, x[4 * k + 3] * inv, w, true);
      c.w[k] = static_cast<uint32_t>(w);
    }
  }
  return c;
}

// The values that codes stand for: code * s, rounded once to float32.
template <int V>
__device__ __forceinline__ void decode(int format, const Codes<V>& c, float s, float (&x)[V]) {
  if (format == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      x[k] = static_cast<float>(static_cast<int8_t>(c.w[k / 4] >> (8 * (k & 3)))) * s;
  } else {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      const rf2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.w[k]), false);
      const rf2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c.w[k]), true);
      x[4 * k] = a[0] * s;
      x[4 * k + 1] = a[1] * s;
      x[4 * k + 2] = b[0] * s;
      x[4 * k + 3] = b[1] * s;
    }
  }
}

// Largest |x| of the 2^lb lanes that share a scale block, as bits.  The lanes
// of a block are aligned to 2^lb within their wave.
template <int V>
__device__ __forceinline__ uint32_t block_amax(const float (&x)[V], int lb) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const uint32_t b = as_bits(x[k]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return static_cast<uint32_t>(over_lanes(static_cast<int>(m), lb, [](int a, int b) { return a > b ? a : b; }));
}

// ---------------------------------------------------------------- activations

constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;

// 1 / (1 + e^-u): the hardware exponential and reciprocal, each within an
// ulp.  Below zero the argument's rounding and its constant's add 1.25 |u| 2^-24
// relative: 2^-20 at u = -10, where the result is 5e-5.
__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504088896341f));
}

// e^(-u^2 / 2), and the normal distribution's tail from it:
//   1 - Phi(|u|) = e^(-u^2 / 2) (a1 t + ... + an t^n),  t = 1 / (1 + p |u|),
// the form of formula 7.1.26 in Abramowitz and Stegun's Handbook of
// Mathematical Functions.  Its constants there bound the absolute error of erf
// and leave the tail 5e-5 off at |u| = 3 and 2e-2 at 10, relative to itself;
// those below were fitted to the tail's relative error over |u| <= 14.5, since
// u Phi(u) below zero is as small as the tail.  What is left, relative to it:
//   FINE  (float32)  1.7e-7 everywhere, eight terms
//   else  (16 bits)  2.9e-7 (1 + 4 u^2), six terms: 1e-5 at |u| = 2, 1.5e-4 at 13,
//         where half a step of float16 is 4.9e-4
// and float32's roundings, (16 + 1.5 u^2) 2^-24, the second term the bell's
// argument's.  A bell whose argument keeps what its products round off, and nine
// terms, leave 2^-21 of float32 at 4 to 6 us more of VALU work on [8192, 4096]
// float32 (norm and GELU 57 us for 53, with five terms 51; GELU and its backward
// pass, saved in i8, 107 for 101, 100).
// Past |u| = 13.2 the bell is below float32's normal range and so is the tail.
__device__ __forceinline__ float normal_bell(float u) {
  return __builtin_amdgcn_exp2f(u * u * -0.721347520444481704f);
}

// 1 - Phi(|u|)
template <bool FINE>
__device__ __forceinline__ float normal_tail(float u, float bell) {
  constexpr int N = FINE ? 8 : 6;
  constexpr float kP = FINE ? 0.3f : 0.42f;
  constexpr float k[8] = {FINE ? 0.119632013f : 0.166697279f,   FINE ? 0.120712139f : 0.179843664f,
                          FINE ? 0.100175977f : 0.0705016926f,  FINE ? 0.127691671f : 0.260967582f,
                          FINE ? -0.0520338044f : -0.23618038f, FINE ? 0.204556525f : 0.0581701808f,
                          -0.156158313f,                        0.0354237035f};
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(u), kP, 1.0f));
  float q = k[N - 1];
#pragma unroll
  for (int e = N - 2; e >= 0; --e) q = __builtin_fmaf(t, q, k[e]);
  return q * (t * bell);
}

// Phi(u)
__device__ __forceinline__ float normal_cdf(float u, float tail) { return u < 0.0f ? tail : 1.0f - tail; }

// act(u).  FINITE: u is no infinity, and u Phi(u) = max(u, 0) - |u| (1 -
// Phi(|u|)) takes two operations less of the VALU time that bounds a large
// norm with GELU ([128, 500, 1024] float16 2 to 4 % faster, timed in turn).
// FINE: as normal_tail's.
template <int ACT, bool FINITE, bool FINE>
__device__ __forceinline__ float act_value(float u) {
  if constexpr (ACT == kActSilu) return u * sigmoid(u);
  if constexpr (ACT == kActGelu) {
    const float tail = normal_tail<FINE>(u, normal_bell(u));
    if constexpr (FINITE) return __builtin_fmaf(-__builtin_fabsf(u), tail, __builtin_fmaxf(u, 0.0f));
    return u * normal_cdf(u, tail);
  }
  return u;
}

// act(u) and act'(u)
template <int ACT, bool FINE>
__device__ __forceinline__ void act_both(float u, float* value, float* slope) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(u);
    *value = u * s;
    *slope = s * (1.0f + u * (1.0f - s));
  } else if constexpr (ACT == kActGelu) {
    const float bell = normal_bell(u), tail = normal_tail<FINE>(u, bell);
    const float cdf = normal_cdf(u, tail);
    *value = u * cdf;
    *slope = __builtin_fmaf(u * 0.398942280401432678f, bell, cdf);
  } else {
    *value = u;
    *slope = 1.0f;
  }
}

// a chunk of float32, whose results keep what a 16-bit type rounds off
template <int V>
constexpr bool kFine = V == kChunk<float>;

template <int ACT, int V, bool FINITE = true>
__device__ __forceinline__ void act_values(float (&u)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) u[k] = act_value<ACT, FINITE, kFine<V>>(u[k]);
}

template <int V>
__device__ __forceinline__ void act_values(int act, float (&u)[V]) {
  if (act == kActSilu) act_values<kActSilu, V, false>(u);
  else if (act == kActGelu) act_values<kActGelu, V, false>(u);
}

// value = act(u) and slope = act'(u), channel by channel
template <int V>
__device__ __forceinline__ void act_pairs(int act, const float (&u)[V], float (&value)[V], float (&slope)[V]) {
  if (act == kActSilu) {
#pragma unroll
    for (int k = 0; k < V; ++k) act_both<kActSilu, kFine<V>>(u[k], &value[k], &slope[k]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int k = 0; k < V; ++k) act_both<kActGelu, kFine<V>>(u[k], &value[k], &slope[k]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) act_both<kActNone, kFine<V>>(u[k], &value[k], &slope[k]);
  }
}

}  // namespace dev
}  // namespace acp
