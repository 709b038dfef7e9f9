// Device side of attention over a paged cache: rows' places, keys' addresses,
// the 8-bit codes as matrix operands, and the form for rows that need care.
#pragma once

#include "acp_attn.hpp"
#include "acp_dev_cache.hpp"
#include "acp_dev_heads.hpp"
#include "acp_dev_walk.hpp"

namespace acp {
namespace dev {

typedef _Float16 ah8 __attribute__((ext_vector_type(8)));
typedef __bf16 ab8 __attribute__((ext_vector_type(8)));
typedef _Float16 ah2 __attribute__((ext_vector_type(2)));
typedef __bf16 ab2 __attribute__((ext_vector_type(2)));
typedef float af4 __attribute__((ext_vector_type(4)));
typedef float af16 __attribute__((ext_vector_type(16)));
typedef short as4 __attribute__((ext_vector_type(4)));
typedef int ai2 __attribute__((ext_vector_type(2)));
#define ACP_LDS __attribute__((address_space(3)))

// ---------------------------------------------------------------- tiles

// The kernel's arguments, read anew: what a tile's work needs of them is not
// kept in registers from one tile to the next.
__device__ __forceinline__ const AttendArgs& attend_args() {
  auto p = (const __attribute__((address_space(4))) AttendArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttendArgs*)p;
}
// Likewise the lane's number.
__device__ __forceinline__ uint32_t thread_again() {
  uint32_t t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

__device__ __forceinline__ char* head_row(const AttendArgs& A, const HeadTensor& t, uint32_t token, uint32_t head) {
  const uint32_t i = divide(token, A.n2);
  return t.p + i * t.s[0] + (token - i * A.n2.d) * t.s[1] + head * t.s[2];
}

// Where a tile's rows go, if not to the output: their partial results, of rows
// that `index` counts from the workgroup's and the tile's place.
struct Partial {
  bool wanted;
  uint64_t row;  // of the first

  template <int M, uint32_t CUT, bool SHARES>
  __device__ __forceinline__ Partial(const AttendArgs& A, const Walk<M, CUT, SHARES>& w, const Tile& t, uint32_t kv) {
    if constexpr (!SHARES) {
      wanted = false;
      row = 0;
      return;
    }
    wanted = !(w.head && w.tail);
    row = ((static_cast<uint64_t>(w.share) * A.kv_heads.d + kv) * 2u + (w.head ? 1u : 0u)) *
          (static_cast<uint32_t>(M) << A.side_log2);
    if (w.head && threadIdx.x == 0) {
      uint32_t* j = A.joins + 2 * ((Tile::slot_of<M>(A, t.seq) + w.tile) * static_cast<uint64_t>(A.kv_heads.d) + kv);
      j[0] = w.share;
      j[1] = w.tail ? 1u : w.meets(A);
    }
  }
  __device__ __forceinline__ float* part(const AttendArgs& A, uint32_t index) const {
    return wanted ? A.part + (row + index) * A.dim : nullptr;
  }
  __device__ __forceinline__ float* stat(const AttendArgs& A, uint32_t index) const { return A.stat + 2 * (row + index); }
};

// Page and index of a key that is below tile.keys; -1: it has no page.
__device__ __forceinline__ int32_t key_page(const AttendArgs& A, uint32_t seq, uint32_t key, uint32_t* index) {
  const uint32_t n = divide(key, A.batch.page);
  *index = key - n * A.batch.page.d;
  return page_of(A.batch, seq, n);
}

// The same in two parts, for loops over keys: the load, at an address that is
// right for any key (keys > 0), and what it says, once it is needed.  A test in
// between would wait for all that was loaded before.
__device__ __forceinline__ int32_t page_entry(const AttendArgs& A, uint32_t seq, uint32_t key, uint32_t keys) {
  const uint32_t n = divide(key < keys ? key : keys - 1u, A.batch.page);
  return A.batch.pages[static_cast<uint64_t>(seq) * A.batch.max_pages + n];
}
__device__ __forceinline__ int32_t entry_page(const AttendArgs& A, int32_t entry, uint32_t key, uint32_t keys) {
  return key < keys && static_cast<uint32_t>(entry) < A.batch.page_count ? entry : -1;
}

// Lane `src`'s value.
__device__ __forceinline__ int64_t from_lane(int64_t v, uint32_t src) {
  const int lo = __builtin_amdgcn_ds_bpermute(static_cast<int>(src * 4u), static_cast<int>(v));
  const int hi = __builtin_amdgcn_ds_bpermute(static_cast<int>(src * 4u), static_cast<int>(v >> 32));
  return static_cast<int64_t>(static_cast<uint32_t>(lo)) | static_cast<int64_t>(hi) << 32;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The two halves of lanes that hold one row's values 16 or 32 lanes apart.
template <int STEP>
__device__ __forceinline__ float max_step(float v) {
  return as_float(static_cast<uint32_t>(lane_step<STEP>(static_cast<int>(as_bits(v)), [](int a, int b) {
    return static_cast<int>(
        as_bits(__builtin_fmaxf(as_float(static_cast<uint32_t>(a)), as_float(static_cast<uint32_t>(b)))));
  })));
}
template <int STEP>
__device__ __forceinline__ float sum_step(float v) {
  return as_float(static_cast<uint32_t>(lane_step<STEP>(static_cast<int>(as_bits(v)), [](int a, int b) {
    return static_cast<int>(as_bits(as_float(static_cast<uint32_t>(a)) + as_float(static_cast<uint32_t>(b))));
  })));
}

// ---------------------------------------------------------------- operands

template <class T>
__device__ __forceinline__ af4 mfma16(const rw4& a, const rw4& b, af4 c) {
  if constexpr (std::is_same_v<T, _Float16>)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(ah8, a), __builtin_bit_cast(ah8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(ab8, a), __builtin_bit_cast(ab8, b), c, 0, 0, 0);
}
template <class T>
__device__ __forceinline__ af16 mfma32(const rw4& a, const rw4& b, af16 c) {
  if constexpr (std::is_same_v<T, _Float16>)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(ah8, a), __builtin_bit_cast(ah8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(ab8, a), __builtin_bit_cast(ab8, b), c, 0, 0, 0);
}

// Eight weights in two parts of T.  The first is cut off towards zero, so that the
// other is above zero too: an infinite value times both is infinite, and not the
// difference of two.  Its least keeps it from zero where the first part is the
// whole weight; 8-bit values are finite, and need none.
template <class T, int FMT>
__device__ __forceinline__ void two_parts(const float (&p)[8], rw4* first, rw4* second) {
  constexpr bool kHalf = std::is_same_v<T, _Float16>;
  constexpr float kLeast = FMT != kCacheSame ? 0.0f : kHalf ? 5.9604644775390625e-8f : 7.888609052210118e-31f;  // 2^-24, 2^-100
  float rest[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = p[2 * k], b = p[2 * k + 1];
    float c, d;
    if constexpr (kHalf) {
      // less the least, so that small weights are rounded to nearest and not up
      constexpr bool small = FMT == kCacheSame;
      const auto w = __builtin_amdgcn_cvt_pkrtz(small ? __builtin_fmaxf(a - kLeast, 0.0f) : a,
                                                small ? __builtin_fmaxf(b - kLeast, 0.0f) : b);
      (*first)[k] = __builtin_bit_cast(uint32_t, w);
      c = static_cast<float>(w[0]);
      d = static_cast<float>(w[1]);
    } else {
      (*first)[k] = __builtin_amdgcn_perm(as_bits(b), as_bits(a), 0x07060302u);
      c = as_float(as_bits(a) & 0xFFFF0000u);
      d = as_float(as_bits(b) & 0xFFFF0000u);
    }
    // between the least and the weight: zero where that is, the least where both are infinite
    rest[2 * k] = __builtin_amdgcn_fmed3f(a - c, kLeast, a);
    rest[2 * k + 1] = __builtin_amdgcn_fmed3f(b - d, kLeast, b);
  }
  *second = narrow(rest, static_cast<const T*>(nullptr));
}

// 16 bytes for each lane from its address to LDS: lane l's come to offset + 16 l.
// The waits are the caller's (s_nop: between the write of M0 and its use).
__device__ __forceinline__ void to_lds(const char* from, uint32_t offset) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(offset) : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ACP_LDS const char*)p));
}

// l plus the two values of T in w.
template <class T>
__device__ __forceinline__ float add_pair(uint32_t w, float l) {
  if constexpr (std::is_same_v<T, _Float16>) {
    const ah2 one = {static_cast<_Float16>(1.0f), static_cast<_Float16>(1.0f)};
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(ah2, w), one, l, false);
  } else {
    const ab2 one = {static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)};
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(ab2, w), one, l, false);
  }
}

// Eight codes as values of T: all of them are exact in either type.
//   e4m3  the conversion of gfx950, scale 1
//   i8    u = code + 128 as an unsigned byte; float16: 1024 + u is the bits 0x6400
//         | u, less 1152; bfloat16: through float32, whose low half is zero
template <class T, int FMT>
__device__ __forceinline__ rw4 codes_to(uint32_t lo, uint32_t hi) {
  rw4 r;
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (FMT == kCacheE4M3) {
      if constexpr (std::is_same_v<T, _Float16>) {
        r[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k], 1.0f, false));
        r[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k], 1.0f, true));
      } else {
        r[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], 1.0f, false));
        r[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], 1.0f, true));
      }
    } else {
      const uint32_t u = w[k] ^ 0x80808080u;
      if constexpr (std::is_same_v<T, _Float16>) {
        const ah2 off = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
        const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);  // bytes: u0, 64, u1, 64
        const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
        r[2 * k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(ah2, a) - off);
        r[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(ah2, b) - off);
      } else {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = static_cast<float>((u >> (8 * i)) & 0xFFu) - 128.0f;
        r[2 * k] = __builtin_amdgcn_perm(as_bits(f[1]), as_bits(f[0]), 0x07060302u);
        r[2 * k + 1] = __builtin_amdgcn_perm(as_bits(f[3]), as_bits(f[2]), 0x07060302u);
      }
    }
  }
  return r;
}

__device__ __forceinline__ float one_code(int fmt, uint8_t c) {
  return fmt == kCacheI8 ? static_cast<float>(static_cast<int8_t>(c)) : __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 0);
}

__device__ __forceinline__ float one_value(const char* p, const _Float16*) {
  return static_cast<float>(*reinterpret_cast<const _Float16*>(p));
}
__device__ __forceinline__ float one_value(const char* p, const bf16_t*) {
  return as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
}
__device__ __forceinline__ void put_value(char* p, float v, const _Float16*) {
  *reinterpret_cast<_Float16*>(p) = static_cast<_Float16>(v);
}
__device__ __forceinline__ void put_value(char* p, float v, const bf16_t*) {
  *reinterpret_cast<__bf16*>(p) = static_cast<__bf16>(v);
}

// The running maximum is taken up only when it grows by 2^kRise or more: weights
// of up to 2^kRise lose nothing, and most steps need no rescaling.  float16 has few
// powers of two below one, and weights under 2^-25 of a step's largest would be
// lost, however many they are: its weights are 2^kRoom times theirs, so that those
// down to 2^-25 of the row's largest keep their digits and others are off by 2^-36
// of it.  (A rise of 8 leaves a room of 7, so 2^-32, and takes as long: prompts of
// [2 x 8192 tokens, 32 / 8 heads, 128] 802 us and 801.)
template <class T, int FMT>
struct Weights {
  static constexpr bool kHalf = FMT == kCacheSame && std::is_same_v<T, _Float16>;
  static constexpr float kRise = kHalf ? 4.0f : 8.0f, kRoom = kHalf ? 11.0f : 0.0f;
};

// float16 weights that carry the scales of 8-bit values: a row's are held in
// units of a power of two of its own, so that its largest product of a weight and
// a scale is from 2^8 to 2^15 of them and the smallest are off by 2^-33 of that.
// Only what the row sees counts: products are zero elsewhere.  The values' scales
// come as kScale of themselves, which keeps products of weights of up to 2^15
// in float32's range.
struct WeightUnit {
  static constexpr int kScaleLog2 = -16;
  static constexpr float kScale = 1.0f / 65536.0f;
  static constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100: what is less is nothing in float16
  float most = kLeast;  // the largest product so far, by the present maximum
  float unit = 2.596148429267414e+33f;  // 2^111: a product times this is its weight

  // The row's maximum rose.
  __device__ __forceinline__ void shrink(float f) { most = __builtin_fmaxf(most * f, kLeast); }
  // A step's largest product, before its weights are formed: whether some lane's
  // unit no longer fits.
  __device__ __forceinline__ bool take(float largest) {
    most = __builtin_fmaxf(most, largest);
    return __builtin_amdgcn_ballot_w64(away()) != 0;
  }
  // Gives those lanes another, and says by which power of two their sums change.
  __device__ __forceinline__ int change() {
    if (!away()) return 0;
    const int before = log2();
    unit = as_float(265u - (as_bits(most) >> 23) << 23);  // 2^11 to 2^12
    return log2() - before;
  }
  // What the sums are multiplied by in the end, as a power of two.
  __device__ __forceinline__ int back() const { return -kScaleLog2 - log2(); }

 private:
  __device__ __forceinline__ bool away() const {
    constexpr uint32_t kLow = 135u << 23, kHigh = 142u << 23;  // 2^8, 2^15
    return as_bits(most * unit) - kLow >= kHigh - kLow;
  }
  __device__ __forceinline__ int log2() const { return static_cast<int>(as_bits(unit) >> 23) - 127; }
};

// ---------------------------------------------------------------- rows that need care

// A weight of zero times a value that is not finite is NaN, so a token's row
// would take on what lies behind it in a product over a whole tile of keys.
// Rows that come out not finite, and that have such a value among the tile's keys
// that they do not see, are computed again by row_by_keys: one wave, one row, one
// key after another.  That takes about half a microsecond a key and row (a NaN in
// the newest value of a prompt of [8192, 32 / 8 heads, 128]: 127 ms); rows that see
// the value themselves are what they should be, and stay.

// Position of the last of a tile's keys [begin, keys) that some of its rows do not
// see and whose value is not finite; -1: none.  A lane looks at a key's row.
template <class T, int FMT>
__device__ __forceinline__ int32_t last_odd_value(const AttendArgs& A, const Tile& t, uint32_t begin, uint32_t keys, uint32_t kv) {
  int32_t last = -1;
  if constexpr (FMT == kCacheI8) return last;  // codes are finite, and hidden keys' scales do not count
  const uint32_t hidden = t.low < 0 ? 0u : static_cast<uint32_t>(t.low) + 1u;
  for (uint32_t key0 = begin > hidden ? begin : hidden; key0 < keys; key0 += 64u) {
    const uint32_t key = key0 + (threadIdx.x & 63u);
    uint32_t index;
    const int32_t page = key < keys ? key_page(A, t.seq, key, &index) : -1;
    bool odd = false;
    if (page >= 0) {
      const char* v = A.v.p + page * A.v.s[0] + index * A.v.s[1] + kv * A.v.s[2];
      for (uint32_t c = 0; c < A.dim; c += 8u) {
        if constexpr (FMT == kCacheSame) {
          const rw4 w = *reinterpret_cast<const rw4_any*>(v + c * 2u);
          constexpr uint32_t kTop = std::is_same_v<T, _Float16> ? 0x7C00u : 0x7F80u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            odd = odd || (w[k] & kTop) == kTop || (w[k] >> 16 & kTop) == kTop;
        } else {
          const rw2 w = *reinterpret_cast<const rw2_any*>(v + c);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int b = 0; b < 32; b += 8) odd = odd || (w[k] >> b & 0x7Fu) == 0x7Fu;
        }
      }
    }
    const uint64_t m = __builtin_amdgcn_ballot_w64(odd);
    if (m != 0u) last = static_cast<int32_t>(key0) + 63 - __builtin_clzll(m);
  }
  return last;
}

// Keys [from, to); part and stat: the row's partial results, or null for the
// output itself.
template <class T, int FMT, int DP>
__device__ __forceinline__ void row_by_keys(const AttendArgs& A, const Tile& t, uint32_t row, uint32_t kv, uint32_t from,
                                            uint32_t to, float* part, float* stat) {
  constexpr int E = DP / 64;
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t token, head;
  t.place(A, row, kv, &token, &head);
  const int32_t last = t.position(A, row);
  const uint32_t kv_heads = A.kv_heads.d << A.side_log2;
  const uint32_t end = last + 1 <= 0 ? 0u : static_cast<uint32_t>(last + 1) < to ? static_cast<uint32_t>(last + 1) : to;
  const char* qr = head_row(A, A.q, token, head);
  float q[E], o[E], m = -__builtin_inff(), l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t c = lane * E + e;
    q[e] = c < A.dim ? one_value(qr + c * 2, static_cast<const T*>(nullptr)) : 0.0f;
    if (A.flip) q[e] = -q[e];
    o[e] = 0.0f;
  }
  for (uint32_t key = from; key < end; ++key) {
    uint32_t index;
    const int32_t page = key_page(A, t.seq, key, &index);
    if (page < 0) continue;
    const char* kr = A.k.p + page * A.k.s[0] + index * A.k.s[1] + kv * A.k.s[2];
    const char* vr = A.v.p + page * A.v.s[0] + index * A.v.s[1] + kv * A.v.s[2];
    const uint64_t scale_at = (static_cast<uint64_t>(page) * A.batch.page.d + index) * kv_heads + kv;
    float v[E], dot = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = lane * E + e;
      float kc = 0.0f;
      v[e] = 0.0f;
      if (c < A.dim) {
        if constexpr (FMT == kCacheSame) {
          kc = one_value(kr + c * 2, static_cast<const T*>(nullptr));
          v[e] = one_value(vr + c * 2, static_cast<const T*>(nullptr));
        } else {
          kc = one_code(FMT, static_cast<uint8_t>(kr[c])) * A.k.scales[scale_at];
          v[e] = one_code(FMT, static_cast<uint8_t>(vr[c])) * A.v.scales[scale_at];
        }
      }
      dot = __builtin_fmaf(q[e], kc, dot);
    }
    const float s = sum_lanes(dot, 6) * A.scale;
    const float top = __builtin_fmaxf(m, s), base = top == -__builtin_inff() ? 0.0f : top;
    const float shrink = exp2_of(m - base), p = exp2_of(s - base);
    l = l * shrink + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(p, v[e], o[e] * shrink);
    m = top;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t c = lane * E + e;
    if (c >= A.dim) continue;
    if (part == nullptr)
      put_value(head_row(A, A.out, token, head) + c * 2, l == 0.0f ? 0.0f : o[e] / l, static_cast<const T*>(nullptr));
    else
      part[c] = o[e];
  }
  if (part != nullptr && lane == 0) {
    stat[0] = m;
    stat[1] = l;
  }
}

__device__ __forceinline__ bool is_finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }

// Workgroup of a launch: the cache's heads (the form for few rows: groups of
// them) are neighbours, so that an XCD, which takes every eighth workgroup and
// has an L2 of its own, sees few heads.  Without shares the last tiles, which see
// most keys, come first.
struct AttendPlace {
  uint32_t kv, index;
  __device__ __forceinline__ AttendPlace(const AttendArgs& A) {
    index = divide(blockIdx.x, A.kv_heads);
    kv = blockIdx.x - index * A.kv_heads.d;
    if (A.shares == 0) index = A.slots.d - 1u - index;
  }
};
inline uint32_t attend_grid(const AttendArgs& a) { return a.kv_heads.d * (a.shares ? a.shares : a.slots.d); }

}  // namespace dev
}  // namespace acp
