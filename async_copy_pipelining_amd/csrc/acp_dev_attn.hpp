// Device side of attention over a paged cache: tiles of rows, keys' addresses,
// the 8-bit codes as matrix operands, and the form for rows that need care.
#pragma once

#include "acp_attn.hpp"
#include "acp_dev_cache.hpp"
#include "acp_dev_heads.hpp"

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

// M rows of one sequence and one of the cache's heads.  All of it is uniform.
struct Tile {
  uint32_t seq, first;  // first row
  int32_t start, news;  // tokens of the sequence
  int32_t rows;         // rows of the sequence
  int32_t behind;       // position of the sequence's token i: behind + i
  int32_t keys;         // keys that some row of the tile sees
  int32_t low;          // position of the tile's first row

  // whether there is a tile in the slot
  template <int M>
  __device__ __forceinline__ bool find(const AttendArgs& A, uint32_t slot) {
    const BatchArgs& B = A.batch;
    uint32_t tile;
    if (B.starts == nullptr) {
      const uint32_t per = (A.group.d + M - 1) / M;
      seq = slot / per;
      tile = slot - seq * per;
      if (seq >= B.sequences || seq >= A.tokens) return false;
      start = static_cast<int32_t>(seq);
      news = 1;
    } else {
      auto base = [&](uint32_t s) {
        return static_cast<uint32_t>(static_cast<uint64_t>(static_cast<uint32_t>(B.starts[s])) * A.group.d / M) + s;
      };
      const uint32_t lane = threadIdx.x & 63u;
      seq = 0;
      for (uint32_t i = 1; i < B.sequences; i += 64u) {
        const bool before = i + lane < B.sequences && base(i + lane) <= slot;
        const uint32_t c = static_cast<uint32_t>(__builtin_popcountll(__builtin_amdgcn_ballot_w64(before)));
        seq += c;
        if (c < 64u) break;
      }
      if (base(seq) > slot) return false;
      tile = slot - base(seq);
      start = B.starts[seq];
      news = B.starts[seq + 1u] - start;
      if (start < 0 || news <= 0) return false;
    }
    behind = B.lengths[seq] - news;
    const int32_t left = static_cast<int32_t>(A.tokens) - start;  // starts past the tokens
    if (left <= 0) return false;
    rows = (news < left ? news : left) * static_cast<int32_t>(A.group.d);
    first = tile * M;
    if (first >= static_cast<uint32_t>(rows)) return false;
    const uint32_t last = first + M <= static_cast<uint32_t>(rows) ? first + M - 1u : static_cast<uint32_t>(rows) - 1u;
    low = position(A, first);
    const int64_t most = static_cast<int64_t>(B.max_pages) * B.page.d;
    const int64_t end = static_cast<int64_t>(position(A, last)) + 1;
    keys = static_cast<int32_t>(end < 0 ? 0 : end < most ? end : most);
    return true;
  }
  __device__ __forceinline__ int32_t position(const AttendArgs& A, uint32_t row) const {
    return behind + static_cast<int32_t>(divide(row, A.group));
  }
  // token and query head of a row
  __device__ __forceinline__ void place(const AttendArgs& A, uint32_t row, uint32_t kv, uint32_t* token,
                                        uint32_t* head) const {
    const uint32_t i = divide(row, A.group);
    *token = static_cast<uint32_t>(start) + i;
    *head = kv * A.group.d + (row - i * A.group.d);
  }
  // partial results that the tile's workgroups leave; 1: the output itself
  __device__ __forceinline__ uint32_t splits(const AttendArgs& A) const {
    const uint32_t n = (static_cast<uint32_t>(keys) + A.chunk - 1u) / A.chunk;
    return n < 1u ? 1u : n < A.splits ? n : A.splits;
  }
};

__device__ __forceinline__ char* head_row(const AttendArgs& A, const HeadTensor& t, uint32_t token, uint32_t head) {
  const uint32_t i = divide(token, A.n2);
  return t.p + i * t.s[0] + (token - i * A.n2.d) * t.s[1] + head * t.s[2];
}

// Page and index of a key that is below tile.keys; -1: it has no page.
__device__ __forceinline__ int32_t key_page(const AttendArgs& A, uint32_t seq, uint32_t key, uint32_t* index) {
  const uint32_t n = divide(key, A.batch.page);
  *index = key - n * A.batch.page.d;
  return page_of(A.batch, seq, n);
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

// ---------------------------------------------------------------- rows that need care

// A weight of zero times a value that is not finite is NaN, so a token's row
// would take on what lies behind it in a product over a whole tile of keys.
// Rows that come out not finite where the tile holds keys that they do not
// see are computed again by this: one wave, one row, one key after another,
// and no others.
template <class T, int FMT, int DP>
__device__ __forceinline__ void row_by_keys(const AttendArgs& A, const Tile& t, uint32_t row, uint32_t kv, uint32_t split,
                                            uint32_t splits) {
  constexpr int E = DP / 64;
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t token, head;
  t.place(A, row, kv, &token, &head);
  const int32_t last = t.position(A, row);
  const uint32_t end = last + 1 < t.keys ? static_cast<uint32_t>(last + 1 < 0 ? 0 : last + 1) : static_cast<uint32_t>(t.keys);
  const char* qr = head_row(A, A.q, token, head);
  float q[E], o[E], m = -__builtin_inff(), l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t c = lane * E + e;
    q[e] = c < A.dim ? one_value(qr + c * 2, static_cast<const T*>(nullptr)) : 0.0f;
    o[e] = 0.0f;
  }
  for (uint32_t from = split * A.chunk; from < end; from += A.splits * A.chunk) {
    const uint32_t to = from + A.chunk < end ? from + A.chunk : end;
    for (uint32_t key = from; key < to; ++key) {
      uint32_t index;
      const int32_t page = key_page(A, t.seq, key, &index);
      if (page < 0) continue;
      const char* kr = A.k.p + page * A.k.s[0] + index * A.k.s[1] + kv * A.k.s[2];
      const char* vr = A.v.p + page * A.v.s[0] + index * A.v.s[1] + kv * A.v.s[2];
      const uint64_t scale_at = (static_cast<uint64_t>(page) * A.batch.page.d + index) * A.kv_heads.d + kv;
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
      if (s == -__builtin_inff()) continue;
      const float top = __builtin_fmaxf(m, s);
      const float shrink = exp2_of(m - top), p = exp2_of(s - top);
      l = l * shrink + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(p, v[e], o[e] * shrink);
      m = top;
    }
  }
  const uint64_t at = (static_cast<uint64_t>(split) * A.tokens + token) * A.heads.d + head;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t c = lane * E + e;
    if (c >= A.dim) continue;
    if (splits == 1u)
      put_value(head_row(A, A.out, token, head) + c * 2, l == 0.0f ? 0.0f : o[e] / l, static_cast<const T*>(nullptr));
    else
      A.part[at * A.dim + c] = o[e];
  }
  if (splits > 1u && lane == 0) {
    A.stat[2 * at] = m;
    A.stat[2 * at + 1] = l;
  }
}

__device__ __forceinline__ bool is_finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }

// Workgroup of a launch: the cache's heads are neighbours (one XCD has the same
// head of every tile), then come tiles, the last ones, which see most keys,
// first, and then the splits.
struct AttendPlace {
  uint32_t kv, slot, split;
  __device__ __forceinline__ AttendPlace(const AttendArgs& A) {
    const uint32_t i = divide(blockIdx.x, A.kv_heads);
    kv = blockIdx.x - i * A.kv_heads.d;
    split = divide(i, A.slots);
    slot = A.slots.d - 1u - (i - split * A.slots.d);
  }
};

}  // namespace dev
}  // namespace acp
