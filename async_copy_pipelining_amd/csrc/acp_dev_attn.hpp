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

// A value that all lanes hold, in scalar registers.
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32)));
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// A sequence's tokens, as far as there are any.
struct Tokens {
  int32_t start, news;  // none: 0
  int32_t behind;       // position of its token i: behind + i
  int32_t rows;         // query heads of one of the cache's heads

  __device__ __forceinline__ Tokens(const AttendArgs& A, uint32_t seq) {
    const BatchArgs& B = A.batch;
    start = static_cast<int32_t>(seq);
    news = 1;
    if (B.starts != nullptr) {
      start = B.starts[seq];
      news = B.starts[seq + 1u] - start;
    }
    const int32_t length = B.lengths[seq];  // below zero as zero: nothing is seen
    behind = (length > 0 ? length : 0) - news;
    const int32_t left = static_cast<int32_t>(A.tokens) - start;  // starts past the tokens
    if (start < 0 || left <= 0 || news < 0) news = 0;
    rows = (news < left ? news : left) * static_cast<int32_t>(A.group.d);
    if (news == 0) rows = 0;
  }
};

// M rows of one sequence and one of the cache's heads.  All of it is uniform.
struct Tile {
  uint32_t seq, first;  // first row
  int32_t start, rows;  // of the sequence
  int32_t behind;
  int32_t keys;         // keys that some row of the tile sees
  int32_t low;          // position of the tile's first row

  // whether the sequence has such a tile
  template <int M>
  __device__ __forceinline__ bool set(const AttendArgs& A, uint32_t sequence, uint32_t tile) {
    const Tokens s(A, sequence);
    seq = sequence;
    first = tile * M;
    start = s.start;
    rows = s.rows;
    behind = s.behind;
    if (first >= static_cast<uint32_t>(rows)) return false;
    const uint32_t last = first + M <= static_cast<uint32_t>(rows) ? first + M - 1u : static_cast<uint32_t>(rows) - 1u;
    low = position(A, first);
    const int64_t most = static_cast<int64_t>(A.batch.max_pages) * A.batch.page.d;
    const int64_t end = static_cast<int64_t>(position(A, last)) + 1;
    keys = static_cast<int32_t>(end < 0 ? 0 : end < most ? end : most);
    return true;
  }
  // whether there is a tile in the slot
  template <int M>
  __device__ __forceinline__ bool find(const AttendArgs& A, uint32_t slot) {
    const BatchArgs& B = A.batch;
    uint32_t s = 0, tile;
    if (B.starts == nullptr) {
      const uint32_t per = (A.group.d + M - 1) / M;
      s = slot / per;
      tile = slot - s * per;
      if (s >= B.sequences) return false;
    } else {
      const uint32_t lane = threadIdx.x & 63u;
      for (uint32_t i = 1; i < B.sequences; i += 64u) {
        const bool before = i + lane < B.sequences && slot_of<M>(A, i + lane) <= slot;
        const uint32_t c = static_cast<uint32_t>(__builtin_popcountll(__builtin_amdgcn_ballot_w64(before)));
        s += c;
        if (c < 64u) break;
      }
      if (slot_of<M>(A, s) > slot) return false;
      tile = slot - slot_of<M>(A, s);
    }
    return set<M>(A, s, tile);
  }
  // the sequence's first slot
  template <int M>
  static __device__ __forceinline__ uint32_t slot_of(const AttendArgs& A, uint32_t s) {
    if (A.batch.starts == nullptr) return s * ((A.group.d + M - 1) / M);
    return static_cast<uint32_t>(static_cast<uint64_t>(static_cast<uint32_t>(A.batch.starts[s])) * A.group.d / M) + s;
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
};

// A workgroup's part of the work: a tile, or its share of all tiles of a head
// (the form with shares).
//
// For the shares the tiles of all sequences stand in a row, tile i of a sequence
// with base + (i + 1) q places, where base is the position of its first new token
// and q the tokens of a tile, rounded up: as many as its keys, or some more where
// the heads of a group do not divide a tile.  Share w has the places from floor(w
// total / shares) on.  Inside a tile the cut is moved down to a multiple of CUT
// keys; places past the tile's keys are no work.
constexpr int kWalkWords = 8;
template <int M, uint32_t CUT, bool SHARES>
struct Walk {
  uint64_t from, to, at;   // places of the share, and of the tile
  uint64_t total;
  uint32_t shares, share;
  uint32_t seq, tile, tiles;
  uint64_t base;

  // the tile's keys [begin, end) that are this workgroup's
  uint32_t begin, end;
  bool head, tail;         // its first key and its last place are

  static __device__ __forceinline__ uint32_t per_tile(const AttendArgs& A) { return (M + A.group.d - 1) / A.group.d; }
  static __device__ __forceinline__ uint64_t places(const AttendArgs& A, uint32_t s, uint32_t* tiles, uint64_t* base) {
    const Tokens t(A, s);
    const uint32_t n = (static_cast<uint32_t>(t.rows) + M - 1) / M;
    const int64_t most = static_cast<int64_t>(A.batch.max_pages) * A.batch.page.d;
    const int64_t b = t.behind < 0 ? 0 : t.behind < most ? t.behind : most;
    *tiles = n;
    *base = static_cast<uint64_t>(b);
    return before(A, n, *base);
  }
  // places of the first n tiles
  static __device__ __forceinline__ uint64_t before(const AttendArgs& A, uint64_t n, uint64_t base) {
    return n * base + n * (n + 1) / 2 * per_tile(A);
  }

  // Workgroups go to the eight XCDs in turn, so one of 1, 2 or 4 heads has every
  // P-th.  Each takes shares that follow one another, whose tiles read the same
  // keys through its L2 (6 chunks of up to 509 tokens over up to 6001, 28 / 4 heads
  // of 128: 191 us, in turn 195; 64 tokens over up to 4096, 32 / 8: 118, 126).
  static __device__ __forceinline__ uint32_t together(const AttendArgs& A, uint32_t index, uint32_t shares) {
    const uint32_t H = A.kv_heads.d;
    const uint32_t log2 = H == 1u ? 3u : H == 2u ? 2u : H == 4u ? 1u : 0u, P = 1u << log2;
    const uint32_t p = index & (P - 1u), rest = shares & (P - 1u);
    return p * (shares >> log2) + (p < rest ? p : rest) + (index >> log2);
  }
  // false: nothing to do.  All lanes of the workgroup take part.
  __device__ __forceinline__ bool begin_at(const AttendArgs& A, uint32_t index, uint64_t* lds) {
    if constexpr (!SHARES) return true;
    const uint32_t S = A.batch.sequences, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t each = (S + kAttendThreads - 1) / kAttendThreads, s0 = threadIdx.x * each;
    uint64_t mine = 0;
    uint32_t n;
    uint64_t b;
    for (uint32_t k = 0; k < each; ++k)
      if (s0 + k < S) mine += places(A, s0 + k, &n, &b);
    uint64_t sum = mine;
#pragma unroll
    for (uint32_t d = 1; d < 64u; d <<= 1) {
      const uint64_t other = __shfl_up(static_cast<unsigned long long>(sum), d);
      if (lane >= d) sum += other;
    }
    if (lane == 63u) lds[wave] = sum;
    __syncthreads();
    uint64_t before_me = sum - mine;
    total = 0;
#pragma unroll
    for (uint32_t k = 0; k < kAttendThreads / 64; ++k) {
      if (k < wave) before_me += lds[k];
      total += lds[k];
    }
    total = uniform(total);
    const uint64_t most = (total + A.least - 1) / A.least;
    shares = static_cast<uint32_t>(most < A.shares ? most : A.shares);
    if (index >= shares) return false;
    share = together(A, index, shares);
    from = total * share / shares;
    to = total * (share + 1u) / shares;
    if (from >= before_me && from < before_me + mine) {
      uint64_t p = before_me;
      for (uint32_t k = 0; k < each; ++k) {
        const uint64_t w = s0 + k < S ? places(A, s0 + k, &n, &b) : 0;
        if (from < p + w) {
          lds[4] = s0 + k;
          lds[5] = p;
          break;
        }
        p += w;
      }
    }
    __syncthreads();
    seq = static_cast<uint32_t>(uniform(lds[4]));
    at = uniform(lds[5]);
    places(A, seq, &tiles, &base);
    // the tile that has place `from`: by the root of its quadratic, then exactly
    const uint64_t r = from - at;
    const float q = static_cast<float>(per_tile(A)), h = static_cast<float>(base) + 0.5f * q;
    float guess = (__builtin_sqrtf(h * h + 2.0f * q * static_cast<float>(r)) - h) / q;
    guess = guess > 0.0f ? guess : 0.0f;
    tile = static_cast<uint32_t>(guess);
    if (tile >= tiles) tile = tiles - 1u;
    while (tile > 0u && before(A, tile, base) > r) --tile;
    while (tile + 1u < tiles && before(A, tile + 1u, base) <= r) ++tile;
    at += before(A, tile, base);
    return true;
  }
  __device__ __forceinline__ uint64_t width(const AttendArgs& A) const {
    return base + static_cast<uint64_t>(tile + 1u) * per_tile(A);
  }
  // which keys of the tile, whose places begin at `at`
  __device__ __forceinline__ void cut(const AttendArgs& A, uint32_t keys) {
    head = tail = true;
    begin = 0;
    end = keys;
    if constexpr (!SHARES) return;
    head = from <= at;
    tail = at + width(A) <= to;
    const uint64_t b = head ? 0 : (from - at) / CUT * CUT, e = tail ? keys : (to - at) / CUT * CUT;
    begin = static_cast<uint32_t>(b < keys ? b : keys);
    end = static_cast<uint32_t>(e < keys ? e : keys);
  }
  // shares that the tile's places meet, of which this is the first
  __device__ __forceinline__ uint32_t meets(const AttendArgs& A) const {
    return static_cast<uint32_t>(((at + width(A)) * shares - 1u) / total) - share + 1u;
  }
  // Across a tile's work the walk waits in LDS: it would take the scalar
  // registers that the loops over keys need.
  __device__ __forceinline__ void put(uint64_t* lds) const {
    if (threadIdx.x != 0) return;
    const uint64_t v[kWalkWords] = {from, to, at, total, base, pair(shares, share), pair(seq, tile), tiles};
#pragma unroll
    for (int k = 0; k < kWalkWords; ++k) lds[k] = v[k];
  }
  __device__ __forceinline__ void take(const uint64_t* lds) {
    uint64_t v[kWalkWords];
#pragma unroll
    for (int k = 0; k < kWalkWords; ++k) v[k] = uniform(lds[k]);
    from = v[0];
    to = v[1];
    at = v[2];
    total = v[3];
    base = v[4];
    shares = static_cast<uint32_t>(v[5]);
    share = static_cast<uint32_t>(v[5] >> 32);
    seq = static_cast<uint32_t>(v[6]);
    tile = static_cast<uint32_t>(v[6] >> 32);
    tiles = static_cast<uint32_t>(v[7]);
  }
  static __device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return static_cast<uint64_t>(b) << 32 | a; }

  // on to the next tile; false: the share has no more
  __device__ __forceinline__ bool next(const AttendArgs& A) {
    if constexpr (!SHARES) return false;
    at += width(A);
    ++tile;
    if (at >= to) return false;
    while (tile >= tiles) {
      tile = 0;
      if (++seq >= A.batch.sequences) return false;
      places(A, seq, &tiles, &base);
    }
    return true;
  }
};

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

// ---------------------------------------------------------------- rows that need care

// A weight of zero times a value that is not finite is NaN, so a token's row
// would take on what lies behind it in a product over a whole tile of keys.
// Rows that come out not finite where the tile holds keys that they do not
// see are computed again by this: one wave, one row, one key after another,
// and no others.
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
    if (s == -__builtin_inff()) continue;
    const float top = __builtin_fmaxf(m, s);
    const float shrink = exp2_of(m - top), p = exp2_of(s - top);
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
