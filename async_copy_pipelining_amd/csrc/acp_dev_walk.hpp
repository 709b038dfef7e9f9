// How the tiles of attention are numbered and dealt out: a sequence's tokens, a
// tile's rows and keys, a workgroup's walk over its share.  Nothing here touches
// a tensor, and it compiles for the host too, where a test runs it.  Included
// after divide() is declared.
#pragma once

#include "acp_attn.hpp"

namespace acp {
namespace dev {

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
    __syncthreads();  // put() writes there
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

}  // namespace dev
}  // namespace acp
