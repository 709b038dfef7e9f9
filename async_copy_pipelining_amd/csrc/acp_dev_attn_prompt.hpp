// Attention of many rows for each of the cache's heads: chunks and prompts.
// Bound by the matrix instructions and the exponentials.
//
// 32 rows a wave, 128 or 256 a workgroup, as columns of S^T = K Q^T and
// O^T = V^T P^T (32x32x16 matrix instructions): a row's scores lie in two lanes,
// its maximum and its sum need one exchange, and the weights are the second
// product's operand as they are.  The waves share tiles of 64 keys in LDS, two of
// them, so that the next one comes while this one is read and there is one
// barrier a tile.  16-bit rows go there straight from memory; 8-bit codes become
// 16-bit values in registers on the way, as do rows of odd alignment.
//
// [2 x 8192 tokens, 32 / 8 heads, 128] bfloat16: 746 to 767 us, 975 to 1003 TFLOP/s
// of the tokens' own scores and values (single launches under a trace 757 to 816),
// where a product of 8192^3 by the library reaches 1227.  With 32 rows a wave the LDS has as many cycles of reads as there
// are of matrix instructions, and the exponentials have half as many again; two
// waves a SIMD overlap them as they come.  Not better: one of the two half a tile
// late, so that scores meet values (788 us, a barrier more a tile); pieces sent
// for between the matrix instructions (840); more operands read ahead than four
// (equal); rows' places worked out by scalar instructions (880, where 811 then).
#pragma once

#include "acp_dev_attn.hpp"

namespace acp {
namespace dev {

template <int FMT, int DP, bool DIRECT, int W>
struct PromptShape {
  static constexpr uint32_t kWaves = W;
  static constexpr int kKeys = 64;                    // of a tile, in two blocks of 32
  static constexpr int kRow = DP * 2;
  static constexpr int kPieces = kRow / 16;
  static constexpr int kTile = kKeys * kRow;          // bytes of K or V
  using Piece = std::conditional_t<FMT == kCacheSame, rw4, rw2>;  // 8 channels
  static constexpr int kRegs = kTile / 16 / (64 * W);  // pieces of K or V that a lane brings
  // Operands of K, and groups of 16 keys of V, that are read ahead: as many as
  // registers last for.  More take nothing off the time.
  static constexpr uint32_t kKAhead = 4, kVAhead = DP == 256 && !DIRECT ? 0 : 1;
};

// f(integral_constant i) for i = I .. N - 1
template <uint32_t N, uint32_t I = 0, class F>
__device__ __forceinline__ void unroll(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<uint32_t, I>{});
    unroll<N, I + 1>(f);
  }
}

// Where piece c of row r lies.  K is read as 16 bytes of 32 rows: pieces are
// permuted by the row.  V's transposing reads take 64 bytes of four rows at a
// time: units of that size are.
template <int DP>
__device__ __forceinline__ constexpr uint32_t k_at(uint32_t row, uint32_t piece) {
  constexpr uint32_t kPieces = DP / 8, kRows = kPieces >= 16 ? 1u : 16u / kPieces;
  return row * (DP * 2u) + (piece ^ ((row / kRows) & (kPieces - 1u) & 15u)) * 16u;
}
template <int DP>
__device__ __forceinline__ constexpr uint32_t v_at(uint32_t row, uint32_t piece) {
  constexpr uint32_t kRows = DP >= 128 ? 1u : 128u / DP, kUnits = DP / 32;
  return row * (DP * 2u) + (piece ^ (((row / kRows) & 3u & (kUnits - 1u)) << 2)) * 16u;
}

// The wave's rows: row col, channel 32 d + 8 (i / 4) + 4 half + i % 4 in o[d][i].
template <class T, int FMT, int DP>
__device__ __forceinline__ void prompt_rows(const AttendArgs& A, const Tile& t, const Partial& to, uint32_t begin,
                                            uint32_t keys, uint32_t kv, const af16 (&o)[DP / 32], float m, float l) {
  const uint32_t thread = thread_again();
  const uint32_t lane = thread & 63u, wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(thread >> 6));
  const uint32_t col = lane & 31u, half = lane >> 5;
  const uint32_t row0 = t.first + wave * 32u, row = row0 + col;
  const bool real = row < static_cast<uint32_t>(t.rows);
  uint32_t token, head;
  t.place(A, real ? row : t.first, kv, &token, &head);
  uint64_t odd = 0;
  if (t.low + 1 < t.keys) {
    bool fine = is_finite(l);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) fine = fine && is_finite(o[d][i]);
    odd = __builtin_amdgcn_ballot_w64(!fine && real && t.position(A, row) + 1 < t.keys);
    if (odd != 0u) {
      const int32_t last = last_odd_value<T, FMT>(A, t, begin, keys, kv);
      odd &= __builtin_amdgcn_ballot_w64(t.position(A, row) < last);
    }
    odd = (odd | odd >> 32) & 0xFFFFFFFFu;
  }
  if (real && !(odd >> col & 1u)) {
    if (!to.wanted) {
      char* y = head_row(A, A.out, token, head);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = l == 0.0f ? 0.0f : o[d][i + e] * inv;
          const rw4 w = narrow(f, static_cast<const T*>(nullptr));
          const uint32_t c = 32u * d + 2u * i + 4u * half;
          if (c < A.dim) *reinterpret_cast<rw2_any*>(y + c * 2) = rw2{w[0], w[1]};
          if (c + 8u < A.dim) *reinterpret_cast<rw2_any*>(y + (c + 8u) * 2) = rw2{w[2], w[3]};
        }
    } else {
      float* y = to.part(A, wave * 32u + col);
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const uint32_t c = 32u * d + 2u * i + 4u * half;
          if (c < A.dim) *reinterpret_cast<af4*>(y + c) = af4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        }
      if (half == 0) {
        float* z = to.stat(A, wave * 32u + col);
        z[0] = m;
        z[1] = l;
      }
    }
  }
  for (uint32_t k = 0; k < 32u; ++k)
    if (odd >> k & 1u)
      row_by_keys<T, FMT, DP>(A, t, row0 + k, kv, begin, keys, to.part(A, wave * 32u + k), to.stat(A, wave * 32u + k));
}

// A tile's keys [begin, keys) for one of the cache's heads.
//
// DIRECT: 16-bit rows at 16-byte aligned addresses go straight to LDS, in
// instructions of 64 pieces of 16 bytes that lie one after another there, the
// pieces' places permuted on the global side.  They take no registers, so that a
// whole tile is on its way while another is computed.  Pieces past the channels
// are never written: they were cleared once.  Else (8-bit codes, other
// alignments) pieces wait in registers.
template <class T, int FMT, int DP, bool DIRECT, int W>
__device__ __forceinline__ void prompt_tile(const AttendArgs& A, const Tile& t, const Partial& to, uint32_t begin,
                                            uint32_t keys, uint32_t kv, char (*lds)[2][PromptShape<FMT, DP, DIRECT, W>::kTile],
                                            float (*scales)[2][PromptShape<FMT, DP, DIRECT, W>::kKeys]) {
  using S = PromptShape<FMT, DP, DIRECT, W>;
  constexpr uint32_t kBlock = 32u * DP * 2u;  // bytes of a block of 32 keys in LDS
  const uint32_t thread = thread_again();
  const uint32_t lane = thread & 63u, wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(thread >> 6));
  const uint32_t col = lane & 31u, half = lane >> 5;

  const uint32_t row = t.first + wave * 32u + col;
  const bool real = row < static_cast<uint32_t>(t.rows);
  const int32_t sees = real ? t.position(A, row) : -1;
  // positions of the wave's first and last rows
  const uint32_t row0 = t.first + wave * 32u;
  const bool any = row0 < static_cast<uint32_t>(t.rows);
  const int32_t low = any ? t.position(A, row0) : -1;
  const uint32_t row9 = row0 + 31u < static_cast<uint32_t>(t.rows) ? row0 + 31u : static_cast<uint32_t>(t.rows) - 1u;
  const int32_t high = any ? t.position(A, row9) : -1;

  rw4 q[DP / 16];
  {
    uint32_t token, head;
    t.place(A, real ? row : t.first, kv, &token, &head);
    const char* qr = head_row(A, A.q, token, head);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const uint32_t c = 16u * s + 8u * half;
      q[s] = rw4{0u, 0u, 0u, 0u};
      if (real && c < A.dim) q[s] = *reinterpret_cast<const rw4_any*>(qr + c * 2) ^ A.flip;
    }
  }
  af16 o[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  constexpr bool kUnits = FMT != kCacheSame && std::is_same_v<T, _Float16>;
  WeightUnit row_unit;  // kUnits

  // Each wave finds the rows of all the tile's keys: lane j has key j.
  auto entry_at = [&](uint32_t key0) { return page_entry(A, t.seq, key0 + lane, keys); };
  auto page_at = [&](uint32_t key0, int32_t entry) { return entry_page(A, entry, key0 + lane, keys); };
  // An instruction of a wave has 64 pieces: rows of kRowsEach keys, instruction i
  // of wave w those from (4 i + w) kRowsEach on.  Piece `slot` of a row in LDS is
  // piece kp (vp) of the row in memory: V's is the same for all i.
  constexpr uint32_t kRowsEach = 64u / S::kPieces, kEach = S::kRegs;
  static_assert(kEach * S::kWaves * kRowsEach == S::kKeys);
  const uint32_t slot = lane % S::kPieces, line = lane / S::kPieces, row_in = wave * kRowsEach + line;
  static_assert(v_at<DP>(S::kWaves * kRowsEach, 0) == S::kWaves * kRowsEach * S::kRow);
  const uint32_t kp0 = (k_at<DP>(row_in, slot) - row_in * S::kRow) / 16u;
  const uint32_t vp = (v_at<DP>(row_in, slot) - row_in * S::kRow) / 16u;
  auto kp = [&](uint32_t i) { return kp0 ^ (k_at<DP>(i * S::kWaves * kRowsEach, 0) - i * S::kWaves * kRowsEach * S::kRow) / 16u; };
  // Where the rows of the tile after this one lie.  The lanes of a row's pieces
  // need kEach rows each, the same ones: the lanes of a quad work out one row each
  // (two, where there are eight) and pass it on.
  constexpr uint32_t kOwn = kEach < 4u ? kEach : 4u, kSets = kEach / kOwn;
  const char* k_head = A.k.p + kv * A.k.s[2];
  const char* v_head = A.v.p + kv * A.v.s[2];
  const char *k_row[kSets], *v_row[kSets];
  auto rows_at = [&](uint32_t key0, int32_t page) {
#pragma unroll
    for (uint32_t n = 0; n < kSets; ++n) {
      const uint32_t j = (n * 4u + (lane & (kOwn - 1u))) * S::kWaves * kRowsEach + row_in, key = key0 + j;
      const uint32_t index = key - divide(key, A.batch.page) * A.batch.page.d;
      const int p = __builtin_amdgcn_ds_bpermute(static_cast<int>(j * 4u), page);
      const uint32_t g = p < 0 ? 0u : static_cast<uint32_t>(p);
      k_row[n] = k_head + (g * A.k.s[0] + index * A.k.s[1]);
      v_row[n] = v_head + (g * A.v.s[0] + index * A.v.s[1]);
    }
  };
  auto row_of = [&](const char* const (&own)[kSets], auto I) {
    constexpr int i = decltype(I)::value;
    const uint64_t p = reinterpret_cast<uint64_t>(own[i / 4]);
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(p), i % 4 * 0x55, 0xF, 0xF, true));
    const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(p >> 32), i % 4 * 0x55, 0xF, 0xF, true));
    return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
  };
  auto bring = [&](uint32_t b, uint64_t here) {
    const uint32_t kt = lds_offset(lds[b][0]) + wave * 1024u, vt = lds_offset(lds[b][1]) + wave * 1024u;
    if (here == ~uint64_t(0) && A.dim == DP) {
      unroll<kEach>([&](auto I) {
        constexpr uint32_t i = decltype(I)::value;
        to_lds(row_of(k_row, I) + kp(i) * 16u, kt + i * S::kWaves * 1024u);
        to_lds(row_of(v_row, I) + vp * 16u, vt + i * S::kWaves * 1024u);
      });
    } else {
      unroll<kEach>([&](auto I) {
        constexpr uint32_t i = decltype(I)::value;
        const char* kr = row_of(k_row, I) + kp(i) * 16u;
        const char* vr = row_of(v_row, I) + vp * 16u;
        if (!(here >> (i * S::kWaves * kRowsEach) >> row_in & 1u)) {
          *reinterpret_cast<rw4*>(lds[b][0] + (i * S::kWaves + wave) * 1024u + lane * 16u) = rw4{0u, 0u, 0u, 0u};
          *reinterpret_cast<rw4*>(lds[b][1] + (i * S::kWaves + wave) * 1024u + lane * 16u) = rw4{0u, 0u, 0u, 0u};
        } else {
          if (kp(i) * 8u < A.dim) to_lds(kr, kt + i * S::kWaves * 1024u);
          if (vp * 8u < A.dim) to_lds(vr, vt + i * S::kWaves * 1024u);
        }
      });
    }
  };
  // not DIRECT: the lane's pieces of a tile
  typename S::Piece kw[S::kRegs], vw[S::kRegs];
  auto load = [&](uint64_t here) {
    using P = typename S::Piece;
    typedef P P_any __attribute__((aligned(1)));
    unroll<kEach>([&](auto I) {
      constexpr uint32_t i = decltype(I)::value;
      const char* kr = row_of(k_row, I) + slot * sizeof(P);
      const char* vr = row_of(v_row, I) + slot * sizeof(P);
      kw[i] = vw[i] = P{};
      if (slot * 8u < A.dim && (here >> (i * S::kWaves * kRowsEach) >> row_in & 1u)) {
        kw[i] = *reinterpret_cast<const P_any*>(kr);
        vw[i] = *reinterpret_cast<const P_any*>(vr);
      }
    });
  };
  auto value = [](const typename S::Piece& w) {
    if constexpr (FMT == kCacheSame) return w;
    else return codes_to<T, FMT>(w[0], w[1]);
  };
  auto put = [&](uint32_t b) {
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      const uint32_t j = i * S::kWaves * kRowsEach + row_in;
      *reinterpret_cast<rw4*>(lds[b][0] + k_at<DP>(j, slot)) = value(kw[i]);
      *reinterpret_cast<rw4*>(lds[b][1] + v_at<DP>(j, slot)) = value(vw[i]);
    }
  };
  // 8-bit rows: the scales of the tile's keys
  float ks = 0.0f, vs = 0.0f;
  auto load_scales = [&](uint32_t key0, int32_t page) {
    if constexpr (FMT != kCacheSame) {
      ks = vs = 0.0f;
      const uint32_t key = key0 + lane;
      if (page >= 0) {
        const uint32_t index = key - divide(key, A.batch.page) * A.batch.page.d;
        const uint64_t s = (static_cast<uint64_t>(page) * A.batch.page.d + index) * A.kv_heads.d + kv;
        ks = A.k.scales[s];
        vs = A.v.scales[s];
      }
    }
  };
  auto put_scales = [&](uint32_t b) {
    if constexpr (FMT != kCacheSame) {
      if (thread < S::kKeys) {
        scales[b][0][thread] = ks;
        scales[b][1][thread] = kUnits ? vs * WeightUnit::kScale : vs;
      }
    }
  };

  // Reads: K's piece 2 i + half of row 32 h + col; V's channels 32 d .. of rows
  // 32 h + 16 k + 8 e + 4 half .., group g of 16 lanes channels 16 (g % 2) of them
  const uint32_t ka = k_at<DP>(col, half);
  const uint32_t va = v_at<DP>(4u * half + (lane & 15u) / 4u, 2u * (lane >> 4 & 1u) + (lane & 3u) / 2u) + (lane & 1u) * 8u;

  // Three tiles at once: one is computed, the next one's rows load, the pages of
  // the one after are known (`page`), and of the fourth they load (`entry`).
  uint32_t now = begin, b = 0;
  int32_t page = -1, entry = -1;
  uint64_t here = 0, next_here = 0;
  if constexpr (DIRECT) {
    if (A.dim != DP) {  // channels that no row has
#pragma unroll 1
      for (uint32_t i = thread * 16u; i < 4u * S::kTile; i += S::kWaves * 1024u)
        *reinterpret_cast<rw4*>(lds[0][0] + i) = rw4{0u, 0u, 0u, 0u};
      __syncthreads();
    }
  }
  if (now < keys) {
    const int32_t first = entry_at(now), second = entry_at(now + S::kKeys);
    entry = entry_at(now + 2u * S::kKeys);
    page = page_at(now, first);
    here = __builtin_amdgcn_ballot_w64(page >= 0);
    rows_at(now, page);
    if constexpr (DIRECT) {
      page = page_at(now + S::kKeys, second);
      bring(0, here);
    } else {
      load(here);
      load_scales(now, page);
      page = page_at(now + S::kKeys, second);
      put(0);
      put_scales(0);
    }
    next_here = __builtin_amdgcn_ballot_w64(page >= 0);
    rows_at(now + S::kKeys, page);
  }
  while (now < keys) {
    const uint32_t next = now + S::kKeys;
    const bool more = next < keys;
    // this tile has arrived, and all waves are done with the other one
    if constexpr (DIRECT) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if constexpr (!DIRECT) {
      if (more) load_scales(next, page);
    }
    page = page_at(next + S::kKeys, entry);
    entry = entry_at(next + 2u * S::kKeys);
    if (more) {
      if constexpr (DIRECT) bring(b ^ 1u, next_here);
      else load(next_here);
    }
    if (static_cast<int32_t>(now) <= high) {
      const char* kt = lds[b][0];
      const char* vt = lds[b][1];
      af16 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[h][i] = 0.0f;
      // 16 keys' values, the first ones read while the scores are computed
      auto values_of = [&](uint32_t n, rw4 (&a)[DP / 32]) {
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const as4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (ACP_LDS as4*)(vt + (va ^ (64u * d)) + (16u * n + 8u * e) * S::kRow));
            const rw2 x = __builtin_bit_cast(rw2, u);
            a[d][2 * e] = x[0];
            a[d][2 * e + 1] = x[1];
          }
      };
      rw4 a[DP / 32];
      {
        constexpr uint32_t kSteps = DP / 8, kAhead = S::kKAhead;
        rw4 w[kSteps];
        auto read = [&](uint32_t n) {
          return *reinterpret_cast<const rw4*>(kt + n % 2u * kBlock + (ka ^ (32u * (n / 2u))));
        };
#pragma unroll
        for (uint32_t n = 0; n < kAhead; ++n) w[n] = read(n);
        unroll<kSteps>([&](auto N) {
          constexpr uint32_t n = decltype(N)::value;
          if constexpr (n + kAhead < kSteps) w[n + kAhead] = read(n + kAhead);
          s[n % 2u] = mfma32<T>(w[n], q[n / 2u], s[n % 2u]);
          if constexpr (S::kVAhead && n == kSteps / 2u) values_of(0, a);
        });
        asm volatile("" ::: "memory");
      }
      // key of s[h][i]: 32 h + 8 (i / 4) + 4 half + i % 4
      if constexpr (FMT != kCacheSame) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const af4 x = *reinterpret_cast<const af4*>(&scales[b][0][32 * h + 2 * i + 4 * half]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][i + e] *= x[e];
          }
      }
      if (here != ~uint64_t(0) || static_cast<int32_t>(now + S::kKeys - 1u) > low) {
        // both in the lane's own terms, so that the bit and the bound are constants
        const int32_t left = sees - static_cast<int32_t>(now + 4u * half);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t mine = static_cast<uint32_t>(here >> (32 * h)) >> (4u * half);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 8 * (i / 4) + (i & 3);
            if (32 * h + j > left || !(mine & (1u << j))) s[h][i] = -__builtin_inff();
          }
        }
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[h][i]);
      top = max_step<5>(top) * A.scale;
      if (__builtin_amdgcn_ballot_w64(top > m + Weights<T, FMT>::kRise)) {
        const float up = __builtin_fmaxf(m, top);
        const float shrink = exp2_of(m - (up == -__builtin_inff() ? 0.0f : up));
        m = up;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) o[d] *= shrink;
        if constexpr (kUnits) row_unit.shrink(shrink);
      }
      const float base = m == -__builtin_inff() ? 0.0f : m - Weights<T, FMT>::kRoom;
      // float16 over 8-bit values: all of the tile's products, and the unit that holds them
      if constexpr (kUnits) {
        float big = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const af4 x = *reinterpret_cast<const af4*>(&scales[b][1][32 * h + 2 * i + 4 * half]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = exp2_of(__builtin_fmaf(s[h][i + e], A.scale, -base));
              l += p;
              s[h][i + e] = p > 0.0f ? p * x[e] : 0.0f;
              big = __builtin_fmaxf(big, __builtin_fabsf(s[h][i + e]));
            }
          }
        if (row_unit.take(max_step<5>(big))) {
          const int by = row_unit.change();
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = __builtin_amdgcn_ldexpf(o[d][i], by);
        }
      }
      unroll<4>([&](auto N) {
        constexpr uint32_t n = decltype(N)::value;
        if constexpr (!S::kVAhead) values_of(n, a);
        float p[8];
        if constexpr (kUnits) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = s[n / 2u][8 * (n & 1u) + i] * row_unit.unit;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = exp2_of(__builtin_fmaf(s[n / 2u][8 * (n & 1u) + i], A.scale, -base));
        }
        if constexpr (FMT != kCacheSame && !kUnits) {
#pragma unroll
          for (int i = 0; i < 8; ++i) l += p[i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const af4 x = *reinterpret_cast<const af4*>(&scales[b][1][16u * n + 8 * e + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * e + i] = p[4 * e + i] > 0.0f ? p[4 * e + i] * x[i] : 0.0f;
          }
        }
        // Rounded to the type: half a step of each weight, as the output's own
        // rounding.  In two parts, as the form for few rows has them, the values'
        // products would double (prompts of [2 x 8192 tokens, 32 / 8 heads, 128]
        // 1035 us, so 759).
        const rw4 weights = narrow(p, static_cast<const T*>(nullptr));
        if constexpr (FMT == kCacheSame) {
          // the sum of the weights as they were rounded
#pragma unroll
          for (int i = 0; i < 4; ++i) l = add_pair<T>(weights[i], l);
        }
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) o[d] = mfma32<T>(a[d], weights, o[d]);
        if constexpr (S::kVAhead && n < 3u) values_of(n + 1u, a);
      });
    }
    const uint64_t after_here = __builtin_amdgcn_ballot_w64(page >= 0);
    rows_at(next + S::kKeys, page);
    if constexpr (!DIRECT) {
      if (more) {
        put(b ^ 1u);
        put_scales(b ^ 1u);
      }
    }
    now = next;
    here = next_here;
    next_here = after_here;
    b ^= 1u;
  }
  if constexpr (kUnits) {
    const int by = row_unit.back();
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = __builtin_amdgcn_ldexpf(o[d][i], by);
  }
  l = sum_step<5>(l);
  m -= Weights<T, FMT>::kRoom;
  if (!any) return;
  prompt_rows<T, FMT, DP>(attend_args(), t, to, begin, keys, kv, o, m, l);
}

template <class T, int FMT, int DP, bool SHARES, bool DIRECT, int W>
__global__ __launch_bounds__(64 * W, DP == 256 ? 1 : 2) void attend_prompt_kernel(const AttendArgs A) {
  using S = PromptShape<FMT, DP, DIRECT, W>;
  __shared__ __attribute__((aligned(16))) char lds[2][2][S::kTile];
  __shared__ __attribute__((aligned(16))) float scales[2][2][S::kKeys];
  const AttendPlace at(A);
  Walk<32 * W, kCutPrompt, SHARES> walk;
  if constexpr (!SHARES) {
    Tile t;
    if (!t.find<32 * W>(A, at.index)) return;
    walk.cut(A, static_cast<uint32_t>(t.keys));
    const Partial to(A, walk, t, at.kv);
    prompt_tile<T, FMT, DP, DIRECT, W>(A, t, to, walk.begin, walk.end, at.kv, lds, scales);
  } else {
    __shared__ uint64_t walk_space[kWalkWords];
    if (!walk.begin_at(A, at.index, walk_space)) return;
    bool more;
    do {
      Tile t;
      if (t.set<32 * W>(A, walk.seq, walk.tile)) {
        walk.cut(A, static_cast<uint32_t>(t.keys));
        const Partial to(A, walk, t, at.kv);
        walk.put(walk_space);
        prompt_tile<T, FMT, DP, DIRECT, W>(attend_args(), t, to, walk.begin, walk.end, at.kv, lds, scales);
      }
      __syncthreads();  // the next tile's keys and sums go where this one's were
      walk.take(walk_space);
      more = walk.next(A);
      __syncthreads();
    } while (more);
  }
}

template <class T, int FMT, int DP, bool DIRECT>
const void* attend_prompt_of(bool shares) {
  constexpr int W = prompt_waves(DP);
  return shares ? reinterpret_cast<const void*>(attend_prompt_kernel<T, FMT, DP, true, DIRECT, W>)
                : reinterpret_cast<const void*>(attend_prompt_kernel<T, FMT, DP, false, DIRECT, W>);
}
template <class T>
hipError_t attend_prompt_for(int cache, int padded, const AttendArgs& a, hipStream_t s) {
  const void* f = nullptr;
#define ACP_PROMPT(FMT, DP)                                                        \
  if (cache == FMT && padded == DP)                                                \
  f = FMT == kCacheSame && a.direct ? attend_prompt_of<T, kCacheSame, DP, true>(a.shares) \
                                    : attend_prompt_of<T, FMT, DP, false>(a.shares)
  ACP_PROMPT(kCacheSame, 64);
  ACP_PROMPT(kCacheSame, 128);
  ACP_PROMPT(kCacheSame, 256);
  ACP_PROMPT(kCacheI8, 64);
  ACP_PROMPT(kCacheI8, 128);
  ACP_PROMPT(kCacheI8, 256);
  ACP_PROMPT(kCacheE4M3, 64);
  ACP_PROMPT(kCacheE4M3, 128);
  ACP_PROMPT(kCacheE4M3, 256);
#undef ACP_PROMPT
  if (f == nullptr) return hipErrorInvalidValue;
  AttendArgs copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(f, dim3(attend_grid(a)), dim3(64 * prompt_waves(padded)), args, 0, s);
}

}  // namespace dev
}  // namespace acp
