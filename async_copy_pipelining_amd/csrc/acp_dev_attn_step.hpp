// Attention of few rows for each of the cache's heads: single tokens, short
// chunks.  Bound by reading the cache.
//
// The rows that share keys, padded to 16, are columns of the products
// S^T = K Q^T and O^T = V^T P^T (16x16x32 matrix instructions), so that a row's
// scores lie in one lane's registers and three others', and the weights of S^T
// are the second product's operand as they are: its sum over keys takes them in
// the order in which the first leaves them.
//
// Each of the four waves takes every fourth step of 32 keys with sums of its
// own; they meet once, at the end.  A lane loads its part of K straight into
// the first product's operand.  V goes through LDS, where the transposing reads
// turn rows of channels into columns of keys; only the wave itself reads what
// it wrote, so there is no barrier in the loop.  The next step's rows load
// while this one is computed: 16 KiB a wave for 128 channels of 16 bits, and
// eight waves a CU keep twice the bytes in flight that its share of HBM needs.
//
// [32 tokens over up to 32768 positions, 32 / 8 heads, 128] bfloat16: 401 us,
// 6.5 TB/s; 64 over up to 8192 in 8 bits 135 us, 5.0 TB/s, where codes and scales
// are most of the work.  Two steps ahead, or three workgroups a CU, are no faster.
// Weights in two 16-bit parts, which leave 2^-16 of each (float16 2^-22) where one
// part leaves 2^-8 (2^-11), take next to no time: 401 us, with one part 401; in 8
// bits 135, 134; 3 tokens over up to 700 positions 9.3, 9.0.
#pragma once

#include "acp_dev_attn.hpp"

namespace acp {
namespace dev {

template <class T, int FMT, int DP>
struct StepShape {
  static constexpr int kBytes = FMT == kCacheSame ? 2 : 1;      // of a channel
  static constexpr int kRow = DP * kBytes;                      // of a row in LDS
  static constexpr int kPieces = kRow / 16;                     // 16-byte pieces of a row
  static constexpr int kSteps = DP / 32;                        // of the first product
  static constexpr int kKRegs = DP * kBytes / 64;               // pieces of K a lane has of one of its two keys
  static constexpr int kVRows = 64 / kPieces;                   // rows that one load of the wave covers
  static constexpr int kVRegs = kStepKeys / kVRows;
  static constexpr int kWaveBytes = kStepKeys * kRow;
  // the waves' sums meet there afterwards, 128 channels at a time
  static constexpr int kJoinPitch = 132;
  static constexpr int kJoinBytes = 4 * kStepRows * kJoinPitch * 4;
  // 8-bit rows: the scales of a wave's keys, behind all waves' rows
  static constexpr int kScaleBytes = FMT == kCacheSame ? 0 : 2 * kStepKeys * 4;
  static constexpr int kLds = 4 * (kWaveBytes + kScaleBytes) > kJoinBytes ? 4 * (kWaveBytes + kScaleBytes) : kJoinBytes;
};

// Where piece c of row r lies in a wave's rows of V.  A transposing read takes
// 32 bytes (16 channels) of eight rows, or 16 bytes of sixteen (8-bit codes), in
// one of its turns: units of that size are permuted by the row, so that these
// fill the 64 banks.
template <class S, int FMT>
__device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t piece) {
  constexpr uint32_t kRows = S::kRow >= 256 ? 1u : 256u / S::kRow;  // rows side by side in the banks
  uint32_t p;
  if constexpr (FMT == kCacheSame) {
    constexpr uint32_t kUnits = S::kPieces / 2;
    p = ((piece >> 1) ^ ((row / kRows) & 7u & (kUnits - 1u))) << 1 | (piece & 1u);
  } else {
    p = piece ^ ((row / kRows) & (S::kPieces - 1u));
  }
  return row * S::kRow + p * 16u;
}

// Channels 128 h + jc .. + 8 of row jr of each of the workgroup's heads, from the
// sums of the waves that shared the head's keys; rows that are odd are left out.
template <class T, class S, int WIDE>
__device__ __forceinline__ void join_out(const AttendArgs& A, const Tile& t, const Partial& to, uint32_t kv0, int h,
                                         const float* stage, const float (*stat)[kStepRows][2], const uint32_t* odd,
                                         uint32_t jr, uint32_t jc, bool real) {
  const uint32_t c = 128u * h + jc, side = 1u << A.side_log2, turns = 4u >> A.side_log2;
  if (!real || jc >= WIDE || c >= A.dim) return;
  for (uint32_t g = 0; g < side; ++g) {
    if (odd[g] >> jr & 1u) continue;
    float best = -__builtin_inff(), total = 0.0f, sum[8];
    for (uint32_t k = 0; k < turns; ++k) best = __builtin_fmaxf(best, stat[k * side + g][jr][0]);
    const float base = best == -__builtin_inff() ? 0.0f : best;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    for (uint32_t k = 0; k < turns; ++k) {
      const uint32_t w = k * side + g;
      const float f = exp2_of(stat[w][jr][0] - base);
      total = __builtin_fmaf(f, stat[w][jr][1], total);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(f, stage[(w * kStepRows + jr) * S::kJoinPitch + jc + i], sum[i]);
    }
    if (!to.wanted) {
      uint32_t token, head;
      t.place(A, t.first + jr, kv0 + g, &token, &head);
      char* y = head_row(A, A.out, token, head);
      const float inv = 1.0f / total;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = total == 0.0f ? 0.0f : sum[i] * inv;
      *reinterpret_cast<rw4_any*>(y + c * 2) = narrow(sum, static_cast<const T*>(nullptr));
    } else {
      const uint32_t index = g * kStepRows + jr;
      float* y = to.part(A, index) + c;
      *reinterpret_cast<af4*>(y) = af4{sum[0], sum[1], sum[2], sum[3]};
      *reinterpret_cast<af4*>(y + 4) = af4{sum[4], sum[5], sum[6], sum[7]};
      if (c == 0) {
        float* z = to.stat(A, index);
        z[0] = best;
        z[1] = total;
      }
    }
  }
}

// The waves' sums: row col, channel 16 d + 4 quarter + i in o[d][i].  A lane
// joins eight channels of a row, head after head.
template <class T, int FMT, int DP>
__device__ __forceinline__ void step_rows(const AttendArgs& A, const Tile& t, const Partial& to, uint32_t begin,
                                          uint32_t keys, uint32_t kv0, const af4 (&o)[DP / 16], float m, float l, char* lds,
                                          float (*join_stat)[kStepRows][2], uint32_t* odd_rows) {
  using S = StepShape<T, FMT, DP>;
  const uint32_t thread = thread_again();
  const uint32_t lane = thread & 63u, wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(thread >> 6));
  const uint32_t col = lane & 15u, quarter = lane >> 4, side = 1u << A.side_log2;
  if (quarter == 0) {
    join_stat[wave][col][0] = m;
    join_stat[wave][col][1] = l;
  }
  if (thread < 4) odd_rows[thread] = 0;
  const uint32_t jr = thread / 16u, jc = thread % 16u * 8u;
  constexpr int kParts = (DP + 127) / 128, kWide = DP < 128 ? DP : 128;
  float* stage = reinterpret_cast<float*>(lds);
  const uint32_t my_row = t.first + jr;
  const bool row_real = my_row < static_cast<uint32_t>(t.rows);
  const bool mixed = t.low + 1 < t.keys;  // rows that see less than others
  // Of the rows that are not finite those that do not see a value that is not.
  // The workgroup takes part.
  auto look_again = [&] {
    __syncthreads();
    uint32_t any = 0;
    for (uint32_t g = 0; g < side; ++g) any |= odd_rows[g];
    if (any == 0u) return;
    __syncthreads();
    if (wave < side) {
      const int32_t last = last_odd_value<T, FMT>(A, t, begin, keys, kv0 + wave);
      const uint64_t m = __builtin_amdgcn_ballot_w64(lane < kStepRows && t.position(A, t.first + lane) < last);
      if (lane == 0) odd_rows[wave] &= static_cast<uint32_t>(m);
    }
    __syncthreads();
  };
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kWide / 16; ++d)
      *reinterpret_cast<af4*>(stage + (wave * kStepRows + col) * S::kJoinPitch + 16 * d + 4 * quarter) = o[8 * h + d];
    __syncthreads();
    if (mixed) {
      // a row is odd by its sum or any of its channels, which other lanes have
      if (row_real && t.position(A, my_row) + 1 < t.keys) {
        for (uint32_t w = 0; w < 4u; ++w) {
          bool fine = is_finite(join_stat[w][jr][1]);
          if (jc < kWide) {
#pragma unroll
            for (int i = 0; i < 8; ++i) fine = fine && is_finite(stage[(w * kStepRows + jr) * S::kJoinPitch + jc + i]);
          }
          if (!fine) atomicOr(&odd_rows[w & (side - 1u)], 1u << jr);
        }
      }
    }
    if (kParts > 1 && mixed) continue;  // written below, once all channels were looked at
    if (mixed) look_again();
    join_out<T, S, kWide>(A, t, to, kv0, h, stage, join_stat, odd_rows, jr, jc, row_real);
  }
  if (kParts > 1 && mixed) {
    look_again();
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      __syncthreads();
#pragma unroll
      for (int d = 0; d < kWide / 16; ++d)
        *reinterpret_cast<af4*>(stage + (wave * kStepRows + col) * S::kJoinPitch + 16 * d + 4 * quarter) = o[8 * h + d];
      __syncthreads();
      join_out<T, S, kWide>(A, t, to, kv0, h, stage, join_stat, odd_rows, jr, jc, row_real);
    }
  }
  if (mixed) {
    for (uint32_t g = 0; g < side; ++g)
      for (uint32_t k = wave; k < kStepRows; k += 4u)
        if (odd_rows[g] >> k & 1u) {
          const uint32_t index = g * kStepRows + k;
          row_by_keys<T, FMT, DP>(A, t, t.first + k, kv0 + g, begin, keys, to.part(A, index), to.stat(A, index));
        }
  }
}

// A tile's keys [begin, keys) for the workgroup's heads.
template <class T, int FMT, int DP>
__device__ __forceinline__ void step_tile(const AttendArgs& A, const Tile& t, const Partial& to, uint32_t begin,
                                          uint32_t keys, uint32_t kv0, char* lds, float (*join_stat)[kStepRows][2],
                                          uint32_t* odd_rows) {
  using S = StepShape<T, FMT, DP>;
  const uint32_t thread = thread_again();
  const uint32_t lane = thread & 63u, wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(thread >> 6));
  const uint32_t col = lane & 15u, quarter = lane >> 4;
  // Waves side by side have `side` heads of the same keys, and 4 / side of them
  // take a head's steps in turn.
  const uint32_t side = 1u << A.side_log2, turn = wave >> A.side_log2, stride = (4u >> A.side_log2) * kStepKeys;
  const uint32_t kv = kv0 + (wave & (side - 1u));
  const bool exact = A.dim == DP;
  char* mine = lds + wave * S::kWaveBytes;
  float* my_scales = reinterpret_cast<float*>(lds + 4 * S::kWaveBytes + wave * S::kScaleBytes);

  // the lane's row, and its part of Q: channel order as K's pieces have it
  const uint32_t row = t.first + col;
  const bool real = row < static_cast<uint32_t>(t.rows);
  const int32_t sees = real ? t.position(A, row) : -1;
  rw4 q[S::kSteps];
  {
    uint32_t token, head;
    t.place(A, real ? row : t.first, kv, &token, &head);
    const char* qr = head_row(A, A.q, token, head);
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      const uint32_t c = FMT == kCacheSame ? 32u * s + 8u * quarter : 64u * (s / 2) + 16u * quarter + 8u * (s & 1);
      q[s] = rw4{0u, 0u, 0u, 0u};
      if (real && c < A.dim) q[s] = *reinterpret_cast<const rw4_any*>(qr + c * 2) ^ A.flip;
    }
  }

  af4 o[DP / 16];
#pragma unroll
  for (int d = 0; d < DP / 16; ++d) o[d] = af4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -__builtin_inff(), l = 0.0f;
  using W = Weights<T, FMT>;
  constexpr bool kUnits = FMT != kCacheSame && std::is_same_v<T, _Float16>;
  WeightUnit row_unit;  // kUnits

  // Lanes 0..31 (and again 32..63) have a key each: its page, or -1
  auto entry_at = [&](uint32_t key0) { return page_entry(A, t.seq, key0 + (lane & 31u), keys); };
  struct Rows {  // of the lane's key
    int64_t k, v;
    uint32_t here;  // keys that have a page, by bits: uniform
    float ks, vs;
  };
  auto rows_at = [&](uint32_t key0, int32_t entry) {
    Rows r;
    const uint32_t key = key0 + (lane & 31u);
    const int32_t page = entry_page(A, entry, key, keys);
    const uint32_t index = key - divide(key, A.batch.page) * A.batch.page.d;
    const int64_t g = page < 0 ? 0 : page;
    r.k = g * A.k.s[0] + index * A.k.s[1];
    r.v = g * A.v.s[0] + index * A.v.s[1];
    r.here = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(page >= 0));
    r.ks = r.vs = 0.0f;
    if constexpr (FMT != kCacheSame) {
      if (page >= 0) {
        const uint64_t s = (static_cast<uint64_t>(page) * A.batch.page.d + index) * (A.kv_heads.d << A.side_log2) + kv;
        r.ks = A.k.scales[s];
        r.vs = A.v.scales[s];
      }
    }
    return r;
  };
  const char* kbase = A.k.p + kv * A.k.s[2];
  const char* vbase = A.v.p + kv * A.v.s[2];
  rw4 kr[2][S::kKRegs], vr[S::kVRegs];
  // where a piece of 16 bytes at byte c of a row holds channels: all of it, or (codes) its first 8
  const uint32_t row_bytes = A.dim * S::kBytes;
  auto piece_of = [&](const char* p, uint32_t c, bool there) {
    rw4 w{0u, 0u, 0u, 0u};
    if (there && c + 16u <= row_bytes) {
      w = *reinterpret_cast<const rw4_any*>(p);
    } else if (FMT != kCacheSame && there && c < row_bytes) {
      const rw2 u = *reinterpret_cast<const rw2_any*>(p);
      w = rw4{u[0], u[1], 0u, 0u};
    }
    return w;
  };
  auto load_k = [&](const Rows& r) {
    const char* p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) p[h] = kbase + from_lane(r.k, 16u * h + col) + 16u * quarter;
    if (exact && r.here == 0xFFFFFFFFu && A.once) {
      asm volatile("");  // keeps the branches apart: joined, the loads would lose their policy
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::kKRegs; ++i)
          kr[h][i] = __builtin_nontemporal_load(reinterpret_cast<const rw4_any*>(p[h] + 64 * i));
      asm volatile("");
    } else if (exact && r.here == 0xFFFFFFFFu) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::kKRegs; ++i) kr[h][i] = *reinterpret_cast<const rw4_any*>(p[h] + 64 * i);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < S::kKRegs; ++i)
          kr[h][i] = piece_of(p[h] + 64 * i, 64u * i + 16u * quarter, r.here >> (16u * h + col) & 1u);
    }
  };
  auto load_v = [&](const Rows& r) {
    const uint32_t piece = lane % S::kPieces, first = lane / S::kPieces;
    const char* p[S::kVRegs];
#pragma unroll
    for (int i = 0; i < S::kVRegs; ++i) p[i] = vbase + from_lane(r.v, first + i * S::kVRows) + piece * 16u;
    if (exact && r.here == 0xFFFFFFFFu && A.once) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < S::kVRegs; ++i) vr[i] = __builtin_nontemporal_load(reinterpret_cast<const rw4_any*>(p[i]));
      asm volatile("");
    } else if (exact && r.here == 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < S::kVRegs; ++i) vr[i] = *reinterpret_cast<const rw4_any*>(p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < S::kVRegs; ++i)
        vr[i] = piece_of(p[i], piece * 16u, r.here >> (first + i * S::kVRows) & 1u);
    }
  };

  // The wave's steps: this one and the next, whose rows load meanwhile; the page
  // numbers of the one after are on their way too.
  uint32_t now = begin + turn * kStepKeys, next = now + stride;
  int32_t entry = -1;
  Rows r{};
  if (now < keys) {
    const int32_t first = entry_at(now);
    entry = entry_at(next);
    r = rows_at(now, first);
    load_k(r);
    load_v(r);
  }
  while (now < keys) {
    const Rows rn = rows_at(next, entry);
    entry = entry_at(next + stride);
    const bool more = next < keys;

    if constexpr (FMT != kCacheSame) my_scales[lane] = lane < 32u ? r.ks : kUnits ? r.vs * WeightUnit::kScale : r.vs;
    af4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = af4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) {
        if constexpr (FMT == kCacheSame) s[h] = mfma16<T>(kr[h][i], q[i], s[h]);
        else
          s[h] = mfma16<T>(codes_to<T, FMT>(kr[h][i / 2][2 * (i & 1)], kr[h][i / 2][2 * (i & 1) + 1]), q[i], s[h]);
      }
    }
    if (more) load_k(rn);

    // scores in powers of two, and what is hidden
    float x[8], ws[8];
    if constexpr (FMT != kCacheSame) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (FMT == kCacheSame) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * h + i] = s[h][i] * A.scale;
      } else {
        const af4 k = *reinterpret_cast<const af4*>(my_scales + 16u * h + 4u * quarter);
        const af4 v = *reinterpret_cast<const af4*>(my_scales + 32u + 16u * h + 4u * quarter);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[4 * h + i] = s[h][i] * A.scale * k[i];
          ws[4 * h + i] = v[i];
        }
      }
    }
    if (r.here != 0xFFFFFFFFu || static_cast<int32_t>(now + kStepKeys - 1u) > t.low) {
      // both in the lane's own terms, so that the bit and the bound are constants
      const int32_t left = sees - static_cast<int32_t>(now + 4u * quarter);
      const uint32_t mine = r.here >> (4u * quarter);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = 16 * (k / 4) + (k & 3);
        if (j > left || !(mine & (1u << j))) x[k] = -__builtin_inff();
      }
    }
    float top = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) top = __builtin_fmaxf(top, x[k]);
    top = max_step<5>(max_step<4>(top));
    if (__builtin_amdgcn_ballot_w64(top > m + W::kRise)) {
      const float to = __builtin_fmaxf(m, top);
      const float shrink = exp2_of(m - (to == -__builtin_inff() ? 0.0f : to));
      m = to;
      l *= shrink;
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) o[d] *= shrink;
      if constexpr (kUnits) row_unit.shrink(shrink);
    }
    const float base = m == -__builtin_inff() ? 0.0f : m - W::kRoom;
    float p[8], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      p[k] = exp2_of(x[k] - base);
      sum += p[k];
    }
    l += sum;
    if constexpr (FMT != kCacheSame) {
      // the values' scales go into the weights
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = p[k] > 0.0f ? p[k] * ws[k] : 0.0f;
      if constexpr (kUnits) {
        float big = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) big = __builtin_fmaxf(big, __builtin_fabsf(p[k]));
        if (row_unit.take(max_step<5>(max_step<4>(big)))) {
          const int by = row_unit.change();
#pragma unroll
          for (int d = 0; d < DP / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][i] = __builtin_amdgcn_ldexpf(o[d][i], by);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] *= row_unit.unit;
      }
    }
    // each weight in two parts: the matrix instructions have time to spare
    rw4 weights, rest;
    two_parts<T, FMT>(p, &weights, &rest);

    // V: rows of channels to columns of keys
    {
      const uint32_t piece = lane % S::kPieces, first = lane / S::kPieces;
#pragma unroll
      for (int i = 0; i < S::kVRegs; ++i)
        *reinterpret_cast<rw4*>(mine + v_at<S, FMT>(first + i * S::kVRows, piece)) = vr[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (more) load_v(rn);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
      rw4 a;
      if constexpr (FMT == kCacheSame) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k = 16u * h + 4u * quarter + col / 4u;
          const uint32_t piece = 2u * d + (col & 3u) / 2u;
          const as4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (ACP_LDS as4*)(mine + v_at<S, FMT>(k, piece) + (col & 1u) * 8u));
          const rw2 u = __builtin_bit_cast(rw2, w);
          a[2 * h] = u[0];
          a[2 * h + 1] = u[1];
        }
      } else {
        const uint32_t j = col / 2u;
        const uint32_t k = 16u * (j / 4u) + 4u * quarter + (j & 3u);
        const ai2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((ACP_LDS ai2*)(mine + v_at<S, FMT>(k, d) + (col & 1u) * 8u));
        a = codes_to<T, FMT>(static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[1]));
      }
      o[d] = mfma16<T>(a, rest, mfma16<T>(a, weights, o[d]));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    now = next;
    next += stride;
    r = rn;
  }
  if constexpr (kUnits) {
    const int by = row_unit.back();
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[d][i] = __builtin_amdgcn_ldexpf(o[d][i], by);
  }
  l = sum_step<5>(sum_step<4>(l));
  m -= W::kRoom;

  step_rows<T, FMT, DP>(attend_args(), t, to, begin, keys, kv0, o, m, l, lds, join_stat, odd_rows);
}

template <class T, int FMT, int DP, bool SHARES>
__global__ __launch_bounds__(kAttendThreads, DP == 256 ? 1 : 2) void attend_step_kernel(const AttendArgs A) {
  __shared__ __attribute__((aligned(16))) char lds[StepShape<T, FMT, DP>::kLds];
  __shared__ float join_stat[4][kStepRows][2];
  __shared__ uint32_t odd_rows[4];
  const AttendPlace at(A);
  Walk<kStepRows, kCutStep, SHARES> walk;
  if constexpr (!SHARES) {
    Tile t;
    if (!t.find<kStepRows>(A, at.index)) return;
    walk.cut(A, static_cast<uint32_t>(t.keys));
    const Partial to(A, walk, t, at.kv);
    step_tile<T, FMT, DP>(A, t, to, walk.begin, walk.end, at.kv << A.side_log2, lds, join_stat, odd_rows);
  } else {
    __shared__ uint64_t walk_space[kWalkWords];
    if (!walk.begin_at(A, at.index, walk_space)) return;
    bool more;
    do {
      Tile t;
      if (t.set<kStepRows>(A, walk.seq, walk.tile)) {
        walk.cut(A, static_cast<uint32_t>(t.keys));
        const Partial to(A, walk, t, at.kv);
        walk.put(walk_space);
        step_tile<T, FMT, DP>(attend_args(), t, to, walk.begin, walk.end, at.kv << A.side_log2, lds, join_stat, odd_rows);
      }
      __syncthreads();  // the next tile's keys and sums go where this one's were
      walk.take(walk_space);
      more = walk.next(A);
      __syncthreads();
    } while (more);
  }
}

template <class T>
hipError_t attend_step_for(int cache, int padded, const AttendArgs& a, hipStream_t s) {
  const void* f = nullptr;
#define ACP_STEP(FMT, DP)                                                                       \
  if (cache == FMT && padded == DP)                                                            \
    f = a.shares ? reinterpret_cast<const void*>(attend_step_kernel<T, FMT, DP, true>)          \
                 : reinterpret_cast<const void*>(attend_step_kernel<T, FMT, DP, false>)
  ACP_STEP(kCacheSame, 64);
  ACP_STEP(kCacheSame, 128);
  ACP_STEP(kCacheSame, 256);
  ACP_STEP(kCacheI8, 64);
  ACP_STEP(kCacheI8, 128);
  ACP_STEP(kCacheI8, 256);
  ACP_STEP(kCacheE4M3, 64);
  ACP_STEP(kCacheE4M3, 128);
  ACP_STEP(kCacheE4M3, 256);
#undef ACP_STEP
  if (f == nullptr) return hipErrorInvalidValue;
  AttendArgs copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(f, dim3(attend_grid(a)), dim3(kAttendThreads), args, 0, s);
}

}  // namespace dev
}  // namespace acp
