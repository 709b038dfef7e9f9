// Attention of many rows for each of the cache's heads: chunks and prompts.
// Bound by the matrix instructions and the exponentials.
//
// 128 rows a workgroup, 32 a wave, as columns of S^T = K Q^T and O^T = V^T P^T
// (32x32x16 matrix instructions): a row's scores lie in two lanes, its maximum
// and its sum need one exchange, and the weights are the second product's
// operand as they are.  The waves share tiles of keys in LDS, two of them, so
// that the next one is written while this one is read and there is one barrier
// a tile.  A tile's rows are loaded a tile ahead into registers, at any
// alignment, and 8-bit codes become 16-bit values on the way.
#pragma once

#include "acp_dev_attn.hpp"

namespace acp {
namespace dev {

template <int FMT, int DP>
struct PromptShape {
  static constexpr int kKeys = DP <= 128 ? 64 : 32;   // of a tile: 64 KiB of LDS, two workgroups a CU
  static constexpr int kRow = DP * 2;
  static constexpr int kPieces = kRow / 16;
  static constexpr int kTile = kKeys * kRow;          // bytes of K or V
  static constexpr int kRegs = kTile / 16 / kAttendThreads;
  static constexpr int kStride = kAttendThreads / kPieces;  // rows between a lane's pieces
};

// Where piece c of row r lies.  K is read as 16 bytes of 32 rows: pieces are
// permuted by the row.  V's transposing reads take 64 bytes of four rows at a
// time: units of that size are.
template <int DP>
__device__ __forceinline__ uint32_t k_at(uint32_t row, uint32_t piece) {
  constexpr uint32_t kPieces = DP / 8, kRows = kPieces >= 16 ? 1u : 16u / kPieces;
  return row * (DP * 2u) + (piece ^ ((row / kRows) & (kPieces - 1u) & 15u)) * 16u;
}
template <int DP>
__device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t piece) {
  constexpr uint32_t kRows = DP >= 128 ? 1u : 128u / DP, kUnits = DP / 32;
  return row * (DP * 2u) + (piece ^ (((row / kRows) & 3u & (kUnits - 1u)) << 2)) * 16u;
}

template <class T, int FMT, int DP>
__global__ __launch_bounds__(kAttendThreads, DP == 256 ? 1 : 2) void attend_prompt_kernel(const AttendArgs A) {
  using S = PromptShape<FMT, DP>;
  constexpr int NB = S::kKeys / 32;  // blocks of 32 keys
  __shared__ __attribute__((aligned(16))) char lds[2][2][S::kTile];
  __shared__ __attribute__((aligned(16))) float scales[2][2][S::kKeys];
  const AttendPlace at(A);
  Tile t;
  if (!t.find<kPromptRows>(A, at.slot)) return;
  const uint32_t splits = t.splits(A);
  if (at.split >= splits) return;
  const uint32_t lane = threadIdx.x & 63u, wave = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const uint32_t col = lane & 31u, half = lane >> 5;
  const uint32_t keys = static_cast<uint32_t>(t.keys);

  const uint32_t row = t.first + wave * 32u + col;
  const bool real = row < static_cast<uint32_t>(t.rows);
  const int32_t sees = real ? t.position(A, row) : -1;
  uint32_t token, head;
  t.place(A, real ? row : t.first, at.kv, &token, &head);
  // positions of the wave's first and last rows
  const uint32_t row0 = t.first + wave * 32u;
  const bool any = row0 < static_cast<uint32_t>(t.rows);
  const int32_t low = any ? t.position(A, row0) : -1;
  const uint32_t row9 = row0 + 31u < static_cast<uint32_t>(t.rows) ? row0 + 31u : static_cast<uint32_t>(t.rows) - 1u;
  const int32_t high = any ? t.position(A, row9) : -1;

  rw4 q[DP / 16];
  {
    const char* qr = head_row(A, A.q, token, head);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const uint32_t c = 16u * s + 8u * half;
      q[s] = rw4{0u, 0u, 0u, 0u};
      if (real && c < A.dim) q[s] = *reinterpret_cast<const rw4_any*>(qr + c * 2);
    }
  }
  af16 o[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  int v_exp = -200;  // as in the form for few rows

  // The lane's pieces of a tile: piece `piece` of rows first, first + kStride, ...
  const uint32_t piece = threadIdx.x % S::kPieces, first = threadIdx.x / S::kPieces;
  const char* kbase = A.k.p + at.kv * A.k.s[2] + piece * (FMT == kCacheSame ? 16u : 8u);
  const char* vbase = A.v.p + at.kv * A.v.s[2] + piece * (FMT == kCacheSame ? 16u : 8u);
  const bool holds = piece * 8u < A.dim;
  rw4 kr[S::kRegs], vr[S::kRegs];
  // Each wave finds the pages of all the tile's keys: lane j has key j
  auto page_at = [&](uint32_t key0) -> int32_t {
    const uint32_t key = key0 + (lane & (S::kKeys - 1u));
    uint32_t index;
    return key < keys ? key_page(A, t.seq, key, &index) : -1;
  };
  float ks = 0.0f, vs = 0.0f;  // of the lane's key in the tile that is loading
  auto load = [&](uint32_t key0, int32_t page) {
    const uint64_t here = __builtin_amdgcn_ballot_w64(page >= 0);
    if constexpr (FMT != kCacheSame) {
      ks = vs = 0.0f;
      const uint32_t key = key0 + (lane & (S::kKeys - 1u));
      if (page >= 0) {
        const uint32_t index = key - divide(key, A.batch.page) * A.batch.page.d;
        const uint64_t s = (static_cast<uint64_t>(page) * A.batch.page.d + index) * A.kv_heads.d + at.kv;
        ks = A.k.scales[s];
        vs = A.v.scales[s];
      }
    }
#pragma unroll
    for (int i = 0; i < S::kRegs; ++i) {
      const uint32_t j = first + i * S::kStride;
      const uint32_t key = key0 + j;
      const int64_t g = __builtin_amdgcn_ds_bpermute(static_cast<int>(j * 4u), page);
      const uint32_t index = key - divide(key, A.batch.page) * A.batch.page.d;
      const char* kp = kbase + g * A.k.s[0] + index * A.k.s[1];
      const char* vp = vbase + g * A.v.s[0] + index * A.v.s[1];
      kr[i] = vr[i] = rw4{0u, 0u, 0u, 0u};
      if (holds && (here >> j & 1u)) {
        if constexpr (FMT == kCacheSame) {
          kr[i] = *reinterpret_cast<const rw4_any*>(kp);
          vr[i] = *reinterpret_cast<const rw4_any*>(vp);
        } else {
          const rw2 a = *reinterpret_cast<const rw2_any*>(kp), b = *reinterpret_cast<const rw2_any*>(vp);
          kr[i] = rw4{a[0], a[1], 0u, 0u};
          vr[i] = rw4{b[0], b[1], 0u, 0u};
        }
      }
    }
    return here;
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < S::kRegs; ++i) {
      const uint32_t j = first + i * S::kStride;
      if constexpr (FMT == kCacheSame) {
        *reinterpret_cast<rw4*>(lds[b][0] + k_at<DP>(j, piece)) = kr[i];
        *reinterpret_cast<rw4*>(lds[b][1] + v_at<DP>(j, piece)) = vr[i];
      } else {
        *reinterpret_cast<rw4*>(lds[b][0] + k_at<DP>(j, piece)) = codes_to<T, FMT>(kr[i][0], kr[i][1]);
        *reinterpret_cast<rw4*>(lds[b][1] + v_at<DP>(j, piece)) = codes_to<T, FMT>(vr[i][0], vr[i][1]);
      }
    }
    if constexpr (FMT != kCacheSame) {
      if (threadIdx.x < S::kKeys) {
        scales[b][0][threadIdx.x] = ks;
        scales[b][1][threadIdx.x] = vs;
      }
    }
  };

  const uint32_t per = A.chunk / S::kKeys;
  uint32_t now = at.split * A.chunk, n = 0;
  auto after = [&](uint32_t key, uint32_t* k) {
    key += S::kKeys;
    if (++*k == per) {
      *k = 0;
      key += (A.splits - 1u) * A.chunk;
    }
    return key;
  };
  uint64_t here = 0;
  uint32_t next = after(now, &n);
  int32_t next_page = -1;
  if (now < keys) {
    const int32_t page = page_at(now);
    next_page = page_at(next);
    here = load(now, page);
    put(0);
  }
  __syncthreads();
  int b = 0;
  while (now < keys) {
    uint32_t n2 = n;
    const uint32_t then = after(next, &n2);
    uint64_t next_here = 0;
    const bool more = next < keys;
    if (more) next_here = load(next, next_page);
    next_page = page_at(then);

    if (static_cast<int32_t>(now) <= high) {
      const char* kt = lds[b][0];
      const char* vt = lds[b][1];
      af16 s[NB];
#pragma unroll
      for (int h = 0; h < NB; ++h) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[h][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          const rw4 a = *reinterpret_cast<const rw4*>(kt + k_at<DP>(32u * h + col, 2u * i + half));
          s[h] = mfma32<T>(a, q[i], s[h]);
        }
      }
      // key of s[h][i]: 32 h + 8 (i / 4) + 4 half + i % 4
      float top = -__builtin_inff();
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][i + e] *= A.scale;
          if constexpr (FMT != kCacheSame) {
            const af4 w = *reinterpret_cast<const af4*>(&scales[b][0][32 * h + 2 * i + 4 * half]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][i + e] *= w[e];
          }
        }
      constexpr uint64_t kAll = S::kKeys == 64 ? ~uint64_t(0) : (uint64_t(1) << (S::kKeys & 63)) - 1;
      if ((here & kAll) != kAll || static_cast<int32_t>(now + S::kKeys - 1u) > low) {
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t j = 32u * h + 8u * (i / 4) + 4u * half + (i & 3);
            if (static_cast<int32_t>(now + j) > sees || !(here >> j & 1u)) s[h][i] = -__builtin_inff();
          }
      }
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[h][i]);
      top = max_step<5>(top);
      // taken up only when it grows by 2^8 or more, as in the form for few rows
      if (__builtin_amdgcn_ballot_w64(top > m + 8.0f)) {
        const float to = __builtin_fmaxf(m, top);
        const float shrink = exp2_of(m - (to == -__builtin_inff() ? 0.0f : to));
        m = to;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) o[d] *= shrink;
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;
      float unit = 1.0f;
      if constexpr (FMT != kCacheSame && std::is_same_v<T, _Float16>) {
        float big = scales[b][1][lane & (S::kKeys - 1)];
        const uint32_t most = static_cast<uint32_t>(
            over_lanes(static_cast<int>(as_bits(__builtin_fmaxf(big, 0.0f))), 6, [](int x, int y) { return x > y ? x : y; }));
        const int e = static_cast<int>(most >> 23) - 126;  // big < 2^e
        const int up = __builtin_amdgcn_readfirstlane(e > v_exp ? e : v_exp);
        if (up > v_exp) {
          const float down = v_exp - up < -126 ? 0.0f : as_float(static_cast<uint32_t>(127 + v_exp - up) << 23);
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) o[d] *= down;
          v_exp = up;
        }
        unit = __builtin_amdgcn_ldexpf(1.0f, -v_exp);
      }
      float sum = 0.0f;
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        rw4 weights[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = exp2_of(s[h][8 * k + i] - base);
            sum += p[i];
          }
          if constexpr (FMT != kCacheSame) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const af4 w = *reinterpret_cast<const af4*>(&scales[b][1][32 * h + 16 * k + 8 * e + 4 * half]);
#pragma unroll
              for (int i = 0; i < 4; ++i) p[4 * e + i] = p[4 * e + i] > 0.0f ? p[4 * e + i] * (w[i] * unit) : 0.0f;
            }
          }
          weights[k] = narrow(p, static_cast<const T*>(nullptr));
        }
        // group g of 16 lanes reads rows 4 (g / 2) .. and channels 16 (g % 2) ..
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) {
            rw4 a;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t r = 32u * h + 16u * k + 8u * e + 4u * half + (lane & 15u) / 4u;
              const uint32_t c = 4u * d + 2u * (lane >> 4 & 1u) + (lane & 3u) / 2u;
              const as4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ACP_LDS as4*)(vt + v_at<DP>(r, c) + (lane & 1u) * 8u));
              const rw2 u = __builtin_bit_cast(rw2, w);
              a[2 * e] = u[0];
              a[2 * e + 1] = u[1];
            }
            o[d] = mfma32<T>(a, weights[k], o[d]);
          }
      }
      l += sum;
    }
    if (more) put(b ^ 1);
    __syncthreads();
    b ^= 1;
    here = next_here;
    now = next;
    next = then;
    n = n2;
  }
  if constexpr (FMT != kCacheSame && std::is_same_v<T, _Float16>) {
    const float unit = __builtin_amdgcn_ldexpf(1.0f, v_exp);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) o[d] *= unit;
  }
  l = sum_step<5>(l);
  if (!any) return;

  // row col, channel 32 d + 8 (i / 4) + 4 half + i % 4 in o[d][i]
  uint64_t odd = 0;
  if (low + 1 < t.keys) {
    bool fine = is_finite(l);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) fine = fine && is_finite(o[d][i]);
    odd = __builtin_amdgcn_ballot_w64(!fine && real && sees + 1 < t.keys);
    odd = (odd | odd >> 32) & 0xFFFFFFFFu;
  }
  if (real && !(odd >> col & 1u)) {
    if (splits == 1u) {
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
      const uint64_t r0 = (static_cast<uint64_t>(at.split) * A.tokens + token) * A.heads.d + head;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const uint32_t c = 32u * d + 2u * i + 4u * half;
          if (c < A.dim)
            *reinterpret_cast<af4*>(A.part + r0 * A.dim + c) = af4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
        }
      if (half == 0) {
        A.stat[2 * r0] = m;
        A.stat[2 * r0 + 1] = l;
      }
    }
  }
  for (uint32_t k = 0; k < 32u; ++k)
    if (odd >> k & 1u) row_by_keys<T, FMT, DP>(A, t, row0 + k, at.kv, at.split, splits);
}

template <class T>
hipError_t attend_prompt_for(int cache, int padded, const AttendArgs& a, hipStream_t s) {
  const void* f = nullptr;
#define ACP_PROMPT(FMT, DP) \
  if (cache == FMT && padded == DP) f = reinterpret_cast<const void*>(attend_prompt_kernel<T, FMT, DP>)
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
  return hipLaunchKernel(f, dim3(a.kv_heads.d * a.slots.d * a.splits), dim3(kAttendThreads), args, 0, s);
}

}  // namespace dev
}  // namespace acp
