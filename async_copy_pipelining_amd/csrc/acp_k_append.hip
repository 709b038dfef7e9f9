// Appending to a paged cache: new keys, turned, and new values go to the pages
// of their positions, as they are or in 8 bits with one scale a row; queries
// are turned in the same launch.
//
// Each row is read and written once.  A wave has one token: its sequence, its
// position and its page are found once for all heads.
#include "acp_dev_cache.hpp"
#include "acp_dev_heads.hpp"

namespace acp {
namespace dev {

constexpr int kPassesInFlight = 4;

// Where a pass's rows go: an output tensor, or a cache's page.
template <class T, bool PAIRS, bool WHOLE, bool PACK, bool TURN>
__device__ __forceinline__ void rows_through(const HeadsCore& A, const char* x, int64_t x_head, char* y, int64_t y_head,
                                             float* scales, int format, uint32_t heads, uint32_t slot,
                                             const Unit<T, PAIRS>& u, const Waves<kChunk<T>>& w, uint32_t from,
                                             uint32_t to) {
  constexpr int V = kChunk<T>, U = kPassesInFlight;
  for (uint32_t p = from; p < to; p += U) {
    Piece<T, PAIRS, WHOLE> piece[U];
    uint32_t head[U];
    bool there[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      head[k] = ((p + k) << A.heads_log2) + slot;
      there[k] = p + k < to && head[k] < heads;
      piece[k].load(x + head[k] * x_head, u, there[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (p + k >= to) break;
      if constexpr (!TURN && !PACK && WHOLE) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          store_chunk<T, false>(y + head[k] * y_head + u.at[j] * static_cast<int>(sizeof(T)), there[k] ? u.n[j] : 0,
                                piece[k].raw[j]);
        continue;
      }
      float a[V], b[V];
      piece[k].values(u, there[k], a, b);
      if constexpr (TURN) turn<PAIRS>(a, b, w, u.turned);
      if constexpr (!PACK) {
        piece[k].store(y + head[k] * y_head, u, there[k], a, b);
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t c = as_bits(a[i]) & 0x7FFFFFFFu, d = as_bits(b[i]) & 0x7FFFFFFFu;
          m = c > m ? c : m;
          m = d > m ? d : m;
        }
        m = static_cast<uint32_t>(
            over_lanes(static_cast<int>(m), A.lanes_log2, [](int c, int d) { return c > d ? c : d; }));
        const float s = block_scale(format, m);
        const Codes<V> ca = encode<T, V>(format, a, s), cb = encode<T, V>(format, b, s);
        char* row = y + head[k] * y_head;
        store_codes<V, !WHOLE>(row + u.at[0], there[k] ? u.n[0] : 0, ca);
        store_codes<V, !WHOLE>(row + u.at[1], there[k] ? u.n[1] : 0, cb);
        if (there[k] && u.at[0] == 0 && u.n[0] > 0) scales[head[k]] = s;
      }
    }
  }
}

template <class T, bool PAIRS, bool WHOLE, bool PACK>
__global__ __launch_bounds__(kHeadThreads) void append_kernel(const AppendArgs A) {
  const uint32_t wave = wave_index();
  if (wave >= A.groups * A.parts.d) return;
  const HeadPlace at(A, wave);  // a wave has one token: at.group
  const uint32_t token = at.group;
  const Unit<T, PAIRS> u(A, at.unit);
  const uint32_t seq = sequence_of(A.batch, token);
  if (seq >= A.batch.sequences) return;
  int32_t behind = 1;  // tokens of the sequence from this one on
  if (A.batch.starts != nullptr) {
    if (static_cast<int32_t>(token) < A.batch.starts[seq]) return;
    behind = A.batch.starts[seq + 1u] - static_cast<int32_t>(token);
  }
  const int32_t position = A.batch.lengths[seq] - behind;
  uint32_t from = at.pass, to = from + A.per_wave;
  Waves<kChunk<T>> w;
  if (A.rotated && from < A.q.passes + A.k.passes) w.template at<WHOLE>(A, u.first, u.turned, position);
  const uint32_t q_end = to < A.q.passes ? to : A.q.passes;
  if (from < q_end) {
    if (A.rotated)
      rows_through<T, PAIRS, WHOLE, false, true>(A, token_row(A, A.q.x, token), A.q.x.s[2], token_row(A, A.q.y, token),
                                                 A.q.y.s[2], nullptr, 0, A.q.heads, at.slot, u, w, from, q_end);
    else
      rows_through<T, PAIRS, WHOLE, false, false>(A, token_row(A, A.q.x, token), A.q.x.s[2], token_row(A, A.q.y, token),
                                                  A.q.y.s[2], nullptr, 0, A.q.heads, at.slot, u, w, from, q_end);
  }
  from = from > A.q.passes ? from - A.q.passes : 0u;
  to = to > A.q.passes ? to - A.q.passes : 0u;
  if (to == 0 || position < 0) return;
  const uint32_t index = divide(static_cast<uint32_t>(position), A.batch.page);
  const int32_t page = page_of(A.batch, seq, index);
  if (page < 0) return;
  const uint32_t slot = static_cast<uint32_t>(position) - index * A.batch.page.d;
  const uint64_t row = static_cast<uint64_t>(page) * A.batch.page.d + slot;
  const uint32_t k_end = to < A.k.passes ? to : A.k.passes;
  if (from < k_end) {
    char* y = A.ck.p + page * A.ck.s[0] + slot * A.ck.s[1];
    float* scales = PACK ? A.ck.scales + row * A.k.heads : nullptr;
    if (A.rotated)
      rows_through<T, PAIRS, WHOLE, PACK, true>(A, token_row(A, A.k.x, token), A.k.x.s[2], y, A.ck.s[2], scales,
                                                A.format, A.k.heads, at.slot, u, w, from, k_end);
    else
      rows_through<T, PAIRS, WHOLE, PACK, false>(A, token_row(A, A.k.x, token), A.k.x.s[2], y, A.ck.s[2], scales,
                                                 A.format, A.k.heads, at.slot, u, w, from, k_end);
  }
  from = from > A.k.passes ? from - A.k.passes : 0u;
  to = to > A.k.passes ? to - A.k.passes : 0u;
  const uint32_t v_end = to < A.v.passes ? to : A.v.passes;
  if (from < v_end)
    rows_through<T, PAIRS, WHOLE, PACK, false>(A, token_row(A, A.v.x, token), A.v.x.s[2],
                                               A.cv.p + page * A.cv.s[0] + slot * A.cv.s[1], A.cv.s[2],
                                               PACK ? A.cv.scales + row * A.v.heads : nullptr, A.format, A.v.heads,
                                               at.slot, u, w, from, v_end);
}

}  // namespace dev

namespace {

template <class T, bool PACK>
const void* append_kernel_for(const HeadsShape& k) {
  using namespace dev;
  return k.pairs ? (k.whole ? reinterpret_cast<const void*>(append_kernel<T, true, true, PACK>)
                            : reinterpret_cast<const void*>(append_kernel<T, true, false, PACK>))
                 : (k.whole ? reinterpret_cast<const void*>(append_kernel<T, false, true, PACK>)
                            : reinterpret_cast<const void*>(append_kernel<T, false, false, PACK>));
}

template <class T>
const void* append_kernel_for(const HeadsShape& k, bool pack) {
  return pack ? append_kernel_for<T, true>(k) : append_kernel_for<T, false>(k);
}

}  // namespace

hipError_t append_launch(const HeadsShape& k, int cache, const AppendArgs& a, hipStream_t s) {
  const bool pack = cache != kCacheSame;
  const void* f = k.dt == kRowF16    ? append_kernel_for<_Float16>(k, pack)
                  : k.dt == kRowBF16 ? append_kernel_for<dev::bf16_t>(k, pack)
                                     : append_kernel_for<float>(k, pack);
  constexpr uint32_t kWaves = kHeadThreads / 64;
  AppendArgs copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(f, dim3((a.groups * a.parts.d + kWaves - 1) / kWaves), dim3(kHeadThreads), args, 0, s);
}

}  // namespace acp
