// Appending to a paged cache: new keys, turned, and new values go to the pages
// of their positions, as they are or in 8 bits with one scale a row; queries
// are turned in the same launch.
//
// Each row is read and written once.  A wave has one token: its sequence, its
// position and its page are found once for all heads.  20480 new tokens of 32 + 8
// + 8 heads of 128 bfloat16, half the channels turned: 104 us, 4.8 TB/s.  A step of
// 64 tokens: 5.7 us, the chain of look-ups.
#include "acp_dev_cache.hpp"
#include "acp_dev_heads.hpp"

namespace acp {
namespace dev {

// Passes in flight: of the queries, which mostly have several times the heads,
// and of keys and of values.
constexpr int kPassesQ = 4, kPassesKV = 2;

// Passes [from, to) of a tensor, of which the first U are loaded.  y: an output's
// row of the token, or a page's.
template <class T, bool PAIRS, bool WHOLE, bool PACK, bool TURN, int U>
__device__ __forceinline__ void rows_through(const HeadsCore& A, Passes<T, PAIRS, WHOLE, U>& in, const char* x,
                                             int64_t x_head, char* y, int64_t y_head, float* scales, int format,
                                             uint32_t heads, uint32_t slot, const Unit<T, PAIRS>& u,
                                             const Waves<kChunk<T>>& w, uint32_t from, uint32_t to) {
  constexpr int V = kChunk<T>;
  for (uint32_t p = from; p < to; p += U) {
    if (p != from) in.load(A, x, x_head, u, heads, slot, p, to);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (p + k >= to) break;
      const uint32_t head = in.head(A, p + k, slot);
      const bool there = head < heads;
      Piece<T, PAIRS, WHOLE>& piece = in.piece[k];
      if constexpr (!TURN && !PACK && WHOLE) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          store_whole<T, false>(y + head * y_head + u.at[j] * static_cast<int>(sizeof(T)), there ? u.n[j] : 0, piece.raw[j],
                                A.keep);
        continue;
      }
      float a[V], b[V];
      piece.values(u, there, a, b);
      if constexpr (TURN) turn<PAIRS>(a, b, w, u.turned);
      if constexpr (!PACK) {
        piece.store(A.keep, y + head * y_head, u, there, a, b);
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
        char* row = y + head * y_head;
        store_whole_codes<V, !WHOLE>(row + u.at[0], there ? u.n[0] : 0, ca);
        store_whole_codes<V, !WHOLE>(row + u.at[1], there ? u.n[1] : 0, cb);
        if (there && u.at[0] == 0 && u.n[0] > 0) scales[head] = s;
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
  // the wave's passes of q, k and v, which follow one another
  const uint32_t first = at.pass, last = first + A.per_wave, k0 = A.q.passes, v0 = k0 + A.k.passes;
  auto within = [](uint32_t p, uint32_t from, uint32_t n) { return p < from ? 0u : p - from < n ? p - from : n; };
  const uint32_t q_from = within(first, 0, A.q.passes), q_to = within(last, 0, A.q.passes);
  const uint32_t k_from = within(first, k0, A.k.passes), k_to = within(last, k0, A.k.passes);
  const uint32_t v_from = within(first, v0, A.v.passes), v_to = within(last, v0, A.v.passes);
  const char *xq = token_row(A, A.q.x, token), *xk = token_row(A, A.k.x, token), *xv = token_row(A, A.v.x, token);
  Passes<T, PAIRS, WHOLE, kPassesQ> q;
  Passes<T, PAIRS, WHOLE, kPassesKV> k, v;
  q.load(A, xq, A.q.x.s[2], u, A.q.heads, at.slot, q_from, q_to);
  k.load(A, xk, A.k.x.s[2], u, A.k.heads, at.slot, k_from, k_to);
  v.load(A, xv, A.v.x.s[2], u, A.v.heads, at.slot, v_from, v_to);
  const uint32_t seq = sequence_of(A.batch, token);
  if (seq >= A.batch.sequences) return;
  int32_t behind = 1;  // tokens of the sequence from this one on
  if (A.batch.starts != nullptr) {
    if (static_cast<int32_t>(token) < A.batch.starts[seq]) return;
    behind = A.batch.starts[seq + 1u] - static_cast<int32_t>(token);
  }
  const int32_t length = A.batch.lengths[seq];
  const int32_t position = (length > 0 ? length : 0) - behind;
  int32_t page = -1;
  uint32_t slot = 0;
  if (position >= 0) {
    const uint32_t index = divide(static_cast<uint32_t>(position), A.batch.page);
    slot = static_cast<uint32_t>(position) - index * A.batch.page.d;
    page = page_of(A.batch, seq, index);
  }
  Waves<kChunk<T>> w;
  if (A.rotated && first < v0) w.template at<WHOLE>(A, u, position);
  if (q_from < q_to) {
    char* y = token_row(A, A.q.y, token);
    if (A.rotated)
      rows_through<T, PAIRS, WHOLE, false, true>(A, q, xq, A.q.x.s[2], y, A.q.y.s[2], nullptr, 0, A.q.heads, at.slot, u, w,
                                                 q_from, q_to);
    else
      rows_through<T, PAIRS, WHOLE, false, false>(A, q, xq, A.q.x.s[2], y, A.q.y.s[2], nullptr, 0, A.q.heads, at.slot, u,
                                                  w, q_from, q_to);
  }
  if (page < 0) return;
  const uint64_t row = static_cast<uint64_t>(page) * A.batch.page.d + slot;
  if (k_from < k_to) {
    char* y = A.ck.p + page * A.ck.s[0] + slot * A.ck.s[1];
    float* scales = PACK ? A.ck.scales + row * A.k.heads : nullptr;
    if (A.rotated)
      rows_through<T, PAIRS, WHOLE, PACK, true>(A, k, xk, A.k.x.s[2], y, A.ck.s[2], scales, A.format, A.k.heads, at.slot,
                                                u, w, k_from, k_to);
    else
      rows_through<T, PAIRS, WHOLE, PACK, false>(A, k, xk, A.k.x.s[2], y, A.ck.s[2], scales, A.format, A.k.heads, at.slot,
                                                 u, w, k_from, k_to);
  }
  if (v_from < v_to)
    rows_through<T, PAIRS, WHOLE, PACK, false>(A, v, xv, A.v.x.s[2], A.cv.p + page * A.cv.s[0] + slot * A.cv.s[1],
                                               A.cv.s[2], PACK ? A.cv.scales + row * A.v.heads : nullptr, A.format,
                                               A.v.heads, at.slot, u, w, v_from, v_to);
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
