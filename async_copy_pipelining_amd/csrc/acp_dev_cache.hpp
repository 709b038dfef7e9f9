// Device side of paged caches: the sequence of a token, the page of a position.
#pragma once

#include "acp_heads.hpp"

namespace acp {
namespace dev {

// The sequence that holds `token` (uniform in the wave): how many of
// starts[1 ..] do not lie past it, counted 64 at a time.  sequences: none.
__device__ __forceinline__ uint32_t sequence_of(const BatchArgs& B, uint32_t token) {
  if (B.starts == nullptr) return token < B.sequences ? token : B.sequences;
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t n = 0;
  for (uint32_t i = 0; i < B.sequences; i += 64u) {
    const bool before = i + lane < B.sequences && B.starts[i + lane + 1u] <= static_cast<int32_t>(token);
    const uint32_t c = static_cast<uint32_t>(__builtin_popcountll(__builtin_amdgcn_ballot_w64(before)));
    n += c;
    if (c < 64u) break;
  }
  return n;
}

// Page of position p of a sequence; -1: the position has none.
__device__ __forceinline__ int32_t page_of(const BatchArgs& B, uint32_t sequence, uint32_t index) {
  if (index >= B.max_pages) return -1;
  const int32_t g = B.pages[static_cast<uint64_t>(sequence) * B.max_pages + index];
  return static_cast<uint32_t>(g) < B.page_count ? g : -1;
}

}  // namespace dev
}  // namespace acp
