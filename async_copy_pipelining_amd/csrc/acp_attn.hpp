// Attention of new tokens over a paged cache: argument block and launchers
// shared by the host entry points and the kernels.
//
// The query heads that share a cache's head are rows of one product: row r of
// a sequence with n new tokens (r < n * group) is head r % group of its token
// r / group.  Tiles of M rows never join two sequences.  Tile slots are
// numbered so that a workgroup finds its sequence without a sum over the batch:
// the tiles of sequence s begin at floor(starts[s] * group / M) + s, which leaves
// room for ceil(n * group / M) of them before the next sequence's.
//
// Keys are cut into chunks of `chunk`; workgroup `split` of a tile takes the
// chunks split, split + splits, ...  A tile whose keys fill one chunk writes its
// output, others leave partial results, which a second kernel joins.
#pragma once

#include "acp_heads.hpp"

namespace acp {

struct AttendArgs {
  HeadTensor q, out;
  CacheTensor k, v;
  BatchArgs batch;
  Div n2;               // token dims, as HeadsCore has them
  Div group;            // query heads of a cache's head
  Div kv_heads;
  Div slots;            // tile slots
  Div heads;            // query heads
  uint32_t tokens, dim;
  uint32_t chunk, splits;
  float scale;          // of a score, times log2 e: exponentials are powers of two
  float* part;          // [splits][token][head][dim] sums of weighted values
  float* stat;          // [splits][token][head][2] largest score and sum of weights
};

// dt: kRowF16 or kRowBF16; cache: kCacheSame, kCacheI8 or kCacheE4M3; dim padded to 64, 128 or 256
hipError_t attend_step_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_join_launch(int dt, int tile_rows, const AttendArgs& a, hipStream_t s);

hipError_t attend_step_f16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_step_bf16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_f16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_bf16(int cache, int padded, const AttendArgs& a, hipStream_t s);

constexpr int kAttendThreads = 256;
constexpr int kStepRows = 16;      // rows of a tile of few rows
constexpr int kPromptRows = 128;   // rows of a tile of many
constexpr int kStepKeys = 32;      // keys that a wave takes at a time
constexpr uint32_t kChunkUnit = 128;  // chunks are whole multiples: the keys of a step's four waves, tiles of a prompt

}  // namespace acp
