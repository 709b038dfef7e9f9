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
// A launch has a workgroup for each tile and head, or (`shares` > 0) deals the
// work out evenly: the keys of all tiles of a head, one after another, are cut
// into equal shares, whatever the lengths are, and a tile that a cut goes through
// leaves partial results, which a second kernel joins.
#pragma once

#include "acp_heads.hpp"

namespace acp {

struct AttendArgs {
  HeadTensor q, out;
  CacheTensor k, v;
  BatchArgs batch;
  Div n2;               // token dims, as HeadsCore has them
  Div group;            // query heads of a cache's head
  Div kv_heads;         // heads of the cache, in groups of 2^side_log2 of them
  int side_log2;        // heads of a workgroup: 0 for many rows
  Div slots;            // tile slots
  uint32_t tokens, dim;
  uint32_t shares;      // of a head's work, at most; 0: a workgroup a tile
  uint32_t least;       // keys of a share, at least
  uint32_t once;        // few rows: no two tiles read the same keys, but for some sequences
  uint32_t direct;      // many rows: the cache's rows are 16-byte aligned 16-bit values
  float scale;          // of a score, times log2 e: exponentials are powers of two; > 0
  uint32_t flip;        // the queries' sign bits, where it was below zero
  // partial results: a workgroup leaves up to two, of its first and its last tile.
  // [workgroup][2][2^side_log2 * M rows]
  float* part;          // [...][dim] sums of weighted values
  float* stat;          // [...][2] largest score and sum of weights
  uint32_t* joins;      // [slots][kv_heads][2] first share and number of shares of a tile
};

// dt: kRowF16 or kRowBF16; cache: kCacheSame, kCacheI8 or kCacheE4M3; dim padded to 64, 128 or 256
hipError_t attend_step_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_launch(int dt, int cache, int padded, const AttendArgs& a, hipStream_t s);
// How a workgroup of the join is laid out: lanes of a row, groups of them that
// share its splits, workgroups for the rows of a tile.
struct JoinShape {
  int lanes_log2, shares_log2;
  Div blocks;
};
hipError_t attend_join_launch(int dt, int tile_rows, const AttendArgs& a, const JoinShape& k, hipStream_t s);

hipError_t attend_step_f16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_step_bf16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_f16(int cache, int padded, const AttendArgs& a, hipStream_t s);
hipError_t attend_prompt_bf16(int cache, int padded, const AttendArgs& a, hipStream_t s);

constexpr int kAttendThreads = 256;
constexpr int kStepRows = 16;      // rows of a tile of few rows
// Waves of a tile of many rows, which has 32 rows a wave: eight for 128 channels,
// which halves what a tile's keys cost in loads (prompts of [2 x 8192 tokens, 32 /
// 8 heads, 128] 751 us, four waves 767); four for 64, of which a CU holds more than
// one workgroup (87 us against 96), and for 256, whose registers leave no room.
constexpr int prompt_waves(int padded) { return padded == 128 ? 8 : 4; }
constexpr int kStepKeys = 32;      // keys that a wave takes at a time
constexpr uint32_t kCutStep = 4 * kStepKeys, kCutPrompt = 64;  // cuts lie at multiples

}  // namespace acp
