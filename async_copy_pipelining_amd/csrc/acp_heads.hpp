// Head operators of acp: rotary positions, norms of queries and keys for each
// head, and appending keys and values to a paged cache.  Argument blocks and
// launchers shared by the host entry points and the kernels.
//
// A tensor is seen as tokens of `heads` rows of `dim` contiguous channels.  A
// row is cut into units of two chunks of 16 bytes, chosen so that both
// channels of every turned pair lie in one unit; a lane has the same unit of
// every row that it handles, and 2^lanes_log2 neighbouring lanes have a row.
#pragma once

#include "acp_rows.hpp"

namespace acp {

// A float tensor: token t starts at p + t / n2 * s[0] + t % n2 * s[1] bytes,
// its head h s[2] bytes further for each head.
struct HeadTensor {
  char* p;
  int64_t s[3];
};

struct HeadsCore {
  const double* frequencies;  // rotated / 2, radians a position; nullptr: nothing is turned
  const int32_t* positions;   // nullptr: token % span (rotation without a cache)
  uint32_t tokens;
  Div n2, span;
  uint32_t dim, rotated;
  uint32_t turn_units, units;  // units of turned channels, and of the row
  int lanes_log2;
  int heads_log2;              // heads that a wave handles side by side
  uint32_t per_wave;           // passes over the heads of a wave's tokens that the wave makes
  Div parts;                   // waves that share the passes of one group of tokens
  uint32_t keep;               // stores stay in the L2s for a while, as store_whole says
  uint32_t groups;             // groups of tokens: the wave's lanes hold 2^(6 - lanes_log2 - heads_log2)
  float turn_scale, sign;      // of cos and sin; -1: turned back
  float eps;
};

// One side of a call: the rows of queries or of keys.
struct HeadSide {
  HeadTensor x, y;
  const float* weight;  // nullptr: 1
  uint32_t heads;
  uint32_t passes;      // 0: not there
};
struct HeadsForward : HeadsCore {
  HeadSide side[2];
};

struct HeadGradSide {
  HeadTensor x, dy, dx;
  const float* weight;
  float* part;          // its columns of the partial weight gradients; nullptr: not wanted
  uint32_t heads;
  uint32_t passes;
};
struct HeadsBackward : HeadsCore {
  HeadGradSide side[2];
  uint32_t part_pitch;  // floats between two workgroups' parts
};

// The weight gradients of both sides from the workgroups' parts.
struct HeadColumns {
  const float* part;
  float* out[2];        // nullptr: not wanted
  uint32_t dim, rows, pitch;
};

// A batch of sequences and their pages.  Sequence s has tokens
// starts[s] .. starts[s + 1] (starts nullptr: token s), the last of its
// lengths[s] positions.
struct BatchArgs {
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* pages;   // [sequences, max_pages]
  uint32_t sequences, max_pages;
  Div page;               // positions of a page
  uint32_t page_count;    // of the cache
};

// Rows of a cache: position i of page g and head h starts at
// p + g * s[0] + i * s[1] + h * s[2] bytes; its scale (8-bit forms) likewise.
struct CacheTensor {
  char* p;
  int64_t s[3];
  float* scales;          // packed [page_count, page, heads]
};

struct AppendArgs : HeadsCore {
  BatchArgs batch;
  HeadSide q;             // passes 0: not there
  HeadSide k, v;          // x only
  CacheTensor ck, cv;
  int format;             // 8-bit caches
};

enum { kCacheSame = 0, kCacheI8 = 1, kCacheE4M3 = 2 };

// dt: kRowF16, kRowBF16 or kRowF32; whole: every unit is two whole chunks
struct HeadsShape {
  int dt;
  bool whole, pairs;
};
hipError_t rotate_launch(const HeadsShape& k, const HeadsForward& a, hipStream_t s);
hipError_t head_norm_launch(const HeadsShape& k, const HeadsForward& a, hipStream_t s);
hipError_t head_norm_backward_launch(const HeadsShape& k, const HeadsBackward& a, uint32_t workgroups, hipStream_t s);
hipError_t head_columns_launch(const HeadColumns& a, hipStream_t s);
hipError_t append_launch(const HeadsShape& k, int cache, const AppendArgs& a, hipStream_t s);

constexpr int kHeadThreads = 256;
constexpr int kHeadColumns = 16;  // columns that a workgroup adds up

}  // namespace acp
