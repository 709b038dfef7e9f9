// Row operators of acp: 8-bit checkpoints, activations, and group norm with
// an activation (channels last).  Argument blocks and launchers shared by the
// host entry points and the kernels.
//
// A tensor is seen as rows of C contiguous channels.  A lane handles one
// chunk of 16 bytes of a row: V = 16 / element size channels, whatever the
// row's alignment (the global loads and stores of gfx950 take any address);
// a row's last chunk may hold fewer channels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace acp {

// One tensor's rows: index (i0, i1, i2) of the collapsed outer dims starts at
// p + i0 * s[0] + i1 * s[1] + i2 * s[2] bytes.
struct RowTensor {
  char* p;
  int64_t s[3];
};

// n / d for n < 2^31 (magic_for).
struct Div {
  uint32_t d, mag, sh;
};

// The 8-bit form of a tensor: codes and one float32 scale per `block` channels.
struct Packed {
  RowTensor codes;
  float* scales;
};

// Elementwise row operators: chunk i of the launch is chunk i % cpr of row
// i / cpr, and row r is index (r / (n1 * n2), r / n2 % n1, r % n2).  cpr is a
// whole number of scale blocks, so block i >> lb_log2 has chunk i.
struct RowsArgs {
  RowTensor x, z, y, dy, dx, dz;
  Packed px, pz;
  int64_t c;        // channels of a row
  uint32_t total;   // chunks, those past a row's end included
  Div cpr, n1, n2;
  int lb_log2;      // log2 of the chunks in a scale block
  int format, act;
};

// Group norm.  A workgroup covers `lanes` chunks of a row (channel block
// blk) and `row_lanes` rows at a time, over one of the runs of `run_rows`
// rows that a sample's rows are split into.
struct NormArgs {
  RowTensor x, y, dy, dx;   // s[0] per sample; row r of a sample at r / row2.d * s[1] + r % row2.d * s[2]
  RowTensor codes, scales;  // the saved form of x, written (forward) or read (backward)
  const float* gamma;       // nullptr: 1
  const float* beta;        // nullptr: 0
  float* mean;              // [samples, groups]
  float* rstd;
  float* dgamma;            // [c]
  float* dbeta;
  float* part;              // workspace: partial statistics or partial sums of the parts
  float* coef;              // workspace: two coefficients for each sample and group
  uint32_t samples, rows, c, groups, per_group;
  Div row2, lanes, blocks;  // blocks: channel blocks of a row
  uint32_t row_lanes;
  Div runs;                 // runs of this pass
  uint32_t run_rows;
  uint32_t parts, part_rows;  // runs of the pass that left the parts, and their rows
  uint32_t pieces;          // channel blocks that one group may reach into
  uint32_t main_grid;       // workgroups before those that sum columns
  uint32_t col_rows;        // rows of partial column sums
  int lb_log2, group_lanes_log2, format, act;
  float eps;
};

// How a pass runs, beside its type.
struct NormShape {
  int dt;
  bool linear;   // rows one stride apart, a run's bytes within 31 bits
  bool whole;    // a chunk's channels are of one group
  bool packed;   // forward: saves x in 8 bits; backward: x is its 8-bit form
  uint32_t threads;
};

enum { kRowF16 = 0, kRowBF16 = 1, kRowF32 = 2 };

// dt: kRowF16, kRowBF16 or kRowF32
hipError_t pack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t unpack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t act_forward_launch(int dt, bool gated, bool save, const RowsArgs& a, hipStream_t s);
hipError_t act_backward_launch(int dt, bool gated, const RowsArgs& a, hipStream_t s);

// forward: one row a sample; a sample's slab on chip; by parts (two passes)
hipError_t norm_row_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_slab_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_stats_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_apply_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
// backward, and the sums of columns that follow
hipError_t norm_row_backward_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_slab_backward_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_sums_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_coef_launch(const NormArgs& a, hipStream_t s);
hipError_t norm_dx_launch(const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s);

constexpr int kRowThreads = 256;      // workgroup size, but for small calls and slabs
constexpr int kRowUnroll = 4;         // chunks a lane has in flight
constexpr int kSlabRows = 8;          // chunks that a lane of a forward slab holds
constexpr int kSlabRowsBackward = 4;  // ... of a backward slab
constexpr int kSlabThreads = 1024;    // largest workgroup of a forward slab
constexpr int kSlabThreadsBackward = 512;

}  // namespace acp
