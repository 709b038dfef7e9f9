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
// blk) and `row_lanes` rows at a time.  Sample n's rows are split into
// `chunks` runs of `rpc` rows; row r of a sample is (r / row2.d, r % row2.d).
struct NormArgs {
  RowTensor x, y, dy, dx;   // s[0] per sample, s[1] and s[2] per row index
  Packed px;                // the saved form of x, written (forward) or read (backward)
  const float* gamma;       // nullptr: 1
  const float* beta;        // nullptr: 0
  float* mean;              // [samples, groups]
  float* rstd;
  float* dgamma;            // [c]
  float* dbeta;
  float* part;              // workspace: partial statistics or partial sums
  float* coef;              // workspace: two coefficients for each sample and group
  uint32_t samples, rows, c, groups, per_group;
  Div row2, lanes;
  uint32_t row_lanes, blocks;  // channel blocks of a row
  uint32_t chunks, rpc;
  uint32_t pieces;          // channel blocks that one group may reach into
  uint32_t main_grid;       // workgroups before those that sum columns
  uint32_t col_rows;        // rows of partial column sums
  int lb_log2, group_lanes_log2, format, act;
  float eps;
};

enum { kRowF16 = 0, kRowBF16 = 1, kRowF32 = 2 };

// dt: kRowF16, kRowBF16 or kRowF32
hipError_t pack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t unpack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t act_forward_launch(int dt, bool gated, bool save, const RowsArgs& a, hipStream_t s);
hipError_t act_backward_launch(int dt, bool gated, const RowsArgs& a, hipStream_t s);

hipError_t norm_stats_launch(int dt, const NormArgs& a, hipStream_t s);
hipError_t norm_apply_launch(int dt, bool per_row, bool save, const NormArgs& a, hipStream_t s);
hipError_t norm_sums_launch(int dt, bool packed, const NormArgs& a, hipStream_t s);
hipError_t norm_coef_launch(const NormArgs& a, hipStream_t s);
hipError_t norm_dx_launch(int dt, bool per_row, bool packed, const NormArgs& a, hipStream_t s);
hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s);

constexpr int kRowThreads = 256;   // workgroup size of every row kernel
constexpr int kRowUnroll = 4;      // chunks a lane has in flight

}  // namespace acp
