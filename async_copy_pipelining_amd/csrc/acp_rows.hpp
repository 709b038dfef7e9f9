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

// A launch writes its kernel's arguments to memory that the host reaches
// slowly, at about 2.4 ns a byte (a launch with 540 bytes takes 3.7 us, with
// 110 bytes 2.6): each kernel takes the tensors that it uses and no others.

// Elementwise row operators: chunk i of the launch is chunk i % cpr of row
// i / cpr, and row r is index (r / (n1 * n2), r / n2 % n1, r % n2).  cpr is a
// whole number of scale blocks, so block i >> lb_log2 has chunk i.
struct RowsCore {
  int64_t c;        // channels of a row
  uint32_t total;   // chunks, those past a row's end included
  Div cpr, n1, n2;
  int lb_log2;      // log2 of the chunks in a scale block
  int format, act;
};

// What the host fills in, and a kernel's own arguments: NT float tensors and
// NP 8-bit forms.
struct RowsArgs : RowsCore {
  RowTensor x, z, y, dy, dx, dz;
  Packed px, pz;
};
template <int NT, int NP>
struct RowsUse : RowsCore {
  RowTensor t[NT];
  Packed p[NP > 0 ? NP : 1];
};
template <int NT>
struct RowsUse<NT, 0> : RowsCore {
  RowTensor t[NT];
};

// Group norm.  A workgroup covers `lanes` chunks of a row (channel block
// blk) and `row_lanes` rows at a time; such steps are dealt out to the runs
// that a sample's rows are split into.
struct NormCore {
  const float* gamma;       // nullptr: 1
  const float* beta;        // nullptr: 0
  float* mean;              // [samples, groups]
  float* rstd;
  float* dgamma;            // [c]
  float* dbeta;
  float* part;              // workspace: partial statistics or partial sums of the parts
  float* coef;              // workspace: partial sums of the groups' two coefficients
  uint32_t samples, rows, c, groups, per_group;
  Div row2, lanes, blocks;  // blocks: channel blocks of a row
  Div per;                  // per_group
  uint32_t row_lanes;
  Div runs;                 // runs of this pass
  uint32_t parts;           // runs of the pass that left the parts
  uint32_t pieces;          // channel blocks that one group may reach into
  uint32_t main_grid;       // workgroups beside those that sum columns
  uint32_t col_rows;        // rows of partial column sums
  int lb_log2, group_lanes_log2;
  float eps;
};

// What the host fills in.  Tensors: s[0] per sample; row r of a sample at
// r / row2.d * s[1] + r % row2.d * s[2].  codes and scales: the saved form of
// x, written (forward) or read (backward).
struct NormArgs : NormCore {
  RowTensor x, y, dy, dx, codes, scales;
};

// A kernel's own arguments.
struct NormStats : NormCore {
  RowTensor x;
};
struct NormForward : NormCore {
  RowTensor x, y;
};
struct NormForwardSaved : NormForward {
  RowTensor codes, scales;
};
struct NormBackward : NormCore {
  RowTensor dy, dx, x;
};
struct NormBackwardSaved : NormCore {
  RowTensor dy, dx, codes, scales;
};

// What a chunk may hold and how its row is found: channels of one group; whole
// chunks that groups may divide; anything (rows that end inside a chunk, rows
// more than one stride apart, or so far that a step passes 31 bits).
enum NormKind { kNormWhole = 0, kNormSplit = 1, kNormAny = 2 };

enum NormOp { kNormOpRow, kNormOpSlab, kNormOpStats, kNormOpApply,                     // forward
              kNormOpRowBackward, kNormOpSlabBackward, kNormOpSums, kNormOpDx };       // backward

// The kernel of a pass.
struct NormShape {
  int dt;
  NormKind kind;
  int packed;    // 0 none, 1 i8, 2 e4m3: the form of x that is written (forward) or read (backward)
  int act;
  uint32_t threads;
};

enum { kRowF16 = 0, kRowBF16 = 1, kRowF32 = 2 };

// dt: kRowF16, kRowBF16 or kRowF32
hipError_t pack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t unpack8_launch(int dt, const RowsArgs& a, hipStream_t s);
hipError_t act_forward_launch(int dt, bool gated, bool save, const RowsArgs& a, hipStream_t s);
hipError_t act_backward_launch(int dt, bool gated, const RowsArgs& a, hipStream_t s);

// One pass of a group norm: forward, one row a sample; a sample's slab on
// chip; by parts, the statistics and then the result.  Backward likewise; by
// parts the sums, and then dx with the sums of columns.
hipError_t norm_launch(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_launch_f16(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_launch_bf16(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_launch_f32(NormOp op, const NormShape& k, const NormArgs& a, hipStream_t s);
hipError_t norm_columns_launch(const NormArgs& a, hipStream_t s);
uint32_t norm_column_grid(const NormArgs& a);  // workgroups that sum columns: 0 if nothing wants them

constexpr int kRowThreads = 256;      // workgroup size, but for small calls and slabs
constexpr int kRowUnroll = 4;         // chunks a lane has in flight
constexpr int kSlabRows = 8;          // chunks that a lane of a forward slab holds
constexpr int kSlabRowsBackward = 4;  // ... of a backward slab
constexpr int kSlabThreads = 1024;    // largest workgroup of a forward slab
constexpr int kSlabThreadsBackward = 512;
constexpr int kRowThreadsBackward = 512;
constexpr uint32_t kColumns = 16;     // columns that a workgroup adds up

}  // namespace acp
