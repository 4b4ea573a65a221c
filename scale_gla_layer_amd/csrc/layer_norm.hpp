// Launch parameters of the layer norm.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct LnRows {
  char* p;
  int64_t sb, st;  // byte strides of a sequence and of a position
};

struct LnParams {
  LnRows x, y, dy, dx;
  const float *weight, *bias;
  float *mean, *rstd;               // forward: written, may be NULL
  const float *mean_in, *rstd_in;   // backward
  float *dweight, *dbias;
  float* part;  // [parts][2][D] sums of dy xh and of dy over a workgroup's rows, formed in 64 bits
  int parts;
  int64_t rows;
  int L, D;
  float eps;
};

constexpr int LN_MAX_WIDTH = 16384;  // 1024 lanes of four pieces, in fp32
// Rows up to this many 16-byte pieces keep the sums for dweight and dbias in
// registers while dx is formed; wider ones form them in a kernel of their own.
constexpr int LN_WIDE = 1024;
// Workgroups that the rows of a backward are dealt to, at most: each leaves its sums
// (B = 8, L = 2048, D = 1024, while sums were kept in 32 bits: 24.0 us, with 256 26.7, with 1024 27.7).
constexpr int LN_PARTS = 512;
// Workgroups of a forward, at most: rows of later rounds are under way meanwhile
// (B = 8, L = 2048, D = 1024: 16.3 us, with 512 20.3).
constexpr int LN_GRID = 2048;
// Columns and threads of a workgroup of the kernels that sum over rows, and over their
// parts (B = 8, L = 2048, D = 1024: 25.2 us; with 64 columns for the parts 25.8, with 16 25.3, but
// 49 for 46 us at B = 4, D = 4096).
constexpr int LN_COLS = 64, LN_JOIN_COLS = 32, LN_COL_THREADS = 1024;

struct LnShape {
  int lanes, pieces, threads;  // lanes of a row, 16-byte pieces of a lane, threads of a workgroup
};
LnShape ln_shape(int64_t bytes_of_row, int es);
int ln_groups(int64_t rows, int64_t bytes_of_row, int es);  // workgroups of the backward
int ln_parts(int64_t rows, int64_t bytes_of_row, int es);   // parts of its sums
int ln_grid(int64_t rows, int64_t bytes_of_row, int es);  // of the forward

hipError_t launch_layer_norm(const LnParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_layer_norm_backward(const LnParams& P, bool bf16_path, hipStream_t st);

}  // namespace msgla
