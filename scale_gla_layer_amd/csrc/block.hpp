// Launch parameters of the block selection and the attention over the selected
// blocks.  Strides are in bytes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_plan.hpp"

namespace msgla {

struct BlkHeads {
  char* p;
  int64_t sb, st, sh;  // a sequence, a position, a head
};

constexpr int BLK_KEYS = 32;     // keys of a step
constexpr int BLK_PIECE = 256;   // blocks whose scores are in LDS at once

struct BlkParams {
  BlkHeads q, k, v, o, dout, dq, dk, dv;
  BlkHeads kt, vt;  // the step's new key and value
  const int32_t* sel;
  int32_t* sel_out;
  const int32_t* start;
  const int32_t* lens;
  const int32_t* from;
  float* means;
  float* lse;
  const float* lse_in;
  float* delta;
  int B, L, S, Hq, Hkv, G, dkw, dvw;  // dkw, dvw: head widths
  int lgT, n, n_first, n_recent, nb;  // block of 2^lgT positions, nb = blocks of S
  float scale;
  // tiles of 16 rows: QT queries of all G heads, or GT tiles of 16 heads of one query
  int QT, GT, tiles_per_seq;
  int64_t tiles;
  int parts;     // workgroups a tile's blocks are dealt to
  float* po;     // [tile][part][16][DVP] partial outputs; backward [..][2][DKP] partial sums for dq
  float* pm;     // [tile][part][16][2] their maxima (in units of log 2) and sums; backward [..] delta's errors
  // queries of each block
  int seg, W, max_items, max_parts;  // queries of a work item, 64-query words, bounds per (sequence, head)
  uint64_t* bits;   // [B Hkv][W][nb]; a step's scores [B Hkv][nb]
  int32_t* cnt;     // [B Hkv][nb]
  int32_t* off;     // [B Hkv][nb]
  int32_t* slot;    // [B Hkv][nb] first partial of a block of several items
  int32_t* list;    // [B Hkv][L n]
  int2* items;      // [B Hkv][max_items] block, first query of its list
  int32_t* n_items; // [B Hkv]
  float* part;      // [B Hkv][max_parts][T][DKP + DVP]
};

hipError_t launch_block_means(const BlkParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_block_select(const BlkParams& P, bool bf16_path, hipStream_t st);
// the step: puts the token into the caches and selects its blocks
// Caches of more blocks have their scores spread over workgroups (and in memory: `bits`).
constexpr int BLK_STEP_ONE = 128;
inline bool blk_step_spread(const BlkParams& P) { return P.nb > BLK_STEP_ONE; }
hipError_t launch_block_step(const BlkParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_block_forward(const BlkParams& P, bool bf16_path, hipStream_t st);
// many queries: keys and values shared by a workgroup; nb at most BLK_TILES_MAX
hipError_t launch_block_tiles(const BlkParams& P, bool gradient, bool bf16_path, hipStream_t st);
hipError_t launch_block_dq(const BlkParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_block_dkdv(const BlkParams& P, bool bf16_path, hipStream_t st);

// padded head widths of the kernels
inline int blk_dkp(int dk) { return dk <= 64 ? 64 : 128; }
inline int blk_dvp(int dv) { return dv <= 64 ? 64 : dv <= 128 ? 128 : 256; }

}  // namespace msgla
