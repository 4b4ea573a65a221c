// Launch parameters of the sliding-window attention.  Strides are in bytes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace msgla {

struct WinHeads {
  char* p;
  int64_t sb, st, sh;  // a sequence, a position, a head
};

constexpr int WIN_ROWS = 32;   // (query, head) rows of a wave: one MFMA tile
constexpr int WIN_SINK = 32;   // keys of one that takes first tokens alone, of one pair
constexpr int WIN_FEW_ROWS = 16, WIN_FEW_WAVES = 4, WIN_FEW_KEYS = 32;

struct WinParams {
  WinHeads q, k, v, o, dout, dq, dk, dv;
  WinHeads kt, vt;  // a step's, or an append's, new keys and values
  const int32_t* start;
  const int32_t* lens;
  const int32_t* pos;  // a step's, or an append's, number of tokens before
  const float* lse_in;
  float *lse;
  float *delta, *nref;  // [B][Hq][L] what dq leaves for dk and dv: delta, and minus lse in units of log 2
  int B, L, S, Hq, Hkv, G, dkw, dvw;
  int window, n_sink;
  float scale;
  // tiles of `tile_rows` rows: QT queries of all G heads, or GT tiles of heads a query
  int tile_rows, QT, GT, tiles_per_seq;
  int64_t tiles;
  int parts;  // few rows: workgroups that a tile's keys are dealt to
  float* po;  // [tile][part][16][DVP] partial outputs
  float* pm;  // [tile][part][16][2] their maxima (in units of log 2) and sums
  // dk and dv: key tiles of key_tile keys, the parts of their queries, and what is joined
  int key_tile, key_tiles, key_parts, sink_tiles, sink_parts, joined;  // joined: key tiles that have partial sums
  float* part;  // [B Hkv][joined][key_parts][key_tile][DKP + DVP], then [B Hkv][sink_tiles][sink_parts][32][DKP + DVP]
  float* sink_part;
};

constexpr int WIN_TILES = 4;   // tiles of a workgroup of the forward, one a wave
// Pairs of waves of a workgroup of the gradients, each with a tile of 32 rows (dq) or
// keys (dk and dv): four, or one where three stages of LDS leave no more room and a
// wave needs more than 256 registers.  es: bytes of an element; dvp: padded width.
constexpr int win_pairs(int es, int dvp) { return es == 4 && dvp == 256 ? 1 : 4; }
inline int win_dkp(int dk) { return dk <= 64 ? 64 : 128; }
inline int win_dvp(int dv) { return dv <= 64 ? 64 : dv <= 128 ? 128 : 256; }

hipError_t launch_window(const WinParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_window_dq(const WinParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_window_few(const WinParams& P, bool step, bool bf16_path, hipStream_t st);
hipError_t launch_window_dkdv(const WinParams& P, bool bf16_path, hipStream_t st);
hipError_t launch_window_append(const WinParams& P, bool bf16_path, hipStream_t st);

}  // namespace msgla
