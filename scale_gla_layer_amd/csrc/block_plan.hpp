// The workgroups of k_block_tiles and their LDS, as plain arithmetic: the launch
// and a check on the host go by the same rule.
#pragma once
namespace msgla {

constexpr int BLK_ROWS = 16;     // (query, head) rows of a tile: one MFMA tile
constexpr int BLK_MAX_SEL = 64;  // largest n_select
constexpr int BLK_TILES_MAX = 16384;  // blocks of the keys that shared tiles can hold
constexpr int BLK_TILES_MANY = 4096;  // tiles from which on workgroups are large

struct TileShape {
  int keys, tiles;  // keys of a unit; tiles of a workgroup
};

// A workgroup of 15 tiles has a CU to itself, two of 3 share one.  15 share keys
// among more, but need 4096 tiles to fill the chip (forward of 8 / 2 heads of 64
// with 3 and 15: 2048 tiles 33 and 36 us, 3500 tiles 66 and 48; of 16 / 4 heads of
// 128: 1024 tiles 18 and 28, 3500 tiles 70 and 70, 8192 in fp32 1.26 and 1.08 ms;
// gradients at 8192 tiles in bf16 606 and 505 us).
// 15 tiles leave 128 registers a wave, 11 leave 168, 3 leave 256.  Units of 64
// keys fit the first in the forward at d_v up to 128 (227 us at B = 8, L = 2048,
// 16 / 4 heads of 128, against 233 with 32 keys, 234 with 11 tiles and 279 with 7);
// in the gradient they spill (B = 2, L = 4096: 246 and 284 us), and d_v of 256
// spills with 15 tiles (one sequence of 16384, 8 / 2 heads: forward 509 us with 15,
// 501 with 11, backward 1207 and 1115).  fp32 with wide heads takes 3 tiles for
// their registers.
// es: bytes of an element; dkp, dvp: padded head widths.
constexpr TileShape tile_shape(int es, int dkp, int dvp, bool gradient, int block, bool many) {
  if (!many) return {es == 4 ? 16 : 32, 3};
  if (es == 4) return {16, dvp == 256 || (gradient && dkp == 128) ? 3 : 15};
  return {!gradient && dvp <= 128 && block > 32 ? 64 : 32, dvp == 256 ? 11 : 15};
}

// Workgroups, for `heads` sequences and key-value heads: XCDs take equal numbers of those.
constexpr long long tile_grid(int tiles, int tiles_per_seq, long long heads) {
  return (heads >= 8 ? (heads + 7) / 8 * 8 : heads) * ((tiles_per_seq + tiles - 1) / tiles);
}

struct TileLds {
  int stages, bytes;  // of the ring; all dynamic LDS
};

constexpr int TILE_STATIC = 1024;  // kept free for the kernel's own variables (fewer than 128 bytes)
// LDS of one workgroup on a CU, or of two
constexpr int tile_lds_limit(int tiles) { return (tiles > 3 ? 160 : 80) * 1024; }
constexpr int tile_stage(TileShape s, int es, int dkp, int dvp) { return s.keys * (dkp + dvp) * es; }

// Beside the ring: maps of nb blocks for all tiles and each one, and lists of n + 1
// 16-bit entries for the queries, qt of them a tile, or gt tiles a query.
constexpr TileLds tile_lds(TileShape s, int stage, int nb, int n, int qt, int gt) {
  const int queries = gt > 1 ? s.tiles / gt + 2 : s.tiles * qt;
  const int rest = (s.tiles + 1) * ((nb + 31) / 32 * 4) + queries * (n + 1) * 2;
  const int room = (tile_lds_limit(s.tiles) - TILE_STATIC - rest) / stage, stages = room < 8 ? room : 8;
  return {stages, stages * stage + rest};
}

}  // namespace msgla
