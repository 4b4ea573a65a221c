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
// with 3 and 15: 2048 tiles 60 and 77 us, 3500 tiles 119 and 95; of 16 / 4 heads of
// 128: 1024 tiles 29 and 50, 3500 tiles 108 and 107, 8192 in fp32 1.29 and 1.12 ms).
// 15 tiles leave 128 registers a wave, 11 leave 168, 7 and 3 leave 256.  Forward:
// units of 64 keys fit the first up to d_v of 128, but for 3 registers (237 us at
// B = 8, L = 2048, 16 / 4 heads of 128, against 240 with 32 keys, 239 with 11 tiles
// and 289 with 7); d_v of 256 takes units of 32 and 11 tiles (L = 16384, 8 / 2 heads:
// 529 us; 7 tiles 643).  The bf16 gradient has a second sum beside that of dq and
// takes as many tiles as hold both (B = 2, L = 4096, 16 / 4 heads of 128: 550 us with
// 11, 580 with 7, 606 with 3; d_v of 256 at L = 16384: 1.32 ms with 7, 1.38 with 3).
// fp32 with wide heads takes 3 tiles for their registers.
// es: bytes of an element; dkp, dvp: padded head widths.
constexpr TileShape tile_shape(int es, int dkp, int dvp, bool gradient, int block, bool many) {
  if (!many) return {es == 4 ? 16 : 32, 3};
  if (es == 4) return {16, dvp == 256 || (gradient && dkp == 128) ? 3 : 15};
  if (gradient) return {32, dkp == 128 ? (dvp == 256 ? 7 : 11) : dvp == 256 ? 11 : 15};
  return {dvp <= 128 && block > 32 ? 64 : 32, dvp == 256 ? 11 : 15};
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
