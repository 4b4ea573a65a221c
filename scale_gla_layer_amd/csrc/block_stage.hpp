// LDS stages of the block attention kernels: rows that asynchronous copies bring
// in, their 16-byte pieces XOR-swizzled by the row, so that both readers are
// free of bank conflicts: 16 rows at one piece (a row-major MFMA operand), and
// 16 rows' columns (a transposed one, through the transpose read).
#pragma once
#include "async_copy.hpp"
#include "block_device.hpp"

namespace msgla {

// A stage tile of rows of W pieces: piece p of row r lies at p ^ tile_key(r).
// Rows r .. r + 3 differ in bits that keep neighbouring pieces together, so the
// 16 lanes of one transpose read (four rows, two pieces) meet eight different
// 16-byte units, as do eight consecutive rows at one piece.
template <int W> __device__ __forceinline__ constexpr int tile_key(int r) {
  return W == 8 ? (r >> 1 & 1) << 1 | (r >> 2 & 1) << 2 | (r >> 3 & 1) : (r & 3) << 1 | (r >> 2 & 1) << 3 | (r >> 3 & 1);
}

// Column reader: slab s's rows at columns 16 t .. + 15 (layout of blk_column).
template <typename T, int W> struct Columns;
template <int W> struct Columns<bf16, W> {
  int at;
  __device__ Columns(int lane) {
    const int a = lane >> 4, e = (lane >> 2) & 3, c = lane & 3, r = 4 * a + e;
    at = r * W * 16 + (((c >> 1) ^ tile_key<W>(r)) * 16) + 8 * (c & 1);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    const char* p = lds + (at ^ (32 * t)) + s * 32 * W * 16;
    const blk_v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)p);
    const blk_v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)(p + 16 * W * 16));
    const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
    return u32x4{x[0], x[1], y[0], y[1]};
  }
};
template <int W> struct Columns<float, W> {
  static_assert(W >= 16, "swizzle of four bits");
  int at[4];
  __device__ Columns(int lane) {
    const int a = lane >> 4, c = lane & 15;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * a + j;
      at[j] = r * W * 16 + (((c >> 2) ^ tile_key<W>(r)) * 16) + 4 * (c & 3);
    }
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(lds + (at[j] ^ (64 * t)) + s * 16 * W * 16);
    return v;
  }
};

// Row reader: slab w of rows 16 kt + l % 16.
template <int W> struct Rows {
  int at;
  __device__ Rows(int lane) {
    const int c = lane & 15, a = lane >> 4;
    at = c * W * 16 + ((a ^ tile_key<W>(c)) * 16);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int kt, int w) const {
    return ld16(lds + (at ^ (64 * w)) + kt * 16 * W * 16);
  }
};

}  // namespace msgla
