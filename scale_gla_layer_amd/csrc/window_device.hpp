// Device helpers of the window attention: products of 32 x 32 tiles and the LDS
// readers of their operands.
//
// A "slab" is 32 bytes of each of 32 rows, 16 a lane: lane l has bytes
// 16 (l / 32) .. of row l % 32.  For bf16 it is 16 k-values and one
// v_mfma_f32_32x32x16_bf16, for fp32 8 and four v_mfma_f32_32x32x2_f32.  The
// result's lane l holds, of column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4,
// i = 0 .. 15: in turn the B operand of a product over those rows, 8 (bf16) or 4
// values a slab, whose A operand wants columns over the same rows.
#pragma once
#include <type_traits>

#include "block_stage.hpp"
#include "window.hpp"

namespace msgla {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;

__device__ __forceinline__ f32x16 zero_tile() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

template <typename T> __device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
    return c;
  }
}

// Tiles of rows of W 16-byte pieces, piece p of row r at p ^ tile_key(r).
// Slab s of rows 32 t + l % 32.
template <int W> struct Rows32 {
  int at;
  __device__ Rows32(int lane) {
    const int r = lane & 31;
    at = r * W * 16 + (((lane >> 5) ^ tile_key<W>(r)) * 16);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int t, int s) const { return ld16(lds + (at ^ (32 * s)) + t * 32 * W * 16); }
};

// Columns 32 t .. + 31 over slab s's positions.
template <typename T, int W> struct Columns32;
template <int W> struct Columns32<bf16, W> {
  int at0, at1;
  __device__ Columns32(int lane) {
    const int g = lane >> 4, e = (lane >> 2) & 3, c = lane & 3, r = 4 * (g >> 1) + e, p = 2 * (g & 1) + (c >> 1);
    at0 = r * W * 16 + ((p ^ tile_key<W>(r)) * 16) + 8 * (c & 1);
    at1 = (r + 8) * W * 16 + ((p ^ tile_key<W>(r + 8)) * 16) + 8 * (c & 1);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    const char* base = lds + s * 16 * W * 16;
    const blk_v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)(base + (at0 ^ (64 * t))));
    const blk_v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)(base + (at1 ^ (64 * t))));
    const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
    return u32x4{x[0], x[1], y[0], y[1]};
  }
};
template <int W> struct Columns32<float, W> {
  static_assert(W >= 16, "swizzle of four bits");
  int at[4];
  __device__ Columns32(int lane) {
    const int h = lane >> 5, c = lane & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * h + j;
      at[j] = r * W * 16 + (((c >> 2) ^ tile_key<W>(r)) * 16) + 4 * (c & 3);
    }
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    u32x4 v;  // row bit 3 changes bit 0 of the key
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const uint32_t*>(lds + (at[j] ^ (128 * t) ^ ((s & 1) << 4)) + s * 8 * W * 16);
    return v;
  }
};

// Copies of units of KT rows of W pieces into stage tiles, dealt to a workgroup's
// waves: a unit's rows from one address on, or each chosen by `key`.  Pieces behind
// the rows' width repeat the first one: they meet zeroes or columns that are not
// stored.
template <int W, int KT, int WAVES> struct UnitCopy {
  static constexpr int ALL = KT * W / 64, N = (ALL + WAVES - 1) / WAVES;  // copy instructions, and a wave's
  static_assert(KT * W % 64 == 0, "whole copy instructions");
  const char* base;
  int64_t st;
  uint32_t off[N];  // from the unit's first row
  __device__ UnitCopy(const char* b, int64_t stride, int width, int wave, int lane) : base(b), st(stride) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = 64 * (wave + WAVES * i) + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
      off[i] = (uint32_t)r * (uint32_t)st + (p * 16 < width ? p * 16 : 0);
    }
  }
  // whether 32 bits hold the offsets
  __device__ __forceinline__ bool near() const { return st <= 0x7fffffff / KT; }
  __device__ __forceinline__ void whole(int64_t k0, char* lds, int wave) const {
    const char* first = base + k0 * st;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ALL % WAVES == 0 || wave + WAVES * i < ALL) dma16(first + off[i], lds + 1024 * (wave + WAVES * i));
  }
  template <class Key> __device__ __forceinline__ void chosen(int width, char* lds, int wave, int lane, Key key) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = 64 * (wave + WAVES * i) + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
      if (ALL % WAVES == 0 || wave + WAVES * i < ALL)
        dma16(base + key(r) * st + (p * 16 < width ? p * 16 : 0), lds + 1024 * (wave + WAVES * i));
    }
  }
};

// Two values as one or (bf16) two operand words: hi + lo.
__device__ __forceinline__ uint32_t win_pair(float a, float b) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
  return __builtin_bit_cast(uint32_t, bf16x2{(bf16)a, (bf16)b});
}

// A tile of 32 x 32 weights as the B operands of a product over its rows.
template <typename T> struct Weights;
template <> struct Weights<bf16> {
  static constexpr int SLABS = 2;
  uint32_t hi[8], lo[8];
  __device__ __forceinline__ void set(int i, float a, float b) {  // rows 2 i and 2 i + 1 of the lane's
    hi[i] = win_pair(a, b);
    lo[i] = win_pair(a - u2f(hi[i] << 16), b - u2f(hi[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set_hi(int i, float a, float b) { hi[i] = win_pair(a, b); }
  // a product with the weights as they are, and with their higher halves alone
  __device__ __forceinline__ f32x16 mma_hi(u32x4 f, int s, f32x16 c) const {
    return mma32<bf16>(f, u32x4{hi[4 * s], hi[4 * s + 1], hi[4 * s + 2], hi[4 * s + 3]}, c);
  }
  __device__ __forceinline__ f32x16 mma(u32x4 f, int s, f32x16 c) const {
    c = mma32<bf16>(f, u32x4{hi[4 * s], hi[4 * s + 1], hi[4 * s + 2], hi[4 * s + 3]}, c);
    return mma32<bf16>(f, u32x4{lo[4 * s], lo[4 * s + 1], lo[4 * s + 2], lo[4 * s + 3]}, c);
  }
};
template <> struct Weights<float> {
  static constexpr int SLABS = 4;
  float v[16];
  __device__ __forceinline__ void set(int i, float a, float b) { v[2 * i] = a, v[2 * i + 1] = b; }
  __device__ __forceinline__ f32x16 mma(u32x4 f, int s, f32x16 c) const {
    return mma32<float>(f, u32x4{f2u(v[4 * s]), f2u(v[4 * s + 1]), f2u(v[4 * s + 2]), f2u(v[4 * s + 3])}, c);
  }
};

// A tile of results that one wave of a pair leaves for the other, lane by lane.
constexpr int TILE_BYTES = 64 * 64;
__device__ __forceinline__ void tile_put(char* lds, const f32x16& t, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) st16(lds + (i * 64 + lane) * 16, u32x4{f2u(t[4 * i]), f2u(t[4 * i + 1]), f2u(t[4 * i + 2]), f2u(t[4 * i + 3])});
}
__device__ __forceinline__ f32x16 tile_get(const char* lds, int lane) {
  f32x16 t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 v = __builtin_bit_cast(f32x4, ld16(lds + (i * 64 + lane) * 16));
#pragma unroll
    for (int e = 0; e < 4; ++e) t[4 * i + e] = v[e];
  }
  return t;
}

// 4 consecutive columns of a result tile: 32 t + 8 i + 4 (l / 32)
__device__ __forceinline__ int win_column(int t, int i, int lane) { return 32 * t + 8 * i + 4 * (lane >> 5); }

// A query's position, or -1 for padding: behind the sequence's keys, or before its start.
__device__ __forceinline__ int win_position(const WinParams& P, int b, int i) {
  if (i >= P.L) return -1;
  const int64_t p = (P.start ? (int64_t)P.start[b] : 0) + i;
  const int len = P.lens ? min(P.lens[b], P.S) : P.S;
  return p >= 0 && p < len ? (int)p : -1;
}

// What a lane knows of its row of a tile.
struct WinRow {
  int i, head, p;  // query, query head, position
  bool in;         // a row of the problem (of padding, if p < 0)
  __device__ WinRow(const WinParams& P, int b, int h, int t, int r) {
    const int i0 = P.GT > 1 ? t / P.GT : t * P.QT, g0 = P.GT > 1 ? (t % P.GT) * P.tile_rows : 0;
    const int qi = P.GT > 1 ? 0 : r / P.G, g = P.GT > 1 ? g0 + r : r - qi * P.G;
    i = i0 + qi;
    head = h * P.G + g;
    in = (P.GT > 1 || qi < P.QT) && g < P.G && i < P.L;
    p = in ? win_position(P, b, i) : -1;
  }
};

__device__ __forceinline__ const char* win_at(const WinHeads& t, int64_t b, int64_t i, int64_t h) {
  return t.p + b * t.sb + i * t.st + h * t.sh;
}
__device__ __forceinline__ char* win_out(const WinHeads& t, int64_t b, int64_t i, int64_t h) {
  return t.p + b * t.sb + i * t.st + h * t.sh;
}

// Wait states for the result of the last matrix product (16 passes at most), where
// results that do not fit in vector registers are moved about behind a branch: hipcc
// 7.2 leaves out some on the shortest way there.
__device__ __forceinline__ void products_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 3");
  __builtin_amdgcn_sched_barrier(0);
}

// Whether a row at a position from pmin to pmax does not attend all of the n keys from
// j0 on.  Operators that take both sides make one branch of it: where a branch in two
// steps follows a matrix product, hipcc 7.2 counts the wait states that the product's
// result needs along the longer way alone.
__device__ __forceinline__ bool win_edge(const WinParams& P, int j0, int n, int pmin, int pmax) {
  return (j0 + n - 1 > pmin) | ((j0 <= pmax - P.window) & (j0 + n > P.n_sink));
}
// Whether a row at position p, whose window begins behind `low`, does not attend key j.
__device__ __forceinline__ bool win_out_of(const WinParams& P, int j, int p, int low) {
  return (j > p) | ((j <= low) & (j >= P.n_sink));
}

__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = min(v, __shfl_xor(v, o));
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, __shfl_xor(v, o));
  return __builtin_amdgcn_readfirstlane(v);
}

}  // namespace msgla
