// Device helpers of the block attention kernels.
//
// A tile is 16 rows, a row one (query, head) pair: neighbouring queries with
// all their heads of one key-value head, which share its blocks.  Scores are
// formed transposed, S^T = K Q^T (A = keys, B = rows), so that lane l holds, of
// row l % 16, the four keys 4 (l / 16) + i of every 16-key tile: a row's
// softmax needs two lane exchanges, and the lane's values are already the B
// operand of O^T = V^T P^T.  The A operand of that product, V^T, wants a
// column's values over the same keys: from LDS rows by transpose reads (bf16)
// or by element reads (fp32).
#pragma once
#include "block.hpp"
#include "device_common.hpp"

namespace msgla {

constexpr float BLK_LOG2E = 1.4426950408889634f, BLK_LN2 = 0.6931471805599453f;
constexpr int BLK_END = 0x7fffffff;

typedef short blk_v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) blk_v4s blk_lds_v4s;

// LDS row pitch: 32 (bf16) or 16 (fp32) bytes of padding spread the rows that
// one transpose or element read touches over all banks
template <typename T, int D> constexpr int blk_pitch() { return D * (int)sizeof(T) + (sizeof(T) == 2 ? 32 : 16); }
// positions of one product slab
template <typename T> constexpr int blk_slab() { return 64 / (int)sizeof(T); }

// Column 16 ct + l % 16 of slab rows r0 + 4 (l / 16) + i (and + 16 for bf16).
template <typename T> __device__ __forceinline__ u32x4 blk_column(const char* lds, int pitch, int r0, int ct, int lane);
template <> __device__ __forceinline__ u32x4 blk_column<bf16>(const char* lds, int pitch, int r0, int ct, int lane) {
  const int a = lane >> 4, e = (lane >> 2) & 3, c = lane & 3;
  const char* p = lds + (r0 + 4 * a + e) * pitch + 32 * ct + 8 * c;
  const blk_v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)p);
  const blk_v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)(p + 16 * pitch));
  const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
  return u32x4{x[0], x[1], y[0], y[1]};
}
template <> __device__ __forceinline__ u32x4 blk_column<float>(const char* lds, int pitch, int r0, int ct, int lane) {
  const char* p = lds + (r0 + 4 * (lane >> 4)) * pitch + (16 * ct + (lane & 15)) * 4;
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(p + j * pitch);
  return v;
}

// The B operand of slab s from the lane's values p[16-position tile][i].
template <typename T> __device__ __forceinline__ u32x4 blk_pack(const float (*p)[4], int s) {
  if constexpr (sizeof(T) == 2) {
    const float v[8] = {p[2 * s][0], p[2 * s][1], p[2 * s][2], p[2 * s][3],
                        p[2 * s + 1][0], p[2 * s + 1][1], p[2 * s + 1][2], p[2 * s + 1][3]};
    return pack16<bf16>(v);
  } else {
    return pack16<float>(p[s]);
  }
}

// The same as a sum of two operands: with bf16 what the first one's rounding leaves
// goes through the product as well, so that 16 bits of a weight count (fp32: lo is 0).
template <typename T> __device__ __forceinline__ void blk_split(const float (*p)[4], int s, u32x4& hi, u32x4& lo) {
  if constexpr (sizeof(T) == 2) {
    const float v[8] = {p[2 * s][0], p[2 * s][1], p[2 * s][2], p[2 * s][3],
                        p[2 * s + 1][0], p[2 * s + 1][1], p[2 * s + 1][2], p[2 * s + 1][3]};
    split_bf16(v, hi, lo);
  } else {
    hi = pack16<float>(p[s]);
    lo = zero16();
  }
}
template <typename T> __device__ __forceinline__ f32x4 blk_mma_split(u32x4 a, u32x4 hi, u32x4 lo, f32x4 c) {
  c = mma_slab<T>(a, hi, c);
  if constexpr (sizeof(T) == 2) c = mma_slab<T>(a, lo, c);
  return c;
}

// 16 bytes at byte offset `at` of a row of `width` bytes, zero behind its end
__device__ __forceinline__ u32x4 blk_ld(const char* row, int at, int width) {
  return at < width ? ld16(row + at) : zero16();
}

// Copies rows [0, n) of D elements (width bytes of them given, the rest zero)
// to LDS; a row of a NULL pointer is zero.  THREADS threads take part.
template <typename T, int D, int THREADS, class Row>
__device__ __forceinline__ void blk_stage(char* lds, int n, int width, int tid, Row row) {
  constexpr int PC = D * (int)sizeof(T) / 16;
  for (int i = tid; i < n * PC; i += THREADS) {
    const int r = i / PC, at = (i % PC) * 16;
    const char* p = row(r);
    st16(lds + r * blk_pitch<T, D>() + at, p ? blk_ld(p, at, width) : zero16());
  }
}

// A query's position, or -1 for padding: behind the sequence's keys, or before its start.
__device__ __forceinline__ int blk_position(const BlkParams& P, int b, int i) {
  if (i >= P.L) return -1;
  const int64_t p = (P.start ? (int64_t)P.start[b] : 0) + i;
  const int len = P.lens ? min(P.lens[b], P.S) : P.S;
  return p >= 0 && p < len ? (int)p : -1;
}

// The blocks a query attends, from its row of `sel`: an entry counts where it
// names a block at or before the query's own and is greater than every entry
// that counted before it.  Returns their number; f gets each.
template <class F> __device__ __forceinline__ int blk_chosen(const BlkParams& P, const int32_t* sel, int p, F f) {
  int last = -1, n = 0;
  if (p < 0) return 0;
  const int own = p >> P.lgT;
  for (int e = 0; e < P.n; ++e) {
    const int j = sel[e];
    if (j > last && j <= own) f(n++, last = j);
  }
  return n;
}

// What a lane knows of its tile row.
struct BlkRow {
  int b, h, i, head, p;  // sequence, key-value head, query, query head, position
  bool in;               // a row of the problem (of padding, if p < 0)
};

struct BlkTile {
  int b, h, i0, g0;
  __device__ BlkTile(const BlkParams& P, int64_t tile) {
    const int bh = (int)(tile / P.tiles_per_seq), t = (int)(tile - (int64_t)bh * P.tiles_per_seq);
    b = bh / P.Hkv;
    h = bh - b * P.Hkv;
    i0 = P.GT > 1 ? t / P.GT : t * P.QT;
    g0 = P.GT > 1 ? (t % P.GT) * BLK_ROWS : 0;
  }
  // local query and head of row r
  __device__ BlkRow row(const BlkParams& P, int r) const {
    BlkRow w;
    const int qi = P.GT > 1 ? 0 : r / P.G, g = P.GT > 1 ? g0 + r : r - qi * P.G;
    w.b = b;
    w.h = h;
    w.i = i0 + qi;
    w.head = h * P.G + g;
    w.in = qi < P.QT && g < P.G && w.i < P.L;
    w.p = w.in ? blk_position(P, b, w.i) : -1;
    return w;
  }
};

// The lists of a tile's queries in LDS, each ended by BLK_END: one wave.
constexpr int BLK_LIST = BLK_MAX_SEL + 1;
__device__ __forceinline__ void blk_lists(const BlkParams& P, const BlkTile& t, int* lists, int* raw, int lane) {
  const int rows = min(P.QT, P.L - t.i0);
  const int32_t* sel = P.sel + (((int64_t)t.b * P.Hkv + t.h) * P.L + t.i0) * P.n;
  for (int i = lane; i < rows * P.n; i += 64) raw[i] = sel[i];
  __syncthreads();
  if (lane < P.QT) {
    const int p = blk_position(P, t.b, t.i0 + lane);
    int* l = lists + lane * BLK_LIST;
    l[blk_chosen(P, raw + lane * P.n, p, [&](int n, int j) { l[n] = j; })] = BLK_END;
  }
}

__device__ __forceinline__ float blk_quad_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float blk_quad_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ int blk_row_min(int v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = min(v, __shfl_xor(v, o));
  return v;
}

// 4 consecutive elements of a row
template <typename T> __device__ __forceinline__ void blk_st4(char* p, const float* v) {
  if constexpr (sizeof(T) == 2) st8(p, pack8<bf16>(v));
  else st16(p, pack16<float>(v));
}

// The backward counts each block's queries; its first kernel clears the counts.
__device__ __forceinline__ void blk_clear_counts(const BlkParams& P, int tid, int threads) {
  const int64_t n = (int64_t)P.B * P.Hkv * P.nb;
  for (int64_t i = (int64_t)blockIdx.x * threads + tid; i < n; i += (int64_t)gridDim.x * threads) P.cnt[i] = 0;
}

// sum of the products of 16 bytes of elements
template <typename T> __device__ __forceinline__ float blk_dot(u32x4 x, u32x4 y) {
  constexpr int N = 16 / sizeof(T);
  float u[N], v[N], s = 0.f;
  unpack16<T>(x, u);
  unpack16<T>(y, v);
#pragma unroll
  for (int i = 0; i < N; ++i) s = __builtin_fmaf(u[i], v[i], s);
  return s;
}

}  // namespace msgla
