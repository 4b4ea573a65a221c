// Attention over each query's selected blocks: forward, and the gradient of
// the queries.  o = softmax(scale q K^T) V over the keys at or before the query
// in its blocks, by one pass with a running maximum and sum.
//
// For single queries, for a few over long sequences, and for more blocks than the
// kernel of shared tiles holds.  One wave takes a tile of 16 rows and walks the
// union of its queries' blocks, 32 keys a step; a row that has not chosen a block
// is masked there.  A tile's blocks are dealt to several waves, whose partial
// outputs a second kernel joins.  Bound by the latency of a wave's chain of loads,
// hence the many parts: single queries of 16 sequences, 16 / 4 heads of 128, 16
// blocks of 64 keys take 15 us for 34 MB, and the join 7; 64 tiles of a chunk at
// 8192 positions 54.
#include "block_device.hpp"

namespace msgla {

namespace {

template <typename T, int DKP> struct Qfrag {
  static constexpr int N = DKP * (int)sizeof(T) / 64;
  u32x4 f[N];
  __device__ void load(const char* row, int width, int lane, bool in) {
#pragma unroll
    for (int s = 0; s < N; ++s) f[s] = in ? blk_ld(row, 64 * s + 16 * (lane >> 4), width) : zero16();
  }
};

__device__ __forceinline__ const char* at(const BlkHeads& t, int64_t b, int64_t i, int64_t h) {
  return t.p + b * t.sb + i * t.st + h * t.sh;
}
__device__ __forceinline__ char* out_at(const BlkHeads& t, int64_t b, int64_t i, int64_t h) {
  return t.p + b * t.sb + i * t.st + h * t.sh;
}

// What a wave holds of its tile of rows, and one step of 32 keys.
template <typename T, int DKP, int DVP> struct FwdTile {
  Qfrag<T, DKP> q;
  float m = -__builtin_inff(), l = 0.f;  // running maximum (in units of log 2) and sum
  f32x4 acc[DVP / 16];

  __device__ FwdTile() {
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) acc[d] = zero4();
  }
  // keys k0 .. k0 + 31 for rows at position p (take: the row attends their block); keys behind
  // `last` have weight 0 in every row: zeroes stand in, whatever is there
  __device__ __forceinline__ void step(const BlkParams& P, int b, int h, int k0, int last, int p, bool take, char* vs, int lane) {
    const int r = lane & 15, a = lane >> 4, vw = P.dvw * (int)sizeof(T), kw = P.dkw * (int)sizeof(T);
    const float sc = P.scale * BLK_LOG2E;
    u32x4 kf[2][Qfrag<T, DKP>::N];  // under way before the values are waited for
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const char* kr = at(P.k, b, min(k0 + 16 * kt + r, P.S - 1), h);
#pragma unroll
      for (int c = 0; c < Qfrag<T, DKP>::N; ++c) kf[kt][c] = blk_ld(kr, 64 * c + 16 * a, kw);
    }
    __syncthreads();
    blk_stage<T, DVP, 64>(vs, BLK_KEYS, vw, lane, [&](int i) { return k0 + i <= last ? at(P.v, b, k0 + i, h) : nullptr; });
    float w[2][4];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      f32x4 s = zero4();
#pragma unroll
      for (int c = 0; c < Qfrag<T, DKP>::N; ++c) s = mma_slab<T>(kf[kt][c], q.f[c], s);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[kt][i] = take && k0 + 16 * kt + 4 * a + i <= p ? s[i] * sc : -__builtin_inff();
    }
    float mx = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(w[0][i], w[1][i]));
    mx = blk_quad_max(mx);
    const float ref = mx == -__builtin_inff() ? 0.f : mx;  // nothing to attend yet
    const float corr = __builtin_amdgcn_exp2f(m - ref);
    m = mx;
    l *= corr;
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[kt][i] = __builtin_amdgcn_exp2f(w[kt][i] - ref);
        l += w[kt][i];
      }
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) acc[d] *= corr;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < BLK_KEYS / blk_slab<T>(); ++s) {
      u32x4 x, lo;
      blk_split<T>(w, s, x, lo);
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d)
        acc[d] = blk_mma_split<T>(blk_column<T>(vs, blk_pitch<T, DVP>(), s * blk_slab<T>(), d, lane), x, lo, acc[d]);
    }
  }
  __device__ __forceinline__ void store(const BlkParams& P, const BlkRow& row, int64_t tile, int part, int lane) {
    const int r = lane & 15, a = lane >> 4;
    l = blk_quad_sum(l);
    if (!row.in) return;
    if (P.parts > 1) {
      const int64_t pr = (tile * P.parts + part) * BLK_ROWS + r;
      if (a == 0) {
        P.pm[2 * pr] = m;
        P.pm[2 * pr + 1] = l;
      }
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d) {
        const float v[4] = {acc[d][0], acc[d][1], acc[d][2], acc[d][3]};
        st16(P.po + pr * DVP + 16 * d + 4 * a, pack16<float>(v));
      }
      return;
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // no key: 0; a NaN stays
    char* o = out_at(P.o, row.b, row.i, row.head);
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) {
      const int c = 16 * d + 4 * a;
      const float v[4] = {acc[d][0] * inv, acc[d][1] * inv, acc[d][2] * inv, acc[d][3] * inv};
      if (c < P.dvw) blk_st4<T>(o + c * sizeof(T), v);
    }
    if (P.lse && a == 0)
      P.lse[((int64_t)row.b * P.Hq + row.head) * P.L + row.i] = l == 0.f ? -__builtin_inff() : m * BLK_LN2 + logf(l);
  }
};

template <typename T, int DKP, int DVP>
__global__ __launch_bounds__(64, 2) void k_block_forward(const BlkParams P) {
  __shared__ int lists[BLK_ROWS * BLK_LIST], raw[BLK_ROWS * BLK_MAX_SEL];
  __shared__ __attribute__((aligned(16))) char vs[BLK_KEYS * blk_pitch<T, DVP>()];
  const int lane = threadIdx.x, r = lane & 15;
  const int64_t tile = (int64_t)blockIdx.x / P.parts;
  const int part = (int)((int64_t)blockIdx.x - tile * P.parts);
  const BlkTile t(P, tile);
  const BlkRow row = t.row(P, r);
  blk_lists(P, t, lists, raw, lane);
  FwdTile<T, DKP, DVP> f;
  f.q.load(at(P.q, row.b, row.in ? row.i : 0, row.in ? row.head : 0), P.dkw * sizeof(T), lane, row.in);
  __syncthreads();
  const int* mine = lists + (row.i - t.i0) * BLK_LIST;
  int cur = row.in && row.p >= 0 ? *mine : BLK_END, seen = 0;
  int last = row.p;  // the tile's last position
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) last = max(last, __shfl_xor(last, o));
  for (;;) {
    const int j = blk_row_min(cur);
    if (j == BLK_END) break;
    const bool member = cur == j;
    if (member) cur = *++mine;
    const int first = j << P.lgT;
    for (int k0 = first; k0 < first + (1 << P.lgT) && k0 <= last; k0 += BLK_KEYS) {
      if (P.parts > 1 && seen++ % P.parts != part) continue;
      f.step(P, t.b, t.h, k0, last, row.p, member, vs, lane);
    }
  }
  f.store(P, row, tile, part, lane);
}

// One query a sequence (L = 1), its rows the heads of a group: unit u of 32 keys
// of its list goes to part u mod parts, found by scalar steps.  Four waves a SIMD
// hold all parts at once (128 sequences, 16 / 4 heads, the step: 76 us against 94
// at three).
template <typename T, int DKP, int DVP>
__global__ __launch_bounds__(64, sizeof(T) == 2 && DVP <= 128 ? 4 : 2) void k_block_decode(const BlkParams P) {
  __shared__ __attribute__((aligned(16))) char vs[BLK_KEYS * blk_pitch<T, DVP>()];
  const int lane = threadIdx.x;
  const int64_t tile = (int64_t)blockIdx.x / P.parts;
  const int part = (int)((int64_t)blockIdx.x - tile * P.parts);
  const BlkTile t(P, tile);
  const int mine = lane < P.n ? P.sel[((int64_t)t.b * P.Hkv + t.h) * P.n + lane] : -1;
  const BlkRow row = t.row(P, lane & 15);
  FwdTile<T, DKP, DVP> f;
  f.q.load(at(P.q, row.b, 0, row.in ? row.head : 0), P.dkw * sizeof(T), lane, row.in);
  const int last = __builtin_amdgcn_readfirstlane(blk_position(P, t.b, 0));  // the query's position
  if (last >= 0) {
    const int own = last >> P.lgT, lg_units = P.lgT - 5;
    int before = -1, chosen = 0;  // the rule of blk_chosen
    for (int e = 0; e < P.n; ++e) {
      const int j = __builtin_amdgcn_readlane(mine, e);
      if (j <= before || j > own) continue;
      before = j;
      for (int s = 0; s < 1 << lg_units; ++s) {
        const int k0 = (j << P.lgT) + BLK_KEYS * s;
        if (((chosen << lg_units) + s) % P.parts == part && k0 <= last) f.step(P, t.b, t.h, k0, last, row.p, true, vs, lane);
      }
      ++chosen;
    }
  }
  f.store(P, row, tile, part, lane);
}

// Joins a row's partial outputs.
template <typename T, int DVP> __global__ __launch_bounds__(64) void k_block_join(const BlkParams P) {
  const int64_t tile = blockIdx.x / BLK_ROWS;
  const int r = (int)(blockIdx.x % BLK_ROWS), lane = threadIdx.x;
  const BlkRow row = BlkTile(P, tile).row(P, r);
  if (!row.in) return;
  const int64_t pr = tile * P.parts * BLK_ROWS + r;
  float m = -__builtin_inff(), l = 0.f, o[DVP / 64];
#pragma unroll 4
  for (int k = 0; k < P.parts; ++k) m = fmaxf(m, P.pm[2 * (pr + k * BLK_ROWS)]);
  const float ref = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
  for (int d = 0; d < DVP / 64; ++d) o[d] = 0.f;
#pragma unroll 4
  for (int k = 0; k < P.parts; ++k) {
    const int64_t at = pr + k * BLK_ROWS;
    const float w = __builtin_amdgcn_exp2f(P.pm[2 * at] - ref);
    l += w * P.pm[2 * at + 1];
#pragma unroll
    for (int d = 0; d < DVP / 64; ++d) o[d] += w * P.po[at * DVP + 64 * d + lane];
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  T* out = reinterpret_cast<T*>(out_at(P.o, row.b, row.i, row.head));
#pragma unroll
  for (int d = 0; d < DVP / 64; ++d)
    if (64 * d + lane < P.dvw) out[64 * d + lane] = from_f32<T>(o[d] * inv);
  if (P.lse && lane == 0)
    P.lse[((int64_t)row.b * P.Hq + row.head) * P.L + row.i] = l == 0.f ? -__builtin_inff() : m * BLK_LN2 + logf(l);
}

// dq = scale sum_j p_j (do . v_j - delta) k_j, by the tiles, steps and parts of
// the forward; delta = do . o is the softmax's share.  For bf16 the weights'
// gradients go through the product as a sum of two bf16 values, and delta, which
// comes from the rounded output, is put right (without both, dq is off by 1.6
// times its own rounding): with e = sum_j p_j (do . v_j - delta), its error (the weights sum to 1),
// dq loses scale e sum_j p_j k_j, and delta + e is what dk and dv then use.
template <typename T, int DKP, int DVP> __global__ __launch_bounds__(64) void k_block_dq(const BlkParams P) {
  constexpr bool EXACT = sizeof(T) == 2;
  __shared__ int lists[BLK_ROWS * BLK_LIST], raw[BLK_ROWS * BLK_MAX_SEL];
  __shared__ __attribute__((aligned(16))) char ks[BLK_KEYS * blk_pitch<T, DKP>()];
  const int lane = threadIdx.x, r = lane & 15, a = lane >> 4;
  const int64_t tile = (int64_t)blockIdx.x / P.parts;
  const int part = (int)((int64_t)blockIdx.x - tile * P.parts);
  const BlkTile t(P, tile);
  const BlkRow row = t.row(P, r);
  blk_lists(P, t, lists, raw, lane);
  Qfrag<T, DKP> q;
  Qfrag<T, DVP> g;
  const int vw = P.dvw * (int)sizeof(T), kw = P.dkw * (int)sizeof(T);
  const bool live = row.in && row.p >= 0;
  q.load(at(P.q, row.b, live ? row.i : 0, live ? row.head : 0), kw, lane, live);
  g.load(at(P.dout, row.b, live ? row.i : 0, live ? row.head : 0), vw, lane, live);
  __syncthreads();
  const int* mine = lists + (row.i - t.i0) * BLK_LIST;
  int cur = live ? *mine : BLK_END, seen = 0;
  int last = row.p;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) last = max(last, __shfl_xor(last, o));
  const int64_t lr = ((int64_t)row.b * P.Hq + row.head) * P.L + row.i;
  const float lse = live ? P.lse_in[lr] * BLK_LOG2E : 0.f;
  float delta = 0.f;
  {
    Qfrag<T, DVP> o;
    o.load(at(P.o, row.b, live ? row.i : 0, live ? row.head : 0), vw, lane, live);
#pragma unroll
    for (int c = 0; c < Qfrag<T, DVP>::N; ++c) delta += blk_dot<T>(g.f[c], o.f[c]);
    delta = blk_quad_sum(delta);
  }
  if (live && a == 0 && part == 0) P.delta[lr] = delta;
  blk_clear_counts(P, lane, 64);
  f32x4 acc[DKP / 16], mean[EXACT ? DKP / 16 : 1];  // mean: sum_j p_j k_j
#pragma unroll
  for (int d = 0; d < DKP / 16; ++d) acc[d] = zero4();
#pragma unroll
  for (int d = 0; d < (EXACT ? DKP / 16 : 1); ++d) mean[d] = zero4();
  float off = 0.f;
  const float sc = P.scale * BLK_LOG2E;
  for (;;) {
    const int j = blk_row_min(cur);
    if (j == BLK_END) break;
    const bool member = cur == j;
    if (member) cur = *++mine;
    const int first = j << P.lgT;
    for (int k0 = first; k0 < first + (1 << P.lgT) && k0 <= last; k0 += BLK_KEYS) {
      if (P.parts > 1 && seen++ % P.parts != part) continue;
      __syncthreads();
      blk_stage<T, DKP, 64>(ks, BLK_KEYS, kw, lane, [&](int i) {
        return k0 + i <= last ? at(P.k, t.b, k0 + i, t.h) : nullptr;
      });
      __syncthreads();
      float w[2][4], ds[2][4];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const char* kr = ks + (16 * kt + r) * blk_pitch<T, DKP>();
        const char* vr = at(P.v, t.b, min(k0 + 16 * kt + r, P.S - 1), t.h);
        f32x4 s = zero4(), dp = zero4();
#pragma unroll
        for (int c = 0; c < Qfrag<T, DKP>::N; ++c) s = mma_slab<T>(ld16(kr + 64 * c + 16 * a), q.f[c], s);
#pragma unroll
        for (int c = 0; c < Qfrag<T, DVP>::N; ++c) dp = mma_slab<T>(blk_ld(vr, 64 * c + 16 * a, vw), g.f[c], dp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool on = member && k0 + 16 * kt + 4 * a + i <= row.p;
          w[kt][i] = on ? __builtin_amdgcn_exp2f(s[i] * sc - lse) : 0.f;
          ds[kt][i] = on ? w[kt][i] * (dp[i] - delta) : 0.f;
          off += ds[kt][i];
        }
      }
#pragma unroll
      for (int s = 0; s < BLK_KEYS / blk_slab<T>(); ++s) {
        u32x4 x, lo, y = zero16();
        blk_split<T>(ds, s, x, lo);
        if constexpr (EXACT) y = blk_pack<T>(w, s);
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) {
          const u32x4 f = blk_column<T>(ks, blk_pitch<T, DKP>(), s * blk_slab<T>(), d, lane);
          acc[d] = blk_mma_split<T>(f, x, lo, acc[d]);
          if constexpr (EXACT) mean[d] = mma_slab<T>(f, y, mean[d]);
        }
      }
    }
  }
  if (!row.in) return;
  off = EXACT ? blk_quad_sum(off) : 0.f;
  if (P.parts > 1) {
    const int64_t pr = (tile * P.parts + part) * BLK_ROWS + r;
    if (a == 0) P.pm[pr] = off;
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) {
      st16(P.po + pr * 2 * DKP + 16 * d + 4 * a, __builtin_bit_cast(u32x4, acc[d]));
      if constexpr (EXACT) st16(P.po + (pr * 2 + 1) * DKP + 16 * d + 4 * a, __builtin_bit_cast(u32x4, mean[d]));
    }
    return;
  }
  if (EXACT && live && a == 0) P.delta[lr] = delta + off;
  char* o = out_at(P.dq, row.b, row.i, row.head);
#pragma unroll
  for (int d = 0; d < DKP / 16; ++d) {
    const int c = 16 * d + 4 * a;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (acc[d][e] - (EXACT ? off * mean[EXACT ? d : 0][e] : 0.f)) * P.scale;
    if (c < P.dkw) blk_st4<T>(o + c * sizeof(T), v);
  }
}

// Joins a row's partial gradients.
template <typename T, int DKP> __global__ __launch_bounds__(64) void k_block_dq_join(const BlkParams P) {
  constexpr bool EXACT = sizeof(T) == 2;
  const int64_t tile = blockIdx.x / BLK_ROWS;
  const int r = (int)(blockIdx.x % BLK_ROWS), lane = threadIdx.x;
  const BlkRow row = BlkTile(P, tile).row(P, r);
  if (!row.in) return;
  const int64_t pr = tile * P.parts * BLK_ROWS + r;
  float off = 0.f, g[DKP / 64], m[DKP / 64];
#pragma unroll
  for (int d = 0; d < DKP / 64; ++d) g[d] = m[d] = 0.f;
#pragma unroll 4
  for (int k = 0; k < P.parts; ++k) {
    const int64_t at = pr + k * BLK_ROWS;
    off += P.pm[at];
#pragma unroll
    for (int d = 0; d < DKP / 64; ++d) {
      g[d] += P.po[at * 2 * DKP + 64 * d + lane];
      if (EXACT) m[d] += P.po[(at * 2 + 1) * DKP + 64 * d + lane];
    }
  }
  if (EXACT && row.p >= 0 && lane == 0) P.delta[((int64_t)row.b * P.Hq + row.head) * P.L + row.i] += off;
  T* out = reinterpret_cast<T*>(out_at(P.dq, row.b, row.i, row.head));
#pragma unroll
  for (int d = 0; d < DKP / 64; ++d)
    if (64 * d + lane < P.dkw) out[64 * d + lane] = from_f32<T>((g[d] - off * m[d]) * P.scale);
}

template <typename T, int DKP, int DVP> struct Run {
  static void forward(const BlkParams& P, hipStream_t st) {
    const dim3 grid((unsigned)(P.tiles * P.parts));
    if (P.L == 1) hipLaunchKernelGGL((k_block_decode<T, DKP, DVP>), grid, dim3(64), 0, st, P);
    else hipLaunchKernelGGL((k_block_forward<T, DKP, DVP>), grid, dim3(64), 0, st, P);
    if (P.parts > 1)
      hipLaunchKernelGGL((k_block_join<T, DVP>), dim3((unsigned)(P.tiles * BLK_ROWS)), dim3(64), 0, st, P);
  }
  static void dq(const BlkParams& P, hipStream_t st) {
    hipLaunchKernelGGL((k_block_dq<T, DKP, DVP>), dim3((unsigned)(P.tiles * P.parts)), dim3(64), 0, st, P);
    if (P.parts > 1)
      hipLaunchKernelGGL((k_block_dq_join<T, DKP>), dim3((unsigned)(P.tiles * BLK_ROWS)), dim3(64), 0, st, P);
  }
};

template <typename T, int DKP, class F> void by_dv(int dv, F f) {
  if (blk_dvp(dv) == 64) f(Run<T, DKP, 64>());
  else if (blk_dvp(dv) == 128) f(Run<T, DKP, 128>());
  else f(Run<T, DKP, 256>());
}
template <class F> void dispatch(const BlkParams& P, bool bf16_path, F f) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? by_dv<bf16, 64>(P.dvw, f) : by_dv<bf16, 128>(P.dvw, f);
  else k64 ? by_dv<float, 64>(P.dvw, f) : by_dv<float, 128>(P.dvw, f);
}

}  // namespace

hipError_t launch_block_forward(const BlkParams& P, bool bf16_path, hipStream_t st) {
  dispatch(P, bf16_path, [&](auto r) { r.forward(P, st); });
  return hipGetLastError();
}

hipError_t launch_block_dq(const BlkParams& P, bool bf16_path, hipStream_t st) {
  dispatch(P, bf16_path, [&](auto r) { r.dq(P, st); });
  return hipGetLastError();
}

}  // namespace msgla
