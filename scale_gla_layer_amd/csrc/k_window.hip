// Attention with a sliding window and first tokens that stay visible, forward, for
// many queries.  A query at position p attends the keys j <= p with j > p - window or
// j < n_sink:   o = softmax(scale q K^T) V.
//
// A workgroup takes tiles of 32 (query, head) rows, one a wave: neighbouring
// queries with all their heads of one key-value head, which share its keys, so
// that with groups of heads the tile's queries lie close together and few keys
// are outside of a row's own window.  It walks the units of KT keys that any of its
// rows attends, first those of the first tokens, then the window's, each copied once
// into one of two LDS stages while the other one is worked on.
//   Scores are formed transposed, S^T = K Q^T, whose result is the operand of
// O^T = V^T P^T: a row's values stay in two lanes, and a row's maximum takes one
// exchange.  One pass with a running maximum, which follows a row's true one only
// when that has grown by more than 8 in units of log 2 (weights stay below 2^8).
//   bf16 weights enter their product as two bf16 values each (16 bits; rounded once
// they put outputs 1.3 times as far off as the output's own rounding does), which
// makes three products of the formula's two.  Bound by the matrix cores: 0.95 PFLOP/s
// with those three at L = 16384, 8 / 2 heads of 128 and 256, window 4096 (a large
// library product takes 1.2), 0.74 at B = 8, L = 2048, 16 / 4 heads of 128, window 512.
// fp32: 0.10 of 0.154 at B = 4 of the latter (301 us).
//   Four waves, two workgroups a CU that take turns at the vector and the matrix
// instructions.  At the latter size, and for two sequences of 4096 with 32 / 8 heads of
// 128 and a window of 4096, that takes 122 and 416 us; with units of 32 keys 126 and 454, with
// three such workgroups a CU 119 and 448.  When the former took 128: eight waves with a barrier
// in common 140, units of 128 keys 240, and a wave that forms a tile's weights between the
// products of the one before it 149: it waits for every LDS read of its own.
#include "window_device.hpp"

namespace msgla {

namespace {

constexpr float GROWTH = 8.f;

template <typename T, int DKP, int DVP, int KT>
__global__ __launch_bounds__(64 * WIN_TILES, sizeof(T) == 4 && DVP == 256 ? 1 : 2) void k_window(const WinParams P) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, WAVES = WIN_TILES;
  constexpr int NK = DKP * ES / 32, NO = DVP / 32, TILES = KT / 32, SLABS = Weights<T>::SLABS;
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16;
  // variables of their own, so that reads of one need not wait for copies to another
  __shared__ __attribute__((aligned(1024))) char stage0[STAGE], stage1[STAGE];
  __shared__ int smin[WAVES], smax[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // an XCD takes neighbouring tiles, which share keys
  const int total = P.B * P.Hkv * P.tiles_per_seq, per = (total + N_XCD - 1) / N_XCD;
  const int w = remap_xcd(blockIdx.x, per);
  if (w >= total) return;
  const int bh = w / P.tiles_per_seq, t = w - bh * P.tiles_per_seq, b = bh / P.Hkv, h = bh - b * P.Hkv;
  const WinRow row(P, b, h, t, WIN_ROWS * wave + (lane & 31));
  const bool live = row.in && row.p >= 0;
  const int pmin = wave_min(live ? row.p : 0x7fffffff), pmax = wave_max(live ? row.p : -1);
  if (lane == 0) smin[wave] = pmin, smax[wave] = pmax;
  __syncthreads();
  int first = 0x7fffffff, last = -1;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) first = min(first, smin[i]), last = max(last, smax[i]);
  first = __builtin_amdgcn_readfirstlane(first);
  last = __builtin_amdgcn_readfirstlane(last);
  const int low = last < 0 ? 0 : max(0, first - P.window + 1);  // the first key of a window
  // units: [0, sinks), then from `from` on
  const int hi = last < 0 ? -1 : last / KT;
  const int sinks = min(hi + 1, (P.n_sink + KT - 1) / KT), from = max(sinks, low / KT);
  const int units = sinks + max(0, hi - from + 1);

  const int kw = P.dkw * ES, vw = P.dvw * ES;
  const UnitCopy<WK, KT, WAVES> kc(P.k.p + b * P.k.sb + h * P.k.sh, P.k.st, kw, wave, lane);
  const UnitCopy<WV, KT, WAVES> vc(P.v.p + b * P.v.sb + h * P.v.sh, P.v.st, vw, wave, lane);
  auto unit_key = [&](int u) { return (u < sinks ? u : from + u - sinks) * KT; };
  // the unit's rows; those that no row of the workgroup attends are replaced by one that is
  auto fetch = [&](int u, char* stage) {
    const int k0 = unit_key(u);
    if (k0 + KT - 1 <= last && (k0 >= low || k0 + KT <= P.n_sink) && kc.near() && vc.near()) {
      kc.whole(k0, stage, wave);
      vc.whole(k0, stage + KB, wave);
    } else {
      auto key = [&](int r) {
        const int j = k0 + r;
        return (int64_t)(j <= last && (j >= low || j < P.n_sink) ? j : last);
      };
      kc.chosen(kw, stage, wave, lane, key);
      vc.chosen(vw, stage + KB, wave, lane, key);
    }
  };
  if (units > 0) fetch(0, stage0);

  u32x4 q[NK];
  {
    const char* qr = win_at(P.q, b, live ? row.i : 0, live ? row.head : 0);
#pragma unroll
    for (int s = 0; s < NK; ++s) q[s] = live ? blk_ld(qr, 32 * s + 16 * h2, kw) : zero16();
  }
  f32x16 acc[NO];
#pragma unroll
  for (int d = 0; d < NO; ++d) acc[d] = zero_tile();
  float nref = 0.f, l = 0.f;             // minus the reference maximum, the sum
  const float sc = P.scale * BLK_LOG2E, per_sc = 1.f / sc;
  float grown = -__builtin_inff();       // a score above this moves the reference
  const Rows32<WK> krow(lane);
  const Columns32<T, WV> col(lane);
  const int wlow = pmin - P.window + 1;  // the wave's first window's first key
  const int rlow = row.p - P.window;     // keys behind this are in the row's window

  auto unit = [&](int u, char* stage, char* next) {
    if (u + 1 < units) fetch(u + 1, next);
    const int k0 = unit_key(u);
    const char* vs = stage + KB;
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
      const int j0 = k0 + 32 * x;
      // a tile that none of the wave's rows attends
      if (j0 > pmax || (j0 + 31 < wlow && j0 >= P.n_sink)) continue;
      f32x16 s = zero_tile();
#pragma unroll
      for (int c = 0; c < NK; ++c) s = mma32<T>(krow.read(stage, x, c), q[c], s);
      if (win_edge(P, j0, 32, pmin, pmax)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = j0 + 8 * (i >> 2) + 4 * h2 + (i & 3);
          s[i] = win_out_of(P, j, row.p, rlow) ? -__builtin_inff() : s[i];
        }
      }
      float mx = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
      if (__any(mx > grown)) {
        const float m = grown == -__builtin_inff() ? grown : -nref;  // nothing yet: minus infinity
        const float top = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)) * sc);
        if (top != -__builtin_inff()) {
          const float corr = __builtin_amdgcn_exp2f(m - top);
          nref = -top;
          grown = (top + GROWTH) * per_sc;
          l *= corr;
#pragma unroll
          for (int d = 0; d < NO; ++d) acc[d] *= corr;
        }
      }
      Weights<T> wt;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], sc, nref));
        const float c = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], sc, nref));
        l += a;
        l += c;
        wt.set(i, a, c);
      }
#pragma unroll
      for (int c = 0; c < SLABS; ++c)
#pragma unroll
        for (int d = 0; d < NO; ++d) acc[d] = wt.mma(col.read(vs, x * SLABS + c, d), c, acc[d]);
    }
    __syncthreads();
  };
  __syncthreads();
  for (int u = 0; u < units; u += 2) {
    unit(u, stage0, stage1);
    if (u + 1 < units) unit(u + 1, stage1, stage0);
  }
  l += __shfl_xor(l, 32);
  if (!row.in) return;
  char* out = win_out(P.o, b, row.i, row.head);
  const float mul = l > 0.f ? 1.f / l : l;  // a NaN stays
#pragma unroll
  for (int d = 0; d < NO; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = win_column(d, i, lane);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = live ? acc[d][4 * i + e] * mul : 0.f;
      if (c < P.dvw) blk_st4<T>(out + c * ES, v);
    }
  if (P.lse && h2 == 0)
    P.lse[((int64_t)b * P.Hq + row.head) * P.L + row.i] = live ? logf(l) - nref * BLK_LN2 : -__builtin_inff();
}

// Keys of a unit: 64 for bf16 values of up to 128, whose two stages leave LDS for two
// workgroups a CU, and 32 elsewhere.
template <typename T, int DKP, int DVP> void launch_t(const WinParams& P, hipStream_t st) {
  constexpr int KT = sizeof(T) == 2 && DVP <= 128 ? 64 : 32;
  const int64_t total = (int64_t)P.B * P.Hkv * P.tiles_per_seq;
  hipLaunchKernelGGL((k_window<T, DKP, DVP, KT>), dim3((unsigned)((total + N_XCD - 1) / N_XCD * N_XCD)),
                     dim3(64 * WIN_TILES), 0, st, P);
}
template <typename T, int DKP> void by_dv(const WinParams& P, hipStream_t st) {
  if (win_dvp(P.dvw) == 64) launch_t<T, DKP, 64>(P, st);
  else if (win_dvp(P.dvw) == 128) launch_t<T, DKP, 128>(P, st);
  else launch_t<T, DKP, 256>(P, st);
}

}  // namespace

hipError_t launch_window(const WinParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = win_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? by_dv<bf16, 64>(P, st) : by_dv<bf16, 128>(P, st);
  else k64 ? by_dv<float, 64>(P, st) : by_dv<float, 128>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
