// Attention with a sliding window and first tokens that stay visible, for many
// queries: forward, and the gradient of the queries.  A query at position p
// attends the keys j <= p with j > p - window or j < n_sink:
//   o = softmax(scale q K^T) V,   dq = scale sum_j p_j (do . v_j - delta) k_j
//
// A workgroup takes tiles of 32 (query, head) rows, one a wave: neighbouring
// queries with all their heads of one key-value head, which share its keys, so
// that with groups of heads the tile's queries lie close together and few keys
// are outside of a row's own window.  It walks the units of KT keys that any of its
// rows attends, first those of the first tokens, then the window's; each unit is
// copied once into one of two LDS stages while the other is worked on.  One pass
// with a running maximum, which follows a row's true one only when that has grown
// by more than 8 in units of log 2 (weights stay below 2^8).
//   Scores are formed transposed, S^T = K Q^T, whose result is the operand of
// O^T = V^T P^T: a row's values stay in two lanes, and a row's maximum takes one
// exchange.  Only units at the window's edges are masked.
//   bf16: softmax weights and their gradients enter their products as two bf16
// values each (16 bits; rounded once they put outputs 1.3 times as far off as the
// output's own rounding does).  delta = do . o inherits the rounding of o and is put
// right: e = sum_j p_j (do . v_j - delta) is its error (the weights sum to 1), dq
// loses scale e sum_j p_j k_j, and delta + e is what dk and dv then use.
#include "window_device.hpp"

namespace msgla {

namespace {

constexpr float GROWTH = 8.f;

template <typename T, int DKP, int DVP, int KT, bool GRAD>
__global__ __launch_bounds__(64 * win_waves(sizeof(T), DKP, DVP, GRAD), win_waves(sizeof(T), DKP, DVP, GRAD) / 4) void k_window(const WinParams P) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, WAVES = win_waves(ES, DKP, DVP, GRAD), THREADS = 64 * WAVES;
  constexpr int NK = DKP * ES / 32, NV = DVP * ES / 32, TILES = KT / 32, SLABS = 32 / win_slab<T>();
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16;
  constexpr int CK = (KT * WK + THREADS - 1) / THREADS, CV = (KT * WV + THREADS - 1) / THREADS;  // pieces a thread copies
  constexpr int OUT = GRAD ? DKP : DVP;    // width of the accumulated rows
  constexpr bool EXACT = GRAD && ES == 2;  // delta put right
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];
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
  const char *kb = P.k.p + b * P.k.sb + h * P.k.sh, *vb = P.v.p + b * P.v.sb + h * P.v.sh;
  u32x4 kr[CK], vr[CV];
  // the unit's rows; those that no row of the workgroup attends are replaced by one that is
  auto fetch = [&](int u) {
    const int k0 = (u < sinks ? u : from + u - sinks) * KT;
    auto key = [&](int r) {
      const int j = k0 + r;
      return j <= last && (j >= low || j < P.n_sink) ? j : last;
    };
#pragma unroll
    for (int i = 0; i < CK; ++i) {
      const int p = tid + THREADS * i, r = p / WK, at = p % WK * 16;
      if (KT * WK % THREADS == 0 || r < KT) kr[i] = blk_ld(kb + key(r) * P.k.st, at, kw);
    }
#pragma unroll
    for (int i = 0; i < CV; ++i) {
      const int p = tid + THREADS * i, r = p / WV, at = p % WV * 16;
      if (KT * WV % THREADS == 0 || r < KT) vr[i] = blk_ld(vb + key(r) * P.v.st, at, vw);
    }
  };
  auto put = [&](char* st) {
#pragma unroll
    for (int i = 0; i < CK; ++i) {
      const int p = tid + THREADS * i, r = p / WK;
      if (KT * WK % THREADS == 0 || r < KT) st16(st + (r * WK + ((p % WK) ^ tile_key<WK>(r))) * 16, kr[i]);
    }
#pragma unroll
    for (int i = 0; i < CV; ++i) {
      const int p = tid + THREADS * i, r = p / WV;
      if (KT * WV % THREADS == 0 || r < KT) st16(st + KB + (r * WV + ((p % WV) ^ tile_key<WV>(r))) * 16, vr[i]);
    }
  };
  if (units > 0) fetch(0);

  u32x4 q[NK], g[GRAD ? NV : 1];
  float nref = 0.f, l = 0.f;  // forward: minus the reference maximum, the sum; gradient: minus lse, delta
  const int64_t li = live ? row.i : 0, hd = live ? row.head : 0, lr = ((int64_t)b * P.Hq + hd) * P.L + li;
  {
    const char* qr = win_at(P.q, b, li, hd);
#pragma unroll
    for (int s = 0; s < NK; ++s) q[s] = live ? blk_ld(qr, 32 * s + 16 * h2, kw) : zero16();
    if constexpr (GRAD) {
      const char *gr = win_at(P.dout, b, li, hd), *orow = win_at(P.o, b, li, hd);
#pragma unroll
      for (int s = 0; s < NV; ++s) g[s] = live ? blk_ld(gr, 32 * s + 16 * h2, vw) : zero16();
      nref = live ? -P.lse_in[lr] * BLK_LOG2E : 0.f;
#pragma unroll
      for (int s = 0; s < NV; ++s) l += blk_dot<T>(g[s], live ? blk_ld(orow, 32 * s + 16 * h2, vw) : zero16());
      l += __shfl_xor(l, 32);
    }
  }
  f32x16 acc[OUT / 32], mean[EXACT ? OUT / 32 : 1];  // mean: sum_j p_j k_j
#pragma unroll
  for (int d = 0; d < OUT / 32; ++d) acc[d] = zero_tile();
#pragma unroll
  for (int d = 0; d < (EXACT ? OUT / 32 : 1); ++d) mean[d] = zero_tile();
  float off = 0.f;
  const float sc = P.scale * BLK_LOG2E, per_sc = 1.f / sc;
  float grown = -__builtin_inff();  // a score above this moves the reference
  const Rows32<WK> krow(lane);
  const Rows32<WV> vrow(lane);
  const Columns32<T, GRAD ? WK : WV> col(lane);
  const int wlow = pmin - P.window + 1;  // the wave's first window's first key
  const int rlow = row.p - P.window;     // keys behind this are in the row's window

  if (units > 0) put(smem);
  if (units > 1) fetch(1);
  __syncthreads();
  for (int u = 0; u < units; ++u) {
    const int k0 = (u < sinks ? u : from + u - sinks) * KT;
    const char *ks = smem + (u & 1) * STAGE, *vs = ks + KB;
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
      const int j0 = k0 + 32 * x;
      // a tile that none of the wave's rows attends
      if (j0 > pmax || (j0 + 31 < wlow && j0 >= P.n_sink)) continue;
      f32x16 s = zero_tile();
#pragma unroll
      for (int c = 0; c < NK; ++c) s = mma32<T>(krow.read(ks, x, c), q[c], s);
      if (j0 + 31 > pmin || (j0 <= pmax - P.window && j0 + 32 > P.n_sink)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = j0 + 8 * (i >> 2) + 4 * h2 + (i & 3);
          if (j > row.p || (j <= rlow && j >= P.n_sink)) s[i] = -__builtin_inff();
        }
      }
      f32x16 wt;
      if constexpr (!GRAD) {
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
            for (int d = 0; d < OUT / 32; ++d) acc[d] *= corr;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], sc, nref));
          l += s[i];
        }
      } else {
        f32x16 dp = zero_tile();
#pragma unroll
        for (int c = 0; c < NV; ++c) dp = mma32<T>(vrow.read(vs, x, c), g[c], dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], sc, nref));
          wt[i] = p;
          s[i] = p * (dp[i] - l);
          if constexpr (EXACT) off += s[i];
        }
      }
#pragma unroll
      for (int c = 0; c < SLABS; ++c) {
        u32x4 hi_, lo_, y = zero16();
        win_split<T>(s, c, hi_, lo_);
        if constexpr (EXACT) y = win_pack<T>(wt, c);
#pragma unroll
        for (int d = 0; d < OUT / 32; ++d) {
          const u32x4 f = col.read(GRAD ? ks : vs, x * SLABS + c, d);
          acc[d] = mma32<T>(f, hi_, acc[d]);
          if constexpr (ES == 2) acc[d] = mma32<T>(f, lo_, acc[d]);
          if constexpr (EXACT) mean[d] = mma32<T>(f, y, mean[d]);
        }
      }
    }
    if (u + 1 < units) put(smem + ((u + 1) & 1) * STAGE);
    if (u + 2 < units) fetch(u + 2);
    __syncthreads();
  }
  if constexpr (!GRAD) l += __shfl_xor(l, 32);
  if constexpr (EXACT) {
    off += __shfl_xor(off, 32);
#pragma unroll
    for (int d = 0; d < OUT / 32; ++d) acc[d] -= mean[d] * off;
  }
  if (!row.in) return;
  if (GRAD && live && h2 == 0) P.delta[lr] = l + off;
  char* out = win_out(GRAD ? P.dq : P.o, b, row.i, row.head);
  const int width = GRAD ? P.dkw : P.dvw;
  // a row without a key is 0; a NaN stays
  const float mul = !live ? 0.f : GRAD ? P.scale : l > 0.f ? 1.f / l : l;
#pragma unroll
  for (int d = 0; d < OUT / 32; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = win_column(d, i, lane);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = live ? acc[d][4 * i + e] * mul : 0.f;
      if (c < width) blk_st4<T>(out + c * ES, v);
    }
  if (!GRAD && P.lse && h2 == 0)
    P.lse[((int64_t)b * P.Hq + row.head) * P.L + row.i] = live ? logf(l) - nref * BLK_LN2 : -__builtin_inff();
}

// Keys of a unit: as many as two stages of LDS and the registers leave room for.
template <typename T, int DKP, int DVP, bool GRAD> void launch_t(const WinParams& P, hipStream_t st) {
  constexpr int KT = !GRAD && sizeof(T) == 2 && DKP + DVP <= 256 ? 64 : 32;
  const int64_t total = (int64_t)P.B * P.Hkv * P.tiles_per_seq;
  hipLaunchKernelGGL((k_window<T, DKP, DVP, KT, GRAD>), dim3((unsigned)((total + N_XCD - 1) / N_XCD * N_XCD)),
                     dim3(64 * win_waves(sizeof(T), DKP, DVP, GRAD)), 0, st, P);
}
template <typename T, int DKP, bool GRAD> void by_dv(const WinParams& P, hipStream_t st) {
  if (win_dvp(P.dvw) == 64) launch_t<T, DKP, 64, GRAD>(P, st);
  else if (win_dvp(P.dvw) == 128) launch_t<T, DKP, 128, GRAD>(P, st);
  else launch_t<T, DKP, 256, GRAD>(P, st);
}
template <bool GRAD> void dispatch(const WinParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = win_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? by_dv<bf16, 64, GRAD>(P, st) : by_dv<bf16, 128, GRAD>(P, st);
  else k64 ? by_dv<float, 64, GRAD>(P, st) : by_dv<float, 128, GRAD>(P, st);
}

}  // namespace

hipError_t launch_window(const WinParams& P, bool gradient, bool bf16_path, hipStream_t st) {
  gradient ? dispatch<true>(P, bf16_path, st) : dispatch<false>(P, bf16_path, st);
  return hipGetLastError();
}

}  // namespace msgla
