// Gradient of the queries of the window attention:
//   dq = scale sum_j p_j (do . v_j - delta) k_j,   delta = do . o.
//
// The forward's tiles and units, 32 keys each, and three products: S^T = K Q^T,
// dP^T = V dO^T and dQ^T = K^T dS^T.  A pair of waves shares a tile of rows, which
// halves what each keeps in registers, so that two waves share a SIMD: the first one
// forms the weights and leaves them in LDS, the second one, a unit behind, their
// gradients and dQ.
//   bf16: the weights' gradients enter their product as two bf16 values each, and
// delta, which inherits the rounding of the stored o, is put right: with e =
// sum_j p_j (do . v_j - delta), its error (the weights sum to 1), dq loses scale e
// sum_j p_j k_j, a sum that the first wave forms beside its weights, and delta + e is
// what dk and dv then use: five products.
//   Bound by LDS reads (1.1 KB for each matrix instruction, counted, where a CU delivers 1
// in the time of one on each SIMD) and the matrix cores: 2 x 16 / 4 heads of 128, 4096 positions,
// window 1024 take 181 us in a long run of calls, 215 in a short one (a wave that does
// it all 246, workgroups of one pair 281).  fp32, 2 x 2048, window 512: 245.
#include "window_device.hpp"

namespace msgla {

namespace {

template <typename T, int DKP, int DVP, int PAIRS>
__global__ __launch_bounds__(128 * PAIRS, PAIRS == 4 ? 2 : 1) void k_window_dq(const WinParams P) {
  constexpr int KT = 32, ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, WAVES = 2 * PAIRS;
  constexpr int NK = DKP * ES / 32, NV = DVP * ES / 32, NO = DKP / 32;
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16;
  // variables of their own, so that reads of one need not wait for copies to another
  __shared__ __attribute__((aligned(1024))) char stage0[STAGE], stage1[STAGE], stage2[STAGE];
  __shared__ __attribute__((aligned(16))) char weights[2][PAIRS][TILE_BYTES];
  __shared__ int smin[WAVES], smax[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // an XCD takes neighbouring tiles, which share keys
  const int total = P.B * P.Hkv * P.tiles_per_seq, per = (total + N_XCD - 1) / N_XCD;
  const int w = remap_xcd(blockIdx.x, per);
  if (w >= total) return;
  const int bh = w / P.tiles_per_seq, t = w - bh * P.tiles_per_seq, b = bh / P.Hkv, h = bh - b * P.Hkv;
  const int pair = wave % PAIRS;
  const WinRow row(P, b, h, t, WIN_ROWS * pair + (lane & 31));
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
  auto fetch = [&](int u, char* stage) __attribute__((always_inline)) {
    const int k0 = unit_key(u);
    if (k0 + KT - 1 <= last && (k0 >= low || k0 + KT <= P.n_sink) && kc.near() && vc.near()) {
      kc.whole(k0, stage, wave);
      vc.whole(k0, stage + KB, wave);
    } else {
      auto key = [&](int r) __attribute__((always_inline)) {
        const int j = k0 + r;
        return (int64_t)(j <= last && (j >= low || j < P.n_sink) ? j : last);
      };
      kc.chosen(kw, stage, wave, lane, key);
      vc.chosen(vw, stage + KB, wave, lane, key);
    }
  };
  if (units > 0) fetch(0, stage0);

  constexpr bool EXACT = ES == 2;  // delta put right
  const int64_t li = live ? row.i : 0, hd = live ? row.head : 0, lr = ((int64_t)b * P.Hq + hd) * P.L + li;
  const float nref = live ? -P.lse_in[lr] * BLK_LOG2E : 0.f, sc = P.scale * BLK_LOG2E;
  const Rows32<WK> krow(lane);
  const Rows32<WV> vrow(lane);
  const Columns32<T, WK> col(lane);
  const int wlow = pmin - P.window + 1;  // the tile's first window's first key
  const int rlow = row.p - P.window;     // keys behind this are in the row's window
  f32x16 acc[NO];                        // sum_j p_j k_j, or dq
#pragma unroll
  for (int d = 0; d < NO; ++d) acc[d] = zero_tile();
  // work(u, stage) for each unit, `lag` units behind the copies, that some of the tile's rows attend
  auto walk = [&](auto lag, auto work) __attribute__((always_inline)) {
    auto one = [&](int u, const char* stage) __attribute__((always_inline)) {
      const int j0 = unit_key(u);
      if (j0 <= pmax && (j0 + 31 >= wlow || j0 < P.n_sink)) {
        work(u, j0, stage);
        if constexpr (PAIRS == 1) products_done();
      }
    };
    auto unit = [&](int u, const char* stage, const char* before, char* next) __attribute__((always_inline)) {
      if (u > units) return;
      if (u + 1 < units) fetch(u + 1, next);
      if constexpr (lag() == 0) {
        if (u < units) one(u, stage);
      } else {
        if (u > 0) one(u - 1, before);
      }
      __syncthreads();
    };
    __syncthreads();
    for (int u = 0; u <= units; u += 3) {
      unit(u, stage0, stage2, stage1);
      unit(u + 1, stage1, stage0, stage2);
      unit(u + 2, stage2, stage1, stage0);
    }
  };

  if (wave < PAIRS) {  // the weights
    u32x4 q[NK];
    const char* qr = win_at(P.q, b, li, hd);
#pragma unroll
    for (int s = 0; s < NK; ++s) q[s] = live ? blk_ld(qr, 32 * s + 16 * h2, kw) : zero16();
    walk(std::integral_constant<int, 0>(), [&](int u, int j0, const char* ks) __attribute__((always_inline)) {
      f32x16 s = zero_tile();
#pragma unroll
      for (int c = 0; c < NK; ++c) s = mma32<T>(krow.read(ks, 0, c), q[c], s);
      if (win_edge(P, j0, 32, pmin, pmax)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = j0 + 8 * (i >> 2) + 4 * h2 + (i & 3);
          s[i] = win_out_of(P, j, row.p, rlow) ? -__builtin_inff() : s[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], sc, nref));
      tile_put(weights[u & 1][pair], s, lane);
      if constexpr (EXACT) {
        Weights<T> wt;
#pragma unroll
        for (int i = 0; i < 8; ++i) wt.set_hi(i, s[2 * i], s[2 * i + 1]);
#pragma unroll
        for (int c = 0; c < Weights<T>::SLABS; ++c)
#pragma unroll
          for (int d = 0; d < NO; ++d) acc[d] = wt.mma_hi(col.read(ks, c, d), c, acc[d]);
      }
    });
    if constexpr (EXACT) {
#pragma unroll
      for (int d = 0; d < NO; d += 2) {
        tile_put(weights[0][pair], acc[d], lane);
        tile_put(weights[1][pair], acc[d + 1], lane);
        __syncthreads();
        __syncthreads();
      }
    }
    return;
  }
  // their gradients and dq
  u32x4 g[NV];
  float delta = 0.f, off = 0.f;
  {
    const char *gr = win_at(P.dout, b, li, hd), *orow = win_at(P.o, b, li, hd);
#pragma unroll
    for (int s = 0; s < NV; ++s) g[s] = live ? blk_ld(gr, 32 * s + 16 * h2, vw) : zero16();
#pragma unroll
    for (int s = 0; s < NV; ++s) delta += blk_dot<T>(g[s], live ? blk_ld(orow, 32 * s + 16 * h2, vw) : zero16());
    delta += __shfl_xor(delta, 32);
  }
  walk(std::integral_constant<int, 1>(), [&](int u, int, const char* ks) __attribute__((always_inline)) {
    f32x16 dp = zero_tile();
#pragma unroll
    for (int c = 0; c < NV; ++c) dp = mma32<T>(vrow.read(ks + KB, 0, c), g[c], dp);
    const f32x16 p = tile_get(weights[u & 1][pair], lane);
    Weights<T> ds;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = p[2 * i] * (dp[2 * i] - delta), c = p[2 * i + 1] * (dp[2 * i + 1] - delta);
      if constexpr (EXACT) off += a + c;
      ds.set(i, a, c);
    }
#pragma unroll
    for (int c = 0; c < Weights<T>::SLABS; ++c)
#pragma unroll
      for (int d = 0; d < NO; ++d) acc[d] = ds.mma(col.read(ks, c, d), c, acc[d]);
  });
  if constexpr (EXACT) {
    off += __shfl_xor(off, 32);
#pragma unroll
    for (int d = 0; d < NO; d += 2) {
      __syncthreads();
      acc[d] -= tile_get(weights[0][pair], lane) * off;
      acc[d + 1] -= tile_get(weights[1][pair], lane) * off;
      __syncthreads();
    }
  }
  if (!row.in) return;
  if (live && h2 == 0) P.delta[lr] = delta + off, P.nref[lr] = nref;
  char* out = win_out(P.dq, b, row.i, row.head);
#pragma unroll
  for (int d = 0; d < NO; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = win_column(d, i, lane);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = live ? acc[d][4 * i + e] * P.scale : 0.f;
      if (c < P.dkw) blk_st4<T>(out + c * ES, v);
    }
}

template <typename T, int DKP, int DVP> void launch_t(const WinParams& P, hipStream_t st) {
  const int64_t total = (int64_t)P.B * P.Hkv * P.tiles_per_seq;
  hipLaunchKernelGGL((k_window_dq<T, DKP, DVP, win_pairs(sizeof(T), DVP)>), dim3((unsigned)((total + N_XCD - 1) / N_XCD * N_XCD)),
                     dim3(128 * win_pairs(sizeof(T), DVP)), 0, st, P);
}
template <typename T, int DKP> void by_dv(const WinParams& P, hipStream_t st) {
  if (win_dvp(P.dvw) == 64) launch_t<T, DKP, 64>(P, st);
  else if (win_dvp(P.dvw) == 128) launch_t<T, DKP, 128>(P, st);
  else launch_t<T, DKP, 256>(P, st);
}

}  // namespace

hipError_t launch_window_dq(const WinParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = win_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? by_dv<bf16, 64>(P, st) : by_dv<bf16, 128>(P, st);
  else k64 ? by_dv<float, 64>(P, st) : by_dv<float, 128>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
