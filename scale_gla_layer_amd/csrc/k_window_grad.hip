// Gradients of the keys and values of the window attention:
//   dv_j = sum over the rows that attend j of p_ij do_i,   dk_j = scale sum of p_ij (do_i . v_j - delta_i) q_i.
//
// A workgroup keeps 128 keys and values and their gradients in registers, 32 a pair
// of waves, and streams through the (query, head) rows whose windows hold any of
// them, sets of 32 that copies bring into LDS stages.  A pair's first wave forms the
// weights, leaves them in LDS and adds to dv, the second one, a set behind, forms the
// weights' gradients and adds to dk: each keeps half of what both need, and two waves
// share a SIMD.  First tokens are attended by all later queries as well: the rows
// beyond their windows are walked by workgroups of one pair that holds 32 first
// tokens.  Few key tiles are dealt to several workgroups by their rows.  Such partial
// sums a last kernel adds in order: the result does not vary from call to call.
//   Scores are formed as S = Q K^T, whose result is the operand of dV^T = dO^T P
// and dK^T = Q^T dS.  bf16 weights and their gradients enter these as two bf16 values
// each, as in the other kernels: six products.  2 x 16 / 4 heads of 128, 4096
// positions, window 1024: 235 us in a long run of calls, 283 in a short one (a wave
// that does it all 470, workgroups of one pair 393), first tokens 21, joining 5.  fp32,
// 2 x 2048, window 512: 343, 51 and 16; its instances of 128 values keep 4 or 5 registers
// in scratch memory.
#include "window_device.hpp"

namespace msgla {

namespace {

// The (query, head) rows that a workgroup walks: queries from i0 on, all G heads of
// each.  x / G for x below G + 32 by a product: 2^22 / G, rounded up.
struct Walk {
  int G;
  uint32_t inv;
  __device__ explicit Walk(int g) : G(g), inv((1u << 22) / g + 1) {}
  __device__ __forceinline__ int div(int x) const { return (int)(((uint32_t)x * inv) >> 22); }
};

// Copies of sets of 32 rows of W pieces; rows behind the last one repeat it.
template <int W, int WAVES> struct SetCopy {
  static constexpr int ALL = 32 * W / 64, N = (ALL + WAVES - 1) / WAVES;
  const char* base;  // of the first query and head
  int64_t st, sh;
  uint32_t off[N];   // from a set's first query, where a set is whole queries
  bool even;
  __device__ SetCopy(const char* b, const WinHeads& t, int G, int width, int wave, int lane) : base(b), st(t.st), sh(t.sh) {
    even = 32 % G == 0 && st <= 0x3fffffff / 32 && sh <= 0x3fffffff / 32;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = 64 * (wave + WAVES * i) + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r), qi = r / G;
      off[i] = (uint32_t)qi * (uint32_t)st + (uint32_t)(r - qi * G) * (uint32_t)sh + (p * 16 < width ? p * 16 : 0);
    }
  }
  // set `set`, whose first row is head rem of query q0; `rows` in all
  __device__ __forceinline__ void issue(const Walk& w, int64_t set, int64_t q0, int rem, int64_t rows, int width, char* lds, int wave, int lane) const {
    if (even && set * 32 + 32 <= rows) {
      const char* first = base + q0 * st;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (ALL % WAVES == 0 || wave + WAVES * i < ALL) dma16(first + off[i], lds + 1024 * (wave + WAVES * i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int pc = 64 * (wave + WAVES * i) + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
        const int x = rem + (int)min((int64_t)r, rows - 1 - set * 32), qi = w.div(x);
        if (ALL % WAVES == 0 || wave + WAVES * i < ALL)
          dma16(base + (q0 + qi) * st + (x - qi * w.G) * sh + (p * 16 < width ? p * 16 : 0), lds + 1024 * (wave + WAVES * i));
      }
    }
  }
};

__device__ __forceinline__ void dma4(const void* g, void* lds) {
  __builtin_amdgcn_global_load_lds(g, (lds_void_t*)lds, 4, 0, 0);
}

template <typename T, int DKP, int DVP, int PAIRS, bool SINK>
__global__ __launch_bounds__(128 * PAIRS, PAIRS == 4 ? 2 : 1) void k_window_dkdv(const WinParams P) {
  constexpr int KEYS = 32 * PAIRS, WAVES = 2 * PAIRS, ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, NK = DKP * ES / 32, NV = DVP * ES / 32;
  constexpr int QB = 32 * WK * 16, GB = 32 * WV * 16, SET = QB + GB + 256;  // q, do, nref and delta
  // variables of their own, so that reads of one need not wait for copies to another
  __shared__ __attribute__((aligned(1024))) char stage0[SET], stage1[SET], stage2[SET];
  __shared__ __attribute__((aligned(16))) char weights[2][PAIRS][TILE_BYTES];
  const int tid = threadIdx.x, lane = tid & 63, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), pair = wave % PAIRS;
  const int tiles = SINK ? P.sink_tiles : P.key_tiles, parts = SINK ? P.sink_parts : P.key_parts;
  const int total = P.B * P.Hkv * tiles * parts, per = (total + N_XCD - 1) / N_XCD;
  const int w = remap_xcd(blockIdx.x, per);
  if (w >= total) return;
  const int part = w % parts, tile = w / parts % tiles, bh = w / parts / tiles, b = bh / P.Hkv, h = bh - b * P.Hkv;
  const int k0 = tile * KEYS + 32 * pair;
  const int key = k0 + (lane & 31);
  const int len = P.lens ? max(0, min(P.lens[b], P.S)) : P.S;
  const int64_t start = P.start ? P.start[b] : 0;
  // positions of the rows: those whose windows hold one of the keys, or those behind the first key's window
  const int64_t p0 = SINK ? (int64_t)k0 + P.window : (int64_t)tile * KEYS;
  const int64_t p1 = SINK ? len : min((int64_t)len, p0 + KEYS - 1 + P.window);
  const int64_t i0 = max((int64_t)0, p0 - start), i1 = min((int64_t)P.L, p1 - start);
  const int64_t rows = i1 > i0 ? (i1 - i0) * P.G : 0, sets = (rows + 31) / 32;
  const int64_t begin = sets * part / parts, end = sets * (part + 1) / parts;
  const Walk walk(P.G);

  const int kw = P.dkw * ES, vw = P.dvw * ES;
  const int64_t at0 = rows > 0 ? i0 : 0;
  const SetCopy<WK, WAVES> qc(win_at(P.q, b, at0, h * P.G), P.q, P.G, kw, wave, lane);
  const SetCopy<WV, WAVES> gc(win_at(P.dout, b, at0, h * P.G), P.dout, P.G, vw, wave, lane);
  const float* stats = (lane < 32 ? P.nref : P.delta) + ((int64_t)b * P.Hq + h * P.G) * P.L + at0;
  auto fetch = [&](int64_t set, char* to) __attribute__((always_inline)) {
    const int64_t q0 = set * 32 / P.G;
    const int rem = (int)(set * 32 - q0 * P.G);
    qc.issue(walk, set, q0, rem, rows, kw, to, wave, lane);
    gc.issue(walk, set, q0, rem, rows, vw, to + QB, wave, lane);
    if (wave == 0) {
      const int x = rem + (int)min((int64_t)(lane & 31), rows - 1 - set * 32), qi = walk.div(x);
      dma4(stats + (int64_t)(x - qi * P.G) * P.L + q0 + qi, to + QB + GB);
    }
  };
  if (begin < end) fetch(begin, stage0);

  // whether any row attends the key: what others hold is not used
  const int64_t to_last = min((int64_t)len, start + P.L) - 1;
  const bool is_key = SINK ? key < P.n_sink && max((int64_t)key + P.window, start) <= to_last
                           : max((int64_t)key, start) <= min((int64_t)key + P.window - 1, to_last);
  const float sc = P.scale * BLK_LOG2E;
  const Rows32<WK> qrow(lane);
  const Rows32<WV> grow(lane);
  const Columns32<T, WK> qcol(lane);
  const Columns32<T, WV> gcol(lane);

  // Where a set stands: positions of its first and last row, and the first one's head.
  struct Set {
    int64_t pa, pb;
    int rem;
  };
  // work(set, place, stage) for each set, `lag` sets behind the copies, of which any row holds any of the pair's keys
  auto stream = [&](auto lag, auto work) __attribute__((always_inline)) {
    auto one = [&](int64_t set, const char* stage) __attribute__((always_inline)) {
      const int64_t q0 = set * 32 / P.G;
      Set x;
      x.rem = (int)(set * 32 - q0 * P.G);
      x.pa = start + i0 + q0;
      x.pb = x.pa + walk.div(x.rem + 31);
      if (SINK || (x.pb >= k0 && x.pa <= (int64_t)k0 + 30 + P.window)) work(set, x, stage);
    };
    auto unit = [&](int64_t set, const char* stage, const char* before, char* next) __attribute__((always_inline)) {
      if (set > end) return;
      if (set + 1 < end) fetch(set + 1, next);
      if constexpr (lag() == 0) {
        if (set < end) one(set, stage);
      } else {
        if (set > begin) one(set - 1, before);
      }
      __syncthreads();
    };
    __syncthreads();
    for (int64_t set = begin; set <= end; set += 3) {
      unit(set, stage0, stage2, stage1);
      unit(set + 1, stage1, stage0, stage2);
      unit(set + 2, stage2, stage1, stage0);
    }
  };
  const bool partial = SINK || tile < P.joined;
  const int64_t slot = SINK ? ((int64_t)bh * tiles + tile) * parts + part : (((int64_t)bh * P.joined + tile) * parts + part) * PAIRS + pair;
  float* to = (SINK ? P.sink_part : P.part) + (slot * 32 + (lane & 31)) * (DKP + DVP);
  // N tiles of columns, to column `from` of a partial sum, or to the result
  auto store = [&](auto n_tiles, const f32x16* acc, int from, const WinHeads& result, int width, float mul) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < n_tiles(); ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = win_column(d, i, lane);
        if (partial) {
          st16(to + from + c, u32x4{f2u(acc[d][4 * i]), f2u(acc[d][4 * i + 1]), f2u(acc[d][4 * i + 2]), f2u(acc[d][4 * i + 3])});
        } else if (key < P.S && c < width) {
          const float v[4] = {acc[d][4 * i] * mul, acc[d][4 * i + 1] * mul, acc[d][4 * i + 2] * mul, acc[d][4 * i + 3] * mul};
          blk_st4<T>(win_out(result, b, key, h) + c * ES, v);
        }
      }
  };

  if (wave < PAIRS) {  // the weights and dv
    u32x4 kf[NK];
    const char* kr = win_at(P.k, b, is_key ? key : 0, h);
#pragma unroll
    for (int s = 0; s < NK; ++s) kf[s] = is_key ? blk_ld(kr, 32 * s + 16 * h2, kw) : zero16();
    f32x16 dv[DVP / 32];
#pragma unroll
    for (int d = 0; d < DVP / 32; ++d) dv[d] = zero_tile();
    stream(std::integral_constant<int, 0>(), [&](int64_t set, const Set& x, const char* qs) __attribute__((always_inline)) {
      const float* nref = reinterpret_cast<const float*>(qs + QB + GB) + 4 * h2;
      f32x16 s = zero_tile();
#pragma unroll
      for (int c = 0; c < NK; ++c) s = mma32<T>(qrow.read(qs, 0, c), kf[c], s);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 n = *reinterpret_cast<const f32x4*>(nref + 8 * y);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * y + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * y + e], sc, n[e]));
      }
      // some of the rows do not attend all of the keys
      if (SINK || set * 32 + 32 > rows || k0 + 31 >= len || x.pa < k0 + 31 || x.pb >= (int64_t)k0 + P.window) {
        const int64_t near = SINK ? (int64_t)key + P.window : (int64_t)key, far = SINK ? (int64_t)1 << 62 : (int64_t)key + P.window;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = 8 * (i >> 2) + 4 * h2 + (i & 3);
          const int64_t p = x.pa + walk.div(x.rem + r);
          s[i] = (!is_key | (set * 32 + r >= rows) | (p < near) | (p >= far)) ? 0.f : s[i];
        }
      }
      tile_put(weights[set & 1][pair], s, lane);
      Weights<T> wt;
#pragma unroll
      for (int i = 0; i < 8; ++i) wt.set(i, s[2 * i], s[2 * i + 1]);
#pragma unroll
      for (int c = 0; c < Weights<T>::SLABS; ++c)
#pragma unroll
        for (int d = 0; d < DVP / 32; ++d) dv[d] = wt.mma(gcol.read(qs + QB, c, d), c, dv[d]);
    });
    store(std::integral_constant<int, DVP / 32>(), dv, DKP, P.dv, P.dvw, 1.f);
    return;
  }
  // their gradients and dk
  u32x4 vf[NV];
  const char* vr = win_at(P.v, b, is_key ? key : 0, h);
#pragma unroll
  for (int s = 0; s < NV; ++s) vf[s] = is_key ? blk_ld(vr, 32 * s + 16 * h2, vw) : zero16();
  f32x16 dk[DKP / 32];
#pragma unroll
  for (int d = 0; d < DKP / 32; ++d) dk[d] = zero_tile();
  stream(std::integral_constant<int, 1>(), [&](int64_t set, const Set&, const char* qs) __attribute__((always_inline)) {
    const float* delta = reinterpret_cast<const float*>(qs + QB + GB) + 32 + 4 * h2;
    f32x16 dp = zero_tile();
#pragma unroll
    for (int c = 0; c < NV; ++c) dp = mma32<T>(grow.read(qs + QB, 0, c), vf[c], dp);
    const f32x16 p = tile_get(weights[set & 1][pair], lane);
    Weights<T> ds;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const f32x4 n = *reinterpret_cast<const f32x4*>(delta + 8 * y);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = 4 * y + e;
        ds.set(i / 2, p[i] * (dp[i] - n[e]), p[i + 1] * (dp[i + 1] - n[e + 1]));
      }
    }
#pragma unroll
    for (int c = 0; c < Weights<T>::SLABS; ++c)
#pragma unroll
      for (int d = 0; d < DKP / 32; ++d) dk[d] = ds.mma(qcol.read(qs, c, d), c, dk[d]);
  });
  store(std::integral_constant<int, DKP / 32>(), dk, 0, P.dk, P.dkw, P.scale);
}

// Adds a key's partial gradients: a workgroup a key, its waves a quarter of the
// parts each, then in order.
template <typename T, int DKP, int DVP> __global__ __launch_bounds__(256) void k_window_grad_join(const WinParams P) {
  constexpr int W = DKP + DVP, N = (W + 255) / 256;
  __shared__ f32x4 side[3][N * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, keys = P.joined * P.key_tile;
  const int bh = blockIdx.x / keys, key = blockIdx.x - bh * keys, b = bh / P.Hkv, h = bh - b * P.Hkv;
  if (key >= P.S) return;
  const int more = key < P.n_sink && P.sink_tiles > 0 ? P.sink_parts : 0, all = P.key_parts + more;
  const float* from = P.part + (((int64_t)bh * P.joined + key / P.key_tile) * P.key_parts * P.key_tile + key % P.key_tile) * W;
  const float* sink = P.sink_part + (((int64_t)bh * P.sink_tiles + key / WIN_SINK) * P.sink_parts * WIN_SINK + key % WIN_SINK) * W;
  f32x4 sum[N];
#pragma unroll
  for (int x = 0; x < N; ++x) {
    sum[x] = zero4();
    const int c = 256 * x + 4 * lane;
    if (c < W)
#pragma unroll 4
      for (int k = wave * all / 4; k < (wave + 1) * all / 4; ++k)
        sum[x] += __builtin_bit_cast(f32x4, ld16((k < P.key_parts ? from + (int64_t)k * P.key_tile * W : sink + (int64_t)(k - P.key_parts) * WIN_SINK * W) + c));
    if (wave) side[wave - 1][64 * x + lane] = sum[x];
  }
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const int c = 256 * x + 4 * lane;
    if (c >= W) continue;
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[x] += side[k][64 * x + lane];
    const float mul = c < DKP ? P.scale : 1.f;
    const float v[4] = {sum[x][0] * mul, sum[x][1] * mul, sum[x][2] * mul, sum[x][3] * mul};
    if (c < DKP) {
      if (c < P.dkw) blk_st4<T>(win_out(P.dk, b, key, h) + c * sizeof(T), v);
    } else if (c - DKP < P.dvw) {
      blk_st4<T>(win_out(P.dv, b, key, h) + (c - DKP) * sizeof(T), v);
    }
  }
}

template <typename T, int DKP, int DVP> void launch_t(const WinParams& P, hipStream_t st) {
  constexpr int PAIRS = win_pairs(sizeof(T), DVP);
  auto grid = [](int64_t n) { return dim3((unsigned)((n + N_XCD - 1) / N_XCD * N_XCD)); };
  const int64_t heads = (int64_t)P.B * P.Hkv;
  hipLaunchKernelGGL((k_window_dkdv<T, DKP, DVP, PAIRS, false>), grid(heads * P.key_tiles * P.key_parts), dim3(128 * PAIRS), 0, st, P);
  if (P.sink_tiles > 0)
    hipLaunchKernelGGL((k_window_dkdv<T, DKP, DVP, 1, true>), grid(heads * P.sink_tiles * P.sink_parts), dim3(128), 0, st, P);
  if (P.joined > 0)
    hipLaunchKernelGGL((k_window_grad_join<T, DKP, DVP>), dim3((unsigned)(heads * P.joined * P.key_tile)), dim3(256), 0, st, P);
}
template <typename T, int DKP> void by_dv(const WinParams& P, hipStream_t st) {
  if (win_dvp(P.dvw) == 64) launch_t<T, DKP, 64>(P, st);
  else if (win_dvp(P.dvw) == 128) launch_t<T, DKP, 128>(P, st);
  else launch_t<T, DKP, 256>(P, st);
}
template <typename T> void by_dk(const WinParams& P, hipStream_t st) {
  win_dkp(P.dkw) == 64 ? by_dv<T, 64>(P, st) : by_dv<T, 128>(P, st);
}

}  // namespace

hipError_t launch_window_dkdv(const WinParams& P, bool bf16_path, hipStream_t st) {
  bf16_path ? by_dk<bf16>(P, st) : by_dk<float>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
