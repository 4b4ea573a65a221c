// Gradients of the keys and values of the window attention:
//   dv_j = sum over the rows that attend j of p_ij do_i,   dk_j = scale sum of p_ij (do_i . v_j - delta_i) q_i.
//
// A workgroup keeps 128 keys and values and their gradients in registers, 32 a
// wave, and streams through the (query, head) rows whose windows hold any of them,
// 32 at a time through LDS.  First tokens are attended by all later queries as
// well: the rows beyond their windows are walked by workgroups that hold 32 first
// tokens in each of four waves, which take different rows.  Few key tiles are
// dealt to several workgroups by their rows.  Such partial sums a last kernel adds in
// order: the result does not vary from call to call.
//   Scores are formed as S = Q K^T, whose result is the operand of dV^T = dO^T P
// and dK^T = Q^T dS.  bf16 weights and their gradients enter these as two bf16 values
// each, as in the other kernels.
#include "window_device.hpp"

namespace msgla {

namespace {

template <typename T, int DKP, int DVP, bool SINK>
__global__ __launch_bounds__(256, sizeof(T) == 2 && DKP + DVP <= 128 ? 2 : 1) void k_window_dkdv(const WinParams P) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, NK = DKP * ES / 32, NV = DVP * ES / 32;
  constexpr int QB = 32 * WK * 16, SET = QB + 32 * WV * 16;
  constexpr int SLABS = 32 / win_slab<T>(), SETS = !SINK ? 1 : 4 * SET <= 144 * 1024 ? 4 : 2;  // sets of 32 rows in LDS
  constexpr int CQ = 32 * WK / 256, CV = 32 * WV / 256;
  __shared__ __attribute__((aligned(16))) char smem[SETS * SET];
  __shared__ __attribute__((aligned(16))) float slse[SETS * 32], sdelta[SETS * 32];
  __shared__ int spos[SETS * 32];
  const int tid = threadIdx.x, lane = tid & 63, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = SINK ? P.sink_tiles : P.key_tiles, parts = SINK ? P.sink_parts : P.key_parts;
  const int total = P.B * P.Hkv * tiles * parts, per = (total + N_XCD - 1) / N_XCD;
  const int w = remap_xcd(blockIdx.x, per);
  if (w >= total) return;
  const int part = w % parts, tile = w / parts % tiles, bh = w / parts / tiles, b = bh / P.Hkv, h = bh - b * P.Hkv;
  const int k0 = SINK ? tile * WIN_SINK : tile * WIN_KEYS + 32 * wave;
  const int key = k0 + (lane & 31);
  const int len = P.lens ? max(0, min(P.lens[b], P.S)) : P.S;
  const int64_t start = P.start ? P.start[b] : 0;
  // positions of the rows: those whose windows hold one of the keys, or those behind the first key's window
  const int64_t p0 = SINK ? (int64_t)k0 + P.window : (int64_t)tile * WIN_KEYS;
  const int64_t p1 = SINK ? len : min((int64_t)len, p0 + WIN_KEYS - 1 + P.window);
  const int64_t i0 = max((int64_t)0, p0 - start), i1 = min((int64_t)P.L, p1 - start);
  const int64_t rows = i1 > i0 ? (i1 - i0) * P.G : 0, sets = (rows + 31) / 32;
  const int64_t begin = sets * part / parts, end = sets * (part + 1) / parts;

  const int kw = P.dkw * ES, vw = P.dvw * ES;
  const bool is_key = key < len && (!SINK || key < P.n_sink);
  u32x4 kf[NK], vf[NV];
  {
    const char *kr = win_at(P.k, b, is_key ? key : 0, h), *vr = win_at(P.v, b, is_key ? key : 0, h);
#pragma unroll
    for (int s = 0; s < NK; ++s) kf[s] = is_key ? blk_ld(kr, 32 * s + 16 * h2, kw) : zero16();
#pragma unroll
    for (int s = 0; s < NV; ++s) vf[s] = is_key ? blk_ld(vr, 32 * s + 16 * h2, vw) : zero16();
  }
  f32x16 dk[DKP / 32], dv[DVP / 32];
#pragma unroll
  for (int d = 0; d < DKP / 32; ++d) dk[d] = zero_tile();
#pragma unroll
  for (int d = 0; d < DVP / 32; ++d) dv[d] = zero_tile();
  const float sc = P.scale * BLK_LOG2E;
  const Rows32<WK> qrow(lane);
  const Rows32<WV> grow(lane);
  const Columns32<T, WK> qcol(lane);
  const Columns32<T, WV> gcol(lane);

  u32x4 qr[CQ], gr[CV];
  auto row_of = [&](int64_t r, int64_t& i, int& head) {
    const int64_t qi = r / P.G;
    i = i0 + qi;
    head = h * P.G + (int)(r - qi * P.G);
    return r < rows;
  };
  auto fetch = [&](int64_t set) {
#pragma unroll
    for (int x = 0; x < CQ; ++x) {
      const int p = tid + 256 * x;
      int64_t i;
      int head;
      const bool in = row_of(set * 32 + p / WK, i, head);
      qr[x] = in ? blk_ld(win_at(P.q, b, i, head), p % WK * 16, kw) : zero16();
    }
#pragma unroll
    for (int x = 0; x < CV; ++x) {
      const int p = tid + 256 * x;
      int64_t i;
      int head;
      const bool in = row_of(set * 32 + p / WV, i, head);
      gr[x] = in ? blk_ld(win_at(P.dout, b, i, head), p % WV * 16, vw) : zero16();
    }
  };
  auto put = [&](int64_t set, int at) {
    char* q = smem + at * SET;
#pragma unroll
    for (int x = 0; x < CQ; ++x) {
      const int p = tid + 256 * x, r = p / WK;
      st16(q + (r * WK + ((p % WK) ^ tile_key<WK>(r))) * 16, qr[x]);
    }
#pragma unroll
    for (int x = 0; x < CV; ++x) {
      const int p = tid + 256 * x, r = p / WV;
      st16(q + QB + (r * WV + ((p % WV) ^ tile_key<WV>(r))) * 16, gr[x]);
    }
    if (tid < 32) {
      int64_t i;
      int head;
      const bool in = row_of(set * 32 + tid, i, head);
      const int64_t lr = ((int64_t)b * P.Hq + head) * P.L + i;
      slse[at * 32 + tid] = in ? -P.lse_in[lr] * BLK_LOG2E : -__builtin_inff();  // weights of 0
      sdelta[at * 32 + tid] = in ? P.delta[lr] : 0.f;
      spos[at * 32 + tid] = in ? (int)(start + i) : 0x7fffffff;
    }
  };
  if (!SINK && begin < end) fetch(begin);
  for (int64_t set = begin; set < end; set += SETS) {
    __syncthreads();
    if constexpr (SINK) {
      for (int x = 0; x < SETS; ++x) {
        fetch(set + x < end ? set + x : sets);
        put(set + x < end ? set + x : sets, x);
      }
    } else {
      put(set, 0);
    }
    __syncthreads();
    if (!SINK && set + 1 < end) fetch(set + 1);
    if (SINK && wave >= SETS) continue;
    const int at = SINK ? wave : 0;
    const char *qs = smem + at * SET, *gs = qs + QB;
    f32x16 s = zero_tile(), dp = zero_tile();
#pragma unroll
    for (int c = 0; c < NK; ++c) s = mma32<T>(qrow.read(qs, 0, c), kf[c], s);
#pragma unroll
    for (int c = 0; c < NV; ++c) dp = mma32<T>(grow.read(gs, 0, c), vf[c], dp);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const f32x4 nref = *reinterpret_cast<const f32x4*>(&slse[at * 32 + 8 * y + 4 * h2]);
      const f32x4 delta = *reinterpret_cast<const f32x4*>(&sdelta[at * 32 + 8 * y + 4 * h2]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * y + e, p = spos[at * 32 + 8 * y + 4 * h2 + e];
        const bool on = is_key && (SINK ? key <= p - P.window : key <= p && key > p - P.window);
        const float wt = on ? __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], sc, nref[e])) : 0.f;
        s[i] = wt;
        dp[i] = on ? wt * (dp[i] - delta[e]) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < SLABS; ++c) {
      u32x4 hi, lo;
      win_split<T>(s, c, hi, lo);
#pragma unroll
      for (int d = 0; d < DVP / 32; ++d) {
        const u32x4 f = gcol.read(gs, c, d);
        dv[d] = mma32<T>(f, hi, dv[d]);
        if constexpr (ES == 2) dv[d] = mma32<T>(f, lo, dv[d]);
      }
      win_split<T>(dp, c, hi, lo);
#pragma unroll
      for (int d = 0; d < DKP / 32; ++d) {
        const u32x4 f = qcol.read(qs, c, d);
        dk[d] = mma32<T>(f, hi, dk[d]);
        if constexpr (ES == 2) dk[d] = mma32<T>(f, lo, dk[d]);
      }
    }
  }
  const bool partial = SINK || tile < P.joined;
  if (partial) {
    const int64_t slot = SINK ? (((int64_t)bh * tiles + tile) * parts + part) * 4 + wave
                              : (((int64_t)bh * P.joined + tile) * parts + part) * 4 + wave;
    float* to = (SINK ? P.sink_part : P.part) + (slot * 32 + (lane & 31)) * (DKP + DVP);
#pragma unroll
    for (int d = 0; d < DKP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st16(to + win_column(d, i, lane), u32x4{f2u(dk[d][4 * i]), f2u(dk[d][4 * i + 1]), f2u(dk[d][4 * i + 2]), f2u(dk[d][4 * i + 3])});
#pragma unroll
    for (int d = 0; d < DVP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st16(to + DKP + win_column(d, i, lane), u32x4{f2u(dv[d][4 * i]), f2u(dv[d][4 * i + 1]), f2u(dv[d][4 * i + 2]), f2u(dv[d][4 * i + 3])});
  } else if (key < P.S) {
    char *ko = win_out(P.dk, b, key, h), *vo = win_out(P.dv, b, key, h);
#pragma unroll
    for (int d = 0; d < DKP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = win_column(d, i, lane);
        const float v[4] = {dk[d][4 * i] * P.scale, dk[d][4 * i + 1] * P.scale, dk[d][4 * i + 2] * P.scale, dk[d][4 * i + 3] * P.scale};
        if (c < P.dkw) blk_st4<T>(ko + c * ES, v);
      }
#pragma unroll
    for (int d = 0; d < DVP / 32; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = win_column(d, i, lane);
        const float v[4] = {dv[d][4 * i], dv[d][4 * i + 1], dv[d][4 * i + 2], dv[d][4 * i + 3]};
        if (c < P.dvw) blk_st4<T>(vo + c * ES, v);
      }
  }
}

// Adds a key's partial gradients in order: four keys a workgroup.
template <typename T, int DKP, int DVP> __global__ __launch_bounds__(256) void k_window_grad_join(const WinParams P) {
  constexpr int W = DKP + DVP;
  const int lane = threadIdx.x & 63, keys = P.joined * WIN_KEYS;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int bh = (int)(at / keys), key = (int)(at - (int64_t)bh * keys), b = bh / P.Hkv, h = bh - b * P.Hkv;
  if (bh >= P.B * P.Hkv || key >= P.S) return;
  const int tile = key / WIN_KEYS, r = key % WIN_KEYS;
  const bool sink = key < P.n_sink && P.sink_tiles > 0;
  f32x4 sum[(W + 255) / 256];
#pragma unroll
  for (int x = 0; x < (W + 255) / 256; ++x) {
    sum[x] = zero4();
    const int c = 256 * x + 4 * lane;
    if (c >= W) continue;
    const float* from = P.part + (((int64_t)bh * P.joined + tile) * P.key_parts * WIN_KEYS + r) * W + c;
#pragma unroll 4
    for (int k = 0; k < P.key_parts; ++k) sum[x] += __builtin_bit_cast(f32x4, ld16(from + (int64_t)k * WIN_KEYS * W));
    if (sink) {
      const float* more = P.sink_part + (((int64_t)bh * P.sink_tiles + key / WIN_SINK) * P.sink_parts * 4 * WIN_SINK + key % WIN_SINK) * W + c;
#pragma unroll 4
      for (int k = 0; k < P.sink_parts * 4; ++k) sum[x] += __builtin_bit_cast(f32x4, ld16(more + (int64_t)k * WIN_SINK * W));
    }
    if (c < DKP) {
      const float v[4] = {sum[x][0] * P.scale, sum[x][1] * P.scale, sum[x][2] * P.scale, sum[x][3] * P.scale};
      if (c < P.dkw) blk_st4<T>(win_out(P.dk, b, key, h) + c * sizeof(T), v);
    } else {
      const float v[4] = {sum[x][0], sum[x][1], sum[x][2], sum[x][3]};
      if (c - DKP < P.dvw) blk_st4<T>(win_out(P.dv, b, key, h) + (c - DKP) * sizeof(T), v);
    }
  }
}

template <typename T, int DKP, int DVP> void launch_t(const WinParams& P, hipStream_t st) {
  auto grid = [](int64_t n) { return dim3((unsigned)((n + N_XCD - 1) / N_XCD * N_XCD)); };
  const int64_t heads = (int64_t)P.B * P.Hkv;
  hipLaunchKernelGGL((k_window_dkdv<T, DKP, DVP, false>), grid(heads * P.key_tiles * P.key_parts), dim3(256), 0, st, P);
  if (P.sink_tiles > 0)
    hipLaunchKernelGGL((k_window_dkdv<T, DKP, DVP, true>), grid(heads * P.sink_tiles * P.sink_parts), dim3(256), 0, st, P);
  if (P.joined > 0)
    hipLaunchKernelGGL((k_window_grad_join<T, DKP, DVP>), dim3((unsigned)((heads * P.joined * WIN_KEYS + 3) / 4)), dim3(256), 0, st, P);
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
