// Window attention for few rows: single queries over a cache that may turn over
// (the streaming step), and short chunks of a long sequence.
//
// A tile of 16 (query, head) rows is dealt, units of 32 keys at a time, to the
// waves of several workgroups; a wave keeps the next unit's keys and values under
// way while it works on one.  Four waves' sums meet in LDS, the workgroups' in a
// second launch.  HBM-bound: a step reads every key and value once for all heads
// of its group (16 sequences, 16 / 4 heads of 128, window 4096: 29 us and 4 for joining,
// of a floor of 26).
//   The step puts the new key and value into their slot of the cache and takes
// them from where they came, so that no workgroup waits for another.
#include "window_device.hpp"

namespace msgla {

namespace {

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A step's position, or -1 where its token has no place: a cache too short to turn
// over ends at its last slot.
__device__ __forceinline__ int step_position(const WinParams& P, int b) {
  const int p = P.pos[b];
  return p >= 0 && (p < P.S || P.S - P.n_sink >= P.window) ? p : -1;
}
__device__ __forceinline__ int win_slot(const WinParams& P, int j) {
  return j < P.S ? j : P.n_sink + (j - P.n_sink) % (P.S - P.n_sink);
}

template <typename T, int DKP, int DVP, bool STEP>
__global__ __launch_bounds__(64 * WIN_FEW_WAVES, sizeof(T) == 2 && DVP <= 128 ? 2 : 1) void k_window_few(const WinParams P) {
  constexpr int ES = sizeof(T), NK = DKP * ES / 64, PC = DVP * ES / 16, CV = WIN_FEW_KEYS * PC / 64, VP = blk_pitch<T, DVP>();
  constexpr int ROOM = WIN_FEW_KEYS * VP, SUMS = 16 * DVP * 4;
  __shared__ __attribute__((aligned(16))) char smem[WIN_FEW_WAVES * (ROOM > SUMS ? ROOM : SUMS)];
  __shared__ float sm[WIN_FEW_WAVES][16], sl[WIN_FEW_WAVES][16];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, a = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t tile = (int64_t)blockIdx.x / P.parts;
  const int part = (int)((int64_t)blockIdx.x - tile * P.parts);
  const int bh = (int)(tile / P.tiles_per_seq), t = (int)(tile - (int64_t)bh * P.tiles_per_seq), b = bh / P.Hkv, h = bh - b * P.Hkv;
  WinRow row(P, b, h, t, r16);
  if (STEP) row.p = row.in ? step_position(P, b) : -1;
  const bool live = row.in && row.p >= 0;
  const int first = wave_min(live ? row.p : 0x7fffffff), last = wave_max(live ? row.p : -1);
  const int low = last < 0 ? 0 : max(0, first - P.window + 1);
  // units: [0, sinks), then from `from` on
  const int hi = last < 0 ? -1 : last / WIN_FEW_KEYS;
  const int sinks = min(hi + 1, (P.n_sink + WIN_FEW_KEYS - 1) / WIN_FEW_KEYS), from = max(sinks, low / WIN_FEW_KEYS);
  const int units = sinks + max(0, hi - from + 1);
  const int share = part * WIN_FEW_WAVES + wave, shares = P.parts * WIN_FEW_WAVES;
  const int begin = (int)((int64_t)units * share / shares), end = (int)((int64_t)units * (share + 1) / shares);

  const int kw = P.dkw * ES, vw = P.dvw * ES;
  const char *kb = P.k.p + b * P.k.sb + h * P.k.sh, *vb = P.v.p + b * P.v.sb + h * P.v.sh;
  const char *kn = STEP ? win_at(P.kt, b, 0, h) : nullptr, *vn = STEP ? win_at(P.vt, b, 0, h) : nullptr;
  // where the window's slots begin, and how many there are before they begin again
  const int near = max(P.n_sink, low), turn = P.S - P.n_sink, base = STEP && turn > 0 ? (near - P.n_sink) % turn : 0;
  auto key_row = [&](int j, const char* cache, int64_t st, const char* fresh) {
    j = j <= last && (j >= low || j < P.n_sink) ? j : last;  // keys that no row attends: one that is
    if (STEP) {
      if (j == last) return fresh;
      if (j >= P.n_sink) {
        int s = base + j - near;
        s -= s >= turn ? turn : 0;
        j = P.n_sink + s;
      }
    }
    return cache + j * st;
  };
  u32x4 kf[2][NK], vr[CV];
  auto fetch = [&](int u) {
    const int k0 = (u < sinks ? u : from + u - sinks) * WIN_FEW_KEYS;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const char* kr = key_row(k0 + 16 * x + r16, kb, P.k.st, kn);
#pragma unroll
      for (int c = 0; c < NK; ++c) kf[x][c] = blk_ld(kr, 64 * c + 16 * a, kw);
    }
#pragma unroll
    for (int i = 0; i < CV; ++i) {
      const int p = lane + 64 * i;
      vr[i] = blk_ld(key_row(k0 + p / PC, vb, P.v.st, vn), p % PC * 16, vw);
    }
  };
  if (begin < end) fetch(begin);
  u32x4 q[NK];
  {
    const char* qr = win_at(P.q, b, live ? row.i : 0, live ? row.head : 0);
#pragma unroll
    for (int c = 0; c < NK; ++c) q[c] = live ? blk_ld(qr, 64 * c + 16 * a, kw) : zero16();
  }
  char* vs = smem + wave * (ROOM > SUMS ? ROOM : SUMS);
  float m = -__builtin_inff(), l = 0.f;  // running maximum (in units of log 2) and sum
  f32x4 acc[DVP / 16];
#pragma unroll
  for (int d = 0; d < DVP / 16; ++d) acc[d] = zero4();
  const float sc = P.scale * BLK_LOG2E;
  for (int u = begin; u < end; ++u) {
    const int k0 = (u < sinks ? u : from + u - sinks) * WIN_FEW_KEYS;
    wave_sync();
#pragma unroll
    for (int i = 0; i < CV; ++i) {
      const int p = lane + 64 * i;
      st16(vs + p / PC * VP + p % PC * 16, vr[i]);
    }
    float w[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f32x4 s = zero4();
#pragma unroll
      for (int c = 0; c < NK; ++c) s = mma_slab<T>(kf[x][c], q[c], s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = k0 + 16 * x + 4 * a + i;
        w[x][i] = j <= row.p && (j > row.p - P.window || j < P.n_sink) ? s[i] * sc : -__builtin_inff();
      }
    }
    if (u + 1 < end) fetch(u + 1);
    float mx = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(w[0][i], w[1][i]));
    mx = blk_quad_max(mx);
    const float ref = mx == -__builtin_inff() ? 0.f : mx;  // nothing to attend yet
    const float corr = __builtin_amdgcn_exp2f(m - ref);
    m = mx;
    l *= corr;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[x][i] = __builtin_amdgcn_exp2f(w[x][i] - ref);
        l += w[x][i];
      }
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) acc[d] *= corr;
    wave_sync();
#pragma unroll
    for (int s = 0; s < WIN_FEW_KEYS / blk_slab<T>(); ++s) {
      u32x4 x, lo;
      blk_split<T>(w, s, x, lo);
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d)
        acc[d] = blk_mma_split<T>(blk_column<T>(vs, VP, s * blk_slab<T>(), d, lane), x, lo, acc[d]);
    }
  }
  l = blk_quad_sum(l);
  // the token into its slot: the last unit's wave of the group's first tile
  if (STEP && last >= 0 && share == shares - 1 && t == 0) {
    const int64_t slot = win_slot(P, last);
    char *kc = win_out(P.k, b, slot, h), *vc = win_out(P.v, b, slot, h);
    for (int at = 16 * lane; at < kw; at += 1024) st16(kc + at, ld16(kn + at));
    for (int at = 16 * lane; at < vw; at += 1024) st16(vc + at, ld16(vn + at));
  }
  // the four waves' sums
  __syncthreads();
  if (a == 0) sm[wave][r16] = m, sl[wave][r16] = l;
  float* mine = reinterpret_cast<float*>(vs);
#pragma unroll
  for (int d = 0; d < DVP / 16; ++d) st16(mine + r16 * DVP + 16 * d + 4 * a, __builtin_bit_cast(u32x4, acc[d]));
  __syncthreads();
  for (int i = tid; i < 16 * DVP / 4; i += 64 * WIN_FEW_WAVES) {
    const int r = i / (DVP / 4), c = i % (DVP / 4) * 4;
    float top = sm[0][r], sum = 0.f;
#pragma unroll
    for (int x = 1; x < WIN_FEW_WAVES; ++x) top = fmaxf(top, sm[x][r]);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    f32x4 o = zero4();
#pragma unroll
    for (int x = 0; x < WIN_FEW_WAVES; ++x) {
      const float f = __builtin_amdgcn_exp2f(sm[x][r] - ref);
      sum += f * sl[x][r];
      o += f * __builtin_bit_cast(f32x4, ld16(reinterpret_cast<const float*>(smem + x * (ROOM > SUMS ? ROOM : SUMS)) + r * DVP + c));
    }
    if (P.parts > 1) {
      const int64_t pr = (tile * P.parts + part) * WIN_FEW_ROWS + r;
      if (c == 0) P.pm[2 * pr] = top, P.pm[2 * pr + 1] = sum;
      st16(P.po + pr * DVP + c, __builtin_bit_cast(u32x4, o));
    } else {
      const WinRow to(P, b, h, t, r);
      const float inv = sum > 0.f ? 1.f / sum : sum;  // a NaN stays
      if (to.in && c < P.dvw) {
        float v[4];  // no key: 0, whatever the tile's other rows attend
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = sum == 0.f ? 0.f : o[e] * inv;
        blk_st4<T>(win_out(P.o, b, to.i, to.head) + c * ES, v);
      }
      if (to.in && c == 0 && P.lse)
        P.lse[((int64_t)b * P.Hq + to.head) * P.L + to.i] = sum == 0.f ? -__builtin_inff() : top * BLK_LN2 + logf(sum);
    }
  }
}

// Joins a row's partial outputs.
template <typename T, int DVP> __global__ __launch_bounds__(64) void k_window_join(const WinParams P) {
  const int64_t tile = blockIdx.x / WIN_FEW_ROWS;
  const int r = (int)(blockIdx.x % WIN_FEW_ROWS), lane = threadIdx.x;
  const int bh = (int)(tile / P.tiles_per_seq), t = (int)(tile - (int64_t)bh * P.tiles_per_seq), b = bh / P.Hkv, h = bh - b * P.Hkv;
  const WinRow row(P, b, h, t, r);
  if (!row.in) return;
  const int64_t pr = tile * P.parts * WIN_FEW_ROWS + r;
  float m = -__builtin_inff(), l = 0.f, o[DVP / 64];
#pragma unroll 4
  for (int k = 0; k < P.parts; ++k) m = fmaxf(m, P.pm[2 * (pr + k * WIN_FEW_ROWS)]);
  const float ref = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
  for (int d = 0; d < DVP / 64; ++d) o[d] = 0.f;
#pragma unroll 4
  for (int k = 0; k < P.parts; ++k) {
    const int64_t at = pr + k * WIN_FEW_ROWS;
    const float w = __builtin_amdgcn_exp2f(P.pm[2 * at] - ref);
    l += w * P.pm[2 * at + 1];
#pragma unroll
    for (int d = 0; d < DVP / 64; ++d) o[d] += w * P.po[at * DVP + 64 * d + lane];
  }
  const float inv = l > 0.f ? 1.f / l : l;  // a NaN stays
  T* out = reinterpret_cast<T*>(win_out(P.o, b, row.i, row.head));
#pragma unroll
  for (int d = 0; d < DVP / 64; ++d)
    if (64 * d + lane < P.dvw) out[64 * d + lane] = from_f32<T>(l == 0.f ? 0.f : o[d] * inv);  // no key: 0
  if (P.lse && lane == 0)
    P.lse[((int64_t)b * P.Hq + row.head) * P.L + row.i] = l == 0.f ? -__builtin_inff() : m * BLK_LN2 + logf(l);
}

// A prefill's keys and values into their slots: one wave a position and head.  Of
// the positions that share a slot the last one stays (8 x 2048 positions, 4 heads of 128,
// bf16: 17 us for 67 MB).  A sequence with fewer than 0
// tokens before sits out, as in the step, and so does one whose number of tokens a
// later call could not be told.
__global__ __launch_bounds__(256) void k_window_append(const WinParams P, int es) {
  const int lane = threadIdx.x & 63, h = blockIdx.y;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int b = (int)(row / P.L), i = (int)(row - (int64_t)b * P.L);
  if (b >= P.B) return;
  const int n = P.lens ? min(P.lens[b], P.L) : P.L;  // new tokens
  const int64_t p0 = P.pos ? P.pos[b] : 0, p = p0 + i, end = p0 + n;
  if (i >= n || p0 < 0 || end > 0x7fffffff) return;
  const int turn = P.S - P.n_sink;
  if (p >= P.S && turn < P.window) return;                        // no place for it
  if (turn >= P.window && p >= P.n_sink && p + turn < end) return;  // another one follows in its slot
  const int64_t slot = p < P.S ? p : P.n_sink + (p - P.n_sink) % turn;
  const char *ks = win_at(P.kt, b, i, h), *vs = win_at(P.vt, b, i, h);
  char *kd = win_out(P.k, b, slot, h), *vd = win_out(P.v, b, slot, h);
  for (int at = 16 * lane; at < P.dkw * es; at += 1024) st16(kd + at, ld16(ks + at));
  for (int at = 16 * lane; at < P.dvw * es; at += 1024) st16(vd + at, ld16(vs + at));
}

template <typename T, int DKP, int DVP> void launch_t(const WinParams& P, bool step, hipStream_t st) {
  const dim3 grid((unsigned)(P.tiles * P.parts)), block(64 * WIN_FEW_WAVES);
  if (step) hipLaunchKernelGGL((k_window_few<T, DKP, DVP, true>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((k_window_few<T, DKP, DVP, false>), grid, block, 0, st, P);
  if (P.parts > 1) hipLaunchKernelGGL((k_window_join<T, DVP>), dim3((unsigned)(P.tiles * WIN_FEW_ROWS)), dim3(64), 0, st, P);
}
template <typename T, int DKP> void by_dv(const WinParams& P, bool step, hipStream_t st) {
  if (win_dvp(P.dvw) == 64) launch_t<T, DKP, 64>(P, step, st);
  else if (win_dvp(P.dvw) == 128) launch_t<T, DKP, 128>(P, step, st);
  else launch_t<T, DKP, 256>(P, step, st);
}
template <typename T> void by_dk(const WinParams& P, bool step, hipStream_t st) {
  win_dkp(P.dkw) == 64 ? by_dv<T, 64>(P, step, st) : by_dv<T, 128>(P, step, st);
}

}  // namespace

hipError_t launch_window_few(const WinParams& P, bool step, bool bf16_path, hipStream_t st) {
  bf16_path ? by_dk<bf16>(P, step, st) : by_dk<float>(P, step, st);
  return hipGetLastError();
}

hipError_t launch_window_append(const WinParams& P, bool bf16_path, hipStream_t st) {
  const dim3 grid((unsigned)(((int64_t)P.B * P.L + 3) / 4), (unsigned)P.Hkv);
  hipLaunchKernelGGL(k_window_append, grid, dim3(256), 0, st, P, bf16_path ? 2 : 4);
  return hipGetLastError();
}

}  // namespace msgla
