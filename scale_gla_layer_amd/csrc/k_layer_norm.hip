// Layer norm over the channels of every row, forward and backward.
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mean) rstd
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// A row stays in the registers of the lanes that read it, so it is read once and
// its mean is known before its deviations are squared.  The mean is a sum in 64
// bits: a stored mean near zero keeps its digits, and deviations lose what its
// rounding to 32 bits leaves, which at a mean of 1000 deviations is 2^-14 of one.
//   All loads and stores are 16 bytes a lane whatever the rows' alignment (the
// hardware takes any), so that odd widths cost their last piece only.
//   The backward's workgroups keep their channels' sums of dy xh and dy in
// registers over all their rows, and a second kernel adds the workgroups' sums in
// order: the result does not vary from call to call.  These sums over rows are formed in
// 64 bits and rounded to 32 where a lane's and a workgroup's are left for others: in 32
// bits, equal gradients in each row put dbias off by 1.2e-6 at 32768 rows and by 1.7e-5
// at 2^20 (fp32, D = 2048), now by at most 1.8e-7 at any number.
//   HBM-bound: B = 8, L = 2048, D = 1024 in bf16 takes 16.5 us forward (67 MB, 4.1 TB/s)
// and 21.4 + 4.0 for the gradient (101 MB); a copy reaches 5.1 TB/s.
#include <algorithm>

#include "device_common.hpp"
#include "layer_norm.hpp"

namespace msgla {

namespace {

template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) LnPiece { uint32_t w[4]; };

template <typename T> __device__ __forceinline__ u32x4 ln_ld(const char* p) {
  const LnPiece<T> v = *reinterpret_cast<const LnPiece<T>*>(p);
  return u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
}
template <typename T> __device__ __forceinline__ void ln_st(char* p, u32x4 v) {
  *reinterpret_cast<LnPiece<T>*>(p) = LnPiece<T>{{v[0], v[1], v[2], v[3]}};
}

// Piece c (16 bytes) of a row of D elements, zero behind its end.
template <typename T> __device__ __forceinline__ u32x4 ln_load(const char* row, int c, int D) {
  constexpr int PER = per16<T>();
  const int e = c * PER;
  if (e + PER <= D) return ln_ld<T>(row + 16 * c);
  u32x4 v = zero16();
  if (e < D) {
    float f[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = e + i < D ? to_f32(reinterpret_cast<const T*>(row)[e + i]) : 0.f;
    v = pack16<T>(f);
  }
  return v;
}
template <typename T> __device__ __forceinline__ void ln_store(char* row, int c, int D, const float* f) {
  constexpr int PER = per16<T>();
  const int e = c * PER;
  if (e + PER <= D) {
    ln_st<T>(row + 16 * c, pack16<T>(f));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e + i < D) reinterpret_cast<T*>(row)[e + i] = from_f32<T>(f[i]);
  }
}
// the PER channels of piece c of a vector of D floats
template <int PER> __device__ __forceinline__ void ln_vec(const float* v, int c, int D, float* f) {
  const int e = c * PER;
  if (e + PER <= D) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) unpack16<float>(ln_ld<float>(reinterpret_cast<const char*>(v + e + i)), f + i);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = e + i < D ? v[e + i] : 0.f;
  }
}

template <int CTRL> __device__ __forceinline__ float ln_dpp(float v) {
  return u2f(__builtin_amdgcn_mov_dpp(f2u(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double ln_dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over each group of N lanes (8 .. 64), in all of them: within rows of 16
// lanes by cross-lane moves of the vector unit.
template <int N, typename F> __device__ __forceinline__ F ln_wave_sum(F v) {
  v += ln_dpp<0xB1>(v);   // lane ^ 1
  v += ln_dpp<0x4E>(v);   // lane ^ 2
  v += ln_dpp<0x141>(v);  // mirrored within 8
  if constexpr (N > 8) v += ln_dpp<0x140>(v);  // mirrored within 16
  if constexpr (N > 16) v += __shfl_xor(v, 16);
  if constexpr (N > 32) v += __shfl_xor(v, 32);
  return v;
}

// Sums over the lanes of a row.  Rows wider than a wave have a workgroup to
// themselves: `room` holds its waves' sums and is used in turn.
template <int LANES> struct LnSum {
  static constexpr int WAVES = LANES > 64 ? LANES / 64 : 1;
  double* room;
  int turn = 0;
  __device__ explicit LnSum(double* r) : room(r) {}
  template <typename F> __device__ __forceinline__ F operator()(F v) {
    return two(v, F(0), false).a;
  }
  template <typename F> struct Pair { F a, b; };
  template <typename F> __device__ __forceinline__ Pair<F> two(F a, F b, bool both = true) {
    a = ln_wave_sum<(LANES < 64 ? LANES : 64)>(a);
    if (both) b = ln_wave_sum<(LANES < 64 ? LANES : 64)>(b);
    if constexpr (WAVES > 1) {
      F* r = reinterpret_cast<F*>(room + turn * 2 * WAVES);
      turn ^= 1;  // the waves that still read this sum have not begun to write the next but one
      if ((threadIdx.x & 63) == 0) {
        r[threadIdx.x >> 6] = a;
        if (both) r[WAVES + (threadIdx.x >> 6)] = b;
      }
      __syncthreads();
      a = b = F(0);
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        a += r[i];
        if (both) b += r[WAVES + i];
      }
    }
    return {a, b};
  }
};

// row below 2^28
__device__ __forceinline__ char* ln_row(const LnRows& t, int64_t row, int L) {
  const uint32_t r = (uint32_t)row, b = r / (uint32_t)L;
  return t.p + (int64_t)b * t.sb + (int64_t)(r - b * (uint32_t)L) * t.st;
}

// A row's lanes: THREADS / LANES rows a workgroup and round.
template <typename T, int LANES, int K, int THREADS>
__global__ __launch_bounds__(THREADS) void k_layer_norm(const LnParams P) {
  constexpr int PER = per16<T>(), ROWS = THREADS / LANES;
  __shared__ double room[4 * LnSum<LANES>::WAVES];
  LnSum<LANES> sum(room);
  const int l = threadIdx.x % LANES;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // every lane makes the same number of rounds: wide rows meet at barriers
  const int64_t rounds = (P.rows - 1) / step + 1;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
  u32x4 raw[K];
  auto fetch = [&](int64_t r) {
    const bool in = r < P.rows;
    const char* xr = ln_row(P.x, in ? r : 0, P.L);
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k] = in ? ln_load<T>(xr, l + LANES * k, P.D) : zero16();
  };
  fetch(row);
  for (int64_t n = 0; n < rounds; ++n) {
    const int64_t here = row;
    float v[K][PER];
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack16<T>(raw[k], v[k]);
#pragma unroll
      for (int i = 0; i < PER; ++i) s += (double)v[k][i];
    }
    row += step;
    if (n + 1 < rounds) fetch(row);
    const double exact = sum(s) / P.D;
    const float mean = (float)exact, off = (float)(exact - (double)mean);
    float d2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[k][i] = (l + LANES * k) * PER + i < P.D ? v[k][i] - mean - off : 0.f;
        d2 = __builtin_fmaf(v[k][i], v[k][i], d2);
      }
    const float rstd = 1.f / sqrtf(sum(d2) / (float)P.D + P.eps);
    if (here >= P.rows) continue;
    if (l == 0) {
      if (P.mean) P.mean[here] = mean;
      if (P.rstd) P.rstd[here] = rstd;
    }
    char* yr = ln_row(P.y, here, P.L);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (c * PER >= P.D) continue;
      float w[PER], b[PER], o[PER];
      if (P.weight) ln_vec<PER>(P.weight, c, P.D, w);
      if (P.bias) ln_vec<PER>(P.bias, c, P.D, b);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        o[i] = v[k][i] * rstd;
        if (P.weight) o[i] *= w[i];
        if (P.bias) o[i] += b[i];
      }
      ln_store<T>(yr, c, P.D, o);
    }
  }
}

// dx, and with SUMS the workgroup's part of dweight and dbias.
template <typename T, int LANES, int K, int THREADS, bool SUMS>
__global__ __launch_bounds__(THREADS) void k_layer_norm_dx(const LnParams P) {
  constexpr int PER = per16<T>(), ROWS = THREADS / LANES;
  constexpr bool AHEAD = THREADS < 1024;  // the next row under way meanwhile, where registers hold it
  __shared__ double room[4 * LnSum<LANES>::WAVES];
  LnSum<LANES> sum(room);
  const int l = threadIdx.x % LANES;
  float w[SUMS ? K : 1][PER];
  double dw[SUMS ? K : 1][PER], db[SUMS ? K : 1][PER];
  if constexpr (SUMS) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (P.weight) ln_vec<PER>(P.weight, l + LANES * k, P.D, w[k]);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!P.weight) w[k][i] = 1.f;
        dw[k][i] = db[k][i] = 0.0;
      }
    }
  }
  const float per = 1.f / (float)P.D;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // every lane makes the same number of rounds: wide rows meet at barriers
  const int64_t rounds = (P.rows - 1) / step + 1;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
  u32x4 rx[K], rg[K];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t r) {
    const bool in = r < P.rows;
    const char* xr = ln_row(P.x, in ? r : 0, P.L);
    const char* gr = ln_row(P.dy, in ? r : 0, P.L);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rx[k] = in ? ln_load<T>(xr, l + LANES * k, P.D) : zero16();
      rg[k] = in ? ln_load<T>(gr, l + LANES * k, P.D) : zero16();
    }
    mean = in ? P.mean_in[r] : 0.f;
    rstd = in ? P.rstd_in[r] : 0.f;
  };
  if (AHEAD) fetch(row);
  for (int64_t n = 0; n < rounds; ++n) {
    const int64_t here = row;
    if (!AHEAD) fetch(row);
    const float r = rstd;
    float xh[K][PER], g[K][PER];
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack16<T>(rx[k], xh[k]);
      unpack16<T>(rg[k], g[k]);
      float wk[PER];
      if constexpr (!SUMS) {
        if (P.weight) ln_vec<PER>(P.weight, l + LANES * k, P.D, wk);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        xh[k][i] = (l + LANES * k) * PER + i < P.D ? (xh[k][i] - mean) * r : 0.f;
        if constexpr (SUMS) {
          dw[k][i] = __builtin_fma((double)g[k][i], (double)xh[k][i], dw[k][i]);
          db[k][i] += (double)g[k][i];
          g[k][i] *= w[k][i];
        } else if (P.weight) {
          g[k][i] *= wk[i];
        }
        c1 += g[k][i];
        c2 = __builtin_fmaf(g[k][i], xh[k][i], c2);
      }
    }
    row += step;
    if (AHEAD && n + 1 < rounds) fetch(row);
    const auto c = sum.two(c1, c2);
    c1 = c.a * per;
    c2 = c.b * per;
    if (here >= P.rows) continue;
    char* out = ln_row(P.dx, here, P.L);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = r * (g[k][i] - c1 - xh[k][i] * c2);
      ln_store<T>(out, l + LANES * k, P.D, o);
    }
  }
  if constexpr (SUMS) {
    // rows that a workgroup takes side by side meet in LDS
    constexpr int PITCH = LANES * K + 64 / PER;  // element i of piece c at i PITCH + c: no bank conflicts either way
    float* part = P.part + (int64_t)blockIdx.x * 2 * P.D;
    if constexpr (ROWS == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = (l + LANES * k) * PER + i;
          if (e < P.D) part[e] = (float)dw[k][i], part[P.D + e] = (float)db[k][i];
        }
    } else {
      __shared__ float side[ROWS][PER * PITCH];
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < PER; ++i) side[threadIdx.x / LANES][i * PITCH + l + LANES * k] = (float)(which ? db[k][i] : dw[k][i]);
        __syncthreads();
        for (int e = threadIdx.x; e < P.D; e += THREADS) {
          double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
          for (int j = 0; j < ROWS; ++j) s[j % 4] += (double)side[j][e % PER * PITCH + e / PER];
          part[which * P.D + e] = (float)((s[0] + s[1]) + (s[2] + s[3]));
        }
      }
    }
  }
}

// Sums over rows for rows too wide for the registers: a workgroup takes LN_COLS
// channels and every parts-th group of 16 rows.
template <typename T> __global__ __launch_bounds__(LN_COL_THREADS) void k_layer_norm_columns(const LnParams P) {
  constexpr int ROWS = LN_COL_THREADS / LN_COLS;
  __shared__ double2 side[ROWS][LN_COLS];
  const int c = threadIdx.x % LN_COLS, j = threadIdx.x / LN_COLS, col = blockIdx.x * LN_COLS + c;
  double dw = 0.0, db = 0.0;
  if (col < P.D)
    for (int64_t r = (int64_t)blockIdx.y * ROWS + j; r < P.rows; r += (int64_t)P.parts * ROWS) {
      const float x = to_f32(reinterpret_cast<const T*>(ln_row(P.x, r, P.L))[col]);
      const float g = to_f32(reinterpret_cast<const T*>(ln_row(P.dy, r, P.L))[col]);
      dw = __builtin_fma((double)g, (double)((x - P.mean_in[r]) * P.rstd_in[r]), dw);
      db += (double)g;
    }
  side[j][c] = make_double2(dw, db);
  __syncthreads();
  if (j == 0 && col < P.D) {
    for (int i = 1; i < ROWS; ++i) {
      dw += side[i][c].x;
      db += side[i][c].y;
    }
    float* part = P.part + (int64_t)blockIdx.y * 2 * P.D;
    part[col] = (float)dw;
    part[P.D + col] = (float)db;
  }
}

// dweight and dbias from the parts.
__global__ __launch_bounds__(LN_COL_THREADS) void k_layer_norm_join(const LnParams P) {
  constexpr int ROWS = LN_COL_THREADS / LN_JOIN_COLS;
  __shared__ double side[ROWS][LN_JOIN_COLS];
  float* out = blockIdx.y ? P.dbias : P.dweight;
  if (!out) return;
  const int c = threadIdx.x % LN_JOIN_COLS, j = threadIdx.x / LN_JOIN_COLS, col = blockIdx.x * LN_JOIN_COLS + c;
  double s = 0.0;
  if (col < P.D) {
    const float* p = P.part + (int64_t)blockIdx.y * P.D + col;
#pragma unroll 8
    for (int r = j; r < P.parts; r += ROWS) s += (double)p[(int64_t)r * 2 * P.D];
  }
  side[j][c] = s;
  __syncthreads();
  if (j == 0 && col < P.D) {
    double t[4] = {s, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 1; i < ROWS; ++i) t[i % 4] += side[i][c];
    out[col] = (float)((t[0] + t[1]) + (t[2] + t[3]));
  }
}

// f(lanes, pieces, threads) with the row's shape as constants
template <typename T, class F> void ln_dispatch(int64_t bytes, F f) {
  const LnShape s = ln_shape(bytes, sizeof(T));
#define MSGLA_LN(lanes_, pieces_, threads_) \
  if (s.lanes == lanes_ && s.pieces == pieces_) \
    return f(std::integral_constant<int, lanes_>(), std::integral_constant<int, pieces_>(), std::integral_constant<int, threads_>());
  MSGLA_LN(8, 2, 256)
  MSGLA_LN(32, 2, 256)
  MSGLA_LN(64, 2, 256)
  if constexpr (sizeof(T) == 4) {
    MSGLA_LN(64, 4, 256)
  } else {
    MSGLA_LN(256, 1, 256)
  }
  MSGLA_LN(256, 2, 256)
  MSGLA_LN(256, 4, 256)
  MSGLA_LN(1024, 2, 1024)
  if constexpr (sizeof(T) == 4) {
    MSGLA_LN(1024, 4, 1024)
  }
#undef MSGLA_LN
}

template <typename T> void forward(const LnParams& P, hipStream_t st) {
  ln_dispatch<T>((int64_t)P.D * (int)sizeof(T), [&](auto lanes, auto pieces, auto threads) {
    constexpr int LANES = lanes(), K = pieces(), THREADS = threads();
    hipLaunchKernelGGL((k_layer_norm<T, LANES, K, THREADS>), dim3((unsigned)ln_grid(P.rows, (int64_t)P.D * (int)sizeof(T), sizeof(T))), dim3(THREADS), 0, st, P);
  });
}
template <typename T> void backward(const LnParams& P, hipStream_t st) {
  const int64_t bytes = (int64_t)P.D * (int)sizeof(T);
  const bool sums = P.dweight || P.dbias, wide = bytes > 16 * LN_WIDE;
  const unsigned cols = (unsigned)((P.D + LN_COLS - 1) / LN_COLS);
  // before dx, which may take dy's place
  if (sums && wide) hipLaunchKernelGGL((k_layer_norm_columns<T>), dim3(cols, (unsigned)P.parts), dim3(LN_COL_THREADS), 0, st, P);
  ln_dispatch<T>(bytes, [&](auto lanes, auto pieces, auto threads) {
    constexpr int LANES = lanes(), K = pieces(), THREADS = threads();
    const dim3 grid((unsigned)ln_groups(P.rows, bytes, sizeof(T)));
    if constexpr (LANES * K <= LN_WIDE) {
      if (sums) {
        hipLaunchKernelGGL((k_layer_norm_dx<T, LANES, K, THREADS, true>), grid, dim3(THREADS), 0, st, P);
        return;
      }
    }
    hipLaunchKernelGGL((k_layer_norm_dx<T, LANES, K, THREADS, false>), grid, dim3(THREADS), 0, st, P);
  });
  if (!sums) return;
  hipLaunchKernelGGL(k_layer_norm_join, dim3((unsigned)((P.D + LN_JOIN_COLS - 1) / LN_JOIN_COLS), 2), dim3(LN_COL_THREADS), 0, st, P);
}

}  // namespace

// Rows of a wave as far as its registers hold the sums' channels (gradient of 3 x 4093
// fp32 rows of 1001 elements: 31.7 us with 64 lanes of four pieces, 46 with 256 of one, or
// 36 with twice the workgroups).
LnShape ln_shape(int64_t bytes, int es) {
  const int64_t n = (bytes + 15) / 16;
  if (n <= 16) return {8, 2, 256};
  if (n <= 64) return {32, 2, 256};
  if (n <= 128) return {64, 2, 256};
  if (es == 4 && n <= 256) return {64, 4, 256};
  if (n <= 1024) return {256, n <= 256 ? 1 : n <= 512 ? 2 : 4, 256};
  return {1024, n <= 2048 ? 2 : 4, 1024};
}

static int ln_deal(int64_t rows, int64_t side, int most) { return (int)std::min<int64_t>((rows + side - 1) / side, most); }
static int ln_side(int64_t bytes, int es) { return ln_shape(bytes, es).threads / ln_shape(bytes, es).lanes; }
int ln_groups(int64_t rows, int64_t bytes, int es) { return ln_deal(rows, ln_side(bytes, es), LN_PARTS); }
int ln_parts(int64_t rows, int64_t bytes, int es) {
  return bytes > 16 * LN_WIDE ? ln_deal(rows, LN_COL_THREADS / LN_COLS, LN_PARTS) : ln_groups(rows, bytes, es);
}
int ln_grid(int64_t rows, int64_t bytes, int es) { return ln_deal(rows, ln_side(bytes, es), LN_GRID); }

hipError_t launch_layer_norm(const LnParams& P, bool bf16_path, hipStream_t st) {
  bf16_path ? forward<bf16>(P, st) : forward<float>(P, st);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const LnParams& P, bool bf16_path, hipStream_t st) {
  bf16_path ? backward<bf16>(P, st) : backward<float>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
