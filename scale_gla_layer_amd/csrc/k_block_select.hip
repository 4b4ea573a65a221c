// Block selection: mean keys of whole blocks, and for each query and key-value
// head the blocks it attends.
//
// The score of block j for query t is (sum over the group's heads of q_t) . c_j
// with c_j the block's mean key.  Sums are in 64 bits, where products of the
// inputs are all but exact: the choice is the inputs', not the summation
// order's.  The scores of 16 queries against 16 blocks are a chain of 64-bit
// MFMAs; their ordered bit patterns go to LDS, where one wave finds a row's
// n-th largest by bisection on the bits (a handful of steps: it stops once the
// count is right) and writes the chosen blocks in ascending order.
#include "block_device.hpp"

namespace msgla {

namespace {

typedef double d64x4 __attribute__((ext_vector_type(4)));

// Mean of the 2^lgT rows row(0) .. in 64 bits by one wave, to out (32 bits).
template <typename T, class Row>
__device__ __forceinline__ void block_mean(int lgT, int width, float* out, int lane, Row row) {
  constexpr int PER = per16<T>(), LPR = 128 / PER;  // lanes of a row: 128 elements at most
  const int pc = lane % LPR;
  double s[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) s[e] = 0.0;
  if (pc * 16 < width)
    for (int i = lane / LPR; i < (1 << lgT); i += 64 / LPR) {
      float v[PER];
      unpack16<T>(ld16(row(i) + pc * 16), v);
#pragma unroll
      for (int e = 0; e < PER; ++e) s[e] += (double)v[e];
    }
#pragma unroll
  for (int o = LPR; o < 64; o <<= 1)
#pragma unroll
    for (int e = 0; e < PER; ++e) s[e] += __shfl_xor(s[e], o);
  if (lane < LPR && pc * 16 < width) {
    const double inv = 1.0 / (double)(1 << lgT);
#pragma unroll
    for (int e = 0; e < PER; ++e) out[pc * PER + e] = (float)(s[e] * inv);
  }
}

template <typename T> __global__ __launch_bounds__(64) void k_block_means(const BlkParams P) {
  const int64_t bh = blockIdx.x / P.nb;
  const int j = (int)(blockIdx.x - bh * P.nb), b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  const int64_t end = (int64_t)(j + 1) << P.lgT;
  if (P.from && end <= P.from[b]) return;
  float* out = P.means + (bh * P.nb + j) * P.dkw;
  const int len = P.lens ? min(P.lens[b], P.S) : P.S;
  if (end > len) {
    for (int c = threadIdx.x; c < P.dkw; c += 64) out[c] = 0.f;
    return;
  }
  const char* base = P.k.p + b * P.k.sb + ((int64_t)j << P.lgT) * P.k.st + h * P.k.sh;
  block_mean<T>(P.lgT, P.dkw * (int)sizeof(T), out, threadIdx.x, [&](int i) { return base + i * P.k.st; });
}

// One token's key and value into the caches, and the mean of the block it completes.
template <typename T> __global__ __launch_bounds__(64) void k_block_append(const BlkParams P) {
  const int b = blockIdx.x / P.Hkv, h = blockIdx.x % P.Hkv, lane = threadIdx.x;
  const int p = P.start[b];
  if (p < 0 || p >= P.S) return;
  const char* nk = P.kt.p + b * P.kt.sb + h * P.kt.sh;
  const char* nv = P.vt.p + b * P.vt.sb + h * P.vt.sh;
  char* kr = P.k.p + b * P.k.sb + (int64_t)p * P.k.st + h * P.k.sh;
  char* vr = P.v.p + b * P.v.sb + (int64_t)p * P.v.st + h * P.v.sh;
  for (int c = 16 * lane; c < P.dkw * (int)sizeof(T); c += 1024) st16(kr + c, ld16(nk + c));
  for (int c = 16 * lane; c < P.dvw * (int)sizeof(T); c += 1024) st16(vr + c, ld16(nv + c));
  const int last = (1 << P.lgT) - 1;
  if ((p & last) != last) return;
  const int j = p >> P.lgT;
  const char* base = P.k.p + b * P.k.sb + ((int64_t)j << P.lgT) * P.k.st + h * P.k.sh;
  block_mean<T>(P.lgT, P.dkw * (int)sizeof(T), P.means + (((int64_t)b * P.Hkv + h) * P.nb + j) * P.dkw, lane,
                [&](int i) { return i == last ? nk : base + i * P.k.st; });
}

// Bits whose order as whole numbers is the scores' (a NaN ranks as minus infinity).
__device__ __forceinline__ uint64_t score_key(double s) {
  if (s != s) s = -__builtin_inf();
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  return u >> 63 ? ~u : u | (1ull << 63);
}

constexpr uint64_t FORCED = ~0ull;
constexpr int SEL_WAVES = 4, SEL_ROWS = 16;

template <typename T, int DKP, int PIECE> __global__ __launch_bounds__(64 * SEL_WAVES) void k_block_select(const BlkParams P) {
  __shared__ uint64_t key[SEL_ROWS][PIECE];
  __shared__ uint64_t ckey[SEL_ROWS][BLK_MAX_SEL];  // chosen so far, while pieces remain
  __shared__ int cblk[SEL_ROWS][BLK_MAX_SEL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, a = lane >> 4;
  const int per = (P.L + SEL_ROWS - 1) / SEL_ROWS;
  const int64_t bh = blockIdx.x / per;
  const int i0 = (int)(blockIdx.x - bh * per) * SEL_ROWS, b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  int32_t* out = P.sel_out + (bh * P.L + i0) * P.n;
  // a positions' own blocks: row l % 16 for every lane, and the greatest
  const int mypos = blk_position(P, b, i0 + c16);
  const int myown = mypos < 0 ? -1 : mypos >> P.lgT;
  int top = myown;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor(top, o));
  // the group's query sums, elements 16 g + 4 a .. + 3 of row l % 16
  double q[DKP / 16][4];
  {
    const char* qr = P.q.p + b * P.q.sb + (int64_t)min(i0 + c16, P.L - 1) * P.q.st + (int64_t)h * P.G * P.q.sh;
#pragma unroll
    for (int g = 0; g < DKP / 16; ++g) {
      const int e0 = 16 * g + 4 * a;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[g][e] = 0.0;
      if (e0 < P.dkw && mypos >= 0)
        for (int u = 0; u < P.G; ++u) {
          const T* p = reinterpret_cast<const T*>(qr + u * P.q.sh) + e0;
#pragma unroll
          for (int e = 0; e < 4; ++e) q[g][e] += (double)to_f32(p[e]);
        }
    }
  }
  const float* means = P.means + bh * P.nb * P.dkw;
  for (int i = threadIdx.x; i < SEL_ROWS * BLK_MAX_SEL; i += 64 * SEL_WAVES) ckey[i / BLK_MAX_SEL][i % BLK_MAX_SEL] = 0;
  int carried[SEL_ROWS / SEL_WAVES];
#pragma unroll
  for (int k = 0; k < SEL_ROWS / SEL_WAVES; ++k) carried[k] = 0;
  int piece = 0;
  do {
    const int stop = min(piece + PIECE, top + 1);  // blocks [piece, stop)
    for (int j0 = piece + 16 * wave; j0 < stop; j0 += 16 * SEL_WAVES) {
      const float* m = means + (int64_t)min(j0 + c16, top) * P.dkw;
      d64x4 s = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int g = 0; g < DKP / 16; ++g) {
        const int e0 = 16 * g + 4 * a;
        const bool in = e0 < P.dkw;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s = __builtin_amdgcn_mfma_f64_16x16x4f64(q[g][e], in ? (double)m[e0 + e] : 0.0, s, 0, 0, 0);
      }
      // element i: row l / 16 + 4 i, block l % 16
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = a + 4 * i, own = __shfl(myown, r), j = j0 + c16;
        uint64_t k = score_key(s[i]);
        if (j < P.n_first || j > own - P.n_recent) k = FORCED;
        if (j > own || j >= stop) k = 0;
        key[r][j - piece] = k;
      }
    }
    __syncthreads();
    const bool more = stop <= top;
    constexpr int SLOTS = PIECE / 64 + 1;
#pragma unroll
    for (int rr = 0; rr < SEL_ROWS / SEL_WAVES; ++rr) {
      const int r = wave * (SEL_ROWS / SEL_WAVES) + rr;
      if (i0 + r >= P.L) break;
      uint64_t k[SLOTS];
      const int cb = cblk[r][lane];
      k[0] = lane < carried[rr] ? ckey[r][lane] : 0;
#pragma unroll
      for (int e = 1; e < SLOTS; ++e) {
        const int j = piece + 64 * (e - 1) + lane;
        k[e] = j < stop ? key[r][j - piece] : 0;
      }
      auto count = [&](uint64_t t) {
        int c = 0;
#pragma unroll
        for (int e = 0; e < SLOTS; ++e) c += __popcll(__ballot(k[e] >= t));
        return c;
      };
      // the largest threshold that at least n keys reach (1, if there are no more than n)
      uint64_t t = 1;
      bool exact = true;
      if (count(1) > P.n) {
        t = 0;
        exact = false;
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t want = t | (1ull << bit);
          const int c = count(want);
          if (c >= P.n) {
            t = want;
            if (c == P.n) {
              exact = true;
              break;
            }
          }
        }
      }
      int ties = exact ? 65536 : P.n - count(t + 1);  // of the keys equal to t, the first so many
      int base = 0;
#pragma unroll
      for (int e = 0; e < SLOTS; ++e) {
        const uint64_t eq = __ballot(k[e] == t), below = (1ull << lane) - 1;
        const bool take = k[e] > t || (k[e] == t && (exact || (int)__popcll(eq & below) < ties));
        if (!exact) ties -= min(ties, (int)__popcll(eq));
        const uint64_t took = __ballot(take);
        if (take) {
          const int at = base + (int)__popcll(took & below);
          const int j = e == 0 ? cb : piece + 64 * (e - 1) + lane;
          if (more) {
            ckey[r][at] = k[e];
            cblk[r][at] = j;
          } else {
            out[(int64_t)r * P.n + at] = j;
          }
        }
        base += (int)__popcll(took);
      }
      carried[rr] = base;
      if (!more && lane >= base && lane < P.n) out[(int64_t)r * P.n + lane] = -1;
    }
    __syncthreads();
    piece += PIECE;
  } while (piece <= top);
}

template <typename T, int DKP> void select_t(const BlkParams& P, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)P.B * P.Hkv * ((P.L + SEL_ROWS - 1) / SEL_ROWS))), block(64 * SEL_WAVES);
  // the smaller score buffer lets five workgroups share a CU's LDS instead of two
  if (P.nb <= 128) hipLaunchKernelGGL((k_block_select<T, DKP, 128>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((k_block_select<T, DKP, BLK_PIECE>), grid, block, 0, st, P);
}

}  // namespace

hipError_t launch_block_means(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)P.B * P.Hkv * P.nb));
  if (bf16_path) hipLaunchKernelGGL(k_block_means<bf16>, grid, dim3(64), 0, st, P);
  else hipLaunchKernelGGL(k_block_means<float>, grid, dim3(64), 0, st, P);
  return hipGetLastError();
}

hipError_t launch_block_append(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const dim3 grid((unsigned)(P.B * P.Hkv));
  if (bf16_path) hipLaunchKernelGGL(k_block_append<bf16>, grid, dim3(64), 0, st, P);
  else hipLaunchKernelGGL(k_block_append<float>, grid, dim3(64), 0, st, P);
  return hipGetLastError();
}

hipError_t launch_block_select(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? select_t<bf16, 64>(P, st) : select_t<bf16, 128>(P, st);
  else k64 ? select_t<float, 64>(P, st) : select_t<float, 128>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
