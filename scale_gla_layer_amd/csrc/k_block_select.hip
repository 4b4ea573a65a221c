// Block selection: mean keys of whole blocks, and for each query and key-value
// head the blocks it attends.
//
// The score of block j for query t is (sum over the group's heads of q_t) . c_j
// with c_j the block's mean key.  Sums are in 64 bits, where products of the
// inputs are all but exact: the choice is the inputs', not the summation
// order's.  The scores of 16 queries against 16 blocks are a chain of 64-bit
// MFMAs; their ordered bit patterns go to LDS.  There 16 lanes take a row, four
// rows a wave, and find its n-th largest key by bisection on the upper 32 bits
// (about 20 steps: each lane counts its own keys, four lane exchanges add up; a
// row is done once its count is right), going on to the lower ones only where
// that leaves a tie, and write the chosen blocks in ascending order.
//   At B = 2, L = 8192, 16 / 4 heads of 128, blocks of 64: the means 5.6 us, the
// choice 77, of which the 64-bit products are 15 and the reading of the queries 13;
// the rest is latency between a workgroup's stages, at 4 workgroups a CU.  (A
// bisection that starts between the row's least and greatest score needs half the
// steps and takes as long.)
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
#pragma unroll 8
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

// Bits whose order as whole numbers is the scores' (a NaN ranks as minus infinity).
__device__ __forceinline__ uint64_t score_key(double s) {
  if (s != s) s = -__builtin_inf();
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  return u >> 63 ? ~u : u | (1ull << 63);
}

constexpr uint64_t FORCED = ~0ull;
constexpr int SEL_WAVES = 4, SEL_ROWS = 16;

// Sum over the 16 lanes of a row group (DPP rotations within 16 lanes).
__device__ __forceinline__ int row16_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, false);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, false);
}
// the 16 bits of a wave's ballot that belong to the lane's row group
__device__ __forceinline__ uint32_t row16_ballot(bool v, int lane) {
  const uint64_t m = __ballot(v);
  return ((lane & 32 ? (uint32_t)(m >> 32) : (uint32_t)m) >> (lane & 16)) & 0xffffu;
}

// The largest T that at least n of a row's values reach, found bit by bit;
// count(T) is the number of values >= T.  exact: just n do.
template <class Count> __device__ __forceinline__ uint32_t bisect(int n, bool active, bool& exact, Count count) {
  uint32_t t = 0;
  exact = false;
  for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
    const uint32_t want = t | bit;
    const int c = count(want);
    if (!exact && c >= n) {
      t = want;
      exact = c == n;
    }
    if (__all(exact || !active)) break;
  }
  return t;
}

template <typename T, int DKP, int PIECE> __global__ __launch_bounds__(64 * SEL_WAVES) void k_block_select(const BlkParams P) {
  constexpr bool MULTI = PIECE == BLK_PIECE;  // more blocks than one piece holds, perhaps
  constexpr int CARRY = MULTI ? BLK_MAX_SEL : 1, CS = MULTI ? BLK_MAX_SEL / 16 : 0, SLOTS = CS + PIECE / 16;
  constexpr int QP = DKP + 2, PER = DKP / 16;  // row pitch of the query sums; elements a thread sums
  __shared__ double qsum[SEL_ROWS][QP];
  __shared__ uint64_t key[SEL_ROWS][PIECE];
  __shared__ uint64_t ckey[SEL_ROWS][CARRY];  // chosen so far, while pieces remain
  __shared__ int cblk[SEL_ROWS][CARRY];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, a = lane >> 4;
  const int per = (P.L + SEL_ROWS - 1) / SEL_ROWS;
  const int64_t bh = blockIdx.x / per;
  const int i0 = (int)(blockIdx.x - bh * per) * SEL_ROWS, b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  int32_t* out = P.sel_out + (bh * P.L + i0) * P.n;
  // the positions' own blocks: row l % 16 for every lane, and the greatest
  const int mypos = blk_position(P, b, i0 + c16);
  const int myown = mypos < 0 ? -1 : mypos >> P.lgT;
  int top = myown;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor(top, o));
  {
    // the group's query sums, PER elements of a row each thread
    const int r = threadIdx.x >> 4, e0 = c16 * PER;
    double q[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) q[e] = 0.0;
    if (e0 < P.dkw && blk_position(P, b, i0 + r) >= 0) {
      const char* qr = P.q.p + b * P.q.sb + (int64_t)(i0 + r) * P.q.st + (int64_t)h * P.G * P.q.sh + e0 * sizeof(T);
      for (int u = 0; u < P.G; ++u) {
        const char* p = qr + u * P.q.sh;  // d_k is a multiple of 8
        float f[8];
        if constexpr (PER * sizeof(T) == 8) {
          const u32x2 w = ld8(p);
          unpack16<T>(u32x4{w[0], w[1], 0u, 0u}, f);
        } else {
          unpack16<T>(ld16(p), f);
          if constexpr (PER * sizeof(T) == 32) unpack16<T>(ld16(p + 16), f + 4);
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) q[e] += (double)f[e];
      }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) qsum[r][e0 + e] = q[e];
  }
  const float* means = P.means + bh * P.nb * P.dkw;
  __syncthreads();
  double q[DKP / 16][4];  // elements 16 g + 4 a .. + 3 of row l % 16
#pragma unroll
  for (int g = 0; g < DKP / 16; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) q[g][e] = qsum[c16][16 * g + 4 * a + e];
  int carried = 0, piece = 0;
  do {
    const int stop = min(piece + PIECE, top + 1);  // blocks [piece, stop)
    for (int j0 = piece + 16 * wave; j0 < stop; j0 += 16 * SEL_WAVES) {
      const float* m = means + (int64_t)min(j0 + c16, top) * P.dkw;
      d64x4 s = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int g = 0; g < DKP / 16; ++g) {
        const int e0 = 16 * g + 4 * a;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (e0 < P.dkw) unpack16<float>(ld16(m + e0), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f64_16x16x4f64(q[g][e], (double)f[e], s, 0, 0, 0);
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
    const int r = 4 * wave + a, slots = (stop - piece + 15) >> 4;  // the lane's row; its keys c16, c16 + 16, ..
    uint32_t k[SLOTS];
#pragma unroll
    for (int e = 0; e < CS; ++e) k[e] = 16 * e + c16 < carried ? (uint32_t)(ckey[r][16 * e + c16] >> 32) : 0;
#pragma unroll
    for (int e = CS; e < SLOTS; ++e) k[e] = e - CS < slots ? (uint32_t)(key[r][16 * (e - CS) + c16] >> 32) : 0;
    auto low = [&](int e) -> uint32_t {  // of a key whose upper half is not 0
      return e < CS ? (uint32_t)ckey[r][16 * e + c16] : (uint32_t)key[r][16 * (e - CS) + c16];
    };
    auto count = [&](uint32_t t) {
      int c = 0;
#pragma unroll
      for (int e = 0; e < SLOTS; ++e)
        if (e < CS || e - CS < slots) c += k[e] >= t ? 1 : 0;
      return row16_sum(c);
    };
    // Every score's upper half is above 0 (minus infinity's is 0x000fffff).  With
    // n of them or fewer all are taken.
    uint32_t hi = 1, lo = 0;
    bool all_hi = true, all_lo = true;  // every key with that upper half is taken; every one that reaches (hi, lo)
    int ties = 0;
    const int total = count(1);
    if (__any(total > P.n)) {
      const bool cut = total > P.n;
      bool exact;
      const uint32_t t = bisect(P.n, cut, exact, count);
      if (cut) hi = t, all_hi = exact;
      if (!__all(all_hi)) {
        const int above = hi == ~0u ? 0 : count(hi + 1), want = P.n - above;
        auto count_low = [&](uint32_t t2) {
          int c = 0;
          for (int e = 0; e < SLOTS; ++e)
            if ((e < CS || e - CS < slots) && k[e] == hi) c += low(e) >= t2 ? 1 : 0;
          return row16_sum(c);
        };
        const uint32_t t2 = bisect(want, !all_hi, exact, count_low);
        lo = t2;
        all_lo = exact;
        ties = want - (t2 == ~0u ? 0 : count_low(t2 + 1));
      }
    }
    int base = 0;
#pragma unroll
    for (int e = 0; e < SLOTS; ++e) {
      if (e >= CS && e - CS >= slots) continue;
      bool take = k[e] > hi || (k[e] == hi && all_hi);
      if (!__all(all_hi)) {
        const uint32_t l = k[e] == hi ? low(e) : 0;
        const bool equal = !all_hi && k[e] == hi && l == lo;
        const uint32_t eq = row16_ballot(equal, lane);
        const int before = __popc(eq & ((1u << c16) - 1));
        take = take || (!all_hi && k[e] == hi && l > lo) || (equal && (all_lo || before < ties));
        ties -= min(ties, (int)__popc(eq));
      }
      const uint32_t took = row16_ballot(take, lane);
      if (take) {
        const int at = base + (int)__popc(took & ((1u << c16) - 1));
        const int j = e < CS ? cblk[r][16 * e + c16] : piece + 16 * (e - CS) + c16;
        if (more) {
          // lists only shrink: entry `at` of the next list was read with this slot or before
          ckey[r][at] = e < CS ? ckey[r][16 * e + c16] : key[r][16 * (e - CS) + c16];
          cblk[r][at] = j;
        } else if (i0 + r < P.L) {
          out[(int64_t)r * P.n + at] = j;
        }
      }
      base += (int)__popc(took);
    }
    carried = base;
    if (!more && i0 + r < P.L)
      for (int e = base + c16; e < P.n; e += 16) out[(int64_t)r * P.n + e] = -1;
    __syncthreads();
    piece += PIECE;
  } while (piece <= top);
}

// The streaming step's first half.  A wave puts the token's key and value into
// the caches and renews the mean of the block that this completes (which is the
// query's own: it is not scored); the blocks before are scored, four lanes a
// block; a wave finds the best of up to STEP_PIECE at a time, 64 lanes on the one
// row.  Up to BLK_STEP_ONE blocks, one workgroup a sequence and key-value head
// does it all; of longer caches the scores are spread over more workgroups, and
// the choice is a launch of its own.  (512 blocks, 64 sequences and heads: 10 + 6
// us, in one workgroup each 23; 64 blocks: one launch, whose cost on the host is
// what a second would add.)
constexpr int STEP_WAVES = 8, STEP_PIECE = 512;
static_assert(BLK_STEP_ONE <= STEP_PIECE, "one piece, whose scores fit in LDS");

template <typename T> __device__ __forceinline__ void step_append(const BlkParams& P, int b, int h, int p, int lane) {
  const char* nk = P.kt.p + b * P.kt.sb + h * P.kt.sh;
  const char* nv = P.vt.p + b * P.vt.sb + h * P.vt.sh;
  char* kr = P.k.p + b * P.k.sb + (int64_t)p * P.k.st + h * P.k.sh;
  char* vr = P.v.p + b * P.v.sb + (int64_t)p * P.v.st + h * P.v.sh;
  for (int c = 16 * lane; c < P.dkw * (int)sizeof(T); c += 1024) st16(kr + c, ld16(nk + c));
  for (int c = 16 * lane; c < P.dvw * (int)sizeof(T); c += 1024) st16(vr + c, ld16(nv + c));
  const int last = (1 << P.lgT) - 1, own = p >> P.lgT;
  if ((p & last) == last) {
    const char* base = P.k.p + b * P.k.sb + ((int64_t)own << P.lgT) * P.k.st + h * P.k.sh;
    block_mean<T>(P.lgT, P.dkw * (int)sizeof(T), P.means + (((int64_t)b * P.Hkv + h) * P.nb + own) * P.dkw, lane,
                  [&](int i) { return i == last ? nk : base + i * P.k.st; });
  }
}

// key[j] of the blocks first, first + stride, .. before stop, by four lanes each.
// The whole workgroup comes here; qsum: DKP doubles of LDS.
template <typename T, int DKP>
__device__ __forceinline__ void step_scores(const BlkParams& P, int b, int h, int own, int first, int stride, int stop,
                                            int tid, double* qsum, uint64_t* key) {
  constexpr int PER = DKP / 4;
  const int e0 = (tid & 3) * PER;  // the lane's elements
  const float* means = P.means + ((int64_t)b * P.Hkv + h) * P.nb * P.dkw;
  float m[PER];
  auto load = [&](int j) {
#pragma unroll
    for (int c = 0; c < PER; c += 4)
      if (e0 + c < P.dkw) unpack16<float>(ld16(means + (int64_t)min(j, own) * P.dkw + e0 + c), m + c);
  };
  load(first);
  if (tid < DKP) {  // the group's query sums
    double q = 0.0;
    if (tid < P.dkw) {
      const char* qr = P.q.p + b * P.q.sb + (int64_t)h * P.G * P.q.sh + tid * sizeof(T);
#pragma unroll 8
      for (int u = 0; u < P.G; ++u) q += (double)to_f32(*reinterpret_cast<const T*>(qr + u * P.q.sh));
    }
    qsum[tid] = q;
  }
  __syncthreads();
  for (int j = first; j - ((tid & 63) >> 2) < stop; j += stride) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < PER; ++c)
      if (e0 + c < P.dkw) s += qsum[e0 + c] * (double)m[c];
    if (j + stride - ((tid & 63) >> 2) < stop) load(j + stride);
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    if ((tid & 3) == 0 && j < stop) key[j] = j < P.n_first || j > own - P.n_recent ? FORCED : score_key(s);
  }
}

// A wave's choice among the blocks 0 .. own, in ascending order to out.
__device__ __forceinline__ void step_choose(const BlkParams& P, int own, const uint64_t* key, int32_t* out, int lane) {
  constexpr int SLOTS = STEP_PIECE / 64 + 1;
  __shared__ uint64_t ckey[64];  // chosen so far, while pieces remain
  __shared__ int cblk[64];
  int carried = 0, piece = 0;
  do {
    const int stop = min(piece + STEP_PIECE, own + 1);
    const bool more = stop <= own;
    uint64_t k[SLOTS];
    const int cb = cblk[lane];
    k[0] = lane < carried ? ckey[lane] : 0;
#pragma unroll
    for (int e = 1; e < SLOTS; ++e) {
      const int j = piece + 64 * (e - 1) + lane;
      k[e] = j < stop ? key[j] : 0;
    }
    // as in k_block_select, the row's values in all lanes: the upper halves first,
    // the lower ones where those tie
    auto count = [&](auto reach) {
      int c = 0;
#pragma unroll
      for (int e = 0; e < SLOTS; ++e) c += (int)__popcll(__ballot(reach((uint32_t)(k[e] >> 32), (uint32_t)k[e])));
      return c;
    };
    auto largest = [&](int n, bool& exact, auto reach) {
      uint32_t t = 0;
      exact = false;
      for (uint32_t bit = 1u << 31; bit && !exact; bit >>= 1) {
        const int c = count([&](uint32_t u, uint32_t v) { return reach(u, v, t | bit); });
        if (c >= n) t |= bit, exact = c == n;
      }
      return t;
    };
    uint32_t hi = 1, lo = 0;
    bool all_hi = true, all_lo = true;
    int ties = 0;
    if (count([](uint32_t u, uint32_t) { return u != 0; }) > P.n) {
      hi = largest(P.n, all_hi, [](uint32_t u, uint32_t, uint32_t t) { return u >= t; });
      if (!all_hi) {
        const int want = P.n - count([&](uint32_t u, uint32_t) { return u > hi; });
        lo = largest(want, all_lo, [&](uint32_t u, uint32_t v, uint32_t t) { return u == hi && v >= t; });
        ties = want - count([&](uint32_t u, uint32_t v) { return u == hi && v > lo; });
      }
    }
    int base = 0;
    const uint64_t below = (1ull << lane) - 1, cut = (uint64_t)hi << 32 | lo;
#pragma unroll
    for (int e = 0; e < SLOTS; ++e) {
      const uint32_t u = (uint32_t)(k[e] >> 32);
      const uint64_t eq = __ballot(!all_hi && k[e] == cut);
      const bool take = all_hi ? u >= hi : k[e] > cut || (k[e] == cut && (all_lo || (int)__popcll(eq & below) < ties));
      ties -= min(ties, (int)__popcll(eq));
      const uint64_t took = __ballot(take);
      if (take) {
        const int at = base + (int)__popcll(took & below), j = e == 0 ? cb : piece + 64 * (e - 1) + lane;
        if (more) {
          ckey[at] = k[e];
          cblk[at] = j;
        } else {
          out[at] = j;
        }
      }
      base += (int)__popcll(took);
    }
    carried = base;
    asm volatile("" ::: "memory");  // the wave's own LDS writes, before the next piece's reads
    if (!more && lane >= base && lane < P.n) out[lane] = -1;
    piece += STEP_PIECE;
  } while (piece <= own);
}

// One workgroup a sequence and head: everything (SPREAD false); or gridDim.y - 1
// that score and one that appends, with the choice to come.
template <typename T, int DKP, bool SPREAD> __global__ __launch_bounds__(64 * STEP_WAVES) void k_block_step(const BlkParams P) {
  __shared__ uint64_t lds[SPREAD ? 1 : BLK_STEP_ONE];
  __shared__ double qsum[DKP];
  const int b = blockIdx.x / P.Hkv, h = blockIdx.x % P.Hkv, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int p = P.start[b], own = p >> P.lgT;
  int32_t* out = P.sel_out + (int64_t)blockIdx.x * P.n;
  if (p < 0 || p >= P.S) {
    if (!SPREAD && tid < P.n) out[tid] = -1;
    return;
  }
  const int scorers = SPREAD ? (int)gridDim.y - 1 : 1;
  if (!SPREAD || (int)blockIdx.y < scorers) {
    uint64_t* key = SPREAD ? P.bits + (int64_t)blockIdx.x * P.nb : lds;
    step_scores<T, DKP>(P, b, h, own, (int)blockIdx.y * 16 * STEP_WAVES + (tid >> 2), scorers * 16 * STEP_WAVES,
                        own + 1, tid, qsum, key);
    if constexpr (SPREAD) return;
    __syncthreads();
    if (wave == 0) step_choose(P, own, key, out, lane);
  }
  if (wave == STEP_WAVES - 1) step_append<T>(P, b, h, p, lane);
}

__global__ __launch_bounds__(64) void k_block_choose(const BlkParams P) {
  const int p = P.start[blockIdx.x / P.Hkv], lane = threadIdx.x;
  int32_t* out = P.sel_out + (int64_t)blockIdx.x * P.n;
  if (p >= 0 && p < P.S) step_choose(P, p >> P.lgT, P.bits + (int64_t)blockIdx.x * P.nb, out, lane);
  else if (lane < P.n) out[lane] = -1;
}

template <typename T, int DKP> void step_t(const BlkParams& P, hipStream_t st) {
  const unsigned bh = (unsigned)(P.B * P.Hkv);
  if (blk_step_spread(P)) {
    const dim3 grid(bh, (unsigned)((P.nb + 16 * STEP_WAVES - 1) / (16 * STEP_WAVES) + 1));
    hipLaunchKernelGGL((k_block_step<T, DKP, true>), grid, dim3(64 * STEP_WAVES), 0, st, P);
    hipLaunchKernelGGL(k_block_choose, dim3(bh), dim3(64), 0, st, P);
  } else {
    hipLaunchKernelGGL((k_block_step<T, DKP, false>), dim3(bh), dim3(64 * STEP_WAVES), 0, st, P);
  }
}

template <typename T, int DKP> void select_t(const BlkParams& P, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)P.B * P.Hkv * ((P.L + SEL_ROWS - 1) / SEL_ROWS))), block(64 * SEL_WAVES);
  // the smaller score buffer lets four workgroups share a CU's LDS instead of two (d_k up to 64: six and three)
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

hipError_t launch_block_step(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? step_t<bf16, 64>(P, st) : step_t<bf16, 128>(P, st);
  else k64 ? step_t<float, 64>(P, st) : step_t<float, 128>(P, st);
  return hipGetLastError();
}

hipError_t launch_block_select(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? select_t<bf16, 64>(P, st) : select_t<bf16, 128>(P, st);
  else k64 ? select_t<float, 64>(P, st) : select_t<float, 128>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
