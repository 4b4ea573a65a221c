// Attention over selected blocks for many queries: forward and the gradient of
// the queries with keys and values shared by a workgroup.
//
// A workgroup takes NW * RT neighbouring tiles of 16 (query, head) rows, RT of
// them a wave, and walks the union of all its queries' blocks in ascending
// order, KT keys a unit.  A unit's keys and values are copied asynchronously
// into one of two LDS stages while the other is worked on, with one barrier a
// unit; a wave none of whose rows chose the block goes straight to the next
// barrier.  The tiles' rows keep their outputs in registers throughout, so
// what is paid per unit is one copy from L2 for the workgroup, one pass over
// the LDS stage per wave, and the products.
//
// Stage rows hold their 16-byte pieces XOR-swizzled by the row, so that both
// readers are free of bank conflicts: 16 rows at one piece (the A operand of
// S^T = K Q^T), and 16 rows' columns (the A operand of O^T = V^T P^T, through
// the transpose read).  The running maximum follows a row's true one only when
// that has grown by more than 8 (in units of log 2), so weights stay below 2^8
// and the outputs are rescaled a few times in all instead of every unit.
#include "async_copy.hpp"
#include "block_device.hpp"

namespace msgla {

namespace {

// A stage tile of rows of W pieces.
template <int W> __device__ __forceinline__ constexpr int tile_key(int r) { return W == 8 ? (r >> 1) & 7 : r & 15; }

// A wave's share of the copy of rows key0 .. key0 + KT - 1 (row `last` again
// behind it: rows there have weight 0 and must hold numbers).  Pieces behind
// the head's width repeat its first: they meet zeroes or columns that are not
// stored.
template <int W, int KT, int NW>
__device__ __forceinline__ void copy_rows(const char* base, int64_t st, int key0, int last, int width, char* lds,
                                          int wave, int lane) {
  static_assert(KT * W % (64 * NW) == 0, "whole copy instructions for every wave");
#pragma unroll
  for (int k = 0; k < KT * W / 64 / NW; ++k) {
    const int i = wave + k * NW, pc = 64 * i + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
    dma16(base + (int64_t)min(key0 + r, last) * st + (p * 16 < width ? p * 16 : 0), lds + 1024 * i);
  }
}

// Column reader: slab s's rows at columns 16 t .. + 15 (layout of blk_column).
template <typename T, int W> struct Columns;
template <int W> struct Columns<bf16, W> {
  int at;
  __device__ Columns(int lane) {
    const int a = lane >> 4, e = (lane >> 2) & 3, c = lane & 3, r = 4 * a + e;
    at = r * W * 16 + (((c >> 1) ^ tile_key<W>(r)) * 16) + 8 * (c & 1);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    const char* p = lds + (at ^ (32 * t)) + s * 32 * W * 16;
    const blk_v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)p);
    const blk_v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((blk_lds_v4s*)(p + 16 * W * 16));
    const u32x2 x = __builtin_bit_cast(u32x2, lo), y = __builtin_bit_cast(u32x2, hi);
    return u32x4{x[0], x[1], y[0], y[1]};
  }
};
template <int W> struct Columns<float, W> {
  static_assert(W >= 16, "swizzle of four bits");
  int at[4];
  __device__ Columns(int lane) {
    const int a = lane >> 4, c = lane & 15;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * a + j;
      at[j] = r * W * 16 + (((c >> 2) ^ tile_key<W>(r)) * 16) + 4 * (c & 3);
    }
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int s, int t) const {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(lds + (at[j] ^ (64 * t)) + s * 16 * W * 16);
    return v;
  }
};

// Row reader: slab w of rows 16 kt + l % 16.
template <int W> struct Rows {
  int at;
  __device__ Rows(int lane) {
    const int c = lane & 15, a = lane >> 4;
    at = c * W * 16 + ((a ^ tile_key<W>(c)) * 16);
  }
  __device__ __forceinline__ u32x4 read(const char* lds, int kt, int w) const {
    return ld16(lds + (at ^ (64 * w)) + kt * 16 * W * 16);
  }
};

// The units of a workgroup: the set bits of `map` in ascending order, a block's
// KT-key parts in turn, up to the last position.
struct Units {
  const uint32_t* map;
  int words, w = -1, j = 0, k0 = 0;
  uint32_t bits = 0;
  __device__ bool next(int lgT, int kt, int last) {
    if (w >= 0 && k0 + kt < (j + 1) << lgT && k0 + kt <= last) {
      k0 += kt;
      return true;
    }
    while (!bits) {
      if (++w >= words) return false;
      bits = __builtin_amdgcn_readfirstlane(map[w]);
    }
    j = 32 * w + __builtin_ctz(bits);
    bits &= bits - 1;
    k0 = j << lgT;
    return true;
  }
};

constexpr float GROWTH = 8.f;

template <typename T, int DKP, int DVP, int KT, int RT, int NW, bool GRAD>
__global__ __launch_bounds__(64 * NW) void k_block_tiles(const BlkParams P) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16;
  constexpr int NK = DKP * ES / 64, NV = DVP * ES / 64, KEY_T = KT / 16, SLABS = KT / blk_slab<T>();
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16, NT = NW * RT;
  constexpr int OUT = GRAD ? DKP : DVP;  // width of the accumulated rows
  extern __shared__ __attribute__((aligned(16))) char smem[];
  uint32_t* map = reinterpret_cast<uint32_t*>(smem + 2 * STAGE);
  const int words = (P.nb + 31) / 32, pitch = P.n + 1;
  uint16_t* lists = reinterpret_cast<uint16_t*>(map + words);  // [queries][n + 1], ended by 0xffff
  __shared__ int slast;
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, a = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = (P.tiles_per_seq + NT - 1) / NT;
  // each XCD takes one contiguous range of the groups, whose blocks meet in its L2
  const int64_t work = (int64_t)(blockIdx.x % N_XCD) * (gridDim.x / N_XCD) + blockIdx.x / N_XCD;
  if (work >= (int64_t)P.B * P.Hkv * groups) return;
  const int64_t bh = work / groups;
  // the last tiles, which have the most blocks, first
  const int t0 = (groups - 1 - (int)(work - bh * groups)) * NT;
  const int b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  const int q0 = P.GT > 1 ? t0 / P.GT : t0 * P.QT;  // the first query
  const int qn = P.GT > 1 ? (t0 + NT - 1) / P.GT - q0 + 1 : NT * P.QT;

  // lists and their union: the raw rows of sel through LDS (the stages are not in use yet)
  for (int i = tid; i < words; i += 64 * NW) map[i] = 0;
  if (tid == 0) slast = -1;
  int* raw = reinterpret_cast<int*>(smem);
  {
    const int rows = min(qn, P.L - q0);
    const int32_t* sel = P.sel + (bh * P.L + q0) * P.n;
    for (int i = tid; i < rows * P.n; i += 64 * NW) raw[i] = sel[i];
  }
  __syncthreads();
  for (int s = tid; s < qn; s += 64 * NW) {
    const int p = blk_position(P, b, q0 + s);
    uint16_t* l = lists + s * pitch;
    l[blk_chosen(P, raw + s * P.n, p, [&](int n, int j) {
      l[n] = (uint16_t)j;
      atomicOr(&map[j >> 5], 1u << (j & 31));
    })] = 0xffff;
    if (p >= 0) atomicMax(&slast, p);
  }

  const int kw = P.dkw * ES, vw = P.dvw * ES;
  u32x4 q[RT][NK], g[GRAD ? RT : 1][GRAD ? NV : 1];
  BlkRow row[RT];
  float m[RT], l[RT];  // forward: the reference maximum and the sum; gradient: lse and delta
  const uint16_t* at[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int t = t0 + wave * RT + rt;
    BlkTile tile(P, bh * P.tiles_per_seq + min(t, P.tiles_per_seq - 1));
    row[rt] = tile.row(P, c16);
    if (t >= P.tiles_per_seq) row[rt].in = false, row[rt].p = -1;
    const bool live = row[rt].in && row[rt].p >= 0;
    const int64_t i = live ? row[rt].i : 0, hd = live ? row[rt].head : 0;
    const char* qr = P.q.p + b * P.q.sb + i * P.q.st + hd * P.q.sh;
#pragma unroll
    for (int s = 0; s < NK; ++s) q[rt][s] = live ? blk_ld(qr, 64 * s + 16 * a, kw) : zero16();
    m[rt] = -__builtin_inff();
    l[rt] = 0.f;
    if constexpr (GRAD) {
      const char* gr = P.dout.p + b * P.dout.sb + i * P.dout.st + hd * P.dout.sh;
#pragma unroll
      for (int s = 0; s < NV; ++s) g[rt][s] = live ? blk_ld(gr, 64 * s + 16 * a, vw) : zero16();
      if (live) {
        const int64_t lr = ((int64_t)b * P.Hq + hd) * P.L + i;
        m[rt] = P.lse_in[lr] * BLK_LOG2E;
        l[rt] = P.delta[lr];
      }
    }
    at[rt] = lists + (live ? row[rt].i - q0 : 0) * pitch;
  }
  __syncthreads();
  const int last = __builtin_amdgcn_readfirstlane(slast);
  int cur[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) cur[rt] = row[rt].in && row[rt].p >= 0 ? *at[rt] : 0xffff;
  f32x4 acc[RT][OUT / 16];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int d = 0; d < OUT / 16; ++d) acc[rt][d] = zero4();
  const float sc = P.scale * BLK_LOG2E;
  const char* kbase = P.k.p + b * P.k.sb + h * P.k.sh;
  const char* vbase = P.v.p + b * P.v.sb + h * P.v.sh;
  const Rows<WK> krow(lane);
  const Rows<WV> vrow(lane);
  const Columns<T, GRAD ? WK : WV> col(lane);

  Units u;
  u.map = map;
  u.words = words;
  bool more = u.next(P.lgT, KT, last);
  auto issue = [&](int stage) {
    char* st = smem + stage * STAGE;
    copy_rows<WK, KT, NW>(kbase, P.k.st, u.k0, last, kw, st, wave, lane);
    copy_rows<WV, KT, NW>(vbase, P.v.st, u.k0, last, vw, st + KB, wave, lane);
  };
  if (more) issue(0);
  bool member[RT];
  int block = -1;
  for (int t = 0; more; ++t) {
    const int j = u.j, k0 = u.k0;
    more = u.next(P.lgT, KT, last);
    wait_vmcnt<0>();
    lds_barrier();
    if (more) issue((t + 1) & 1);
    if (j != block) {
      block = j;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        member[rt] = cur[rt] == j;
        if (member[rt]) cur[rt] = *++at[rt];
      }
    }
    bool any = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) any |= member[rt] && k0 <= row[rt].p;
    if (!__any(any)) continue;
    const char *ks = smem + (t & 1) * STAGE, *vs = ks + KB;
    float p[RT][KEY_T][4];
#pragma unroll
    for (int kt = 0; kt < KEY_T; ++kt) {
      f32x4 s[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt] = zero4();
#pragma unroll
      for (int w = 0; w < NK; ++w) {
        const u32x4 f = krow.read(ks, kt, w);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt] = mma_slab<T>(f, q[rt][w], s[rt]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int lim = member[rt] ? row[rt].p - k0 - 16 * kt - 4 * a : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[rt][kt][i] = i <= lim ? s[rt][i] * sc : -__builtin_inff();
      }
    }
    if constexpr (!GRAD) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = -__builtin_inff();
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, p[rt][kt][i]);
        mx = blk_quad_max(mx);
        if (__any(mx > m[rt] + GROWTH)) {  // from minus infinity, anything has grown
          const float n = fmaxf(m[rt], mx), ref = n == -__builtin_inff() ? 0.f : n;
          const float corr = __builtin_amdgcn_exp2f(m[rt] - ref);
          m[rt] = n;
          l[rt] *= corr;
#pragma unroll
          for (int d = 0; d < OUT / 16; ++d) acc[rt][d] *= corr;
        }
        const float ref = m[rt] == -__builtin_inff() ? 0.f : m[rt];
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[rt][kt][i] = __builtin_amdgcn_exp2f(p[rt][kt][i] - ref);
            l[rt] += p[rt][kt][i];
          }
      }
    } else {
#pragma unroll
      for (int kt = 0; kt < KEY_T; ++kt) {
        f32x4 dp[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) dp[rt] = zero4();
#pragma unroll
        for (int w = 0; w < NV; ++w) {
          const u32x4 f = vrow.read(vs, kt, w);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) dp[rt] = mma_slab<T>(f, g[rt][w], dp[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool on = p[rt][kt][i] != -__builtin_inff();
            p[rt][kt][i] = on ? __builtin_amdgcn_exp2f(p[rt][kt][i] - m[rt]) * (dp[rt][i] - l[rt]) * P.scale : 0.f;
          }
      }
    }
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      u32x4 w[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) w[rt] = blk_pack<T>(p[rt], s);
#pragma unroll
      for (int d = 0; d < OUT / 16; ++d) {
        const u32x4 f = col.read(GRAD ? ks : vs, s, d);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt][d] = mma_slab<T>(f, w[rt], acc[rt][d]);
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if constexpr (!GRAD) l[rt] = blk_quad_sum(l[rt]);
    if (!row[rt].in) continue;
    const BlkHeads& o = GRAD ? P.dq : P.o;
    const int width = GRAD ? P.dkw : P.dvw;
    char* out = o.p + row[rt].b * o.sb + (int64_t)row[rt].i * o.st + row[rt].head * o.sh;
    const float inv = GRAD ? 1.f : l[rt] > 0.f ? 1.f / l[rt] : l[rt] == 0.f ? 0.f : l[rt];
#pragma unroll
    for (int d = 0; d < OUT / 16; ++d) {
      const int c = 16 * d + 4 * a;
      const float v[4] = {acc[rt][d][0] * inv, acc[rt][d][1] * inv, acc[rt][d][2] * inv, acc[rt][d][3] * inv};
      if (c < width) blk_st4<T>(out + c * ES, v);
    }
    if (!GRAD && P.lse && a == 0)
      P.lse[((int64_t)row[rt].b * P.Hq + row[rt].head) * P.L + row[rt].i] =
          l[rt] == 0.f ? -__builtin_inff() : m[rt] * BLK_LN2 + logf(l[rt]);
  }
}

template <typename T, int DKP, int DVP, int KT, int RT, int NW, bool GRAD>
hipError_t launch_t(const BlkParams& P, hipStream_t st) {
  constexpr int STAGE = KT * (DKP + DVP) * (int)sizeof(T), NT = NW * RT;
  const int qn = P.GT > 1 ? NT / P.GT + 2 : NT * P.QT;
  static_assert(NT * BLK_ROWS * BLK_MAX_SEL * 4 <= 2 * STAGE, "the raw selection fits the stages");
  const int lds = 2 * STAGE + (P.nb + 31) / 32 * 4 + qn * (P.n + 1) * 2;
  const auto kernel = &k_block_tiles<T, DKP, DVP, KT, RT, NW, GRAD>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t groups = (P.tiles_per_seq + NT - 1) / NT, work = (int64_t)P.B * P.Hkv * groups;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((work + N_XCD - 1) / N_XCD * N_XCD)), dim3(64 * NW), lds, st, P);
  return hipGetLastError();
}

template <typename T, int DKP, int DVP, bool GRAD> hipError_t by_block(const BlkParams& P, hipStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (P.lgT == 5) return launch_t<T, DKP, DVP, 32, 1, 4, GRAD>(P, st);
    return launch_t<T, DKP, DVP, 64, 1, 8, GRAD>(P, st);
  } else {
    return launch_t<T, DKP, DVP, 32, 1, 4, GRAD>(P, st);
  }
}
template <typename T, int DKP, bool GRAD> hipError_t by_dv(const BlkParams& P, hipStream_t st) {
  if (blk_dvp(P.dvw) == 64) return by_block<T, DKP, 64, GRAD>(P, st);
  if (blk_dvp(P.dvw) == 128) return by_block<T, DKP, 128, GRAD>(P, st);
  return by_block<T, DKP, 256, GRAD>(P, st);
}
template <bool GRAD> hipError_t dispatch(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) return k64 ? by_dv<bf16, 64, GRAD>(P, st) : by_dv<bf16, 128, GRAD>(P, st);
  return k64 ? by_dv<float, 64, GRAD>(P, st) : by_dv<float, 128, GRAD>(P, st);
}

}  // namespace

hipError_t launch_block_tiles(const BlkParams& P, bool gradient, bool bf16_path, hipStream_t st) {
  return gradient ? dispatch<true>(P, bf16_path, st) : dispatch<false>(P, bf16_path, st);
}

}  // namespace msgla
