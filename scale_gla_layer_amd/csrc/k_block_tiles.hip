// Attention over selected blocks for many queries: forward and the gradient of
// the queries with keys and values shared by a workgroup.
//
// A workgroup takes 15 (or 11, 7, 3) neighbouring tiles of 16 (query, head) rows, one
// a wave, and walks the union of all its queries' blocks in ascending order, KT
// keys a unit.  One more wave copies each unit's keys and values once,
// asynchronously, into a ring of LDS stages; the tiles' waves work on the units
// that their own rows chose, each at its own pace.  What couples them are two
// kinds of counters in LDS: `filled`, the units copied so far, and done[w], the
// units wave w is finished with or does not need.  (With a barrier a unit
// instead, every unit costs the time of one that all waves need, though with
// selections that differ from query to query only a third of them do.)
//   Every wait ends: a tile's wave waits for a unit only after it has counted all
// earlier ones as done, and the copying wave counts every unit it has issued as
// filled before it waits for a stage, which the waves free in order.
//
// Bound by vector, matrix and LDS instructions, which take turns, and by the copying
// wave, which has one unit under way at a time.  So a unit is as long as a block (up
// to 64 keys), and everything that is one value a unit is kept out of the lanes:
// lists and their unions are bit maps that scalar instructions walk, the running
// maximum follows a row's true one only when that has grown by more than 8 (in
// units of log 2: weights stay below 2^8), and rows that have not chosen a block
// are masked on the packed weights.
#include <algorithm>

#include "block_stage.hpp"

namespace msgla {

namespace {

// One wave's copy of rows key0 .. key0 + KT - 1 (row `last` again behind it: rows
// there have weight 0 and must hold numbers).  Pieces behind the head's width
// repeat its first: they meet zeroes or columns that are not stored.
template <int W, int KT> struct RowCopy {
  static constexpr int N = KT * W / 64;  // copy instructions
  static_assert(KT * W % 64 == 0, "whole copy instructions");
  const char* base;
  int64_t st;
  uint32_t off[N];  // the lane's bytes from the first row, where 32 bits hold them
  __device__ RowCopy(const char* b, int64_t s, int width, int lane) : base(b), st(s) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pc = 64 * i + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
      off[i] = (uint32_t)r * (uint32_t)st + (p * 16 < width ? p * 16 : 0);
    }
  }
  __device__ __forceinline__ void issue(int key0, int last, int width, char* lds, int lane) const {
    if (key0 + KT - 1 <= last && st < (1 << 24)) {
      const char* first = base + (int64_t)key0 * st;
#pragma unroll
      for (int i = 0; i < N; ++i) dma16(first + off[i], lds + 1024 * i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int pc = 64 * i + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
        dma16(base + (int64_t)min(key0 + r, last) * st + (p * 16 < width ? p * 16 : 0), lds + 1024 * i);
      }
    }
  }
};

// The set bits of a map of blocks, in ascending order.
struct Blocks {
  const uint32_t* map;
  int words, w = -1;
  uint32_t bits = 0;
  __device__ Blocks(const uint32_t* m, int n) : map(m), words(n) {}
  __device__ int next() {  // -1 at the end
    while (!bits) {
      if (++w >= words) return -1;
      bits = __builtin_amdgcn_readfirstlane(map[w]);
    }
    const int b = __builtin_ctz(bits);
    bits &= bits - 1;
    return 32 * w + b;
  }
};

constexpr float GROWTH = 8.f;
constexpr int TILE_WAVES_MAX = 15, MIN_STAGES = 2;

// LDS counters between the waves of a workgroup
struct Ring {
  int filled;
  int done[TILE_WAVES_MAX + 1];
};
// one LDS word read or written as it stands (LDS operations of a wave stay in order)
__device__ __forceinline__ int ring_get(const int* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ void ring_put(int* p, int v) {
  asm volatile("" ::: "memory");
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// The copying wave.  Units are copied one after the other: the compiler does not know
// that the counters are apart from the rows that the copies write, and waits for all
// copies before it touches a counter, so the wait for all units before the last one
// leaves none under way, and a unit is announced when the one behind it has landed.
template <typename T, int DKP, int DVP, int KT, int WAVES>
__device__ __forceinline__ void fill_ring(const BlkParams& P, Ring* ring, char* ring_lds, int stages, Blocks blocks,
                                          int last, const char* kbase, const char* vbase, int lane) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16;
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16, COPIES = STAGE / 1024;
  const RowCopy<WK, KT> kc(kbase, P.k.st, P.dkw * ES, lane);
  const RowCopy<WV, KT> vc(vbase, P.v.st, P.dvw * ES, lane);
  wait_vmcnt<0>();
  int n = 0, stage = 0;
  for (int j = blocks.next(); j >= 0; j = blocks.next())
    for (int k0 = j << P.lgT; k0 < (j + 1) << P.lgT && k0 <= last; k0 += KT) {
      auto is_free = [&] { return __all(lane >= WAVES || ring_get(&ring->done[lane]) > n - stages); };
      if (!is_free()) {
        wait_vmcnt<0>();
        if (lane == 0) ring_put(&ring->filled, n);
        do __builtin_amdgcn_s_sleep(1);
        while (!is_free());
      }
      asm volatile("" ::: "memory");
      char* st = ring_lds + stage * STAGE;
      stage = stage + 1 == stages ? 0 : stage + 1;
      kc.issue(k0, last, P.dkw * ES, st, lane);
      vc.issue(k0, last, P.dvw * ES, st + KB, lane);
      wait_vmcnt<COPIES < 64 ? COPIES : 0>();  // all units before this one have landed
      if (lane == 0) ring_put(&ring->filled, n);
      ++n;
    }
  wait_vmcnt<0>();
  if (lane == 0) ring_put(&ring->filled, 0x7fffffff);
}

template <typename T, int DKP, int DVP, int KT, int WAVES, bool GRAD>
__global__ __launch_bounds__(64 * (WAVES + 1), WAVES == TILE_WAVES_MAX ? 4 : WAVES == 11 ? 3 : 2) void k_block_tiles(const BlkParams P, int stages) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16;
  constexpr int NK = DKP * ES / 64, NV = DVP * ES / 64, KEY_T = KT / 16, SLABS = KT / blk_slab<T>();
  constexpr int KB = KT * WK * 16, STAGE = KB + KT * WV * 16, NT = WAVES, THREADS = 64 * (WAVES + 1);
  constexpr int OUT = GRAD ? DKP : DVP;  // width of the accumulated rows
  constexpr bool EXACT = GRAD && ES == 2;  // delta put right
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int words = (P.nb + 31) / 32, pitch = P.n + 1;
  __shared__ int slast;
  __shared__ Ring ring;
  static_assert(sizeof(Ring) + sizeof(int) <= 128, "in TILE_STATIC, with room to align");
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, a = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Work in order of length, the last tiles, which have the most blocks, first;
  // an XCD (block id mod 8) keeps to its own sequences and heads, whose blocks
  // meet in its L2.
  const int groups = (P.tiles_per_seq + NT - 1) / NT, heads = P.B * P.Hkv;
  int bh, rank;
  if (heads >= N_XCD) {
    const int x = blockIdx.x % N_XCD, s = blockIdx.x / N_XCD, mine = (heads - x + N_XCD - 1) / N_XCD;
    rank = s / mine;
    bh = x + N_XCD * (s - rank * mine);
  } else {
    rank = blockIdx.x / heads;
    bh = blockIdx.x - rank * heads;
  }
  if constexpr (GRAD) blk_clear_counts(P, tid, THREADS);
  if (rank >= groups) return;
  const int t0 = (groups - 1 - rank) * NT;
  const int b = bh / P.Hkv, h = bh - b * P.Hkv;
  const int q0 = P.GT > 1 ? t0 / P.GT : t0 * P.QT;  // the first query
  const int qn = P.GT > 1 ? (t0 + NT - 1) / P.GT - q0 + 1 : NT * P.QT;
  // maps of the blocks: all queries', and each tile's (of several tiles of one query: the query's)
  uint32_t* map = reinterpret_cast<uint32_t*>(smem + stages * STAGE);
  uint32_t* tmaps = map + words;
  uint16_t* lists = reinterpret_cast<uint16_t*>(tmaps + NT * words);  // [queries][n + 1], ended by 0xffff

  // the raw rows of sel through LDS (the stages are not in use yet)
  for (int i = tid; i < (NT + 1) * words; i += THREADS) map[i] = 0;
  if (tid == 0) slast = -1, ring.filled = 0;
  if (tid < WAVES) ring.done[tid] = 0;
  int* raw = reinterpret_cast<int*>(smem);
  {
    const int rows = min(qn, P.L - q0);
    const int32_t* sel = P.sel + ((int64_t)bh * P.L + q0) * P.n;
    for (int i = tid; i < rows * P.n; i += THREADS) raw[i] = sel[i];
  }
  __syncthreads();
  for (int s = tid; s < qn; s += THREADS) {
    const int p = blk_position(P, b, q0 + s);
    uint16_t* l = lists + s * pitch;
    uint32_t* own = tmaps + (P.GT > 1 ? s : s / P.QT) * words;
    l[blk_chosen(P, raw + s * P.n, p, [&](int n, int j) {
      l[n] = (uint16_t)j;
      atomicOr(&map[j >> 5], 1u << (j & 31));
      atomicOr(&own[j >> 5], 1u << (j & 31));
    })] = 0xffff;
    if (p >= 0) atomicMax(&slast, p);
  }
  __syncthreads();
  const int last = __builtin_amdgcn_readfirstlane(slast);
  if (wave == WAVES) {
    fill_ring<T, DKP, DVP, KT, WAVES>(P, &ring, smem, stages, Blocks(map, words), last, P.k.p + b * P.k.sb + h * P.k.sh,
                               P.v.p + b * P.v.sb + h * P.v.sh, lane);
    return;
  }

  const int kw = P.dkw * ES, vw = P.dvw * ES, t = t0 + wave;
  BlkRow row = BlkTile(P, (int64_t)bh * P.tiles_per_seq + min(t, P.tiles_per_seq - 1)).row(P, c16);
  if (t >= P.tiles_per_seq) row.in = false, row.p = -1;
  const bool live = row.in && row.p >= 0;
  u32x4 q[NK], g[GRAD ? NV : 1];
  float nref = 0.f, l = 0.f;  // forward: minus the reference maximum, the sum; gradient: minus lse, delta
  {
    const int64_t li = live ? row.i : 0, hd = live ? row.head : 0;
    const char* qr = P.q.p + b * P.q.sb + li * P.q.st + hd * P.q.sh;
#pragma unroll
    for (int s = 0; s < NK; ++s) q[s] = live ? blk_ld(qr, 64 * s + 16 * a, kw) : zero16();
    if constexpr (GRAD) {
      const char* gr = P.dout.p + b * P.dout.sb + li * P.dout.st + hd * P.dout.sh;
#pragma unroll
      for (int s = 0; s < NV; ++s) g[s] = live ? blk_ld(gr, 64 * s + 16 * a, vw) : zero16();
      const int64_t lr = ((int64_t)b * P.Hq + hd) * P.L + li;
      nref = live ? -P.lse_in[lr] * BLK_LOG2E : 0.f;
      const char* orow = P.o.p + b * P.o.sb + li * P.o.st + hd * P.o.sh;
      u32x4 ov[NV];
#pragma unroll
      for (int s = 0; s < NV; ++s) ov[s] = live ? blk_ld(orow, 64 * s + 16 * a, vw) : zero16();
#pragma unroll
      for (int s = 0; s < NV; ++s) l += blk_dot<T>(g[s], ov[s]);
      l = blk_quad_sum(l);
      if (!EXACT && live && a == 0) P.delta[lr] = l;
    }
  }
  const uint16_t* at = lists + (live ? row.i - q0 : 0) * pitch;
  int cur = live ? *at : 0xffff;
  f32x4 acc[OUT / 16];
#pragma unroll
  for (int d = 0; d < OUT / 16; ++d) acc[d] = zero4();
  f32x4 mean[EXACT ? OUT / 16 : 1];  // sum_j p_j k_j
#pragma unroll
  for (int d = 0; d < (EXACT ? OUT / 16 : 1); ++d) mean[d] = zero4();
  float off = 0.f;
  const float sc = P.scale * BLK_LOG2E, per_sc = 1.f / sc;
  float grown = -__builtin_inff();  // a score above this moves the reference
  const Rows<WK> krow(lane);
  const Rows<WV> vrow(lane);
  const Columns<T, GRAD ? WK : WV> col(lane);

  Blocks blocks(tmaps + (P.GT > 1 ? t / P.GT - q0 : wave) * words, words);
  const int lg_units = P.lgT - (KT == 16 ? 4 : KT == 32 ? 5 : 6);  // units of a block
  int before = 0, word = -1;  // blocks of the union in the words before the one that `before` was counted for
  for (int j = blocks.next(); j >= 0; j = blocks.next()) {
    // the block's place in the union
    while (word < blocks.w) {
      if (word >= 0) before += __builtin_popcount(__builtin_amdgcn_readfirstlane(map[word]));
      ++word;
    }
    const int place = before + __builtin_popcount(__builtin_amdgcn_readfirstlane(map[word]) & ((1u << (j & 31)) - 1));
    const bool member = cur == j;
    if (member) cur = *++at;
    const int first = j << P.lgT;
    for (int sub = 0; sub < 1 << lg_units; ++sub) {
      const int n = (place << lg_units) + sub, k0 = first + sub * KT;
      const bool take = member && k0 <= row.p;
      if (!__any(take)) break;
      if (ring_get(&ring.filled) <= n) {
        if (lane == 0) ring_put(&ring.done[wave], n);
        do __builtin_amdgcn_s_sleep(1);
        while (ring_get(&ring.filled) <= n);
      }
      asm volatile("" ::: "memory");
      const char *ks = smem + (n % stages) * STAGE, *vs = ks + KB;
      f32x4 s[KEY_T];
#pragma unroll
      for (int kt = 0; kt < KEY_T; ++kt) s[kt] = zero4();
#pragma unroll
      for (int w = 0; w < NK; ++w)
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt) s[kt] = mma_slab<T>(krow.read(ks, kt, w), q[w], s[kt]);
      if (__any(take && k0 + KT - 1 > row.p)) {  // the own block: keys behind the query
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + 16 * kt + 4 * a + i > row.p) s[kt][i] = -__builtin_inff();
      }
      float p[KEY_T][4], pw[EXACT ? KEY_T : 1][4];
      if constexpr (!GRAD) {
        float mx = s[0][0];
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[kt][i]);
        if (__any(take && mx > grown)) {
          const float m = grown == -__builtin_inff() ? grown : -nref;  // nothing yet: minus infinity
          const float top = take ? fmaxf(m, blk_quad_max(mx) * sc) : m;
          if (top != -__builtin_inff()) {
            const float corr = __builtin_amdgcn_exp2f(m - top);
            nref = -top;
            grown = (top + GROWTH) * per_sc;
            l *= corr;
#pragma unroll
            for (int d = 0; d < OUT / 16; ++d) acc[d] *= corr;
          }
        }
        float sum = 0.f;
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[kt][i] = __builtin_amdgcn_exp2f(s[kt][i] * sc + nref);
            sum += p[kt][i];
          }
        l += take ? sum : 0.f;
      } else {
#pragma unroll
        for (int kt = 0; kt < KEY_T; ++kt) {
          f32x4 dp = zero4();
#pragma unroll
          for (int w = 0; w < NV; ++w) dp = mma_slab<T>(vrow.read(vs, kt, w), g[w], dp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = __builtin_amdgcn_exp2f(s[kt][i] * sc + nref);
            p[kt][i] = w * (dp[i] - l);
            if constexpr (EXACT) {
              pw[kt][i] = w;
              off += take ? p[kt][i] : 0.f;
            }
          }
        }
      }
#pragma unroll
      for (int sl = 0; sl < SLABS; ++sl) {
        u32x4 w, lo, y = zero16();
        blk_split<T>(p, sl, w, lo);
        if constexpr (EXACT) y = blk_pack<T>(pw, sl);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows that have not chosen the block
          w[i] = take ? w[i] : 0u;
          lo[i] = take ? lo[i] : 0u;
          if constexpr (EXACT) y[i] = take ? y[i] : 0u;
        }
#pragma unroll
        for (int d = 0; d < OUT / 16; ++d) {
          const u32x4 f = col.read(GRAD ? ks : vs, sl, d);
          acc[d] = blk_mma_split<T>(f, w, lo, acc[d]);
          if constexpr (EXACT) mean[d] = mma_slab<T>(f, y, mean[d]);
          // without this all reads move ahead of the products, and registers spill
          if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (lane == 0) ring_put(&ring.done[wave], n + 1);
    }
  }
  if (lane == 0) ring_put(&ring.done[wave], 0x7fffffff);
  if constexpr (!GRAD) l = blk_quad_sum(l);
  if constexpr (EXACT) {
    off = blk_quad_sum(off);
    if (live && a == 0) P.delta[((int64_t)row.b * P.Hq + row.head) * P.L + row.i] = l + off;
#pragma unroll
    for (int d = 0; d < OUT / 16; ++d) acc[d] -= mean[d] * off;
  }
  if (!row.in) return;
  const BlkHeads& o = GRAD ? P.dq : P.o;
  const int width = GRAD ? P.dkw : P.dvw;
  char* out = o.p + row.b * o.sb + (int64_t)row.i * o.st + row.head * o.sh;
  const float mul = GRAD ? P.scale : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // no key: 0; a NaN stays
#pragma unroll
  for (int d = 0; d < OUT / 16; ++d) {
    const int c = 16 * d + 4 * a;
    const float v[4] = {acc[d][0] * mul, acc[d][1] * mul, acc[d][2] * mul, acc[d][3] * mul};
    if (c < width) blk_st4<T>(out + c * ES, v);
  }
  if (!GRAD && P.lse && a == 0)
    P.lse[((int64_t)row.b * P.Hq + row.head) * P.L + row.i] = l == 0.f ? -__builtin_inff() : logf(l) - nref * BLK_LN2;
}

template <typename T, int DKP, int DVP, int KT, int WAVES, bool GRAD> hipError_t launch_t(const BlkParams& P, hipStream_t st) {
  constexpr int ES = sizeof(T), NT = WAVES, LIMIT = tile_lds_limit(WAVES);
  constexpr TileShape SHAPE = {KT, WAVES};
  constexpr int STAGE = tile_stage(SHAPE, ES, DKP, DVP);
  constexpr int MOST = (NT + 1) * (BLK_TILES_MAX / 8) + NT * BLK_ROWS * (BLK_MAX_SEL + 1) * 2 + TILE_STATIC;
  static_assert((LIMIT - MOST) / STAGE >= MIN_STAGES && std::min((LIMIT - MOST) / STAGE, 8) * STAGE >= NT * BLK_ROWS * BLK_MAX_SEL * 4,
                "beside the largest maps and lists there is a ring, in which the raw selection fits");
  const TileLds plan = tile_lds(SHAPE, STAGE, P.nb, P.n, P.QT, P.GT);
  const int stages = plan.stages, lds = plan.bytes;
  const auto kernel = &k_block_tiles<T, DKP, DVP, KT, WAVES, GRAD>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  static_assert(N_XCD == 8, "tile_grid's");
  hipLaunchKernelGGL(kernel, dim3((unsigned)tile_grid(NT, P.tiles_per_seq, (int64_t)P.B * P.Hkv)), dim3(64 * (WAVES + 1)), lds, st, P, stages);
  return hipGetLastError();
}

template <typename T, int DKP, int DVP, bool GRAD> hipError_t by_block(const BlkParams& P, hipStream_t st) {
  constexpr int ES = sizeof(T);
  constexpr TileShape FEW = tile_shape(ES, DKP, DVP, GRAD, 32, false), SHORT = tile_shape(ES, DKP, DVP, GRAD, 32, true),
                      LONG = tile_shape(ES, DKP, DVP, GRAD, 64, true);
  if (P.tiles < BLK_TILES_MANY) return launch_t<T, DKP, DVP, FEW.keys, FEW.tiles, GRAD>(P, st);
  return P.lgT == 5 ? launch_t<T, DKP, DVP, SHORT.keys, SHORT.tiles, GRAD>(P, st)
                    : launch_t<T, DKP, DVP, LONG.keys, LONG.tiles, GRAD>(P, st);
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
