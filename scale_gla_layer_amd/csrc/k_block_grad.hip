// Gradients of the keys and values of the block attention:
//   dv_j = sum over the rows that attend j of p_ij do_i,   dk_j = scale sum of p_ij (do_i . v_j - delta_i) q_i.
//
// A workgroup keeps up to 64 keys and values and their gradients in registers,
// KTW tiles of 16 keys a wave, and streams through the queries that chose the
// block: their (query, head) rows of q and do are gathered asynchronously into
// one of two LDS stages while the other is worked on, 32 rows for each group of
// waves that together hold all keys.  The overlap is a part of the step only: the
// threads that bring lse wait for the next stage with it, and the compiler, which
// does not know the two stages apart, waits for all copies before the transposed
// reads.  With KTW = 2 every row that a wave reads
// from LDS meets 32 keys, which is what LDS and the matrix cores take equal time
// for; two groups of waves then take different rows and add up at the end.
//   The lists of those queries come from a bit matrix (block x query) that is
// written without regard to order and read in order, so no sum's order varies.  A
// block that many queries chose (the first one) is cut into work items of `seg`
// queries, whose partial gradients a last kernel adds in order.
//   bf16 weights and their gradients enter the products as two bf16 values each
// (blk_split): rounded once, they put dv and dk 1.4 times as far off as their own
// rounding does, and the whole gradient takes 470 us instead of 508 at B = 2,
// L = 4096, 16 / 4 heads of 128.
//   Bound by LDS and matrix instructions in turn, at as many waves a SIMD as the
// registers allow without spills to speak of.  bf16 heads of 192 elements in sum
// and fewer: three.  Of 256 (gradient at the same size): with two 508 us, with
// three, which spill 4 registers, 501; at blocks of 32, where three spill 22, 389
// and 592.  Of 128 and 256: two, which spill 2 and at blocks of 32 10, 1.13 ms at
// L = 16384 and 8 / 2 heads, one 1.43; at blocks of 32 687 and 667 us.  fp32 heads
// of more than 256 in sum: one (3.1 ms against 4.4 with two at B = 2, L = 4096).
#include "block_stage.hpp"

namespace msgla {

namespace {

constexpr int INV_PIECE = 2048;  // blocks of one workgroup's bit words

// Bit i of word (w, j): query 64 w + i chose block j; and the number of queries of every block.
__global__ __launch_bounds__(256) void k_block_bits(const BlkParams P) {
  __shared__ unsigned long long word[INV_PIECE];
  const int tid = threadIdx.x, w = blockIdx.x % P.W, j0 = blockIdx.y * INV_PIECE;
  const int64_t bh = blockIdx.x / P.W;
  const int n = min(INV_PIECE, P.nb - j0);
  for (int j = tid; j < n; j += 256) word[j] = 0;
  __syncthreads();
  if (tid < 64) {
    const int i = 64 * w + tid;
    const int p = blk_position(P, (int)(bh / P.Hkv), i);
    blk_chosen(P, P.sel + (bh * P.L + min(i, P.L - 1)) * P.n, p, [&](int, int j) {
      if (j >= j0 && j < j0 + n) atomicOr(&word[j - j0], 1ull << tid);
    });
  }
  __syncthreads();
  uint64_t* out = P.bits + (bh * P.W + w) * P.nb + j0;
  for (int j = tid; j < n; j += 256) {
    out[j] = word[j];
    if (word[j]) atomicAdd(P.cnt + bh * P.nb + j0 + j, __popcll(word[j]));  // whole numbers: in any order
  }
}

// A wave writes one block's queries in order, and where its list, its work items
// and its partials begin: sums over the blocks before it, which FILL_WAVES
// neighbours form together (more would write their lists on one CU: 16 take 21 us
// at B = 2, L = 4096, 16 / 4 heads, 4 take 10, and by itself each takes 8 but reads
// four times the counts, which is felt from some ten thousand blocks on).
constexpr int FILL_WAVES = 4;

__global__ __launch_bounds__(64 * FILL_WAVES) void k_block_fill(const BlkParams P) {
  __shared__ int sums[FILL_WAVES][3];
  const int groups = (P.nb + FILL_WAVES - 1) / FILL_WAVES;
  const int64_t bh = blockIdx.x / groups;
  const int j0 = (int)(blockIdx.x - bh * groups) * FILL_WAVES, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = j0 + wave;
  const int32_t* cnt = P.cnt + bh * P.nb;
  auto items_of = [&](int c) { return max(1, (c + P.seg - 1) / P.seg); };
  int off = 0, first = 0, slot = 0;
  auto add = [&](int i) {
    const int c = cnt[i], n = items_of(c);
    off += c;
    first += n;
    slot += n > 1 ? n : 0;
  };
  auto total = [&] {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      off += __shfl_xor(off, o);
      first += __shfl_xor(first, o);
      slot += __shfl_xor(slot, o);
    }
  };
#pragma unroll 4
  for (int i = threadIdx.x; i < j0; i += 64 * FILL_WAVES) add(i);
  total();
  if (lane == 0) sums[wave][0] = off, sums[wave][1] = first, sums[wave][2] = slot;
  __syncthreads();
  if (j >= P.nb) return;
  off = first = slot = 0;
  if (lane < FILL_WAVES) off = sums[lane][0], first = sums[lane][1], slot = sums[lane][2];
  else if (lane - FILL_WAVES < wave) add(j0 + lane - FILL_WAVES);
  total();
  const int items = items_of(cnt[j]);
  for (int s = lane; s < items; s += 64) P.items[bh * P.max_items + first + s] = make_int2(j, s * P.seg);
  if (lane == 0) {
    P.off[bh * P.nb + j] = off;
    P.slot[bh * P.nb + j] = items > 1 ? slot : -1;
    if (j == P.nb - 1) P.n_items[bh] = first + items;
  }
  const uint64_t* bits = P.bits + bh * P.W * P.nb + j;
  int32_t* list = P.list + bh * P.L * P.n + off;
  int base = 0;
  for (int w0 = 0; w0 < P.W; w0 += 64) {
    uint64_t m = w0 + lane < P.W ? bits[(int64_t)(w0 + lane) * P.nb] : 0;
    const int c = __popcll(m);
    int at = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(at, o);
      if (lane >= o) at += v;
    }
    const int total = __shfl(at, 63);
    at += base - c;
    while (m) {
      list[at++] = 64 * (w0 + lane) + __builtin_ctzll(m);
      m &= m - 1;
    }
    base += total;
  }
}

// rr / G for rr < 2^20, G <= 1024, with magic = ceil(2^32 / G)
__device__ __forceinline__ int div_group(int rr, uint32_t magic, int G) { return G == 1 ? rr : (int)__umulhi((uint32_t)rr, magic); }

// Gathers rows row(0) .. row(N - 1) of W pieces with THREADS threads (pieces
// behind the width repeat the first: they meet zeroes or are not stored).
template <int W, int N, int WAVES, class Row>
__device__ __forceinline__ void gather_rows(char* lds, int width, int wave, int lane, Row row) {
  static_assert(N * W % (64 * WAVES) == 0, "whole copy instructions for every wave");
#pragma unroll
  for (int k = 0; k < N * W / 64 / WAVES; ++k) {
    const int i = wave + k * WAVES, pc = 64 * i + lane, r = pc / W, p = (pc % W) ^ tile_key<W>(r);
    dma16(row(r) + (p * 16 < width ? p * 16 : 0), lds + 1024 * i);
  }
}

template <typename T, int DKP, int DVP, int KTW, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 4 && DKP + DVP > 256 ? 1 : sizeof(T) == 2 && KTW == 1 && DKP + DVP <= 192 ? 3 : 2) void k_block_dkdv(const BlkParams P) {
  constexpr int ES = sizeof(T), WK = DKP * ES / 16, WV = DVP * ES / 16, NK = DKP * ES / 64, NV = DVP * ES / 64;
  constexpr int KEYS = WAVES >= 4 ? 64 : 32, KG = KEYS / 16 / KTW, RG = WAVES / KG, ROWS = 32 * RG;
  constexpr int QB = ROWS * WK * 16, STAGE = QB + ROWS * WV * 16, SLABS = 32 / blk_slab<T>();
  static_assert(KG * RG == WAVES && (RG - 1) * KEYS * (DKP + DVP) * 4 <= 2 * STAGE, "the groups' sums meet in the stages");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ float slse[2][ROWS], sdelta[2][ROWS];
  __shared__ int spos[2][ROWS];
  int* slist = reinterpret_cast<int*>(smem + 2 * STAGE);
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, a = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = wave % KG, rg = wave / KG;
  const int sub = 1 << P.lgT >= KEYS ? (1 << P.lgT) / KEYS : 1;  // workgroups of a block
  // one contiguous range of the work for each XCD: a head's queries meet in its L2
  const int64_t id = (int64_t)(blockIdx.x % N_XCD) * (gridDim.x / N_XCD) + blockIdx.x / N_XCD, work = id / sub;
  const int64_t bh = work / P.max_items;
  const int it = (int)(work - bh * P.max_items);
  if (bh >= (int64_t)P.B * P.Hkv || it >= P.n_items[bh]) return;
  const int b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  const int2 item = P.items[bh * P.max_items + it];
  const int j = item.x, nq = min(P.seg, P.cnt[bh * P.nb + j] - item.y);
  {
    const int32_t* list = P.list + bh * P.L * P.n + P.off[bh * P.nb + j] + item.y;
    for (int i = tid; i < nq; i += 64 * WAVES) slist[i] = list[i];
  }
  const int in_block = (int)(id - work * sub) * KEYS + 16 * KTW * kg + c16;
  const int key = (j << P.lgT) + in_block;  // the lane's key of the wave's first tile, as a column
  const int kw = P.dkw * ES, vw = P.dvw * ES;
  u32x4 kf[KTW][NK], vf[KTW][NV];
#pragma unroll
  for (int kt = 0; kt < KTW; ++kt) {
    const int k = key + 16 * kt;
    const bool in = k < P.S;
    const char* kr = P.k.p + b * P.k.sb + (int64_t)(in ? k : 0) * P.k.st + h * P.k.sh;
    const char* vr = P.v.p + b * P.v.sb + (int64_t)(in ? k : 0) * P.v.st + h * P.v.sh;
#pragma unroll
    for (int s = 0; s < NK; ++s) kf[kt][s] = in ? blk_ld(kr, 64 * s + 16 * a, kw) : zero16();
#pragma unroll
    for (int s = 0; s < NV; ++s) vf[kt][s] = in ? blk_ld(vr, 64 * s + 16 * a, vw) : zero16();
  }
  f32x4 dk[KTW][DKP / 16], dv[KTW][DVP / 16];
#pragma unroll
  for (int kt = 0; kt < KTW; ++kt) {
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) dk[kt][d] = zero4();
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) dv[kt][d] = zero4();
  }
  const float sc = P.scale * BLK_LOG2E;
  const int rows = nq * P.G, steps = (rows + ROWS - 1) / ROWS;
  const uint32_t magic = (uint32_t)((0x100000000ull + P.G - 1) / P.G);
  const Rows<WK> qrow(lane);
  const Rows<WV> grow(lane);
  const Columns<T, WK> qcol(lane);
  const Columns<T, WV> gcol(lane);
  const char* qbase = P.q.p + b * P.q.sb + (int64_t)h * P.G * P.q.sh;
  const char* gbase = P.dout.p + b * P.dout.sb + (int64_t)h * P.G * P.dout.sh;
  float rlse = 0.f, rdelta = 0.f;  // of the row that this thread brings in for the next step
  int rpos = 0;
  auto issue = [&](int t) {
    char* st = smem + (t & 1) * STAGE;
    auto at = [&](const char* base, const BlkHeads& x, int r) {  // rows behind the last repeat it, with weight 0
      const int rr = min(t * ROWS + r, rows - 1), i = div_group(rr, magic, P.G);
      return base + (int64_t)slist[i] * x.st + (int64_t)(rr - i * P.G) * x.sh;
    };
    gather_rows<WK, ROWS, WAVES>(st, kw, wave, lane, [&](int r) { return at(qbase, P.q, r); });
    gather_rows<WV, ROWS, WAVES>(st + QB, vw, wave, lane, [&](int r) { return at(gbase, P.dout, r); });
    if (tid < ROWS) {
      const int rr = t * ROWS + tid;
      rlse = -__builtin_inff();
      rdelta = 0.f;
      rpos = -1;
      if (rr < rows) {
        const int g = div_group(rr, magic, P.G), i = slist[g];
        const int64_t lr = ((int64_t)b * P.Hq + h * P.G + rr - g * P.G) * P.L + i;
        rlse = -P.lse_in[lr] * BLK_LOG2E;
        rdelta = P.delta[lr];
        rpos = blk_position(P, b, i);
      }
    }
  };
  __syncthreads();
  if (steps > 0) issue(0);
  const int top = key - c16 + 16 * KTW - 1;  // the wave's last key
  for (int t = 0; t < steps; ++t) {
    wait_vmcnt<0>();
    if (tid < ROWS) {
      slse[t & 1][tid] = rlse;
      sdelta[t & 1][tid] = rdelta;
      spos[t & 1][tid] = rpos;
    }
    lds_barrier();
    if (t + 1 < steps) issue(t + 1);
    const char *qs = smem + (t & 1) * STAGE + rg * 32 * WK * 16, *gs = smem + (t & 1) * STAGE + QB + rg * 32 * WV * 16;
    const float *nlse = slse[t & 1] + rg * 32, *delta = sdelta[t & 1] + rg * 32;
    const int* pos = spos[t & 1] + rg * 32;
    const bool masked = __any(pos[lane & 31] < top);  // queries of this very block: keys behind them
    float p[KTW][2][4], ds[KTW][2][4];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      f32x4 s[KTW], dp[KTW];
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) s[kt] = dp[kt] = zero4();
#pragma unroll
      for (int w = 0; w < NK; ++w) {
        const u32x4 f = qrow.read(qs, rt, w);
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) s[kt] = mma_slab<T>(f, kf[kt][w], s[kt]);
      }
#pragma unroll
      for (int w = 0; w < NV; ++w) {
        const u32x4 f = grow.read(gs, rt, w);
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) dp[kt] = mma_slab<T>(f, vf[kt][w], dp[kt]);
      }
      float nl[4], de[4];
      unpack16<float>(ld16(nlse + 16 * rt + 4 * a), nl);
      unpack16<float>(ld16(delta + 16 * rt + 4 * a), de);
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[kt][rt][i] = __builtin_amdgcn_exp2f(s[kt][i] * sc + nl[i]);
          ds[kt][rt][i] = p[kt][rt][i] * (dp[kt][i] - de[i]);
        }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ps = pos[16 * rt + 4 * a + i];
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt)
            if (key + 16 * kt > ps) p[kt][rt][i] = ds[kt][rt][i] = 0.f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      u32x4 w[KTW], lo[KTW];
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) blk_split<T>(p[kt], s, w[kt], lo[kt]);
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d) {
        const u32x4 f = gcol.read(gs, s, d);
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) dv[kt][d] = blk_mma_split<T>(f, w[kt], lo[kt], dv[kt][d]);
        if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) blk_split<T>(ds[kt], s, w[kt], lo[kt]);
#pragma unroll
      for (int d = 0; d < DKP / 16; ++d) {
        const u32x4 f = qcol.read(qs, s, d);
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) dk[kt][d] = blk_mma_split<T>(f, w[kt], lo[kt], dk[kt][d]);
        if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if constexpr (RG > 1) {  // the row groups' sums, in order
    float* sums = reinterpret_cast<float*>(smem) + ((rg - 1) * KG + kg) * KTW * (DKP + DVP) / 4 * 64;
    __syncthreads();
    if (rg > 0) {
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) {
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) st16(sums + ((kt * (DKP + DVP) / 16 + d) * 64 + lane) * 4, __builtin_bit_cast(u32x4, dk[kt][d]));
#pragma unroll
        for (int d = 0; d < DVP / 16; ++d)
          st16(sums + ((kt * (DKP + DVP) / 16 + DKP / 16 + d) * 64 + lane) * 4, __builtin_bit_cast(u32x4, dv[kt][d]));
      }
    }
    __syncthreads();
    if (rg > 0) return;
#pragma unroll
    for (int o = 1; o < RG; ++o) {
      const float* in = reinterpret_cast<float*>(smem) + ((o - 1) * KG + kg) * KTW * (DKP + DVP) / 4 * 64;
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) {
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) dk[kt][d] += __builtin_bit_cast(f32x4, ld16(in + ((kt * (DKP + DVP) / 16 + d) * 64 + lane) * 4));
#pragma unroll
        for (int d = 0; d < DVP / 16; ++d)
          dv[kt][d] += __builtin_bit_cast(f32x4, ld16(in + ((kt * (DKP + DVP) / 16 + DKP / 16 + d) * 64 + lane) * 4));
      }
    }
  }
  const int slot = P.slot[bh * P.nb + j];
#pragma unroll
  for (int kt = 0; kt < KTW; ++kt) {
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) dk[kt][d] *= P.scale;
    if (slot >= 0) {
      float* out = P.part + (((bh * P.max_parts + slot + item.y / P.seg) << P.lgT) + in_block + 16 * kt) * (DKP + DVP);
#pragma unroll
      for (int d = 0; d < DKP / 16; ++d) st16(out + 16 * d + 4 * a, __builtin_bit_cast(u32x4, dk[kt][d]));
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d) st16(out + DKP + 16 * d + 4 * a, __builtin_bit_cast(u32x4, dv[kt][d]));
      continue;
    }
    const int k = key + 16 * kt;
    if (k >= P.S) continue;
    char* ok = P.dk.p + b * P.dk.sb + (int64_t)k * P.dk.st + h * P.dk.sh;
    char* ov = P.dv.p + b * P.dv.sb + (int64_t)k * P.dv.st + h * P.dv.sh;
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) {
      const float v[4] = {dk[kt][d][0], dk[kt][d][1], dk[kt][d][2], dk[kt][d][3]};
      if (16 * d + 4 * a < P.dkw) blk_st4<T>(ok + (16 * d + 4 * a) * ES, v);
    }
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) {
      const float v[4] = {dv[kt][d][0], dv[kt][d][1], dv[kt][d][2], dv[kt][d][3]};
      if (16 * d + 4 * a < P.dvw) blk_st4<T>(ov + (16 * d + 4 * a) * ES, v);
    }
  }
}

// Adds the partials of blocks of several work items, four elements a thread.
template <typename T, int DKP, int DVP> __global__ __launch_bounds__(256) void k_block_grad_join(const BlkParams P) {
  const int64_t bh = blockIdx.x / P.nb;
  const int j = (int)(blockIdx.x - bh * P.nb), slot = P.slot[bh * P.nb + j];
  if (slot < 0) return;
  const int b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv), T2 = 1 << P.lgT;
  const int n = (P.cnt[bh * P.nb + j] + P.seg - 1) / P.seg;
  constexpr int ROW = DKP + DVP, Q = ROW / 4;
  const float* in = P.part + ((bh * P.max_parts + slot) << P.lgT) * ROW;
  for (int i = threadIdx.x + 256 * blockIdx.y; i < T2 * Q; i += 256 * gridDim.y) {
    const int r = i / Q, c = (i % Q) * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < n; s0 += 4) {
      u32x4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = ld16(in + ((int64_t)min(s0 + k, n - 1) * T2 + r) * ROW + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
        unpack16<float>(u[k], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += s0 + k < n ? f[e] : 0.f;
      }
    }
    const int key = (j << P.lgT) + r;
    if (key >= P.S) continue;
    if (c < DKP) {
      if (c < P.dkw) blk_st4<T>(P.dk.p + b * P.dk.sb + (int64_t)key * P.dk.st + h * P.dk.sh + c * sizeof(T), v);
    } else if (c - DKP < P.dvw) {
      blk_st4<T>(P.dv.p + b * P.dv.sb + (int64_t)key * P.dv.st + h * P.dv.sh + (c - DKP) * sizeof(T), v);
    }
  }
}

template <typename T, int DKP, int DVP, int KTW, int WAVES> hipError_t dkdv_t(const BlkParams& P, int64_t grid, hipStream_t st) {
  constexpr int KEYS = WAVES >= 4 ? 64 : 32, ROWS = 32 * WAVES / (KEYS / 16 / KTW);
  const int lds = 2 * ROWS * (DKP + DVP) * (int)sizeof(T) + P.seg * 4;
  const auto kernel = &k_block_dkdv<T, DKP, DVP, KTW, WAVES>;
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)((grid + N_XCD - 1) / N_XCD * N_XCD)), dim3(64 * WAVES), lds, st, P);
  return hipGetLastError();
}

template <typename T, int DKP, int DVP> hipError_t grad_t(const BlkParams& P, hipStream_t st) {
  const int64_t bh = (int64_t)P.B * P.Hkv;
  hipLaunchKernelGGL(k_block_bits, dim3((unsigned)(bh * P.W), (P.nb + INV_PIECE - 1) / INV_PIECE), dim3(256), 0, st, P);
  hipLaunchKernelGGL(k_block_fill, dim3((unsigned)(bh * ((P.nb + FILL_WAVES - 1) / FILL_WAVES))), dim3(64 * FILL_WAVES), 0,
                     st, P);
  const int64_t work = bh * P.max_items;
  // two key tiles a wave where their gradients fit the registers
  constexpr int KTW = sizeof(T) == 2 && DKP + DVP <= 128 ? 2 : 1;
  const hipError_t e = P.lgT == 5 ? dkdv_t<T, DKP, DVP, KTW, 2>(P, work, st)
                                  : dkdv_t<T, DKP, DVP, KTW, 4>(P, work << (P.lgT - 6), st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_block_grad_join<T, DKP, DVP>), dim3((unsigned)(bh * P.nb), 8), dim3(256), 0, st, P);
  return hipGetLastError();
}

template <typename T, int DKP> hipError_t by_dv(const BlkParams& P, hipStream_t st) {
  if (blk_dvp(P.dvw) == 64) return grad_t<T, DKP, 64>(P, st);
  if (blk_dvp(P.dvw) == 128) return grad_t<T, DKP, 128>(P, st);
  return grad_t<T, DKP, 256>(P, st);
}

}  // namespace

hipError_t launch_block_dkdv(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) return k64 ? by_dv<bf16, 64>(P, st) : by_dv<bf16, 128>(P, st);
  return k64 ? by_dv<float, 64>(P, st) : by_dv<float, 128>(P, st);
}

}  // namespace msgla
