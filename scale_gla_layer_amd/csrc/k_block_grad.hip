// Gradients of the keys and values of the block attention:
//   dv_j = sum over the rows that attend j of p_ij do_i,   dk_j = scale sum of p_ij (do_i . v_j - delta_i) q_i.
//
// A workgroup keeps up to 64 keys and values and their gradients in registers
// and streams through the queries that chose the block, gathered 32 (query,
// head) rows at a time into LDS.  The lists of those queries come from a bit
// matrix (block x query) that is written without regard to order and read in
// order, so no sum's order varies.  A block that many queries chose (the first
// one) is cut into work items of `seg` queries, whose partial gradients a last
// kernel adds in order.
#include "block_device.hpp"

namespace msgla {

namespace {

constexpr int INV_PIECE = 2048;  // blocks of one workgroup's bit words
constexpr int GRAD_ROWS = 32;    // rows of a step

// bit i of word (w, j): query 64 w + i chose block j
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
  for (int j = tid; j < n; j += 256) out[j] = word[j];
}

__global__ __launch_bounds__(64) void k_block_count(const BlkParams P) {
  const int64_t bh = blockIdx.y;
  const int j = blockIdx.x * 64 + threadIdx.x;
  if (j >= P.nb) return;
  const uint64_t* bits = P.bits + bh * P.W * P.nb + j;
  int c = 0;
  for (int w = 0; w < P.W; ++w) c += __popcll(bits[(int64_t)w * P.nb]);
  P.cnt[bh * P.nb + j] = c;
}

// Running sums over the blocks: where each one's list, work items and partials begin.
__global__ __launch_bounds__(1024) void k_block_plan(const BlkParams P) {
  __shared__ int sum[3][1024];
  const int64_t bh = blockIdx.x;
  const int tid = threadIdx.x;
  int before[3] = {0, 0, 0};
  for (int j0 = 0; j0 < P.nb; j0 += 1024) {
    const int j = j0 + tid, c = j < P.nb ? P.cnt[bh * P.nb + j] : 0;
    const int ni = j < P.nb ? max(1, (c + P.seg - 1) / P.seg) : 0;
    const int v[3] = {c, ni, ni > 1 ? ni : 0};
    for (int k = 0; k < 3; ++k) sum[k][tid] = v[k];
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      int add[3] = {0, 0, 0};
      if (tid >= o)
        for (int k = 0; k < 3; ++k) add[k] = sum[k][tid - o];
      __syncthreads();
      for (int k = 0; k < 3; ++k) sum[k][tid] += add[k];
      __syncthreads();
    }
    if (j < P.nb) {
      P.off[bh * P.nb + j] = before[0] + sum[0][tid] - c;
      P.slot[bh * P.nb + j] = ni > 1 ? before[2] + sum[2][tid] - ni : -1;
      for (int s = 0; s < ni; ++s)
        P.items[bh * P.max_items + before[1] + sum[1][tid] - ni + s] = make_int2(j, s * P.seg);
    }
    for (int k = 0; k < 3; ++k) before[k] += sum[k][1023];
    __syncthreads();
  }
  if (tid == 0) P.n_items[bh] = before[1];
}

// A wave writes one block's queries in order.
__global__ __launch_bounds__(64) void k_block_fill(const BlkParams P) {
  const int64_t bh = blockIdx.x / P.nb;
  const int j = (int)(blockIdx.x - bh * P.nb), lane = threadIdx.x;
  const uint64_t* bits = P.bits + bh * P.W * P.nb + j;
  int32_t* list = P.list + bh * P.L * P.n + P.off[bh * P.nb + j];
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

// WAVES waves of 16 keys each.
template <typename T, int DKP, int DVP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_block_dkdv(const BlkParams P) {
  constexpr int KP = blk_pitch<T, DKP>(), VP = blk_pitch<T, DVP>(), KEYS = 16 * WAVES;
  constexpr int NK = DKP * (int)sizeof(T) / 64, NV = DVP * (int)sizeof(T) / 64;
  __shared__ __attribute__((aligned(16))) char qs[GRAD_ROWS * KP], gs[GRAD_ROWS * VP];
  __shared__ float slse[GRAD_ROWS], sdelta[GRAD_ROWS];
  __shared__ int spos[GRAD_ROWS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c16 = lane & 15, a = lane >> 4;
  const int sub = 1 << P.lgT >= KEYS ? (1 << P.lgT) / KEYS : 1;  // workgroups of a block
  const int64_t work = blockIdx.x / sub;
  const int64_t bh = work / P.max_items;
  const int it = (int)(work - bh * P.max_items);
  if (it >= P.n_items[bh]) return;
  const int b = (int)(bh / P.Hkv), h = (int)(bh - (int64_t)b * P.Hkv);
  const int2 item = P.items[bh * P.max_items + it];
  const int j = item.x, count = P.cnt[bh * P.nb + j];
  const int nq = min(P.seg, count - item.y);
  const int32_t* list = P.list + bh * P.L * P.n + P.off[bh * P.nb + j] + item.y;
  const int in_block = (int)(blockIdx.x - work * sub) * KEYS + 16 * wave + c16;
  const int key = (j << P.lgT) + in_block;  // the lane's key, as a column
  const int kw = P.dkw * (int)sizeof(T), vw = P.dvw * (int)sizeof(T);
  u32x4 kf[NK], vf[NV];
  {
    const bool in = key < P.S;
    const char* kr = P.k.p + b * P.k.sb + (int64_t)(in ? key : 0) * P.k.st + h * P.k.sh;
    const char* vr = P.v.p + b * P.v.sb + (int64_t)(in ? key : 0) * P.v.st + h * P.v.sh;
#pragma unroll
    for (int s = 0; s < NK; ++s) kf[s] = in ? blk_ld(kr, 64 * s + 16 * a, kw) : zero16();
#pragma unroll
    for (int s = 0; s < NV; ++s) vf[s] = in ? blk_ld(vr, 64 * s + 16 * a, vw) : zero16();
  }
  f32x4 dk[DKP / 16], dv[DVP / 16];
#pragma unroll
  for (int d = 0; d < DKP / 16; ++d) dk[d] = zero4();
#pragma unroll
  for (int d = 0; d < DVP / 16; ++d) dv[d] = zero4();
  const float sc = P.scale * BLK_LOG2E;
  const int rows = nq * P.G;
  for (int r0 = 0; r0 < rows; r0 += GRAD_ROWS) {
    __syncthreads();
    if (tid < GRAD_ROWS) {
      const int rr = r0 + tid;
      int p = -1;
      if (rr < rows) {
        const int i = list[rr / P.G];
        const int64_t lr = ((int64_t)b * P.Hq + h * P.G + rr % P.G) * P.L + i;
        p = blk_position(P, b, i);
        slse[tid] = P.lse_in[lr] * BLK_LOG2E;
        sdelta[tid] = P.delta[lr];
      }
      spos[tid] = p;
    }
    auto row = [&](const BlkHeads& t, int r) -> const char* {
      const int rr = r0 + r;
      return rr < rows ? t.p + b * t.sb + (int64_t)list[rr / P.G] * t.st + (int64_t)(h * P.G + rr % P.G) * t.sh : nullptr;
    };
    blk_stage<T, DKP, 64 * WAVES>(qs, GRAD_ROWS, kw, tid, [&](int r) { return row(P.q, r); });
    blk_stage<T, DVP, 64 * WAVES>(gs, GRAD_ROWS, vw, tid, [&](int r) { return row(P.dout, r); });
    __syncthreads();
    float p[2][4], ds[2][4];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const char *qr = qs + (16 * rt + c16) * KP + 16 * a, *gr = gs + (16 * rt + c16) * VP + 16 * a;
      f32x4 s = zero4(), dp = zero4();
#pragma unroll
      for (int w = 0; w < NK; ++w) s = mma_slab<T>(ld16(qr + 64 * w), kf[w], s);
#pragma unroll
      for (int w = 0; w < NV; ++w) dp = mma_slab<T>(ld16(gr + 64 * w), vf[w], dp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * rt + 4 * a + i;
        const bool on = key <= spos[r];
        p[rt][i] = on ? __builtin_amdgcn_exp2f(s[i] * sc - slse[r]) : 0.f;
        ds[rt][i] = on ? p[rt][i] * (dp[i] - sdelta[r]) * P.scale : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < GRAD_ROWS / blk_slab<T>(); ++s) {
      const u32x4 wp = blk_pack<T>(p, s), wd = blk_pack<T>(ds, s);
#pragma unroll
      for (int d = 0; d < DVP / 16; ++d) dv[d] = mma_slab<T>(blk_column<T>(gs, VP, s * blk_slab<T>(), d, lane), wp, dv[d]);
#pragma unroll
      for (int d = 0; d < DKP / 16; ++d) dk[d] = mma_slab<T>(blk_column<T>(qs, KP, s * blk_slab<T>(), d, lane), wd, dk[d]);
    }
  }
  const int slot = P.slot[bh * P.nb + j];
  if (slot >= 0) {
    float* out = P.part + (((bh * P.max_parts + slot + item.y / P.seg) << P.lgT) + in_block) * (DKP + DVP);
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) st16(out + 16 * d + 4 * a, __builtin_bit_cast(u32x4, dk[d]));
#pragma unroll
    for (int d = 0; d < DVP / 16; ++d) st16(out + DKP + 16 * d + 4 * a, __builtin_bit_cast(u32x4, dv[d]));
    return;
  }
  if (key >= P.S) return;
  char* ok = P.dk.p + b * P.dk.sb + (int64_t)key * P.dk.st + h * P.dk.sh;
  char* ov = P.dv.p + b * P.dv.sb + (int64_t)key * P.dv.st + h * P.dv.sh;
#pragma unroll
  for (int d = 0; d < DKP / 16; ++d) {
    const float v[4] = {dk[d][0], dk[d][1], dk[d][2], dk[d][3]};
    if (16 * d + 4 * a < P.dkw) blk_st4<T>(ok + (16 * d + 4 * a) * sizeof(T), v);
  }
#pragma unroll
  for (int d = 0; d < DVP / 16; ++d) {
    const float v[4] = {dv[d][0], dv[d][1], dv[d][2], dv[d][3]};
    if (16 * d + 4 * a < P.dvw) blk_st4<T>(ov + (16 * d + 4 * a) * sizeof(T), v);
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
    for (int s = 0; s < n; ++s) {
      float u[4];
      unpack16<float>(ld16(in + ((int64_t)s * T2 + r) * ROW + c), u);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
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

template <typename T, int DKP, int DVP> void grad_t(const BlkParams& P, hipStream_t st) {
  const int64_t bh = (int64_t)P.B * P.Hkv;
  hipLaunchKernelGGL(k_block_bits, dim3((unsigned)(bh * P.W), (P.nb + INV_PIECE - 1) / INV_PIECE), dim3(256), 0, st, P);
  hipLaunchKernelGGL(k_block_count, dim3((P.nb + 63) / 64, (unsigned)bh), dim3(64), 0, st, P);
  hipLaunchKernelGGL(k_block_plan, dim3((unsigned)bh), dim3(1024), 0, st, P);
  hipLaunchKernelGGL(k_block_fill, dim3((unsigned)(bh * P.nb)), dim3(64), 0, st, P);
  const int64_t work = bh * P.max_items;
  if (P.lgT == 5) hipLaunchKernelGGL((k_block_dkdv<T, DKP, DVP, 2>), dim3((unsigned)work), dim3(128), 0, st, P);
  else hipLaunchKernelGGL((k_block_dkdv<T, DKP, DVP, 4>), dim3((unsigned)(work << (P.lgT - 6))), dim3(256), 0, st, P);
  hipLaunchKernelGGL((k_block_grad_join<T, DKP, DVP>), dim3((unsigned)(bh * P.nb), 8), dim3(256), 0, st, P);
}

template <typename T, int DKP> void by_dv(const BlkParams& P, hipStream_t st) {
  if (blk_dvp(P.dvw) == 64) grad_t<T, DKP, 64>(P, st);
  else if (blk_dvp(P.dvw) == 128) grad_t<T, DKP, 128>(P, st);
  else grad_t<T, DKP, 256>(P, st);
}

}  // namespace

hipError_t launch_block_dkdv(const BlkParams& P, bool bf16_path, hipStream_t st) {
  const bool k64 = blk_dkp(P.dkw) == 64;
  if (bf16_path) k64 ? by_dv<bf16, 64>(P, st) : by_dv<bf16, 128>(P, st);
  else k64 ? by_dv<float, 64>(P, st) : by_dv<float, 128>(P, st);
  return hipGetLastError();
}

}  // namespace msgla
