// Linear attention with a decay per head:
//   S_t = gamma S_{t-1} + k_t^T v_t,   out_t = scale q_t S_t
//
// A chunk of 64 positions with the state S before it:
//   out_i = scale (gamma^(i+1) q_i S + sum_{j <= i} gamma^(i-j) (q_i . k_j) v_j)
//   S' = gamma^n S + sum_j gamma^(n-1-j) k_j^T v_j
// so a walk over the chunks is four matrix products each.  A workgroup walks one
// (sequence, head) for 64 or 128 columns of v.  Four of its waves form the outputs, of
// 16 positions each; four or eight others keep the state in their accumulators, an
// equal share of its rows each, and leave it, rounded, in LDS, where it is an operand of
// the next chunk's outputs.  Both work on a chunk at the same time, with half the registers that one
// wave for both would need, while asynchronous copies bring the next one.  All
// exponents of gamma are at least 0, so nothing overflows, and a decay of 0
// (log_decay of minus infinity) is exact.
//   Few sequences and heads: each sequence is cut into segments, what each adds
// to the state is formed first (from zero, without outputs), a small kernel sums up
// the states before the segments, and the walks begin with these.
//   The gradients are walks themselves: with do the output's gradient, dq is that
// of (do, v, k), and from the last token to the first dk is that of (v, do, q) and
// dv that of (k, q, do), whose state is the state's gradient.  Three jobs of a launch.
//   bf16: the weighted q k^T, the state and the decayed keys enter their products
// as two bf16 values each (16 bits); rounded once, each of them would be off by as
// much as the output's own rounding.  Where the last state is wanted, which is fp32,
// the decayed keys enter as three (with two it is off by 2.4e-6).  Sums are fp32.
//   Bound by latency, between barriers, and vector instructions: B = 8, L = 2048, 4 heads
// of 128 and 256, bf16 takes 19.0 us for the segments, 6.5 for their states and 37.8 for the
// walk, whose workgroups' eight chunks have matrix instructions for 8 and LDS reads for
// 15 (counted): 63.3 a call in a long run of calls (77 in the first of them; 89 for 66 with
// 32 x 32 tiles for both, which read half as much from LDS and leave two waves a SIMD).  Its
// gradient takes 153.  fp32 195 and 575: at a large product's rate the walk's matrix
// instructions take 82 of its 138.
//   The products' layouts chain without exchanges between lanes: A^T = K Q^T holds
// a row's weights where out^T = V^T A^T wants them, and S as the sum of K^T V has
// four neighbouring rows a lane, which is 8 bytes of the transposed state in LDS.
#include <algorithm>

#include "block_stage.hpp"
#include "linear.hpp"

namespace msgla {

namespace {

__device__ __forceinline__ float lin_power(int e, float lg2) { return exp2f((float)e * lg2); }

// log2 of the head's decay; minus infinity as a number that no exponent makes finite again
__device__ __forceinline__ float lin_log2(const float* log_decay, int h) {
  const float v = log_decay[h];
  return (v < -1e30f ? -1e30f : v) * BLK_LOG2E;
}

__device__ __forceinline__ int lin_len(const LinParams& P, int b) {
  return P.lens ? max(0, min(P.lens[b], P.L)) : P.L;
}

// Copies of chunks of 64 rows of W pieces into stage tiles, dealt to a workgroup's
// waves: rows of positions that follow one another, or (turned) that go back.  Rows
// behind the last one repeat it, and pieces behind the width the first one: they meet
// zeroes or are not stored.
template <int W, int WAVES> struct ChunkCopy {
  static constexpr int N = W / WAVES;  // copy instructions of a wave
  static_assert(LIN_CHUNK == 64 && W % WAVES == 0, "a row a lane and instruction");
  const char* base;
  int64_t st;
  int32_t off[N];
  int width;
  bool near;
  __device__ ChunkCopy(const char* b, int64_t stride, int w, bool turned, int wave, int lane) : base(b), st(turned ? -stride : stride), width(w) {
    near = stride <= 0x7fffffff / (2 * LIN_CHUNK);
#pragma unroll
    for (int i = 0; i < N; ++i) off[i] = row(i, wave, lane) * (int)st + byte(i, wave, lane);
  }
  __device__ __forceinline__ static int row(int i, int wave, int lane) { return (64 * (wave + WAVES * i) + lane) / W; }
  __device__ __forceinline__ int byte(int i, int wave, int lane) const {
    const int at = ((lane % W) ^ tile_key<W>(row(i, wave, lane))) * 16;
    return at < width ? at : 0;
  }
  // n rows from the position `first` on
  __device__ __forceinline__ void issue(int64_t first, int n, char* lds, int wave, int lane) const {
    const char* p = base + first * (st < 0 ? -st : st);
    if (n >= LIN_CHUNK && near) {
#pragma unroll
      for (int i = 0; i < N; ++i) dma16(p + off[i], lds + 1024 * (wave + WAVES * i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) dma16(p + min(row(i, wave, lane), n - 1) * st + byte(i, wave, lane), lds + 1024 * (wave + WAVES * i));
    }
  }
};

template <typename T, int KWP, int VS> constexpr int state_waves() { return lin_state_waves(sizeof(T), KWP, VS); }
// Waves a SIMD: of one workgroup, or of the two that LDS holds.
template <typename T, int KWP, int VS, bool OUT> constexpr int lin_waves() {
  return sizeof(T) == 4 ? (OUT ? 2 : 1) : state_waves<T, KWP, VS>() == 8 ? (OUT ? 3 : 2) : OUT ? 4 : 3;
}
// Stages of LDS for a chunk's keys and values: two where they fit.
template <typename T, int KWP> constexpr int lin_stages() { return sizeof(T) == 4 && KWP == 256 ? 1 : 2; }

// OUT: the walk; else what a segment adds to the state (the state's waves alone).
template <typename T, int KWP, int VS, bool OUT>
__global__ __launch_bounds__(64 * (state_waves<T, KWP, VS>() + (OUT ? 4 : 0)), (lin_waves<T, KWP, VS, OUT>())) void k_linear(const LinParams P) {
  constexpr int ES = sizeof(T), C = LIN_CHUNK, NSW = state_waves<T, KWP, VS>(), STAGES = lin_stages<T, KWP>();
  constexpr int COPYING = OUT && NSW == 4 ? 8 : NSW;  // waves that copy: all, or of twelve those with the state
  constexpr int NQ = KWP * ES / 64;            // slabs of a row
  constexpr int KT = KWP / 16 / NSW, VT = VS / 16;   // a state wave's tiles
  constexpr int SL = C / blk_slab<T>();        // slabs of a chunk's positions
  constexpr int WK = KWP * ES / 16, WV = VS * ES / 16, KB = C * WK * 16, STAGE = KB + C * WV * 16, SB = VS * WK * 16;
  constexpr bool LO = ES == 2;
  // variables of their own, so that reads of one need not wait for copies to another
  __shared__ __attribute__((aligned(1024))) char stage0[STAGE], stage1[STAGES == 2 ? STAGE : 16];
  __shared__ __attribute__((aligned(16))) char ss[OUT ? (LO ? 2 : 1) * SB : 16];  // state^T [column][row], hi and lo
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, a = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const LinJob& J = P.job[blockIdx.y];
  const int nseg = OUT ? J.segments : J.segments - 1;
  const int total = P.B * P.H * nseg * J.slices, per = (total + N_XCD - 1) / N_XCD;
  // an XCD takes neighbouring slices, which read the same q and k
  const int w = remap_xcd(blockIdx.x, per);
  if (blockIdx.x / N_XCD >= (unsigned)per || w >= total) return;
  const int slice = w % J.slices, seg = w / J.slices % nseg, bh = w / J.slices / nseg, b = bh / P.H, h = bh - b * P.H;
  const int len = lin_len(P, b), v0 = slice * VS;
  const float lg2 = lin_log2(P.log_decay, h);
  const int first = seg * J.seg_chunks * C, past = min(P.L, first + J.seg_chunks * C), end = min(past, len);
  const int kw = J.kw * ES, vw = min(VS, J.vw - v0) * ES;  // bytes of a row, and of its part
  const bool turned = J.turned != 0;
  auto position = [&](int n) { return turned ? len - 1 - n : n; };  // of the walk's n-th token
  const int copier = OUT && NSW == 8 ? wave - 4 : wave;
  const ChunkCopy<WK, COPYING> kc(J.k.p + b * J.k.sb + h * J.k.sh, J.k.st, kw, turned, copier, lane);
  const ChunkCopy<WV, COPYING> vc(J.v.p + b * J.v.sb + h * J.v.sh + v0 * ES, J.v.st, vw, turned, copier, lane);
  auto fetch = [&](int n0, char* to) {
    if (copier < 0) return;
    kc.issue(position(n0), end - n0, to, copier, lane);
    vc.issue(position(n0), end - n0, to + KB, copier, lane);
  };
  if (first < end) fetch(first, stage0);
  const Rows<WK> row(lane);
  const Columns<T, WK> kcol(lane);
  const Columns<T, WV> vcol(lane);

  // Chunk by chunk: before(n0, stage) and after(n0, stage), with a barrier behind each; the first one
  // finds the state before the chunk in LDS, the second one may renew it.
  auto walk = [&](auto before, auto after) __attribute__((always_inline)) {
    auto chunk = [&](int n0, char* stage, char* next) __attribute__((always_inline)) {
      if (STAGES == 2 && n0 + C < end) fetch(n0 + C, next);
      before(n0, stage);
      if constexpr (OUT) lds_barrier();
      after(n0, stage);
      __syncthreads();
      if (STAGES == 1 && n0 + C < end) {
        fetch(n0 + C, stage);
        __syncthreads();
      }
    };
    __syncthreads();
    for (int n0 = first; n0 < end; n0 += STAGES * C) {
      chunk(n0, stage0, STAGES == 2 ? stage1 : stage0);
      if (STAGES == 2 && n0 + C < end) chunk(n0 + C, stage1, stage0);
    }
  };

  if (OUT && wave < 4) {  // the outputs
    const int mine = 16 * wave + c16;  // the lane's row of a chunk
    float within[C / 16][4];           // decays from the positions before it
#pragma unroll
    for (int t = 0; t < C / 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int back = mine - (16 * t + 4 * a + e);
        within[t][e] = back >= 0 ? lin_power(max(back, 0), lg2) : 0.f;
      }
    const float grow = lin_power(mine + 1, lg2), grow_first = lin_power(mine, lg2);
    const char* qb = J.q.p + b * J.q.sb + h * J.q.sh;
    u32x4 q[NQ];
    auto load = [&](int n0) {
      const char* p = qb + (int64_t)position(min(n0 + mine, end - 1)) * J.q.st;
#pragma unroll
      for (int s = 0; s < NQ; ++s) q[s] = ld16(p + (64 * s + 16 * a < kw ? 64 * s + 16 * a : 0));
      if (kw < KWP * ES) {
#pragma unroll
        for (int s = 0; s < NQ; ++s)
          if (64 * s + 16 * a >= kw) q[s] = zero16();
      }
    };
    if (first < end) load(first);
    f32x4 out[VT];
    float A[C / 16][4];
    walk(
        [&](int n0, const char* ks) {
#pragma unroll
          for (int t = 0; t < C / 16; ++t) {
            f32x4 x = zero4();
            if (t <= wave) {
#pragma unroll
              for (int s = 0; s < NQ; ++s) x = mma_slab<T>(row.read(ks, t, s), q[s], x);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) A[t][e] = x[e] * within[t][e];
          }
          const float g = turned && n0 == 0 ? grow_first : grow;
#pragma unroll
          for (int j = 0; j < VT; ++j) {
            out[j] = zero4();
#pragma unroll
            for (int s = 0; s < NQ; ++s) {
              out[j] = mma_slab<T>(row.read(ss, j, s), q[s], out[j]);
              if constexpr (LO) out[j] = mma_slab<T>(row.read(ss + SB, j, s), q[s], out[j]);
            }
            out[j] *= g;
          }
        },
        [&](int n0, const char* ks) {
          const char* vs = ks + KB;
          if (n0 + C < end) load(n0 + C);
#pragma unroll
          for (int s = 0; s < SL; ++s) {
            if (s * blk_slab<T>() > 16 * wave + 15) break;
            u32x4 hi, lo;
            blk_split<T>(A, s, hi, lo);
#pragma unroll
            for (int j = 0; j < VT; ++j) out[j] = blk_mma_split<T>(vcol.read(vs, s, j), hi, lo, out[j]);
          }
          if (n0 + mine < past) {
            const bool token = n0 + mine < len;
            char* o = J.o.p + b * J.o.sb + (int64_t)(token ? position(n0 + mine) : n0 + mine) * J.o.st + h * J.o.sh + v0 * ES;
#pragma unroll
            for (int j = 0; j < VT; ++j) {
              const int c = 16 * j + 4 * a;
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = token ? out[j][e] * P.scale : 0.f;
              if (c * ES < vw) blk_st4<T>(o + c * ES, v);
            }
          }
        });
    // rows behind the sequence's end
    for (int n0 = end > first ? first + (end - first + C - 1) / C * C : first; n0 < past; n0 += C)
      if (n0 + mine < past) {
        char* o = J.o.p + b * J.o.sb + (int64_t)(n0 + mine) * J.o.st + h * J.o.sh + v0 * ES;
        const float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < VT; ++j)
          if ((16 * j + 4 * a) * ES < vw) blk_st4<T>(o + (16 * j + 4 * a) * ES, v);
      }
    return;
  }

  // the state: tiles KT k0 .. of 16 rows
  const int k0 = KT * (OUT ? wave - 4 : wave);
  f32x4 S[KT][VT];
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int j = 0; j < VT; ++j) S[i][j] = zero4();
  // rows 16 (k0 + i) + 4 a + e, column v0 + 16 j + c16
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) f(S[i][j], e, 16 * (k0 + i) + 4 * a + e, v0 + 16 * j + c16);
  };
  const int64_t size = (int64_t)J.kw * J.vw;
  if (OUT && (J.segments > 1 || J.entry)) {
    const bool flip = J.segments == 1 && J.flip_entry;
    const float* p = J.segments > 1 ? J.part + ((int64_t)bh * J.segments + seg) * size : J.entry + bh * size;
    const float mul = J.segments > 1 ? 1.f : J.entry_mul;
    each([&](f32x4& s, int e, int r, int c) {
      const int64_t x = min(r, J.kw - 1), y = min(c, J.vw - 1);
      s[e] = p[flip ? y * J.kw + x : x * J.vw + y];
    });
    each([&](f32x4& s, int e, int r, int c) { s[e] = r < J.kw && c < J.vw ? s[e] * mul : 0.f; });
  }
  auto publish = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int j = 0; j < VT; ++j) {
        const int r = 16 * j + c16, piece = (16 * (k0 + i) + 4 * a) * ES / 16;
        char* p = ss + r * WK * 16 + ((piece ^ tile_key<WK>(r)) * 16) + (LO ? 8 * (a & 1) : 0);
        const float v[4] = {S[i][j][0], S[i][j][1], S[i][j][2], S[i][j][3]};
        if constexpr (LO) {
          const u32x2 hi = pack8<bf16>(v);
          const uint32_t w0 = hi[0], w1 = hi[1];
          const float d[4] = {v[0] - u2f(w0 << 16), v[1] - u2f(w0 & 0xffff0000u), v[2] - u2f(w1 << 16), v[3] - u2f(w1 & 0xffff0000u)};
          st8(p, hi);
          st8(p + SB, pack8<bf16>(d));
        } else {
          st16(p, pack16<float>(v));
        }
      }
  };
  if constexpr (OUT) publish();
  float left[SL][LO ? 8 : 4];  // decays until the chunk's last token, of the positions of a K^T operand
  auto set_left = [&](int n) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SL; ++s)
#pragma unroll
      for (int e = 0; e < (LO ? 8 : 4); ++e) {
        const int j = s * blk_slab<T>() + 4 * a + (e & 3) + 16 * (e >> 2);
        left[s][e] = j < n ? lin_power(max(n - 1 - j, 0), lg2) : 0.f;
      }
  };
  set_left(min(C, end - first));
  float keep = lin_power(min(C, end - first) - (turned && seg == 0 ? 1 : 0), lg2);
  walk(
      [&](int n0, const char* ks) {
        const char* vs = ks + KB;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int j = 0; j < VT; ++j) S[i][j] *= keep;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          u32x4 f[VT];
#pragma unroll
          for (int j = 0; j < VT; ++j) f[j] = vcol.read(vs, s, j);
#pragma unroll
          for (int i = 0; i < KT; ++i) {
            constexpr int N = LO ? 8 : 4;
            float x[N];
            unpack16<T>(kcol.read(ks, s, k0 + i), x);
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] *= left[s][e];
            u32x4 hi, lo = zero16(), rest = zero16();
            if constexpr (LO) {
              split_bf16(x, hi, lo);
              if (J.exit) {
                float y[8], m[8];
                unpack16<bf16>(hi, y);
                unpack16<bf16>(lo, m);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] - y[e] - m[e];
                rest = pack16<bf16>(x);
              }
            } else {
              hi = pack16<float>(x);
            }
#pragma unroll
            for (int j = 0; j < VT; ++j) {
              S[i][j] = mma_slab<T>(hi, f[j], S[i][j]);
              if constexpr (LO) {
                S[i][j] = mma_slab<T>(lo, f[j], S[i][j]);
                if (J.exit) S[i][j] = mma_slab<T>(rest, f[j], S[i][j]);
              }
            }
          }
        }
        // of the next chunk: another decay behind the first one, others in the last one
        const int n = min(C, end - n0 - C);
        if (n > 0 && n < C) set_left(n);
        if (n > 0 && (n < C || n0 == first)) keep = lin_power(n, lg2);
      },
      [&](int n0, const char*) {
        if (OUT && n0 + C < end) publish();
      });
  auto store = [&](float* p, float mul) __attribute__((always_inline)) {
    each([&](f32x4& s, int e, int r, int c) {
      if (r < J.kw && c < J.vw) p[(int64_t)r * J.vw + c] = s[e] * mul;
    });
  };
  if constexpr (!OUT) store(J.part + ((int64_t)bh * J.segments + seg + 1) * size, 1.f);
  else if (J.exit && seg == J.segments - 1) store(J.exit + bh * size, J.exit_mul * (turned && len > 0 ? lin_power(1, lg2) : 1.f));
}

// The states before the segments from what each segment adds: four elements a
// thread, eight segments' loads under way at a time.
__global__ __launch_bounds__(256) void k_linear_scan(const LinParams P) {
  const LinJob& J = P.job[blockIdx.y];
  const int64_t size = (int64_t)J.kw * J.vw, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int bh = (int)(i / size), e = (int)(i - bh * size);  // size is a multiple of 64
  if (bh >= P.B * P.H) return;
  const int len = lin_len(P, bh / P.H), whole = J.seg_chunks * LIN_CHUNK;
  const float lg2 = lin_log2(P.log_decay, bh % P.H), keep = lin_power(whole, lg2);
  float* p = J.part + (int64_t)bh * J.segments * size + e;
  f32x4 s = zero4();
  if (J.entry) {
    const int r = e / J.vw, c = e - r * J.vw;
#pragma unroll
    for (int x = 0; x < 4; ++x) s[x] = J.entry[bh * size + (J.flip_entry ? (int64_t)(c + x) * J.kw + r : e + x)] * J.entry_mul;
  }
  constexpr int AHEAD = 8;
  for (int m0 = 1; m0 < J.segments; m0 += AHEAD) {
    f32x4 add[AHEAD];
#pragma unroll
    for (int m = 0; m < AHEAD; ++m) add[m] = __builtin_bit_cast(f32x4, ld16(p + min(m0 + m, J.segments - 1) * size));
#pragma unroll
    for (int m = 0; m < AHEAD; ++m) {
      if (m0 + m >= J.segments) break;
      st16(p + (m0 + m - 1) * size, __builtin_bit_cast(u32x4, s));
      const int n = max(0, min(len - (m0 + m - 1) * whole, whole));  // tokens of the segment before
      if (n) s = (n == whole && m0 + m > 1 ? keep : lin_power(n - (m0 + m == 1 ? J.turned : 0), lg2)) * s + add[m];
    }
  }
  st16(p + (J.segments - 1) * size, __builtin_bit_cast(u32x4, s));
}

// One token: a workgroup takes LIN_STEP_COLUMNS columns of one state, four a lane.
template <typename T> __global__ __launch_bounds__(LIN_STEP_THREADS) void k_linear_step(const LinParams P) {
  constexpr int LANES = LIN_STEP_COLUMNS / 4, ROWS = LIN_STEP_THREADS / LANES;
  __shared__ float side[LIN_STEP_THREADS / 64][LIN_STEP_COLUMNS];
  const LinJob& J = P.job[0];
  const int bh = blockIdx.x / J.slices, slice = blockIdx.x - bh * J.slices, b = bh / P.H, h = bh - b * P.H;
  const int c = slice * LIN_STEP_COLUMNS + 4 * (threadIdx.x % LANES), r0 = threadIdx.x / LANES;
  const bool on = !P.mask || P.mask[b];
  const float gamma = lin_power(1, lin_log2(P.log_decay, h));
  const T* q = reinterpret_cast<const T*>(J.q.p + b * J.q.sb + h * J.q.sh);
  const T* k = reinterpret_cast<const T*>(J.k.p + b * J.k.sb + h * J.k.sh);
  const T* v = reinterpret_cast<const T*>(J.v.p + b * J.v.sb + h * J.v.sh);
  const int64_t at = (int64_t)bh * J.kw * J.vw + c;
  f32x4 sum = zero4(), vc = zero4();
  const bool in = c < J.vw;
  if (in && on)
#pragma unroll
    for (int e = 0; e < 4; ++e) vc[e] = to_f32(v[c + e]);
  if (in)
#pragma unroll 4
    for (int r = r0; r < J.kw; r += ROWS) {
      f32x4 s = __builtin_bit_cast(f32x4, ld16(J.entry + at + (int64_t)r * J.vw));
      if (on) {
        s = gamma * s + to_f32(k[r]) * vc;
        sum += to_f32(q[r]) * s;
      }
      st16(J.exit + at + (int64_t)r * J.vw, __builtin_bit_cast(u32x4, s));
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = sum[e];
#pragma unroll
    for (int o = LANES; o < 64; o <<= 1) x += __shfl_xor(x, o);
    if ((threadIdx.x & 63) < LANES) side[threadIdx.x >> 6][4 * (threadIdx.x % LANES) + e] = x;
  }
  __syncthreads();
  const int col = slice * LIN_STEP_COLUMNS + threadIdx.x;
  if (threadIdx.x < LIN_STEP_COLUMNS && col < J.vw) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < LIN_STEP_THREADS / 64; ++i) x += side[i][threadIdx.x];
    reinterpret_cast<T*>(J.o.p + b * J.o.sb + h * J.o.sh)[col] = from_f32<T>(on ? x * P.scale : 0.f);
  }
}

template <typename T, int KWP, int VS, bool OUT> void walk_jobs(const LinParams& P, hipStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < P.jobs; ++i) {
    const int64_t n = (int64_t)P.B * P.H * (P.job[i].segments - (OUT ? 0 : 1)) * P.job[i].slices;
    most = n > most ? n : most;
  }
  const int64_t grid = (most + N_XCD - 1) / N_XCD * N_XCD;
  const int threads = 64 * (state_waves<T, KWP, VS>() + (OUT ? 4 : 0));
  hipLaunchKernelGGL((k_linear<T, KWP, VS, OUT>), dim3((unsigned)grid, (unsigned)P.jobs), dim3(threads), 0, st, P);
}

// Jobs of one shape share a launch.
template <typename T, int KWP, int VS> void walk(const LinParams& all, hipStream_t st) {
  LinParams P = all;
  P.jobs = 0;
  for (int i = 0; i < all.jobs; ++i)
    if (lin_kwp(all.job[i].kw) == KWP && all.job[i].columns == VS) P.job[P.jobs++] = all.job[i];
  if (!P.jobs) return;
  if (P.job[0].segments > 1) {
    walk_jobs<T, KWP, VS, false>(P, st);
    int64_t most = 0;
    for (int i = 0; i < P.jobs; ++i) most = std::max(most, (int64_t)P.B * P.H * P.job[i].kw * P.job[i].vw);
    hipLaunchKernelGGL(k_linear_scan, dim3((unsigned)((most / 4 + 255) / 256), (unsigned)P.jobs), dim3(256), 0, st, P);
  }
  walk_jobs<T, KWP, VS, true>(P, st);
}
template <typename T> void walk_all(const LinParams& P, hipStream_t st) {
  walk<T, 64, 64>(P, st);
  walk<T, 128, 64>(P, st);
  walk<T, 256, 64>(P, st);
  if constexpr (sizeof(T) == 2) walk<T, 128, 128>(P, st);
}

}  // namespace

hipError_t launch_linear(const LinParams& P, bool bf16_path, hipStream_t st) {
  bf16_path ? walk_all<bf16>(P, st) : walk_all<float>(P, st);
  return hipGetLastError();
}

hipError_t launch_linear_step(const LinParams& P, bool bf16_path, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)P.B * P.H * P.job[0].slices));
  if (bf16_path) hipLaunchKernelGGL((k_linear_step<bf16>), grid, dim3(LIN_STEP_THREADS), 0, st, P);
  else hipLaunchKernelGGL((k_linear_step<float>), grid, dim3(LIN_STEP_THREADS), 0, st, P);
  return hipGetLastError();
}

}  // namespace msgla
