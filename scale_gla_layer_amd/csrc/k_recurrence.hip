// Gated linear recurrence, forward, backward and streaming step.
//
//   log alpha_t = logsigmoid(z_t + b) / gamma,   h_t = alpha_t h_{t-1} + beta_t x_t
//
// Two affine maps h -> A h + H compose to (A2 A1, A2 H1 + H2), so a workgroup
// reduces its REC_CHUNK positions of 64 VEC channels to one map (decay product
// A, state from zero H) and needs only the state that enters it to finish: its
// positions stay in registers meanwhile, and x and z are read once.  The maps
// pass between workgroups through memory, one 64-bit word {A, H} a channel:
// each workgroup publishes its own, then waits for those before it back to the
// last group boundary (every REC_GROUP chunks) and for the state there, which
// the group's last workgroup publishes.  So a sequence costs one wait per group
// rather than one per chunk, and always the same sums in the same order.
//   Every wait ends: a workgroup learns its chunk from a counter of its chain
// (one sequence's slab of channels), so the chunks before it have workgroups
// that are already running; those publish their maps before they wait, and wait
// only for chunks still further back.
//   The words need no fences: a word is one atomic store that carries all that
// its reader wants, and starts as all ones, which no map is (a NaN decay is
// stored as the quiet NaN).
//   The backward's carry c = alpha_{t+1} dh_{t+1} obeys the same recurrence from
// the other end, c -> A c + R.  It runs first the forward without y, which
// leaves every chunk's entry state, then the chunks from the last to the first.
// Bound by HBM and, nearly as much, by the gate's arithmetic (about 45 vector
// instruction slots an element with NORM), which is why it is worth reading and
// evaluating once.  B = 8, L = 2048, D = 1024 in bf16: forward 37 us (2.7 TB/s; a
// copy of the bytes takes 20), backward 94 (33); in three passes with the maps
// joined between them they took 77 and 286.
#include <type_traits>

#include "device_common.hpp"
#include "recurrence.hpp"

namespace msgla {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// ---- one thread's VEC consecutive channels of a row --------------------------

template <typename T, int VEC> struct RowLoad;
template <> struct RowLoad<bf16, 2> {
  typedef uint32_t raw;
  static __device__ __forceinline__ void unpack(raw r, float* f) {
    f[0] = u2f(r << 16);
    f[1] = u2f(r & 0xffff0000u);
  }
  static __device__ __forceinline__ raw pack(const float* f) {
    typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, bf16x2{(bf16)f[0], (bf16)f[1]});
  }
};
template <> struct RowLoad<float, 2> {
  typedef u32x2 raw;
  static __device__ __forceinline__ void unpack(raw r, float* f) {
    const uint32_t a = r[0], b = r[1];
    f[0] = u2f(a);
    f[1] = u2f(b);
  }
  static __device__ __forceinline__ raw pack(const float* f) { return pack8<float>(f); }
};
template <typename T> struct RowLoad<T, 1> {
  typedef T raw;
  static __device__ __forceinline__ void unpack(raw r, float* f) { f[0] = to_f32(r); }
  static __device__ __forceinline__ raw pack(const float* f) { return from_f32<T>(f[0]); }
};

template <typename T, int VEC>
__device__ __forceinline__ typename RowLoad<T, VEC>::raw load_row(const RecRows& r, int64_t b, int t, int c) {
  const T* p = reinterpret_cast<const T*>(r.p) + b * r.sb + (int64_t)t * r.st + c;
  return *reinterpret_cast<const typename RowLoad<T, VEC>::raw*>(p);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_row(const RecRows& r, int64_t b, int t, int c, const float* f) {
  T* p = reinterpret_cast<T*>(r.p) + b * r.sb + (int64_t)t * r.st + c;
  *reinterpret_cast<typename RowLoad<T, VEC>::raw*>(p) = RowLoad<T, VEC>::pack(f);
}

template <int VEC> __device__ __forceinline__ void load_f32(const float* p, float* f) {
  RowLoad<float, VEC>::unpack(*reinterpret_cast<const typename RowLoad<float, VEC>::raw*>(p), f);
}
template <int VEC> __device__ __forceinline__ void store_f32(float* p, const float* f) {
  *reinterpret_cast<typename RowLoad<float, VEC>::raw*>(p) = RowLoad<float, VEC>::pack(f);
}

// ---- the gate ------------------------------------------------------------------

// -expm1(y) for y <= 0, given e = exp(y): the series to y^6 / 720 above -1/4 (its
// next term is below 2^-24 of the sum there), 1 - e below, where e's rounding is
// less than 2^-21 of the difference.
__device__ __forceinline__ float neg_expm1(float y, float e) {
  float s = y * (1.f / 720.f) + 1.f / 120.f;
  s = s * y + 1.f / 24.f;
  s = s * y + 1.f / 6.f;
  s = s * y + 0.5f;
  s = s * y + 1.f;
  return y > -0.25f ? -y * s : 1.f - e;
}

struct Gate {
  float alpha, beta, rbeta;  // rbeta: 1 / beta, with NORM
};

// With E = exp(-|z|), logsigmoid(z) = min(z, 0) - log(1 + E).  log2(1 + E) / E
// on [0, 1] by a polynomial of degree 8 fitted to its relative error (3e-8), so
// that a small E, which 1 - alpha hangs on, keeps its relative accuracy.
template <int MODE> __device__ __forceinline__ Gate gate(float z, float inv_gamma, float& E) {
  E = __builtin_amdgcn_exp2f(-fabsf(z) * LOG2E);
  float q = 0.007549172880588877f;
  q = q * E - 0.04256702485905678f;
  q = q * E + 0.11285613290977259f;
  q = q * E - 0.1971189186662436f;
  q = q * E + 0.27564138814486205f;
  q = q * E - 0.3584084662973025f;
  q = q * E + 0.48069295654396693f;
  q = q * E - 0.7213402079704885f;
  q = q * E + 1.442694997434065f;
  const float la = (fminf(z, 0.f) * LOG2E - E * q) * inv_gamma;  // log2 alpha; a NaN z comes back through E
  Gate g;
  g.alpha = __builtin_amdgcn_exp2f(la);
  if constexpr (MODE == 0) g.beta = 1.f;
  if constexpr (MODE == 1) g.beta = neg_expm1(la * LN2, g.alpha);
  if constexpr (MODE == 2) {
    const float b2 = neg_expm1(la * (2.f * LN2), g.alpha * g.alpha);
    // b2 runs out of normal numbers before it is 0 (z + b from 74 to 87 at a gamma of 1e6),
    // and the hardware's root takes those for 0: scaled by an even power of two
    g.rbeta = 0x1p12f * __builtin_amdgcn_rsqf(0x1p24f * b2);
    g.beta = b2 == 0.f ? 0.f : b2 * g.rbeta;
  }
  return g;
}

// dbeta / dlog alpha
template <int MODE> __device__ __forceinline__ float slope(const Gate& g) {
  if constexpr (MODE == 0) return 0.f;
  if constexpr (MODE == 1) return -g.alpha;
  return g.beta == 0.f ? 0.f : -g.alpha * g.alpha * g.rbeta;
}

// ---- words between workgroups -----------------------------------------------------

constexpr uint64_t NOT_YET = ~0ull;

__device__ __forceinline__ uint64_t make_word(float a, float h) {
  const uint32_t u = a != a ? 0x7fc00000u : f2u(a);
  return (uint64_t)u << 32 | f2u(h);
}
__device__ __forceinline__ void publish(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t await(uint64_t* p) {
  uint64_t v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  while (v == NOT_YET) {
    __builtin_amdgcn_s_sleep(1);
    v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  return v;
}
__device__ __forceinline__ float word_a(uint64_t v) { return u2f((uint32_t)(v >> 32)); }
__device__ __forceinline__ float word_h(uint64_t v) { return u2f((uint32_t)v); }

// All words of the passes (16 bytes a thread), and their chains' counters.
__global__ __launch_bounds__(256) void k_rec_init(uint64_t* words, int64_t pairs, uint32_t* counters, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < pairs) st16(words + 2 * i, u32x4{~0u, ~0u, ~0u, ~0u});
  if (i < n) counters[i] = 0;
}

// ---- a chunk -------------------------------------------------------------------

// Where a workgroup stands: `step` chunks have begun before it in its chain.
template <int VEC, int NW> struct Place {
  int b, step, lane, wave, c, cl;  // cl: the channel that is loaded where c is past the last
  bool on;
  __device__ Place(const RecParams& P, uint32_t* counters, int nch) {
    __shared__ int ticket;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chains = P.slabs * P.B, chain = blockIdx.x % chains;
    step = 0;
    if (nch > 1) {
      if (threadIdx.x == 0)
        ticket = (int)__hip_atomic_fetch_add(&counters[chain], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      step = __builtin_amdgcn_readfirstlane(ticket);
    }
    b = chain / P.slabs;
    c = ((chain % P.slabs) * 64 + lane) * VEC;
    on = c < P.D;
    cl = on ? c : 0;
  }
};

// bit i: position t0 + i is a token (the same in every lane; lane i looks at its own)
template <int NT> __device__ __forceinline__ uint32_t tokens(const RecParams& P, int b, int t0) {
  const int lane = threadIdx.x & 63, t = t0 + lane;
  const bool in = lane < NT && t < P.L;
  return (uint32_t)__ballot(in && (!P.mask || P.mask[(int64_t)b * P.L + (in ? t : 0)]));
}

// What enters the sequence, for the chunks of the first group.
template <int VEC> __device__ __forceinline__ void load_begin(const float* p, int64_t at, int step, float* begin) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) begin[e] = 0.f;
  if (p && step < REC_GROUP) load_f32<VEC>(p + at, begin);
}

// Before the barrier that a workgroup publishes its map behind: the chunk that writes
// the sequence's result, which may go to the same memory, waits for the maps of all
// chunks that read what enters.  The barrier itself does not wait for loads; a use of
// the values does.
template <int VEC> __device__ __forceinline__ void have_begin(float* begin) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) asm volatile("" : "+v"(begin[e])::"memory");
}

// The value that enters chunk `step` of the chain: the state at the last group
// boundary run through the maps since.  Wave w fetches map w (and w + NW, ..)
// of the group; a barrier; every lane runs them.
template <int VEC, int NW> struct Chain {
  float a[REC_GROUP][64 * VEC], h[REC_GROUP][64 * VEC];

  // maps: {A, H} words [step][D] of this sequence, ends: state words [group][D]
  __device__ void fetch(const RecParams& P, const Place<VEC, NW>& at, uint64_t* maps, uint64_t* ends,
                        const float* begin) {
    const int g = at.step / REC_GROUP, n = at.step % REC_GROUP;
    for (int k = at.wave; k <= n; k += NW)  // k == n: the state at the boundary
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float x = 1.f, y = begin[e];
        if (at.on && k < n) {
          const uint64_t v = await(maps + (int64_t)(g * REC_GROUP + k) * P.D + at.c + e);
          x = word_a(v);
          y = word_h(v);
        } else if (at.on && g > 0) {
          y = word_h(await(ends + (int64_t)(g - 1) * P.D + at.c + e));
        }
        a[k][e * 64 + at.lane] = x;
        h[k][e * 64 + at.lane] = y;
      }
  }
  __device__ void run(const Place<VEC, NW>& at, float* state) const {
    const int n = at.step % REC_GROUP;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float s = h[n][e * 64 + at.lane];
      for (int k = 0; k < n; ++k) s = a[k][e * 64 + at.lane] * s + h[k][e * 64 + at.lane];
      state[e] = s;
    }
  }
};

// ---- forward ---------------------------------------------------------------------

// Y: writes y and h_out.  Otherwise leaves the chunks' entry states for the backward.
template <typename T, int VEC, int MODE, bool Y>
__global__ __launch_bounds__(64 * REC_WAVES) void k_rec_forward(const RecParams P) {
  constexpr int NW = REC_WAVES, NT = REC_NT;
  __shared__ float sA[NW][64 * VEC], sH[NW][64 * VEC];
  __shared__ Chain<VEC, NW> chain;
  const Place<VEC, NW> at(P, P.counters, P.nch);
  const int t0 = at.step * REC_CHUNK + at.wave * NT;
  float bias[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) bias[e] = 0.f;
  if (P.bias) load_f32<VEC>(P.bias + at.cl, bias);
  const uint32_t tok = tokens<NT>(P, at.b, t0);
  float A[VEC], H[VEC], al[NT][VEC], u[NT][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, H[e] = 0.f;
  if (tok) {
    typename RowLoad<T, VEC>::raw rx[NT], rz[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = min(t0 + i, P.L - 1);
      rx[i] = load_row<T, VEC>(P.x, at.b, t, at.cl);
      rz[i] = load_row<T, VEC>(P.z, at.b, t, at.cl);
    }
    auto walk = [&](auto full) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float x[VEC], z[VEC];
        RowLoad<T, VEC>::unpack(rx[i], x);
        RowLoad<T, VEC>::unpack(rz[i], z);
        const bool on = full.value || (tok >> i & 1);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float E;
          const Gate g = gate<MODE>(z[e] + bias[e], P.inv_gamma, E);
          al[i][e] = on ? g.alpha : 1.f;
          u[i][e] = on ? g.beta * x[e] : 0.f;
          A[e] *= al[i][e];
          H[e] = al[i][e] * H[e] + u[i][e];
        }
      }
    };
    if (tok == (1u << NT) - 1) walk(std::true_type());
    else walk(std::false_type());
  }
  float state[VEC], begin[VEC];
  load_begin<VEC>(P.h_in, (int64_t)at.b * P.D + at.cl, at.step, begin);
  have_begin<VEC>(begin);
  uint64_t* maps = P.maps + (int64_t)at.b * P.nch * P.D;
  uint64_t* ends = P.ends + (int64_t)at.b * P.groups * P.D;
#pragma unroll
  for (int e = 0; e < VEC; ++e) sA[at.wave][e * 64 + at.lane] = A[e], sH[at.wave][e * 64 + at.lane] = H[e];
  if (P.nch == 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) state[e] = begin[e];
    __syncthreads();
  } else {
    __syncthreads();
    if (at.wave == 0 && at.step + 1 < P.nch) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float a = A[e], h = H[e];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          const float aw = sA[w][e * 64 + at.lane];
          h = aw * h + sH[w][e * 64 + at.lane];
          a *= aw;
        }
        if (at.on) publish(maps + (int64_t)at.step * P.D + at.c + e, make_word(a, h));
      }
    }
    chain.fetch(P, at, maps, ends, begin);
    __syncthreads();
    chain.run(at, state);
  }
  // the state that leaves the chunk goes out first: others wait for it
  const bool boundary = at.step % REC_GROUP == REC_GROUP - 1 && at.step + 1 < P.nch;
  const bool final = Y && at.step == P.nch - 1 && P.h_out;
  float h[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = state[e];
    for (int w = 0; w < at.wave; ++w) h[e] = sA[w][e * 64 + at.lane] * h[e] + sH[w][e * 64 + at.lane];
  }
  if constexpr (!Y) {
    const int k = at.step * (REC_CHUNK / REC_BCHUNK) + at.wave / REC_BWAVES;
    if (at.wave % REC_BWAVES == 0 && k < P.nchb && at.on) store_f32<VEC>(P.entry + ((int64_t)at.b * P.nchb + k) * P.D + at.c, h);
  }
  if (at.wave == NW - 1 && at.on && (boundary || final)) {
    float end[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      end[e] = A[e] * h[e] + H[e];
      if (boundary) publish(ends + (int64_t)(at.step / REC_GROUP) * P.D + at.c + e, make_word(0.f, end[e]));
    }
    if (final) store_f32<VEC>(P.h_out + (int64_t)at.b * P.D + at.c, end);
  }
  if constexpr (Y) {
    if (!at.on) return;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (tok) h[e] = al[i][e] * h[e] + u[i][e];
        y[e] = tok >> i & 1 ? h[e] : 0.f;
      }
      if (t0 + i < P.L) store_row<T, VEC>(P.y, at.b, t0 + i, at.c, y);
    }
  }
}

// ---- backward --------------------------------------------------------------------

// Chunks from the last to the first; P.entry holds their entry states.
// fp32 with PLAIN and two channels a lane is held to two workgroups a CU, which costs
// it 16 registers in memory (B = 8, L = 2048, D = 1024: 130 -> 110 us); the other fp32
// forms fit by themselves.  So does bf16, which held to them takes 260 us for 250 at
// B = 16, L = 4093.
template <typename T, int VEC, int MODE>
__global__ __launch_bounds__(64 * REC_BWAVES, sizeof(T) == 4 ? 2 : 1) void k_rec_backward(const RecParams P) {
  constexpr int NW = REC_BWAVES, NT = REC_NT;
  __shared__ float sA[NW][64 * VEC], sH[NW][64 * VEC], sR[NW][64 * VEC];
  __shared__ Chain<VEC, NW> chain;
  const Place<VEC, NW> at(P, P.counters + (int64_t)P.slabs * P.B, P.nchb);
  const int chunk = P.nchb - 1 - at.step, t0 = chunk * REC_BCHUNK + at.wave * NT;
  const int64_t seq = (int64_t)at.b * P.D + at.cl, ch = ((int64_t)at.b * P.nchb + chunk) * P.D + at.cl;
  float bias[VEC], state[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) bias[e] = state[e] = 0.f;
  if (P.bias) load_f32<VEC>(P.bias + at.cl, bias);
  if (P.nchb > 1) load_f32<VEC>(P.entry + ch, state);
  else if (P.h_in) load_f32<VEC>(P.h_in + seq, state);
  const uint32_t tok = tokens<NT>(P, at.b, t0);
  // per position: alpha, beta, dbeta/dlog alpha x, sigmoid(-z) / gamma; x and dy stay packed
  float A[VEC], H[VEC], R[VEC], al[NT][VEC], be[NT][VEC], sl[NT][VEC], sg[NT][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, H[e] = R[e] = 0.f;
  typename RowLoad<T, VEC>::raw rx[NT], rd[NT];
  if (tok) {
    typename RowLoad<T, VEC>::raw rz[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = min(t0 + i, P.L - 1);
      rx[i] = load_row<T, VEC>(P.x, at.b, t, at.cl);
      rz[i] = load_row<T, VEC>(P.z, at.b, t, at.cl);
      rd[i] = typename RowLoad<T, VEC>::raw{};
      if (P.dy.p) rd[i] = load_row<T, VEC>(P.dy, at.b, t, at.cl);
    }
    auto walk = [&](auto full) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float x[VEC], z[VEC], d[VEC];
        RowLoad<T, VEC>::unpack(rx[i], x);
        RowLoad<T, VEC>::unpack(rz[i], z);
        RowLoad<T, VEC>::unpack(rd[i], d);
        const bool on = full.value || (tok >> i & 1);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float zb = z[e] + bias[e];
          float E;
          const Gate g = gate<MODE>(zb, P.inv_gamma, E);
          al[i][e] = on ? g.alpha : 1.f;
          be[i][e] = on ? g.beta : 0.f;
          sl[i][e] = on ? slope<MODE>(g) * x[e] : 0.f;
          sg[i][e] = on ? (zb < 0.f ? 1.f : E) * __builtin_amdgcn_rcpf(1.f + E) * P.inv_gamma : 0.f;
          A[e] *= al[i][e];
          H[e] = al[i][e] * H[e] + (on ? g.beta * x[e] : 0.f);
          R[e] += A[e] * (on ? d[e] : 0.f);  // dy_t reaches the front through alpha_{t0} .. alpha_t
        }
      }
    };
    if (tok == (1u << NT) - 1) walk(std::true_type());
    else walk(std::false_type());
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sA[at.wave][e * 64 + at.lane] = A[e];
    sH[at.wave][e * 64 + at.lane] = H[e];
    sR[at.wave][e * 64 + at.lane] = R[e];
  }
  float carry[VEC], begin[VEC];
  load_begin<VEC>(P.dh_out, seq, at.step, begin);
  have_begin<VEC>(begin);
  uint64_t* maps = P.rmaps + (int64_t)at.b * P.nchb * P.D;
  uint64_t* ends = P.rends + (int64_t)at.b * P.groupsb * P.D;
  if (P.nchb == 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) carry[e] = begin[e];
    __syncthreads();
  } else {
    __syncthreads();
    if (at.wave == 0 && at.step + 1 < P.nchb) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float a = A[e], r = R[e];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          r += a * sR[w][e * 64 + at.lane];
          a *= sA[w][e * 64 + at.lane];
        }
        if (at.on) publish(maps + (int64_t)at.step * P.D + at.c + e, make_word(a, r));
      }
    }
    chain.fetch(P, at, maps, ends, begin);
    __syncthreads();
    chain.run(at, carry);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    for (int w = NW - 1; w > at.wave; --w) carry[e] = sA[w][e * 64 + at.lane] * carry[e] + sR[w][e * 64 + at.lane];
  const bool boundary = at.step % REC_GROUP == REC_GROUP - 1 && at.step + 1 < P.nchb;
  const bool final = chunk == 0 && P.dh_in;
  if (at.wave == 0 && at.on && (boundary || final)) {
    float front[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      front[e] = A[e] * carry[e] + R[e];
      if (boundary) publish(ends + (int64_t)(at.step / REC_GROUP) * P.D + at.c + e, make_word(0.f, front[e]));
    }
    if (final) store_f32<VEC>(P.dh_in + seq, front);
  }
  float h[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = state[e];
    for (int w = 0; w < at.wave; ++w) h[e] = sA[w][e * 64 + at.lane] * h[e] + sH[w][e * 64 + at.lane];
    db[e] = 0.f;
  }
  if (tok) {
    // alpha_t h_{t-1} + slope x, then the gradients from the last position to the first
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float x[VEC];
      RowLoad<T, VEC>::unpack(rx[i], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float decayed = al[i][e] * h[e];
        sl[i][e] = (decayed + sl[i][e]) * sg[i][e];
        h[e] = decayed + (tok >> i & 1 ? be[i][e] * x[e] : 0.f);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const int i = NT - 1 - k;
    float dx[VEC], dz[VEC], d[VEC];
    if (tok) RowLoad<T, VEC>::unpack(rd[i], d);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dx[e] = dz[e] = 0.f;
      if (tok) {
        const bool on = tok >> i & 1;
        const float dh = carry[e] + (on ? d[e] : 0.f);
        dx[e] = on ? be[i][e] * dh : 0.f;
        dz[e] = on ? dh * sl[i][e] : 0.f;
        db[e] += dz[e];
        carry[e] = al[i][e] * dh;
      }
    }
    if (at.on && t0 + i < P.L) {
      store_row<T, VEC>(P.dx, at.b, t0 + i, at.c, dx);
      store_row<T, VEC>(P.dz, at.b, t0 + i, at.c, dz);
    }
  }
  if (!P.dbias) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < VEC; ++e) sH[at.wave][e * 64 + at.lane] = db[e];
  __syncthreads();
  if (at.wave == 0 && at.on) {
#pragma unroll
    for (int w = 1; w < NW; ++w)
#pragma unroll
      for (int e = 0; e < VEC; ++e) db[e] += sH[w][e * 64 + at.lane];
    store_f32<VEC>(P.dbp + ch, db);
  }
}

// dbias: the partials of all chunks of all sequences, in 64 bits and a fixed
// order.  16 waves take every 16th row of 64 channels, four loads in flight.
__global__ __launch_bounds__(1024) void k_rec_dbias(const RecParams P) {
  __shared__ double part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  const int64_t n = (int64_t)P.B * P.nchb;
  double s = 0.0;
  if (c < P.D) {
    const float* p = P.dbp + c;
    int64_t i = wave;
    for (; i + 48 < n; i += 64) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = p[(i + 16 * k) * P.D];
#pragma unroll
      for (int k = 0; k < 4; ++k) s += (double)v[k];
    }
    for (; i < n; i += 16) s += (double)p[i * P.D];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave || c >= P.D) return;
  for (int w = 1; w < 16; ++w) s += part[w][lane];
  P.dbias[c] = (float)s;
}

// ---- streaming step --------------------------------------------------------------

template <typename T, int VEC, int MODE> __global__ __launch_bounds__(64) void k_rec_step(const RecParams P) {
  const int slab = blockIdx.x % P.slabs, b = blockIdx.x / P.slabs, c = (slab * 64 + (int)threadIdx.x) * VEC;
  if (c >= P.D) return;
  float bias[VEC], h[VEC], x[VEC], z[VEC], y[VEC];
  const auto rx = load_row<T, VEC>(P.x, b, 0, c), rz = load_row<T, VEC>(P.z, b, 0, c);
#pragma unroll
  for (int e = 0; e < VEC; ++e) bias[e] = 0.f;
  if (P.bias) load_f32<VEC>(P.bias + c, bias);
  load_f32<VEC>(P.h_in + (int64_t)b * P.D + c, h);
  const bool on = !P.mask || P.mask[b];
  RowLoad<T, VEC>::unpack(rx, x);
  RowLoad<T, VEC>::unpack(rz, z);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float E;
    const Gate g = gate<MODE>(z[e] + bias[e], P.inv_gamma, E);
    const float n = g.alpha * h[e] + g.beta * x[e];
    h[e] = on ? n : h[e];
    y[e] = on ? n : 0.f;
  }
  store_row<T, VEC>(P.y, b, 0, c, y);
  store_f32<VEC>(P.h_out + (int64_t)b * P.D + c, h);
}

template <typename T, int VEC, int MODE> struct Launch {
  static dim3 grid(const RecParams& P, int nch) { return dim3((unsigned)((int64_t)P.slabs * nch * P.B)); }
  static void init(const RecParams& P, hipStream_t st) {
    const int64_t pairs = P.words / 2, chains = 2 * (int64_t)P.slabs * P.B;
    const int64_t n = pairs > chains ? pairs : chains;
    hipLaunchKernelGGL(k_rec_init, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, P.maps, pairs, P.counters, chains);
  }
  static void forward(const RecParams& P, hipStream_t st) {
    if (P.nch > 1) init(P, st);
    hipLaunchKernelGGL((k_rec_forward<T, VEC, MODE, true>), grid(P, P.nch), dim3(64 * REC_WAVES), 0, st, P);
  }
  static void backward(const RecParams& P, hipStream_t st) {
    if (P.nchb > 1) {
      init(P, st);
      hipLaunchKernelGGL((k_rec_forward<T, VEC, MODE, false>), grid(P, P.nch), dim3(64 * REC_WAVES), 0, st, P);
    }
    hipLaunchKernelGGL((k_rec_backward<T, VEC, MODE>), grid(P, P.nchb), dim3(64 * REC_BWAVES), 0, st, P);
    if (P.dbias) hipLaunchKernelGGL(k_rec_dbias, dim3((P.D + 63) / 64), dim3(1024), 0, st, P);
  }
  static void step(const RecParams& P, hipStream_t st) {
    hipLaunchKernelGGL((k_rec_step<T, VEC, MODE>), dim3((unsigned)(P.slabs * P.B)), dim3(64), 0, st, P);
  }
};

// f is called with the Launch of the configuration
template <typename T, int VEC, class F> void by_mode(int input, F f) {
  if (input == 0) f(Launch<T, VEC, 0>());
  else if (input == 1) f(Launch<T, VEC, 1>());
  else f(Launch<T, VEC, 2>());
}
template <class F> void dispatch(int input, bool bf16_path, bool vec, F f) {
  if (bf16_path) vec ? by_mode<bf16, 2>(input, f) : by_mode<bf16, 1>(input, f);
  else vec ? by_mode<float, 2>(input, f) : by_mode<float, 1>(input, f);
}

}  // namespace

hipError_t launch_recurrence_forward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st) {
  dispatch(input, bf16_path, vec, [&](auto l) { l.forward(P, st); });
  return hipGetLastError();
}

hipError_t launch_recurrence_backward(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st) {
  dispatch(input, bf16_path, vec, [&](auto l) { l.backward(P, st); });
  return hipGetLastError();
}

hipError_t launch_recurrence_step(const RecParams& P, int input, bool bf16_path, bool vec, hipStream_t st) {
  dispatch(input, bf16_path, vec, [&](auto l) { l.step(P, st); });
  return hipGetLastError();
}

}  // namespace msgla
