// Gated linear recurrence, forward, backward and streaming step.
//
//   log alpha_t = logsigmoid(z_t + b) / gamma,   h_t = alpha_t h_{t-1} + beta_t x_t
//
// Two affine maps h -> A h + H compose to (A2 A1, A2 H1 + H2), so the sequence
// is cut into chunks of REC_CHUNK positions: one pass forms every chunk's map
// (its decay product A and its state H from zero), a short pass runs the maps
// one after the other per channel and leaves each chunk's entry state, and a
// last pass walks the chunks again from those.  The backward's carry
// c = alpha_{t+1} dh_{t+1} obeys the same recurrence from the other end with
// the same decays, c -> A c + R, so its chunks are walked in the same passes.
// A workgroup is one chunk of one slab of channels: wave w holds positions
// 8 w .. 8 w + 7 of it in registers, all loads in flight at once, and the
// waves' maps meet in LDS.  HBM-bound: a few tens of instructions an element
// against 6 (forward) and 10 (backward) bytes of bf16.
#include "device_common.hpp"
#include "recurrence.hpp"

namespace msgla {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// ---- one thread's VEC consecutive channels of a row --------------------------

template <typename T, int VEC> struct RowLoad;
template <> struct RowLoad<bf16, 4> {
  typedef u32x2 raw;
  static __device__ __forceinline__ void unpack(raw r, float* f) {
    const uint32_t a = r[0], b = r[1];
    f[0] = u2f(a << 16);
    f[1] = u2f(a & 0xffff0000u);
    f[2] = u2f(b << 16);
    f[3] = u2f(b & 0xffff0000u);
  }
  static __device__ __forceinline__ raw pack(const float* f) { return pack8<bf16>(f); }
};
template <> struct RowLoad<float, 4> {
  typedef u32x4 raw;
  static __device__ __forceinline__ void unpack(raw r, float* f) { unpack16<float>(r, f); }
  static __device__ __forceinline__ raw pack(const float* f) { return pack16<float>(f); }
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
  if constexpr (VEC == 4) unpack16<float>(ld16(p), f);
  else f[0] = *p;
}
template <int VEC> __device__ __forceinline__ void store_f32(float* p, const float* f) {
  if constexpr (VEC == 4) st16(p, pack16<float>(f));
  else *p = f[0];
}

// ---- the gate ------------------------------------------------------------------

// -expm1(y) for y <= 0: the series to y^8 above -0.5 (its tail is below
// 2^-26 of the sum there), 1 - e elsewhere, with e = exp(y) given.
__device__ __forceinline__ float neg_expm1(float y, float e) {
  float s = 1.f + y * (1.f / 8.f);
  s = 1.f + y * (1.f / 7.f) * s;
  s = 1.f + y * (1.f / 6.f) * s;
  s = 1.f + y * (1.f / 5.f) * s;
  s = 1.f + y * (1.f / 4.f) * s;
  s = 1.f + y * (1.f / 3.f) * s;
  s = 1.f + y * (1.f / 2.f) * s;
  return y > -0.5f ? -y * s : 1.f - e;
}

struct Gate {
  float alpha, beta;
};

// E = exp(-|z|) gives both logs' pieces: logsigmoid(z) = min(z, 0) - log1p(E),
// log1p(E) = 2 atanh(E / (2 + E)) by its series (E / (2 + E) <= 1/3: the terms
// up to the 13th power leave 1e-8 of the sum), so small E keeps its relative
// accuracy, which 1 - alpha hangs on.
template <int MODE> __device__ __forceinline__ Gate gate(float z, float inv_gamma, float& E) {
  E = __builtin_amdgcn_exp2f(-fabsf(z) * LOG2E);
  const float s = E * __builtin_amdgcn_rcpf(2.f + E), w = s * s;
  float q = 1.f / 13.f;
  q = q * w + 1.f / 11.f;
  q = q * w + 1.f / 9.f;
  q = q * w + 1.f / 7.f;
  q = q * w + 1.f / 5.f;
  q = q * w + 1.f / 3.f;
  const float la = (fminf(z, 0.f) - 2.f * (s + s * w * q)) * inv_gamma;
  Gate g;
  g.alpha = __builtin_amdgcn_exp2f(la * LOG2E);
  if constexpr (MODE == 0) g.beta = 1.f;
  if constexpr (MODE == 1) g.beta = neg_expm1(la, g.alpha);
  if constexpr (MODE == 2) g.beta = sqrtf(neg_expm1(2.f * la, g.alpha * g.alpha));
  // fminf drops a NaN z; the sum brings it back
  if (z != z) g.alpha = g.beta = z;
  return g;
}

// dbeta / dlog alpha
template <int MODE> __device__ __forceinline__ float slope(const Gate& g) {
  if constexpr (MODE == 0) return 0.f;
  if constexpr (MODE == 1) return -g.alpha;
  return g.beta == 0.f ? 0.f : -g.alpha * g.alpha / g.beta;
}

// ---- where a thread stands -----------------------------------------------------

template <int VEC> struct Place {
  int b, chunk, t0, c, cl;  // cl: the channel that is loaded where c is past the last
  bool on;
  __device__ Place(const RecParams& P) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slab = blockIdx.x % P.slabs, rest = blockIdx.x / P.slabs;
    chunk = rest % P.nch;
    b = rest / P.nch;
    t0 = chunk * REC_CHUNK + wave * REC_T;
    c = (slab * 64 + lane) * VEC;
    on = c < P.D;
    cl = on ? c : 0;
  }
};

template <int VEC> __device__ __forceinline__ void load_bias(const RecParams& P, int cl, float* bias) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) bias[e] = 0.f;
  if (P.bias) load_f32<VEC>(P.bias + cl, bias);
}

// bit i: position t0 + i is a token
__device__ __forceinline__ uint32_t tokens(const RecParams& P, int b, int t0) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    const int t = t0 + i;
    if (t < P.L && (!P.mask || P.mask[(int64_t)b * P.L + t])) m |= 1u << i;
  }
  return m;
}

// ---- forward ---------------------------------------------------------------------

// OUT: walk the chunk from its entry state and write y; otherwise write its map.
template <typename T, int VEC, int MODE, bool OUT>
__global__ __launch_bounds__(64 * REC_WAVES) void k_rec_forward(const RecParams P) {
  __shared__ float sA[REC_WAVES][64 * VEC], sH[REC_WAVES][64 * VEC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Place<VEC> at(P);
  float bias[VEC], entry[VEC];
  load_bias<VEC>(P, at.cl, bias);
  const int64_t ch = ((int64_t)at.b * P.nch + at.chunk) * P.D + at.cl;
#pragma unroll
  for (int e = 0; e < VEC; ++e) entry[e] = 0.f;
  if constexpr (OUT) {
    if (P.nch > 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) entry[e] = P.agg[2 * (ch + e) + 1];
    } else if (P.h_in) {
      load_f32<VEC>(P.h_in + (int64_t)at.b * P.D + at.cl, entry);
    }
  }
  typename RowLoad<T, VEC>::raw rx[REC_T], rz[REC_T];
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    const int t = min(at.t0 + i, P.L - 1);
    rx[i] = load_row<T, VEC>(P.x, at.b, t, at.cl);
    rz[i] = load_row<T, VEC>(P.z, at.b, t, at.cl);
  }
  const uint32_t tok = tokens(P, at.b, at.t0);
  float A[VEC], H[VEC], al[REC_T][VEC], u[REC_T][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, H[e] = 0.f;
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    float x[VEC], z[VEC];
    RowLoad<T, VEC>::unpack(rx[i], x);
    RowLoad<T, VEC>::unpack(rz[i], z);
    const bool on = tok >> i & 1;
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
#pragma unroll
  for (int e = 0; e < VEC; ++e) sA[wave][e * 64 + lane] = A[e], sH[wave][e * 64 + lane] = H[e];
  __syncthreads();
  if constexpr (!OUT) {
    if (wave != 0 || !at.on) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float a = A[e], h = H[e];
#pragma unroll
      for (int w = 1; w < REC_WAVES; ++w) {
        const float aw = sA[w][e * 64 + lane];
        h = aw * h + sH[w][e * 64 + lane];
        a *= aw;
      }
      P.agg[2 * (ch + e)] = a;
      P.agg[2 * (ch + e) + 1] = h;
    }
  } else {
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      h[e] = entry[e];
      for (int w = 0; w < wave; ++w) h[e] = sA[w][e * 64 + lane] * h[e] + sH[w][e * 64 + lane];
    }
    if (!at.on) return;
#pragma unroll
    for (int i = 0; i < REC_T; ++i) {
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[e] = al[i][e] * h[e] + u[i][e];
        y[e] = tok >> i & 1 ? h[e] : 0.f;
      }
      if (at.t0 + i < P.L) store_row<T, VEC>(P.y, at.b, at.t0 + i, at.c, y);
    }
    if (P.nch == 1 && P.h_out && wave == REC_WAVES - 1) store_f32<VEC>(P.h_out + (int64_t)at.b * P.D + at.c, h);
  }
}

// Runs the chunks' maps per channel: agg's second entry becomes the chunk's
// entry state and, backward, rev the carry that enters it from the right.
template <bool BACKWARD> __global__ __launch_bounds__(64) void k_rec_carry(const RecParams P) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= (int64_t)P.B * P.D) return;
  const int64_t b = i / P.D, c = i - b * P.D;
  float2* agg = reinterpret_cast<float2*>(P.agg) + b * P.nch * P.D + c;
  constexpr int AHEAD = 8;
  if (!BACKWARD || P.nch > 1) {
    float h = P.h_in ? P.h_in[i] : 0.f;
    for (int k0 = 0; k0 < P.nch; k0 += AHEAD) {
      float2 m[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) m[k] = agg[(int64_t)min(k0 + k, P.nch - 1) * P.D];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (k0 + k < P.nch) {
          agg[(int64_t)(k0 + k) * P.D].y = h;
          h = m[k].x * h + m[k].y;
        }
    }
    if (!BACKWARD && P.h_out) P.h_out[i] = h;
  }
  if constexpr (BACKWARD) {
    float* rev = P.rev + b * P.nch * P.D + c;
    float r = P.dh_out ? P.dh_out[i] : 0.f;
    for (int k0 = P.nch - 1; k0 >= 0; k0 -= AHEAD) {
      float a[AHEAD], m[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int64_t at = (int64_t)max(k0 - k, 0) * P.D;
        a[k] = agg[at].x;
        m[k] = rev[at];
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (k0 - k >= 0) {
          rev[(int64_t)(k0 - k) * P.D] = r;
          r = a[k] * r + m[k];
        }
    }
    if (P.dh_in) P.dh_in[i] = r;
  }
}

// ---- backward --------------------------------------------------------------------

template <typename T, int VEC, int MODE, bool OUT>
__global__ __launch_bounds__(64 * REC_WAVES) void k_rec_backward(const RecParams P) {
  __shared__ float sA[REC_WAVES][64 * VEC], sH[REC_WAVES][64 * VEC], sR[REC_WAVES][64 * VEC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Place<VEC> at(P);
  float bias[VEC], entry[VEC], carry[VEC];
  load_bias<VEC>(P, at.cl, bias);
  const int64_t ch = ((int64_t)at.b * P.nch + at.chunk) * P.D + at.cl, bd = (int64_t)at.b * P.D + at.cl;
#pragma unroll
  for (int e = 0; e < VEC; ++e) entry[e] = carry[e] = 0.f;
  if constexpr (OUT) {
    if (P.nch > 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) entry[e] = P.agg[2 * (ch + e) + 1];
      load_f32<VEC>(P.rev + ch, carry);
    } else {
      if (P.h_in) load_f32<VEC>(P.h_in + bd, entry);
      if (P.dh_out) load_f32<VEC>(P.dh_out + bd, carry);
    }
  }
  typename RowLoad<T, VEC>::raw rx[REC_T], rz[REC_T], rd[REC_T];
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    const int t = min(at.t0 + i, P.L - 1);
    rx[i] = load_row<T, VEC>(P.x, at.b, t, at.cl);
    rz[i] = load_row<T, VEC>(P.z, at.b, t, at.cl);
    rd[i] = typename RowLoad<T, VEC>::raw{};
    if (P.dy.p) rd[i] = load_row<T, VEC>(P.dy, at.b, t, at.cl);
  }
  const uint32_t tok = tokens(P, at.b, at.t0);
  const uint32_t tod = P.dy.p ? tok : 0u;  // where dy counts
  float A[VEC], H[VEC], R[VEC], al[REC_T][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, H[e] = R[e] = 0.f;
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    float x[VEC], z[VEC], d[VEC];
    RowLoad<T, VEC>::unpack(rx[i], x);
    RowLoad<T, VEC>::unpack(rz[i], z);
    RowLoad<T, VEC>::unpack(rd[i], d);
    const bool on = tok >> i & 1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float E;
      const Gate g = gate<MODE>(z[e] + bias[e], P.inv_gamma, E);
      const float a = on ? g.alpha : 1.f;
      al[i][e] = a;
      A[e] *= a;
      H[e] = a * H[e] + (on ? g.beta * x[e] : 0.f);
      R[e] += A[e] * (tod >> i & 1 ? d[e] : 0.f);  // dy_t reaches the front through alpha_{t0} .. alpha_t
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sA[wave][e * 64 + lane] = A[e];
    sH[wave][e * 64 + lane] = H[e];
    sR[wave][e * 64 + lane] = R[e];
  }
  __syncthreads();
  if constexpr (!OUT) {
    if (wave != 0 || !at.on) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float a = A[e], h = H[e], r = R[e];
#pragma unroll
      for (int w = 1; w < REC_WAVES; ++w) {
        const float aw = sA[w][e * 64 + lane];
        h = aw * h + sH[w][e * 64 + lane];
        r += a * sR[w][e * 64 + lane];
        a *= aw;
      }
      P.agg[2 * (ch + e)] = a;
      P.agg[2 * (ch + e) + 1] = h;
      P.rev[ch + e] = r;
    }
    return;
  }
  float h[VEC], cr[VEC], hb[REC_T][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = entry[e];
    for (int w = 0; w < wave; ++w) h[e] = sA[w][e * 64 + lane] * h[e] + sH[w][e * 64 + lane];
    cr[e] = carry[e];
    for (int w = REC_WAVES - 1; w > wave; --w) cr[e] = sA[w][e * 64 + lane] * cr[e] + sR[w][e * 64 + lane];
    db[e] = 0.f;
  }
  // states before each position, then the gradients from the last to the first
#pragma unroll
  for (int i = 0; i < REC_T; ++i) {
    float x[VEC], z[VEC];
    RowLoad<T, VEC>::unpack(rx[i], x);
    RowLoad<T, VEC>::unpack(rz[i], z);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float E;
      const Gate g = gate<MODE>(z[e] + bias[e], P.inv_gamma, E);
      hb[i][e] = h[e];
      h[e] = al[i][e] * h[e] + (tok >> i & 1 ? g.beta * x[e] : 0.f);
    }
  }
#pragma unroll
  for (int i = REC_T - 1; i >= 0; --i) {
    float x[VEC], z[VEC], d[VEC], dx[VEC], dz[VEC];
    RowLoad<T, VEC>::unpack(rx[i], x);
    RowLoad<T, VEC>::unpack(rz[i], z);
    RowLoad<T, VEC>::unpack(rd[i], d);
    const bool on = tok >> i & 1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float zb = z[e] + bias[e];
      float E;
      const Gate g = gate<MODE>(zb, P.inv_gamma, E);
      const float sig = (zb < 0.f ? 1.f : E) * __builtin_amdgcn_rcpf(1.f + E);  // sigmoid(-zb)
      const float dh = cr[e] + (tod >> i & 1 ? d[e] : 0.f);
      dx[e] = on ? g.beta * dh : 0.f;
      dz[e] = on ? dh * (g.alpha * hb[i][e] + slope<MODE>(g) * x[e]) * (sig * P.inv_gamma) : 0.f;
      db[e] += dz[e];
      cr[e] = al[i][e] * dh;
    }
    if (at.on && at.t0 + i < P.L) {
      store_row<T, VEC>(P.dx, at.b, at.t0 + i, at.c, dx);
      store_row<T, VEC>(P.dz, at.b, at.t0 + i, at.c, dz);
    }
  }
  if (P.nch == 1 && P.dh_in && wave == 0 && at.on) store_f32<VEC>(P.dh_in + bd, cr);
  if (!P.dbias) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < VEC; ++e) sA[wave][e * 64 + lane] = db[e];
  __syncthreads();
  if (wave == 0 && at.on) {
#pragma unroll
    for (int w = 1; w < REC_WAVES; ++w)
#pragma unroll
      for (int e = 0; e < VEC; ++e) db[e] += sA[w][e * 64 + lane];
    store_f32<VEC>(P.dbp + ch, db);
  }
}

// dbias: the partials of all chunks of all sequences, in 64 bits and a fixed order
__global__ __launch_bounds__(1024) void k_rec_dbias(const RecParams P) {
  __shared__ double part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  const int64_t n = (int64_t)P.B * P.nch;
  double s = 0.0;
  if (c < P.D)
    for (int64_t i = wave; i < n; i += 16) s += (double)P.dbp[i * P.D + c];
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
  load_bias<VEC>(P, c, bias);
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
  static void forward(const RecParams& P, hipStream_t st) {
    const dim3 grid((unsigned)(P.slabs * P.nch * P.B)), block(64 * REC_WAVES);
    if (P.nch > 1) {
      hipLaunchKernelGGL((k_rec_forward<T, VEC, MODE, false>), grid, block, 0, st, P);
      hipLaunchKernelGGL(k_rec_carry<false>, dim3((unsigned)(((int64_t)P.B * P.D + 63) / 64)), dim3(64), 0, st, P);
    }
    hipLaunchKernelGGL((k_rec_forward<T, VEC, MODE, true>), grid, block, 0, st, P);
  }
  static void backward(const RecParams& P, hipStream_t st) {
    const dim3 grid((unsigned)(P.slabs * P.nch * P.B)), block(64 * REC_WAVES);
    if (P.nch > 1) {
      hipLaunchKernelGGL((k_rec_backward<T, VEC, MODE, false>), grid, block, 0, st, P);
      hipLaunchKernelGGL(k_rec_carry<true>, dim3((unsigned)(((int64_t)P.B * P.D + 63) / 64)), dim3(64), 0, st, P);
    }
    hipLaunchKernelGGL((k_rec_backward<T, VEC, MODE, true>), grid, block, 0, st, P);
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
  if (bf16_path) vec ? by_mode<bf16, 4>(input, f) : by_mode<bf16, 1>(input, f);
  else vec ? by_mode<float, 4>(input, f) : by_mode<float, 1>(input, f);
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
