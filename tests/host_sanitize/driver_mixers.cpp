// Host-side exercise of the entry points of layer norm, linear attention and window
// attention for a build whose host code carries AddressSanitizer and
// UndefinedBehaviorSanitizer: size queries over a grid of configurations and sizes,
// the largest accepted and the first rejected ones among them, and the
// argument-error paths of every call.  No call here reaches the GPU: each returns
// before its first HIP call.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "msgla.h"

static int failures = 0;
#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "expectation failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                      \
    }                                                                  \
  } while (0)
#define INVALID(call) EXPECT((call) == MSGLA_ERR_INVALID_ARG)

static const size_t BAD = (size_t)-1;
static char* const FAR = reinterpret_cast<char*>(1 << 20);  // never read
static float* const F = reinterpret_cast<float*>(FAR);
static int32_t* const I = reinterpret_cast<int32_t*>(FAR);
static float* const F2 = reinterpret_cast<float*>(FAR + 2);
static int32_t* const I2 = reinterpret_cast<int32_t*>(FAR + 2);

static const int64_t Bs[] = {INT64_MIN, -1, 0, 1, 3, 4096, 1 << 20, (1 << 20) + 1, INT64_MAX};
static const int64_t Ls[] = {INT64_MIN, 0, 1, 63, 2049, 1 << 24, (1 << 24) + 1, INT64_MAX};

static bool sizes_ok(int64_t B, int64_t L) {
  return B >= 1 && L >= 1 && B <= 1 << 20 && L <= 1 << 24 && B * L <= 1 << 28;
}

static long norms() {
  long n = 0;
  const msgla_rows r = {FAR, 1024, 1024};
  for (int width : {INT32_MIN, 0, 1, 7, 1001, 16384, 16385})
    for (float eps : {0.f, 1e-21f, 1e-20f, 1e-5f, 1.f, 2.f, __builtin_nanf("")})
      for (int dtype = -1; dtype <= 2; ++dtype) {
        const msgla_layer_norm_config c = {width, eps, dtype};
        const bool ok = width >= 1 && width <= 16384 && eps >= 1e-20f && eps <= 1.f && (dtype == 0 || dtype == 1);
        for (int64_t B : Bs)
          for (int64_t L : Ls) {
            const bool fits = ok && sizes_ok(B, L);
            const size_t b = msgla_layer_norm_backward_workspace_bytes(&c, B, L);
            EXPECT(fits == (b != BAD));
            if (fits) {
              EXPECT(b >= (size_t)width * 8);
              EXPECT(msgla_layer_norm_backward(&c, &r, &r, F, F, F, B, L, &r, F, F, FAR, b - 1, 0) == MSGLA_ERR_WORKSPACE);
            } else {
              INVALID(msgla_layer_norm_forward(&c, &r, F, F, B, L, &r, F, F, 0));
              INVALID(msgla_layer_norm_backward(&c, &r, &r, F, F, F, B, L, &r, F, F, FAR, BAD, 0));
            }
            ++n;
          }
      }
  const msgla_layer_norm_config c = {64, 1e-5f, MSGLA_BF16};
  const msgla_rows none = {nullptr, 64, 64}, odd = {FAR + 1, 64, 64}, back = {FAR, -64, 64}, back_t = {FAR, 64, -64};
  for (const msgla_rows* x : {(const msgla_rows*)nullptr, &none, &odd, &back, &back_t}) {
    INVALID(msgla_layer_norm_forward(&c, x, F, F, 2, 30, &r, F, F, 0));
    INVALID(msgla_layer_norm_forward(&c, &r, F, F, 2, 30, x, F, F, 0));
    for (int k = 0; k < 3; ++k)
      INVALID(msgla_layer_norm_backward(&c, k == 0 ? x : &r, k == 1 ? x : &r, F, F, F, 2, 30, k == 2 ? x : &r, F, F, FAR, BAD, 0));
  }
  for (int k = 0; k < 4; ++k)
    INVALID(msgla_layer_norm_forward(&c, &r, k == 0 ? F2 : F, k == 1 ? F2 : F, 2, 30, &r, k == 2 ? F2 : F, k == 3 ? F2 : F, 0));
  for (int k = 0; k < 5; ++k)
    INVALID(msgla_layer_norm_backward(&c, &r, &r, k == 0 ? F2 : F, k == 1 ? F2 : F, k == 2 ? F2 : F, 2, 30, &r, k == 3 ? F2 : F,
                                      k == 4 ? F2 : F, FAR, BAD, 0));
  INVALID(msgla_layer_norm_forward(nullptr, &r, F, F, 2, 30, &r, F, F, 0));
  INVALID(msgla_layer_norm_backward(&c, &r, &r, F, nullptr, F, 2, 30, &r, F, F, FAR, BAD, 0));
  INVALID(msgla_layer_norm_backward(&c, &r, &r, F, F, nullptr, 2, 30, &r, F, F, FAR, BAD, 0));
  INVALID(msgla_layer_norm_backward(&c, &r, &r, F, F, F, 2, 30, &r, F, nullptr, nullptr, BAD, 0));
  INVALID(msgla_layer_norm_backward(&c, &r, &r, F, F, F, 2, 30, &r, nullptr, F, FAR + 8, BAD, 0));
  return n;
}

static const msgla_heads h = {FAR, 4096, 2048, 256}, none = {nullptr, 4096, 2048, 256}, odd = {FAR + 8, 4096, 2048, 256},
                         sb = {FAR, 4, 2048, 256}, st = {FAR, 4096, -2048, 256}, sh = {FAR, 4096, 2048, 9};
static const msgla_heads* const bad[] = {nullptr, &none, &odd, &sb, &st, &sh};

template <class C> struct Configs {
  C good, cs[64];
  bool ok[64];
  int m = 0;
  explicit Configs(const C& g) : good(g) { add(true, [](C&) {}); }
  template <class Set> void add(bool valid, Set set) {
    cs[m] = good;
    set(cs[m]);
    ok[m++] = valid;
  }
  template <class V> void field(V C::*at, std::initializer_list<V> valid, std::initializer_list<V> invalid) {
    for (V v : valid) add(true, [&](C& c) { c.*at = v; });
    for (V v : invalid) add(false, [&](C& c) { c.*at = v; });
  }
};

static long linear() {
  typedef msgla_linear_config C;
  long n = 0;
  Configs<C> all(C{4, 128, 256, 0.088f, MSGLA_BF16});
  all.field(&C::heads, {1, 1024}, {0, -1, 1025});
  all.field(&C::d_k, {8, 72, 256}, {0, 4, 12, 264, -8});
  all.field(&C::d_v, {8, 72, 128}, {0, 4, 12, 264, -8});
  all.field(&C::scale, {1e-30f, 1e30f}, {0.f, -1.f, 2e30f, __builtin_nanf("")});
  all.field(&C::dtype, {(int32_t)MSGLA_F32}, {-1, 2});
  for (int i = 0; i < all.m; ++i)
    for (int64_t B : Bs)
      for (int64_t L : Ls) {
        const C& c = all.cs[i];
        const bool fits = all.ok[i] && sizes_ok(B, L);
        const size_t f = msgla_linear_attention_workspace_bytes(&c, B, L), b = msgla_linear_attention_backward_workspace_bytes(&c, B, L);
        EXPECT(fits == (f != BAD) && fits == (b != BAD));
        if (fits) {
          if (f) EXPECT(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, F, B, L, &h, F, FAR, f - 1, 0) == MSGLA_ERR_WORKSPACE);
          if (b)
            EXPECT(msgla_linear_attention_backward(&c, &h, &h, &h, F, I, F, &h, F, B, L, &h, &h, &h, F, FAR, b - 1, 0) ==
                   MSGLA_ERR_WORKSPACE);
        } else {
          INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, F, B, L, &h, F, FAR, BAD, 0));
          INVALID(msgla_linear_attention_backward(&c, &h, &h, &h, F, I, F, &h, F, B, L, &h, &h, &h, F, FAR, BAD, 0));
        }
        if (!all.ok[i] || B < 1 || B > 1 << 20) INVALID(msgla_linear_attention_step(&c, &h, &h, &h, F, 0, F, B, &h, F, 0));
        ++n;
      }
  const C& c = all.good;
  const int64_t B = 1, L = 4096;
  EXPECT(msgla_linear_attention_workspace_bytes(&c, B, L) > 0);
  for (const msgla_heads* x : bad) {
    auto at = [&](int i, int k) { return i == k ? x : &h; };
    for (int k = 0; k < 4; ++k)
      INVALID(msgla_linear_attention_forward(&c, at(0, k), at(1, k), at(2, k), F, I, F, B, L, at(3, k), F, FAR, BAD, 0));
    for (int k = 0; k < 7; ++k)
      INVALID(msgla_linear_attention_backward(&c, at(0, k), at(1, k), at(2, k), F, I, F, at(3, k), F, B, L, at(4, k), at(5, k),
                                              at(6, k), F, FAR, BAD, 0));
    for (int k = 0; k < 4 && x != &st; ++k)  // stride_t is not read
      INVALID(msgla_linear_attention_step(&c, at(0, k), at(1, k), at(2, k), F, 0, F, 2, at(3, k), F, 0));
  }
  float* const f8 = reinterpret_cast<float*>(FAR + 8);
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, nullptr, I, F, B, L, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F2, I, F, B, L, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I2, F, B, L, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, f8, B, L, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, F, B, L, &h, f8, FAR, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, F, B, L, &h, F, nullptr, BAD, 0));
  INVALID(msgla_linear_attention_forward(&c, &h, &h, &h, F, I, F, B, L, &h, F, FAR + 8, BAD, 0));
  INVALID(msgla_linear_attention_backward(&c, &h, &h, &h, nullptr, I, F, &h, F, B, L, &h, &h, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_backward(&c, &h, &h, &h, F, I, F, &h, f8, B, L, &h, &h, &h, F, FAR, BAD, 0));
  INVALID(msgla_linear_attention_backward(&c, &h, &h, &h, F, I, F, &h, F, B, L, &h, &h, &h, f8, FAR, BAD, 0));
  INVALID(msgla_linear_attention_backward(&c, &h, &h, &h, F, I, F, &h, F, B, L, &h, &h, &h, F, nullptr, BAD, 0));
  INVALID(msgla_linear_attention_step(&c, &h, &h, &h, nullptr, 0, F, 2, &h, F, 0));
  INVALID(msgla_linear_attention_step(&c, &h, &h, &h, F, 0, nullptr, 2, &h, F, 0));
  INVALID(msgla_linear_attention_step(&c, &h, &h, &h, F, 0, F, 2, &h, nullptr, 0));
  INVALID(msgla_linear_attention_step(&c, &h, &h, &h, F, 0, f8, 2, &h, F, 0));
  return n;
}

static long windows() {
  typedef msgla_window_config C;
  long n = 0;
  Configs<C> all(C{16, 4, 128, 128, 512, 4, 0.088f, MSGLA_BF16});
  all.field(&C::heads_q, {4, 1024}, {0, 3, -4, 1028});
  all.field(&C::heads_kv, {1, 16}, {0, 3, 17, -1});
  all.field(&C::d_k, {8, 72}, {0, 4, 12, 136});
  all.field(&C::d_v, {8, 256}, {0, 4, 12, 264});
  all.field(&C::window, {1, 1 << 24}, {0, -1, (1 << 24) + 1, INT32_MAX});
  all.field(&C::n_sink, {0, 1024}, {-1, 1025, INT32_MIN});
  all.field(&C::scale, {1e-30f, 1e30f}, {0.f, -1.f, 2e30f, __builtin_nanf("")});
  all.field(&C::dtype, {(int32_t)MSGLA_F32}, {-1, 2});
  const int64_t Ss[] = {INT64_MIN, 0, 1, 63, 8192, 1 << 24, (1 << 24) + 1, INT64_MAX};
  for (int i = 0; i < all.m; ++i)
    for (int64_t B : Bs)
      for (int64_t L : Ls)
        for (int64_t S : Ss) {
          const C& c = all.cs[i];
          const bool s_ok = all.ok[i] && B >= 1 && B <= 1 << 20 && S >= 1 && S <= 1 << 24, fits = s_ok && sizes_ok(B, L);
          const size_t f = msgla_window_attention_workspace_bytes(&c, B, L, S), t = msgla_window_attention_step_workspace_bytes(&c, B, S);
          const size_t b = msgla_window_attention_backward_workspace_bytes(&c, B, L, S);
          EXPECT(fits == (f != BAD) && fits == (b != BAD) && s_ok == (t != BAD));
          if (!fits) {
            INVALID(msgla_window_attention(&c, &h, &h, &h, I, I, B, L, S, &h, F, FAR, BAD, 0));
            INVALID(msgla_window_attention_backward(&c, &h, &h, &h, I, I, &h, F, &h, B, L, S, &h, &h, &h, FAR, BAD, 0));
            INVALID(msgla_window_attention_append(&c, &h, &h, I, I, B, L, S, &h, &h, 0));
          } else {
            EXPECT(b >= (size_t)B * c.heads_q * L * 8);
            if (f) EXPECT(msgla_window_attention(&c, &h, &h, &h, I, I, B, L, S, &h, F, FAR, f - 1, 0) == MSGLA_ERR_WORKSPACE);
            const msgla_status s = msgla_window_attention_backward(&c, &h, &h, &h, I, I, &h, F, &h, B, L, S, &h, &h, &h, FAR, b - 1, 0);
            EXPECT(s == MSGLA_ERR_WORKSPACE || s == MSGLA_ERR_UNSUPPORTED);
          }
          if (!s_ok) INVALID(msgla_window_attention_step(&c, &h, &h, &h, I, B, S, &h, &h, &h, FAR, BAD, 0));
          else if (t) EXPECT(msgla_window_attention_step(&c, &h, &h, &h, I, B, S, &h, &h, &h, FAR, t - 1, 0) == MSGLA_ERR_WORKSPACE);
          ++n;
        }
  const C& c = all.good;
  const int64_t B = 2, L = 10, S = 4000;  // few queries: the attention has a workspace
  EXPECT(msgla_window_attention_workspace_bytes(&c, B, L, S) > 0 && msgla_window_attention_step_workspace_bytes(&c, B, S) > 0);
  for (const msgla_heads* x : bad) {
    auto at = [&](int i, int k) { return i == k ? x : &h; };
    for (int k = 0; k < 4; ++k)
      INVALID(msgla_window_attention(&c, at(0, k), at(1, k), at(2, k), I, I, B, L, S, at(3, k), F, FAR, BAD, 0));
    for (int k = 0; k < 8; ++k)
      INVALID(msgla_window_attention_backward(&c, at(0, k), at(1, k), at(2, k), I, I, at(3, k), F, at(4, k), B, L, S, at(5, k),
                                              at(6, k), at(7, k), FAR, BAD, 0));
    for (int k = 0; k < 4; ++k) INVALID(msgla_window_attention_append(&c, at(0, k), at(1, k), I, I, B, L, S, at(2, k), at(3, k), 0));
    for (int k = 0; k < 6; ++k)
      if (x != &st || k >= 4)  // stride_t of the four _t tensors is not read
        INVALID(msgla_window_attention_step(&c, at(0, k), at(1, k), at(2, k), I, B, S, at(4, k), at(5, k), at(3, k), FAR, BAD, 0));
  }
  INVALID(msgla_window_attention(&c, &h, &h, &h, I2, I, B, L, S, &h, F, FAR, BAD, 0));
  INVALID(msgla_window_attention(&c, &h, &h, &h, I, I2, B, L, S, &h, F, FAR, BAD, 0));
  INVALID(msgla_window_attention(&c, &h, &h, &h, I, I, B, L, S, &h, F2, FAR, BAD, 0));
  INVALID(msgla_window_attention(&c, &h, &h, &h, I, I, B, L, S, &h, F, nullptr, BAD, 0));
  INVALID(msgla_window_attention(&c, &h, &h, &h, I, I, B, L, S, &h, F, FAR + 8, BAD, 0));
  INVALID(msgla_window_attention_backward(&c, &h, &h, &h, I, I, &h, nullptr, &h, B, L, S, &h, &h, &h, FAR, BAD, 0));
  INVALID(msgla_window_attention_backward(&c, &h, &h, &h, I2, I, &h, F, &h, B, L, S, &h, &h, &h, FAR, BAD, 0));
  INVALID(msgla_window_attention_backward(&c, &h, &h, &h, I, I, &h, F, &h, B, L, S, &h, &h, &h, nullptr, BAD, 0));
  INVALID(msgla_window_attention_backward(&c, &h, &h, &h, I, I, &h, F, &h, B, L, S, &h, &h, &h, FAR + 8, BAD, 0));
  INVALID(msgla_window_attention_append(&c, &h, &h, I2, I, B, L, S, &h, &h, 0));
  INVALID(msgla_window_attention_append(&c, &h, &h, I, I2, B, L, S, &h, &h, 0));
  INVALID(msgla_window_attention_step(&c, &h, &h, &h, nullptr, B, S, &h, &h, &h, FAR, BAD, 0));
  INVALID(msgla_window_attention_step(&c, &h, &h, &h, I2, B, S, &h, &h, &h, FAR, BAD, 0));
  INVALID(msgla_window_attention_step(&c, &h, &h, &h, I, B, S, &h, &h, &h, nullptr, BAD, 0));
  return n;
}

int main() {
  const long a = norms(), b = linear(), c = windows();
  std::printf("%ld norm sizes, %ld linear sizes, %ld window sizes, failures %d\n", a, b, c, failures);
  return failures ? 1 : 0;
}
