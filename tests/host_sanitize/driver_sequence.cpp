// Host-side exercise of the sequence operators' entry points for a build whose
// host code carries AddressSanitizer and UndefinedBehaviorSanitizer: size queries
// over a grid of configurations and sizes, the largest accepted and the first
// rejected ones among them, and the argument-error paths of every call.  No call
// here reaches the GPU: each returns before its first HIP call.
#include <cstdint>
#include <cstdio>

#include "msgla.h"

static int failures = 0;
#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "expectation failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

static const size_t BAD = (size_t)-1;
static char* const FAR = reinterpret_cast<char*>(1 << 20);  // never read
static float* const F = reinterpret_cast<float*>(FAR);
static int32_t* const I = reinterpret_cast<int32_t*>(FAR);

static const int64_t Bs[] = {-1, 0, 1, 3, 4096, 1 << 20, (1 << 20) + 1, INT64_MAX};
static const int64_t Ls[] = {-5, 0, 1, 63, 2049, 1 << 24, (1 << 24) + 1, INT64_MAX};

static long recurrence() {
  long n = 0;
  const int widths[] = {-1, 0, 1, 7, 128, 65536, 65537};
  const float gammas[] = {0.f, 1e-7f, 1e-6f, 16.f, 1e6f, 2e6f, __builtin_nanf("")};
  for (int width : widths)
    for (int input = -1; input <= 3; ++input)
      for (float gamma : gammas)
        for (int dtype = -1; dtype <= 2; ++dtype) {
          const msgla_recurrence_config c = {width, input, gamma, dtype};
          const bool ok = width >= 1 && width <= 65536 && input >= 0 && input <= 2 && gamma >= 1e-6f && gamma <= 1e6f &&
                          (dtype == 0 || dtype == 1);
          for (int64_t B : Bs)
            for (int64_t L : Ls) {
              const bool fits = ok && B >= 1 && L >= 1 && B <= 1 << 20 && L <= 1 << 24 && B * L <= 1 << 28;
              const size_t f = msgla_recurrence_workspace_bytes(&c, B, L), b = msgla_recurrence_backward_workspace_bytes(&c, B, L);
              EXPECT(fits == (f != BAD) && fits == (b != BAD));
              if (fits) EXPECT(b >= f && b >= (size_t)(B * width * 4));
              const msgla_rows r = {FAR, width, width};
              if (!fits) {
                EXPECT(msgla_recurrence_forward(&c, &r, &r, 0, 0, 0, B, L, &r, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
                EXPECT(msgla_recurrence_backward(&c, &r, &r, 0, 0, 0, &r, 0, B, L, &r, &r, 0, 0, FAR, BAD, 0) ==
                       MSGLA_ERR_INVALID_ARG);
              } else {
                if (f) EXPECT(msgla_recurrence_forward(&c, &r, &r, 0, 0, 0, B, L, &r, 0, FAR, f - 1, 0) == MSGLA_ERR_WORKSPACE);
                EXPECT(msgla_recurrence_backward(&c, &r, &r, 0, 0, 0, &r, 0, B, L, &r, &r, 0, 0, FAR, b - 1, 0) ==
                       MSGLA_ERR_WORKSPACE);
              }
              ++n;
            }
        }
  const msgla_recurrence_config c = {64, 2, 16.f, MSGLA_BF16};
  const msgla_rows r = {FAR, 64, 64}, none = {nullptr, 64, 64}, odd = {FAR + 1, 64, 64}, back = {FAR, -64, 64}, back_t = {FAR, 64, -64};
  float* const off = reinterpret_cast<float*>(FAR + 2);
  const msgla_rows* bad[] = {nullptr, &none, &odd, &back, &back_t};
  for (const msgla_rows* x : bad) {
    EXPECT(msgla_recurrence_forward(&c, x, &r, 0, 0, 0, 2, 300, &r, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
    EXPECT(msgla_recurrence_forward(&c, &r, x, 0, 0, 0, 2, 300, &r, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
    EXPECT(msgla_recurrence_forward(&c, &r, &r, 0, 0, 0, 2, 300, x, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
    for (int at = 0; at < 5; ++at)
      if (at != 2 || x)  // dy may be NULL beside dh_out
        EXPECT(msgla_recurrence_backward(&c, at == 0 ? x : &r, at == 1 ? x : &r, 0, 0, 0, at == 2 ? x : &r, F, 2, 300,
                                         at == 3 ? x : &r, at == 4 ? x : &r, 0, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
    for (int at = 0; at < 3; ++at)
      EXPECT(msgla_recurrence_step(&c, at == 0 ? x : &r, at == 1 ? x : &r, 0, 0, F, 0, at == 2 ? x : &r, F, 0) ==
             MSGLA_ERR_INVALID_ARG);
  }
  EXPECT(msgla_recurrence_forward(nullptr, &r, &r, 0, 0, 0, 2, 300, &r, 0, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  for (int at = 0; at < 3; ++at)
    EXPECT(msgla_recurrence_forward(&c, &r, &r, at == 0 ? off : 0, 0, at == 1 ? off : 0, 2, 300, &r, at == 2 ? off : 0, FAR, BAD,
                                    0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_forward(&c, &r, &r, 0, 0, 0, 2, 300, &r, 0, nullptr, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_forward(&c, &r, &r, 0, 0, 0, 2, 300, &r, 0, FAR + 8, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_backward(&c, &r, &r, 0, 0, 0, nullptr, nullptr, 2, 300, &r, &r, 0, 0, FAR, BAD, 0) ==
         MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_backward(&c, &r, &r, 0, 0, 0, &r, 0, 2, 30, &r, &r, 0, 0, nullptr, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_step(&c, &r, &r, 0, 0, nullptr, 2, &r, F, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_step(&c, &r, &r, 0, 0, F, 2, &r, nullptr, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_recurrence_step(&c, &r, &r, 0, 0, F, (1 << 20) + 1, &r, F, 0) == MSGLA_ERR_INVALID_ARG);
  return n;
}

static long blocks() {
  long n = 0;
  // one field off at a time, at its ends
  const msgla_block_config good = {16, 4, 128, 128, 64, 16, 1, 2, 0.088f, MSGLA_BF16};
  msgla_block_config cs[64];
  bool ok[64];
  int m = 0;
  auto add = [&](bool valid, auto set) {
    cs[m] = good;
    set(cs[m]);
    ok[m++] = valid;
  };
  add(true, [](auto&) {});
  for (int v : {0, 3, -4, 1028}) add(false, [v](auto& c) { c.heads_q = v; });
  for (int v : {4, 1024}) add(true, [v](auto& c) { c.heads_q = v; });
  for (int v : {0, 3, 17, -1}) add(false, [v](auto& c) { c.heads_kv = v; });
  for (int v : {1, 16}) add(true, [v](auto& c) { c.heads_kv = v; });
  for (int v : {0, 4, 12, 136}) add(false, [v](auto& c) { c.d_k = v; });
  for (int v : {8, 72}) add(true, [v](auto& c) { c.d_k = v; });
  for (int v : {0, 4, 12, 264}) add(false, [v](auto& c) { c.d_v = v; });
  for (int v : {8, 256}) add(true, [v](auto& c) { c.d_v = v; });
  for (int v : {0, 16, 48, 256}) add(false, [v](auto& c) { c.block = v; });
  for (int v : {32, 128}) add(true, [v](auto& c) { c.block = v; });
  for (int v : {0, 65, 2}) add(false, [v](auto& c) { c.n_select = v; });
  for (int v : {3, 64}) add(true, [v](auto& c) { c.n_select = v; });
  for (int v : {-1, 15, INT32_MAX}) add(false, [v](auto& c) { c.n_first = v; });
  for (int v : {0, 14}) add(true, [v](auto& c) { c.n_first = v; });
  for (int v : {0, -1, 16, INT32_MAX}) add(false, [v](auto& c) { c.n_recent = v; });
  for (float v : {0.f, -1.f, 2e30f, __builtin_nanf("")}) add(false, [v](auto& c) { c.scale = v; });
  for (float v : {1e-30f, 1e30f}) add(true, [v](auto& c) { c.scale = v; });
  for (int v : {-1, 2}) add(false, [v](auto& c) { c.dtype = v; });
  add(true, [](auto& c) { c.dtype = MSGLA_F32; });
  const msgla_heads h = {FAR, 4096, 2048, 256};
  const int64_t Ss[] = {-1, 0, 1, 63, 8192, 1 << 24, (1 << 24) + 1, INT64_MAX};
  for (int i = 0; i < m; ++i)
    for (int64_t B : Bs)
      for (int64_t L : Ls)
        for (int64_t S : Ss) {
          const msgla_block_config& c = cs[i];
          const bool s_ok = ok[i] && B >= 1 && B <= 1 << 20 && S >= 1 && S <= 1 << 24;
          const bool fits = s_ok && L >= 1 && L <= 1 << 24 && B * L <= 1 << 28;
          const size_t f = msgla_block_attention_workspace_bytes(&c, B, L, S);
          const size_t b = msgla_block_attention_backward_workspace_bytes(&c, B, L, S);
          const size_t t = msgla_block_attention_step_workspace_bytes(&c, B, S);
          EXPECT(fits == (f != BAD) && fits == (b != BAD) && s_ok == (t != BAD));
          if (fits) EXPECT(b >= (size_t)B * c.heads_kv * L * c.n_select * 4);  // the lists
          if (s_ok) EXPECT(t >= (size_t)B * c.heads_kv * c.n_select * 4);
          if (!fits) {
            EXPECT(msgla_block_select(&c, &h, F, 0, 0, B, L, S, I, 0) == MSGLA_ERR_INVALID_ARG);
            EXPECT(msgla_block_attention(&c, &h, &h, &h, I, 0, 0, B, L, S, &h, F, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
            EXPECT(msgla_block_attention_backward(&c, &h, &h, &h, I, 0, 0, &h, F, &h, B, L, S, &h, &h, &h, FAR, BAD, 0) ==
                   MSGLA_ERR_INVALID_ARG);
          } else {
            if (f) EXPECT(msgla_block_attention(&c, &h, &h, &h, I, 0, 0, B, L, S, &h, F, FAR, f - 1, 0) == MSGLA_ERR_WORKSPACE);
            EXPECT(msgla_block_attention_backward(&c, &h, &h, &h, I, 0, 0, &h, F, &h, B, L, S, &h, &h, &h, FAR, b - 1, 0) ==
                   MSGLA_ERR_WORKSPACE);
          }
          if (!s_ok) {
            EXPECT(msgla_block_means(&c, &h, 0, 0, B, S, F, 0) == MSGLA_ERR_INVALID_ARG);
            EXPECT(msgla_block_attention_step(&c, &h, &h, &h, I, B, S, &h, &h, F, &h, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
          } else {
            EXPECT(msgla_block_attention_step(&c, &h, &h, &h, I, B, S, &h, &h, F, &h, FAR, t - 1, 0) == MSGLA_ERR_WORKSPACE);
          }
          ++n;
        }
  const msgla_heads none = {nullptr, 4096, 2048, 256}, odd = {FAR + 8, 4096, 2048, 256}, sb = {FAR, 4, 2048, 256},
                    st = {FAR, 4096, -2048, 256}, sh = {FAR, 4096, 2048, 9};
  const msgla_heads* bad[] = {nullptr, &none, &odd, &sb, &st, &sh};
  int32_t* const io = reinterpret_cast<int32_t*>(FAR + 2);
  float* const fo = reinterpret_cast<float*>(FAR + 4);
  const int64_t B = 2, L = 10, S = 200;  // few queries: the attention has a workspace
  for (const msgla_heads* x : bad) {
    auto at = [&](int i, int k) { return i == k ? x : &h; };
    EXPECT(msgla_block_means(&good, x, 0, 0, B, S, F, 0) == MSGLA_ERR_INVALID_ARG);
    EXPECT(msgla_block_select(&good, x, F, 0, 0, B, L, S, I, 0) == MSGLA_ERR_INVALID_ARG);
    for (int k = 0; k < 4; ++k)
      EXPECT(msgla_block_attention(&good, at(0, k), at(1, k), at(2, k), I, 0, 0, B, L, S, at(3, k), F, FAR, BAD, 0) ==
             MSGLA_ERR_INVALID_ARG);
    for (int k = 0; k < 8; ++k)
      EXPECT(msgla_block_attention_backward(&good, at(0, k), at(1, k), at(2, k), I, 0, 0, at(3, k), F, at(4, k), B, L, S, at(5, k),
                                            at(6, k), at(7, k), FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
    for (int k = 0; k < 6; ++k)
      if (x != &st || k >= 4)  // stride_t of the four _t tensors is not read
        EXPECT(msgla_block_attention_step(&good, at(0, k), at(1, k), at(2, k), I, B, S, at(4, k), at(5, k), F, at(3, k), FAR, BAD,
                                          0) == MSGLA_ERR_INVALID_ARG);
  }
  EXPECT(msgla_block_means(&good, &h, 0, 0, B, S, nullptr, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_means(&good, &h, io, 0, B, S, F, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_means(&good, &h, 0, io, B, S, F, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_select(&good, &h, fo, 0, 0, B, L, S, I, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_select(&good, &h, F, 0, 0, B, L, S, nullptr, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_select(&good, &h, F, io, 0, B, L, S, I, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention(&good, &h, &h, &h, nullptr, 0, 0, B, L, S, &h, F, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention(&good, &h, &h, &h, I, 0, io, B, L, S, &h, F, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention(&good, &h, &h, &h, I, 0, 0, B, L, S, &h, F, nullptr, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention_backward(&good, &h, &h, &h, I, 0, 0, &h, nullptr, &h, B, L, S, &h, &h, &h, FAR, BAD, 0) ==
         MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention_backward(&good, &h, &h, &h, I, 0, 0, &h, F, &h, B, L, S, &h, &h, &h, nullptr, BAD, 0) ==
         MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention_step(&good, &h, &h, &h, nullptr, B, S, &h, &h, F, &h, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention_step(&good, &h, &h, &h, I, B, S, &h, &h, nullptr, &h, FAR, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  EXPECT(msgla_block_attention_step(&good, &h, &h, &h, I, B, S, &h, &h, F, &h, nullptr, BAD, 0) == MSGLA_ERR_INVALID_ARG);
  return n;
}

int main() {
  const long r = recurrence(), b = blocks();
  std::printf("%ld recurrence sizes, %ld block sizes, failures %d\n", r, b, failures);
  return failures ? 1 : 0;
}
