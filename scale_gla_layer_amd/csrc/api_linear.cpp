// Host side of linear attention with a decay per head: argument checks, the
// segments, the workspace, and the gradients as walks.
#include "api_internal.hpp"
#include "linear.hpp"

using namespace msgla;
using namespace msgla::host;

namespace {

constexpr size_t BAD = (size_t)-1;
constexpr int N_CU = 256;

bool lin_config_ok(const msgla_linear_config* c) {
  return c && (c->dtype == MSGLA_F32 || c->dtype == MSGLA_BF16) && c->heads >= 1 && c->heads <= 1024 && c->d_k >= 8 &&
         c->d_k <= 256 && c->d_k % 8 == 0 && c->d_v >= 8 && c->d_v <= 256 && c->d_v % 8 == 0 && c->scale >= 1.0e-30f &&
         c->scale <= 1.0e30f;
}
bool lin_sizes_ok(int64_t B, int64_t L) {
  return B >= 1 && L >= 1 && B <= (1 << 20) && L <= (1 << 24) && B * L <= ((int64_t)1 << 28);
}
bool heads_ok(const msgla_heads* t, int es) {
  auto stride = [es](int64_t s) { return s >= 0 && s * es % 16 == 0; };
  return t && t->data && aligned16(t->data) && stride(t->stride_b) && stride(t->stride_t) && stride(t->stride_h);
}
bool heads_t_ok(const msgla_heads* t, int es) {  // the step's tensors of one position: stride_t is not read
  if (!t) return false;
  msgla_heads u = *t;
  u.stride_t = 0;
  return heads_ok(&u, es);
}
bool i32_ok(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
LinHeads heads_of(const msgla_heads* t, int es) {
  return LinHeads{static_cast<char*>(t->data), t->stride_b * es, t->stride_t * es, t->stride_h * es};
}
int es_of(const msgla_linear_config* c) { return c->dtype == MSGLA_BF16 ? 2 : 4; }

// Segments of a sequence, of at least four chunks: no more than fill the CUs once with
// the walks of jobs of this one's shape, which share a launch.
void set_segments(LinParams& P, int es) {
  const int chunks = cdiv(P.L, LIN_CHUNK);
  for (int i = 0; i < P.jobs; ++i) {
    LinJob& J = P.job[i];
    int64_t walks = 0;
    for (int j = 0; j < P.jobs; ++j)
      if (lin_kwp(P.job[j].kw) == lin_kwp(J.kw) && P.job[j].columns == J.columns) walks += (int64_t)P.B * P.H * P.job[j].slices;
    const bool share = es == 2 && lin_state_waves(es, lin_kwp(J.kw), J.columns) == 4;
    const int n = (int)std::max<int64_t>(1, std::min<int64_t>({(share ? 2 * N_CU : N_CU) / walks, (int64_t)LIN_SEGMENTS, (int64_t)chunks / 4}));
    J.seg_chunks = cdiv(chunks, n);
    J.segments = cdiv(chunks, J.seg_chunks);
  }
}

LinParams lin_params(const msgla_linear_config* c, int64_t B, int64_t L, bool gradient) {
  LinParams P{};
  P.B = (int)B;
  P.L = (int)L;
  P.H = c->heads;
  P.scale = c->scale;
  P.jobs = gradient ? 3 : 1;
  for (int i = 0; i < P.jobs; ++i) {  // forward; or dq, dk, dv
    LinJob& J = P.job[i];
    J.kw = gradient && i < 2 ? c->d_v : c->d_k;
    J.vw = gradient && i < 2 ? c->d_k : c->d_v;
    J.turned = gradient && i > 0;
    J.flip_entry = gradient && i < 2;
    J.entry_mul = gradient && i > 0 ? 1.f / c->scale : 1.f;
    J.exit_mul = gradient ? c->scale : 1.f;
  }
  for (int i = 0; i < P.jobs; ++i) {
    LinJob& J = P.job[i];
    int64_t walks = 0;  // of 128 columns, in a launch of their own
    for (int j = 0; j < P.jobs; ++j)
      if (lin_kwp(P.job[j].kw) == lin_kwp(J.kw) && P.job[j].vw > 64) walks += B * c->heads * cdiv(P.job[j].vw, 128);
    J.columns = lin_columns(es_of(c), lin_kwp(J.kw), J.vw, walks, walks * cdiv(P.L, LIN_CHUNK));
    J.slices = cdiv(J.vw, J.columns);
  }
  set_segments(P, es_of(c));
  return P;
}

// The states before the segments: their size, and with a workspace their places.
size_t lin_room(LinParams& P, void* ws) {
  size_t cur = 0;
  for (int i = 0; i < P.jobs; ++i) {
    LinJob& J = P.job[i];
    if (J.segments == 1) continue;
    if (ws) J.part = at<float>(ws, cur);
    cur += align256((size_t)P.B * P.H * J.segments * J.kw * J.vw * 4);
  }
  return cur;
}

bool lin_grid_ok(const LinParams& P) {
  int64_t most = 0;
  for (int i = 0; i < P.jobs; ++i) most = std::max(most, (int64_t)P.B * P.H * P.job[i].segments * P.job[i].slices);
  return launch_ok((most + N_XCD) * P.jobs, 768) && launch_ok((int64_t)P.B * P.H * 64, 256);
}

size_t lin_room_bytes(const msgla_linear_config* cfg, int64_t B, int64_t L, bool gradient) {
  if (!lin_config_ok(cfg) || !lin_sizes_ok(B, L)) return BAD;
  LinParams P = lin_params(cfg, B, L, gradient);
  return lin_room(P, nullptr);
}

}  // namespace

extern "C" {

size_t msgla_linear_attention_workspace_bytes(const msgla_linear_config* cfg, int64_t B, int64_t L) {
  return lin_room_bytes(cfg, B, L, false);
}

size_t msgla_linear_attention_backward_workspace_bytes(const msgla_linear_config* cfg, int64_t B, int64_t L) {
  return lin_room_bytes(cfg, B, L, true);
}

msgla_status msgla_linear_attention_forward(const msgla_linear_config* cfg, const msgla_heads* q, const msgla_heads* k,
                                            const msgla_heads* v, const float* log_decay, const int32_t* lens,
                                            const float* state_in, int64_t B, int64_t L, const msgla_heads* out,
                                            float* state_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!lin_config_ok(cfg) || !lin_sizes_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !heads_ok(k, es) || !heads_ok(v, es) || !heads_ok(out, es) || !log_decay || !i32_ok(log_decay) ||
      !i32_ok(lens) || !aligned16(state_in) || !aligned16(state_out))
    return MSGLA_ERR_INVALID_ARG;
  LinParams P = lin_params(cfg, B, L, false);
  LinJob& J = P.job[0];
  J.q = heads_of(q, es);
  J.k = heads_of(k, es);
  J.v = heads_of(v, es);
  J.o = heads_of(out, es);
  J.entry = state_in;
  J.exit = state_out;
  P.log_decay = log_decay;
  P.lens = lens;
  if (!lin_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  const size_t room = msgla_linear_attention_workspace_bytes(cfg, B, L);
  if (room && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < room) return MSGLA_ERR_WORKSPACE;
  lin_room(P, workspace);
  HIP_TRY(launch_linear(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_linear_attention_backward(const msgla_linear_config* cfg, const msgla_heads* q, const msgla_heads* k,
                                             const msgla_heads* v, const float* log_decay, const int32_t* lens,
                                             const float* state_in, const msgla_heads* dout, const float* dstate_out,
                                             int64_t B, int64_t L, const msgla_heads* dq, const msgla_heads* dk,
                                             const msgla_heads* dv, float* dstate_in, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  if (!lin_config_ok(cfg) || !lin_sizes_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !heads_ok(k, es) || !heads_ok(v, es) || !heads_ok(dout, es) || !heads_ok(dq, es) ||
      !heads_ok(dk, es) || !heads_ok(dv, es) || !log_decay || !i32_ok(log_decay) || !i32_ok(lens) ||
      !aligned16(state_in) || !aligned16(dstate_out) || !aligned16(dstate_in))
    return MSGLA_ERR_INVALID_ARG;
  LinParams P = lin_params(cfg, B, L, true);
  const msgla_heads* in[3][3] = {{dout, v, k}, {v, dout, q}, {k, q, dout}};
  const msgla_heads* grad[3] = {dq, dk, dv};
  for (int i = 0; i < 3; ++i) {
    LinJob& J = P.job[i];
    J.q = heads_of(in[i][0], es);
    J.k = heads_of(in[i][1], es);
    J.v = heads_of(in[i][2], es);
    J.o = heads_of(grad[i], es);
    J.entry = i == 0 ? state_in : dstate_out;
    J.exit = i == 2 ? dstate_in : nullptr;
  }
  P.log_decay = log_decay;
  P.lens = lens;
  if (!lin_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  const size_t room = msgla_linear_attention_backward_workspace_bytes(cfg, B, L);
  if (room && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < room) return MSGLA_ERR_WORKSPACE;
  lin_room(P, workspace);
  HIP_TRY(launch_linear(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_linear_attention_step(const msgla_linear_config* cfg, const msgla_heads* q_t, const msgla_heads* k_t,
                                         const msgla_heads* v_t, const float* log_decay, const uint8_t* mask,
                                         const float* state_in, int64_t B, const msgla_heads* out_t, float* state_out,
                                         void* stream) {
  if (!lin_config_ok(cfg) || !lin_sizes_ok(B, 1)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_t_ok(q_t, es) || !heads_t_ok(k_t, es) || !heads_t_ok(v_t, es) || !heads_t_ok(out_t, es) || !log_decay ||
      !i32_ok(log_decay) || !state_in || !state_out || !aligned16(state_in) || !aligned16(state_out))
    return MSGLA_ERR_INVALID_ARG;
  LinParams P = lin_params(cfg, B, 1, false);
  LinJob& J = P.job[0];
  J.q = heads_of(q_t, es);
  J.k = heads_of(k_t, es);
  J.v = heads_of(v_t, es);
  J.o = heads_of(out_t, es);
  J.entry = state_in;
  J.exit = state_out;
  J.slices = cdiv(cfg->d_v, LIN_STEP_COLUMNS);
  P.log_decay = log_decay;
  P.mask = mask;
  if (!launch_ok((int64_t)P.B * P.H * J.slices, LIN_STEP_THREADS)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_linear_step(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

}  // extern "C"
