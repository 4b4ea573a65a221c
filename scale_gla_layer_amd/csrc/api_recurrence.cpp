// Host side of the gated linear recurrence: argument checks, the workspace
// layout, and the choice between the vector and the element path.
#include "api_internal.hpp"
#include "recurrence.hpp"

using namespace msgla;
using namespace msgla::host;

namespace {

constexpr size_t BAD = (size_t)-1;

bool rec_config_ok(const msgla_recurrence_config* c) {
  return c && c->width >= 1 && c->width <= 65536 && c->input >= 0 && c->input <= 2 &&
         (c->dtype == MSGLA_F32 || c->dtype == MSGLA_BF16) && c->gate_normalizer >= 1e-6f &&
         c->gate_normalizer <= 1e6f;
}

bool rec_batch_ok(int64_t B, int64_t L) {
  return B >= 1 && L >= 1 && B <= (1 << 20) && L <= (1 << 24) && B * L <= ((int64_t)1 << 28);
}

struct RecWs {
  size_t words, counters, entry, dbp, total;
  int nch, groups, nchb, groupsb;
  int64_t row;      // channels of a batch
  int64_t n_words;  // words of all chunks and groups
};

RecWs rec_ws(const msgla_recurrence_config* c, int64_t B, int64_t L, bool backward) {
  RecWs w{};
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur += align256(bytes);
    return o;
  };
  w.nch = (int)((L + REC_CHUNK - 1) / REC_CHUNK);
  w.groups = cdiv(w.nch, REC_GROUP);
  w.nchb = backward ? (int)((L + REC_BCHUNK - 1) / REC_BCHUNK) : 0;
  w.groupsb = cdiv(w.nchb, REC_GROUP);
  const int64_t row = w.row = B * (int64_t)c->width;
  w.n_words = (row * ((int64_t)w.nch + w.groups + w.nchb + w.groupsb) + 1) / 2 * 2;  // an even number is cleared
  if (w.nch > 1 || w.nchb > 1) {
    w.words = take((size_t)w.n_words * 8);
    w.counters = take((size_t)B * cdiv(c->width, 64) * 8);
  }
  if (w.nchb > 1) w.entry = take((size_t)row * w.nchb * 4);
  if (backward) w.dbp = take((size_t)row * w.nchb * 4);
  w.total = cur;
  return w;
}

void set_ws(RecParams& P, const RecWs& w, void* ws) {
  P.nch = w.nch;
  P.groups = w.groups;
  P.nchb = w.nchb;
  P.groupsb = w.groupsb;
  if (w.nch > 1 || w.nchb > 1) {
    P.maps = at<uint64_t>(ws, w.words);
    P.ends = P.maps + w.row * w.nch;
    P.rmaps = P.ends + w.row * w.groups;
    P.rends = P.rmaps + w.row * w.nchb;
    P.words = w.n_words;
    P.counters = at<uint32_t>(ws, w.counters);
  }
  if (w.nchb > 1) P.entry = at<float>(ws, w.entry);
  if (w.nchb > 0) P.dbp = at<float>(ws, w.dbp);
}

bool rows_ok(const msgla_rows* r, int es) {
  return r && r->data && reinterpret_cast<uintptr_t>(r->data) % es == 0 && r->stride_b >= 0 && r->stride_t >= 0;
}

bool f32_ok(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

RecRows rows_of(const msgla_rows* r) { return r ? RecRows{r->data, r->stride_b, r->stride_t} : RecRows{}; }

// Whether every row starts at an even element (loads of 4 or 8 bytes).
bool rows_vec(const msgla_rows* r, int es) {
  return !r || !r->data || (reinterpret_cast<uintptr_t>(r->data) % (2 * es) == 0 && r->stride_b % 2 == 0 && r->stride_t % 2 == 0);
}

bool f32_vec(const void* p) { return reinterpret_cast<uintptr_t>(p) % 8 == 0; }

// One workgroup takes 64 lanes' channels, and a chunk or (the step) a position.
bool forward_grid_ok(const RecParams& P) {
  return launch_ok((int64_t)P.slabs * P.nch * P.B, 64 * REC_WAVES) && launch_ok((P.words / 2 + 255) / 256, 256);
}
bool backward_grid_ok(const RecParams& P) {
  return (P.nchb == 1 || forward_grid_ok(P)) && launch_ok((int64_t)P.slabs * P.nchb * P.B, 64 * REC_BWAVES);
}
bool step_grid_ok(const RecParams& P) { return launch_ok((int64_t)P.slabs * P.B, 64); }

}  // namespace

extern "C" {

size_t msgla_recurrence_workspace_bytes(const msgla_recurrence_config* cfg, int64_t B, int64_t L) {
  return rec_config_ok(cfg) && rec_batch_ok(B, L) ? rec_ws(cfg, B, L, false).total : BAD;
}

size_t msgla_recurrence_backward_workspace_bytes(const msgla_recurrence_config* cfg, int64_t B, int64_t L) {
  return rec_config_ok(cfg) && rec_batch_ok(B, L) ? rec_ws(cfg, B, L, true).total : BAD;
}

msgla_status msgla_recurrence_forward(const msgla_recurrence_config* cfg, const msgla_rows* x,
                                      const msgla_rows* z, const float* bias, const uint8_t* mask,
                                      const float* h_in, int64_t B, int64_t L, const msgla_rows* y,
                                      float* h_out, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (!rec_config_ok(cfg) || !rec_batch_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = cfg->dtype == MSGLA_BF16 ? 2 : 4;
  if (!rows_ok(x, es) || !rows_ok(z, es) || !rows_ok(y, es) || !f32_ok(bias) || !f32_ok(h_in) || !f32_ok(h_out))
    return MSGLA_ERR_INVALID_ARG;
  const RecWs w = rec_ws(cfg, B, L, false);
  if (w.total && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  const bool vec = cfg->width % 2 == 0 && rows_vec(x, es) && rows_vec(z, es) && rows_vec(y, es) &&
                   f32_vec(bias) && f32_vec(h_in) && f32_vec(h_out);
  RecParams P{};
  P.x = rows_of(x);
  P.z = rows_of(z);
  P.y = rows_of(y);
  P.bias = bias;
  P.mask = mask;
  P.h_in = h_in;
  P.h_out = h_out;
  P.B = (int)B;
  P.L = (int)L;
  P.D = cfg->width;
  set_ws(P, w, workspace);
  P.slabs = cdiv(P.D, vec ? 128 : 64);
  P.inv_gamma = 1.0f / cfg->gate_normalizer;
  if (!forward_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_recurrence_forward(P, cfg->input, es == 2, vec, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_recurrence_backward(const msgla_recurrence_config* cfg, const msgla_rows* x,
                                       const msgla_rows* z, const float* bias, const uint8_t* mask,
                                       const float* h_in, const msgla_rows* dy, const float* dh_out,
                                       int64_t B, int64_t L, const msgla_rows* dx,
                                       const msgla_rows* dz, float* dbias, float* dh_in,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!rec_config_ok(cfg) || !rec_batch_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = cfg->dtype == MSGLA_BF16 ? 2 : 4;
  if (!rows_ok(x, es) || !rows_ok(z, es) || (dy && !rows_ok(dy, es)) || (!dy && !dh_out) || !rows_ok(dx, es) ||
      !rows_ok(dz, es) || !f32_ok(bias) || !f32_ok(h_in) || !f32_ok(dh_out) || !f32_ok(dbias) || !f32_ok(dh_in))
    return MSGLA_ERR_INVALID_ARG;
  const RecWs w = rec_ws(cfg, B, L, true);
  if (!workspace || !aligned16(workspace)) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  const bool vec = cfg->width % 2 == 0 && rows_vec(x, es) && rows_vec(z, es) && rows_vec(dy, es) &&
                   rows_vec(dx, es) && rows_vec(dz, es) && f32_vec(bias) && f32_vec(h_in) && f32_vec(dh_out) &&
                   f32_vec(dbias) && f32_vec(dh_in);
  RecParams P{};
  P.x = rows_of(x);
  P.z = rows_of(z);
  P.dy = rows_of(dy);
  P.dx = rows_of(dx);
  P.dz = rows_of(dz);
  P.bias = bias;
  P.mask = mask;
  P.h_in = h_in;
  P.dh_out = dh_out;
  P.dbias = dbias;
  P.dh_in = dh_in;
  set_ws(P, w, workspace);
  P.B = (int)B;
  P.L = (int)L;
  P.D = cfg->width;
  P.slabs = cdiv(P.D, vec ? 128 : 64);
  P.inv_gamma = 1.0f / cfg->gate_normalizer;
  if (!backward_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_recurrence_backward(P, cfg->input, es == 2, vec, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_recurrence_step(const msgla_recurrence_config* cfg, const msgla_rows* x_t,
                                   const msgla_rows* z_t, const float* bias, const uint8_t* mask,
                                   const float* h_in, int64_t B, const msgla_rows* y_t, float* h_out,
                                   void* stream) {
  if (!rec_config_ok(cfg) || !rec_batch_ok(B, 1)) return MSGLA_ERR_INVALID_ARG;
  const int es = cfg->dtype == MSGLA_BF16 ? 2 : 4;
  if (!rows_ok(x_t, es) || !rows_ok(z_t, es) || !rows_ok(y_t, es) || !h_in || !h_out || !f32_ok(bias) ||
      !f32_ok(h_in) || !f32_ok(h_out))
    return MSGLA_ERR_INVALID_ARG;
  auto row_vec = [&](const msgla_rows* r) {  // stride_t is not read
    return reinterpret_cast<uintptr_t>(r->data) % (2 * es) == 0 && r->stride_b % 2 == 0;
  };
  const bool vec = cfg->width % 2 == 0 && row_vec(x_t) && row_vec(z_t) && row_vec(y_t) && f32_vec(bias) &&
                   f32_vec(h_in) && f32_vec(h_out);
  RecParams P{};
  P.x = rows_of(x_t);
  P.z = rows_of(z_t);
  P.y = rows_of(y_t);
  P.bias = bias;
  P.mask = mask;
  P.h_in = h_in;
  P.h_out = h_out;
  P.B = (int)B;
  P.L = 1;
  P.D = cfg->width;
  P.nch = 1;
  P.slabs = cdiv(P.D, vec ? 128 : 64);
  P.inv_gamma = 1.0f / cfg->gate_normalizer;
  if (!step_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_recurrence_step(P, cfg->input, es == 2, vec, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

}  // extern "C"
