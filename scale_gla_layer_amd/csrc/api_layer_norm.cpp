// Host side of the layer norm: argument checks and the backward's workspace.
#include "api_internal.hpp"
#include "layer_norm.hpp"

using namespace msgla;
using namespace msgla::host;

namespace {

constexpr size_t BAD = (size_t)-1;

bool ln_config_ok(const msgla_layer_norm_config* c) {
  return c && c->width >= 1 && c->width <= LN_MAX_WIDTH && (c->dtype == MSGLA_F32 || c->dtype == MSGLA_BF16) &&
         c->eps >= 1e-20f && c->eps <= 1.f;
}
bool ln_batch_ok(int64_t B, int64_t L) {
  return B >= 1 && L >= 1 && B <= (1 << 20) && L <= (1 << 24) && B * L <= ((int64_t)1 << 28);
}
bool rows_ok(const msgla_rows* r, int es) {
  return r && r->data && reinterpret_cast<uintptr_t>(r->data) % es == 0 && r->stride_b >= 0 && r->stride_t >= 0;
}
bool f32_ok(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
LnRows rows_of(const msgla_rows* r, int es) {
  return LnRows{static_cast<char*>(r->data), r->stride_b * es, r->stride_t * es};
}
int es_of(const msgla_layer_norm_config* c) { return c->dtype == MSGLA_BF16 ? 2 : 4; }

int64_t row_bytes(const msgla_layer_norm_config* c) { return (int64_t)c->width * es_of(c); }

size_t ln_room(const msgla_layer_norm_config* c, int64_t B, int64_t L) {
  return align256((size_t)ln_parts(B * L, row_bytes(c), es_of(c)) * 2 * c->width * 4);
}

}  // namespace

extern "C" {

size_t msgla_layer_norm_backward_workspace_bytes(const msgla_layer_norm_config* cfg, int64_t B, int64_t L) {
  return ln_config_ok(cfg) && ln_batch_ok(B, L) ? ln_room(cfg, B, L) : BAD;
}

msgla_status msgla_layer_norm_forward(const msgla_layer_norm_config* cfg, const msgla_rows* x, const float* weight,
                                      const float* bias, int64_t B, int64_t L, const msgla_rows* y, float* mean,
                                      float* rstd, void* stream) {
  if (!ln_config_ok(cfg) || !ln_batch_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!rows_ok(x, es) || !rows_ok(y, es) || !f32_ok(weight) || !f32_ok(bias) || !f32_ok(mean) || !f32_ok(rstd))
    return MSGLA_ERR_INVALID_ARG;
  LnParams P{};
  P.x = rows_of(x, es);
  P.y = rows_of(y, es);
  P.weight = weight;
  P.bias = bias;
  P.mean = mean;
  P.rstd = rstd;
  P.rows = B * L;
  P.L = (int)L;
  P.D = cfg->width;
  P.eps = cfg->eps;
  HIP_TRY(launch_layer_norm(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_layer_norm_backward(const msgla_layer_norm_config* cfg, const msgla_rows* x, const msgla_rows* dy,
                                       const float* weight, const float* mean, const float* rstd, int64_t B, int64_t L,
                                       const msgla_rows* dx, float* dweight, float* dbias, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!ln_config_ok(cfg) || !ln_batch_ok(B, L)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!rows_ok(x, es) || !rows_ok(dy, es) || !rows_ok(dx, es) || !mean || !rstd || !f32_ok(weight) || !f32_ok(mean) ||
      !f32_ok(rstd) || !f32_ok(dweight) || !f32_ok(dbias))
    return MSGLA_ERR_INVALID_ARG;
  if (dweight || dbias) {
    if (!workspace || !aligned16(workspace)) return MSGLA_ERR_INVALID_ARG;
    if (workspace_bytes < ln_room(cfg, B, L)) return MSGLA_ERR_WORKSPACE;
  }
  LnParams P{};
  P.x = rows_of(x, es);
  P.dy = rows_of(dy, es);
  P.dx = rows_of(dx, es);
  P.weight = weight;
  P.mean_in = mean;
  P.rstd_in = rstd;
  P.dweight = dweight;
  P.dbias = dbias;
  P.part = static_cast<float*>(workspace);
  P.rows = B * L;
  P.L = (int)L;
  P.D = cfg->width;
  P.eps = cfg->eps;
  P.parts = ln_parts(P.rows, row_bytes(cfg), es);
  HIP_TRY(launch_layer_norm_backward(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

}  // extern "C"
