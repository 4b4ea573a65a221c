// Host side of the sliding-window attention: argument checks, the tiles, and the
// workspace layouts.
#include "api_internal.hpp"
#include "window.hpp"

using namespace msgla;
using namespace msgla::host;

namespace {

constexpr size_t BAD = (size_t)-1;
constexpr int N_CU = 256;

bool win_config_ok(const msgla_window_config* c) {
  if (!c || (c->dtype != MSGLA_F32 && c->dtype != MSGLA_BF16)) return false;
  if (c->heads_kv < 1 || c->heads_q < c->heads_kv || c->heads_q > 1024 || c->heads_q % c->heads_kv) return false;
  if (c->d_k < 8 || c->d_k > 128 || c->d_k % 8 || c->d_v < 8 || c->d_v > 256 || c->d_v % 8) return false;
  if (c->window < 1 || c->window > (1 << 24) || c->n_sink < 0 || c->n_sink > 1024) return false;
  return c->scale >= 1.0e-30f && c->scale <= 1.0e30f;
}
bool win_sizes_ok(int64_t B, int64_t L, int64_t S) {
  return B >= 1 && L >= 1 && S >= 1 && B <= (1 << 20) && L <= (1 << 24) && S <= (1 << 24) &&
         B * L <= ((int64_t)1 << 28);
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
WinHeads heads_of(const msgla_heads* t, int es) {
  return WinHeads{static_cast<char*>(t->data), t->stride_b * es, t->stride_t * es, t->stride_h * es};
}
int es_of(const msgla_window_config* c) { return c->dtype == MSGLA_BF16 ? 2 : 4; }

void set_tiles(WinParams& P, int rows) {
  P.tile_rows = rows;
  P.QT = P.G <= rows ? rows / P.G : 1;
  P.GT = P.G <= rows ? 1 : cdiv(P.G, rows);
  P.tiles_per_seq = P.GT > 1 ? P.L * P.GT : cdiv(P.L, P.QT);
  P.tiles = (int64_t)P.B * P.Hkv * P.tiles_per_seq;
}
// tiles of the workgroups of k_window
void set_many(WinParams& P) { set_tiles(P, WIN_ROWS * WIN_TILES); }
int pairs_of(const WinParams& P, int es) { return win_pairs(es, win_dvp(P.dvw)); }

WinParams win_params(const msgla_window_config* c, int64_t B, int64_t L, int64_t S) {
  WinParams P{};
  P.B = (int)B;
  P.L = (int)L;
  P.S = (int)S;
  P.Hq = c->heads_q;
  P.Hkv = c->heads_kv;
  P.G = c->heads_q / c->heads_kv;
  P.dkw = c->d_k;
  P.dvw = c->d_v;
  P.window = c->window;
  P.n_sink = c->n_sink;
  P.scale = c->scale;
  return P;
}

struct Take {
  size_t cur = 0;
  size_t operator()(size_t bytes) {
    const size_t o = cur;
    cur += align256(bytes);
    return o;
  }
};

// Few rows: tiles of 16, their keys dealt to as many workgroups as there are CUs, each
// wave a unit of 32 keys at least (a step of 16 sequences with 16 / 4 heads of 128 and
// a window of 4096: 31 us; with twice as many workgroups 33, with four times 38).
struct FewWs {
  size_t po, pm, total;
};
FewWs set_few(WinParams& P) {
  set_tiles(P, WIN_FEW_ROWS);
  const int64_t keys = std::min<int64_t>(P.S, (int64_t)P.window + P.n_sink + P.QT);
  const int64_t units = (keys + WIN_FEW_KEYS - 1) / WIN_FEW_KEYS + 1;
  P.parts = (int)std::max<int64_t>(1, std::min<int64_t>((units + WIN_FEW_WAVES - 1) / WIN_FEW_WAVES, N_CU / P.tiles));
  FewWs w{};
  Take take;
  if (P.parts > 1) {
    w.po = take((size_t)P.tiles * P.parts * WIN_FEW_ROWS * win_dvp(P.dvw) * 4);
    w.pm = take((size_t)P.tiles * P.parts * WIN_FEW_ROWS * 8);
  }
  w.total = take.cur;
  return w;
}
void place_few(WinParams& P, const FewWs& w, void* ws) {
  if (P.parts > 1) {
    P.po = at<float>(ws, w.po);
    P.pm = at<float>(ws, w.pm);
  }
}
bool few_grid_ok(const WinParams& P) {
  return launch_ok(P.tiles * P.parts, 64 * WIN_FEW_WAVES) && launch_ok(P.tiles * WIN_FEW_ROWS, 64) &&
         P.tiles <= INT32_MAX;
}
bool many_grid_ok(const WinParams& P) { return launch_ok(P.tiles + N_XCD, 4 * P.tile_rows); }

// Whether the forward deals keys to workgroups: where the tiles of many rows give work
// to a quarter of the CUs at most (16 / 4 heads of 128, window 512, bf16: 64 tiles take
// 17.4 us dealt and 19.2 whole, 128 tiles 35 and 24; 8 heads of fp32: 32 tiles 26 and
// 74, 64 tiles 50 and 75, 144 tiles of 6 / 2 heads 43 and 34).
bool use_few(WinParams P) {
  set_many(P);
  return P.tiles <= N_CU / 4;
}

struct GradWs {
  size_t delta, nref, part, sink_part, total;
};
GradWs set_grad(WinParams& P, int es) {
  P.key_tile = 32 * pairs_of(P, es);
  set_tiles(P, WIN_ROWS * pairs_of(P, es));
  const int64_t heads = (int64_t)P.B * P.Hkv;
  P.key_tiles = cdiv(P.S, P.key_tile);
  const int64_t queries = std::min<int64_t>(P.L, (int64_t)P.window + P.key_tile - 1);
  const int64_t sets = (queries * P.G + 31) / 32;
  // Workgroups fill a CU each: as many as there are CUs, of four sets of 32 rows at least (fp32, 3 x 6 / 2 heads of
  // 999: 47 us, with two sets 66, with eight 84).
  P.key_parts = (int)std::max<int64_t>(1, std::min<int64_t>((N_CU - 1 + heads * P.key_tiles) / (heads * P.key_tiles), sets / 4));
  const int sinks = std::min(P.n_sink, P.S);
  P.sink_tiles = P.S > P.window ? cdiv(sinks, WIN_SINK) : 0;
  if (P.sink_tiles > 0) {
    // two workgroups a CU, of two sets at least (2 x 16 / 4 heads of 4096 positions: 22 us, with four a CU of four
    // sets 28; fp32, 3 x 6 / 2 heads of 999: 25 and 32)
    const int64_t rows = (int64_t)std::min(P.L, P.S - P.window) * P.G;
    P.sink_parts = (int)std::max<int64_t>(1, std::min<int64_t>((2 * N_CU - 1 + heads * P.sink_tiles) / (heads * P.sink_tiles), rows / 64));
  }
  P.joined = P.key_parts > 1 ? P.key_tiles : P.sink_tiles > 0 ? cdiv(sinks, P.key_tile) : 0;
  const size_t width = (size_t)(win_dkp(P.dkw) + win_dvp(P.dvw)) * 4;
  GradWs w{};
  Take take;
  w.delta = take((size_t)P.B * P.Hq * P.L * 4);
  w.nref = take((size_t)P.B * P.Hq * P.L * 4);
  w.part = take((size_t)heads * P.joined * P.key_parts * P.key_tile * width);
  w.sink_part = take((size_t)heads * P.sink_tiles * P.sink_parts * WIN_SINK * width);
  w.total = take.cur;
  return w;
}
bool grad_grid_ok(const WinParams& P) {
  const int64_t heads = (int64_t)P.B * P.Hkv;
  return many_grid_ok(P) && launch_ok(heads * P.key_tiles * P.key_parts + N_XCD, 4 * P.key_tile) &&
         launch_ok(heads * P.sink_tiles * P.sink_parts + N_XCD, 128) && launch_ok(heads * P.joined * P.key_tile, 256);
}

}  // namespace

extern "C" {

size_t msgla_window_attention_workspace_bytes(const msgla_window_config* cfg, int64_t B, int64_t L, int64_t S) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, L, S)) return BAD;
  WinParams P = win_params(cfg, B, L, S);
  return use_few(P) ? set_few(P).total : 0;
}

size_t msgla_window_attention_backward_workspace_bytes(const msgla_window_config* cfg, int64_t B, int64_t L, int64_t S) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, L, S)) return BAD;
  WinParams P = win_params(cfg, B, L, S);
  return set_grad(P, es_of(cfg)).total;
}

size_t msgla_window_attention_step_workspace_bytes(const msgla_window_config* cfg, int64_t B, int64_t S) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, 1, S)) return BAD;
  WinParams P = win_params(cfg, B, 1, S);
  return set_few(P).total;
}

msgla_status msgla_window_attention(const msgla_window_config* cfg, const msgla_heads* q, const msgla_heads* k,
                                    const msgla_heads* v, const int32_t* start, const int32_t* lens, int64_t B,
                                    int64_t L, int64_t S, const msgla_heads* out, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !heads_ok(k, es) || !heads_ok(v, es) || !heads_ok(out, es) || !i32_ok(start) || !i32_ok(lens) ||
      !i32_ok(lse))
    return MSGLA_ERR_INVALID_ARG;
  WinParams P = win_params(cfg, B, L, S);
  P.q = heads_of(q, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out, es);
  P.start = start;
  P.lens = lens;
  P.lse = lse;
  const bool few = use_few(P);
  if (few) {
    const FewWs w = set_few(P);
    if (!few_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
    if (w.total && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
    if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
    place_few(P, w, workspace);
    HIP_TRY(launch_window_few(P, false, es == 2, static_cast<hipStream_t>(stream)));
    return MSGLA_OK;
  }
  set_many(P);
  if (!many_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_window(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_window_attention_backward(const msgla_window_config* cfg, const msgla_heads* q, const msgla_heads* k,
                                             const msgla_heads* v, const int32_t* start, const int32_t* lens,
                                             const msgla_heads* out, const float* lse, const msgla_heads* dout,
                                             int64_t B, int64_t L, int64_t S, const msgla_heads* dq,
                                             const msgla_heads* dk, const msgla_heads* dv, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !heads_ok(k, es) || !heads_ok(v, es) || !heads_ok(out, es) || !heads_ok(dout, es) ||
      !heads_ok(dq, es) || !heads_ok(dk, es) || !heads_ok(dv, es) || !i32_ok(start) || !i32_ok(lens) || !lse || !i32_ok(lse))
    return MSGLA_ERR_INVALID_ARG;
  WinParams P = win_params(cfg, B, L, S);
  const GradWs w = set_grad(P, es_of(cfg));
  if (!grad_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace)) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  P.q = heads_of(q, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out, es);
  P.dout = heads_of(dout, es);
  P.dq = heads_of(dq, es);
  P.dk = heads_of(dk, es);
  P.dv = heads_of(dv, es);
  P.start = start;
  P.lens = lens;
  P.lse_in = lse;
  P.delta = at<float>(workspace, w.delta);
  P.nref = at<float>(workspace, w.nref);
  P.part = at<float>(workspace, w.part);
  P.sink_part = at<float>(workspace, w.sink_part);
  HIP_TRY(launch_window_dq(P, es == 2, static_cast<hipStream_t>(stream)));
  HIP_TRY(launch_window_dkdv(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_window_attention_append(const msgla_window_config* cfg, const msgla_heads* k_new,
                                           const msgla_heads* v_new, const int32_t* pos, const int32_t* lens,
                                           int64_t B, int64_t L, int64_t S, const msgla_heads* k, const msgla_heads* v,
                                           void* stream) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(k_new, es) || !heads_ok(v_new, es) || !heads_ok(k, es) || !heads_ok(v, es) || !i32_ok(pos) || !i32_ok(lens))
    return MSGLA_ERR_INVALID_ARG;
  WinParams P = win_params(cfg, B, L, S);
  P.kt = heads_of(k_new, es);
  P.vt = heads_of(v_new, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.pos = pos;
  P.lens = lens;
  if (!launch_ok((B * L + 3) / 4 * P.Hkv, 256)) return MSGLA_ERR_UNSUPPORTED;
  HIP_TRY(launch_window_append(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_window_attention_step(const msgla_window_config* cfg, const msgla_heads* q_t, const msgla_heads* k_t,
                                         const msgla_heads* v_t, const int32_t* pos, int64_t B, int64_t S,
                                         const msgla_heads* k, const msgla_heads* v, const msgla_heads* out_t,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!win_config_ok(cfg) || !win_sizes_ok(B, 1, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_t_ok(q_t, es) || !heads_t_ok(k_t, es) || !heads_t_ok(v_t, es) || !heads_t_ok(out_t, es) || !heads_ok(k, es) ||
      !heads_ok(v, es) || !pos || !i32_ok(pos))
    return MSGLA_ERR_INVALID_ARG;
  WinParams P = win_params(cfg, B, 1, S);
  const FewWs w = set_few(P);
  if (!few_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  if (w.total && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  P.q = heads_of(q_t, es);
  P.kt = heads_of(k_t, es);
  P.vt = heads_of(v_t, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out_t, es);
  P.pos = pos;
  place_few(P, w, workspace);
  HIP_TRY(launch_window_few(P, true, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

}  // extern "C"
