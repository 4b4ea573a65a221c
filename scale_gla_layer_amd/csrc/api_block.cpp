// Host side of the block selection and the attention over selected blocks:
// argument checks, the tiles, and the workspace layouts.
#include "api_internal.hpp"
#include "block.hpp"

using namespace msgla;
using namespace msgla::host;

namespace {

constexpr size_t BAD = (size_t)-1;

bool blk_config_ok(const msgla_block_config* c) {
  if (!c || (c->dtype != MSGLA_F32 && c->dtype != MSGLA_BF16)) return false;
  if (c->heads_kv < 1 || c->heads_q < c->heads_kv || c->heads_q > 1024 || c->heads_q % c->heads_kv) return false;
  if (c->d_k < 8 || c->d_k > 128 || c->d_k % 8 || c->d_v < 8 || c->d_v > 256 || c->d_v % 8) return false;
  if (c->block != 32 && c->block != 64 && c->block != 128) return false;
  if (c->n_select < 1 || c->n_select > BLK_MAX_SEL || c->n_first < 0 || c->n_recent < 1) return false;
  if (c->n_first > c->n_select || c->n_recent > c->n_select - c->n_first) return false;
  return c->scale >= 1.0e-30f && c->scale <= 1.0e30f;
}

bool blk_sizes_ok(int64_t B, int64_t L, int64_t S) {
  return B >= 1 && L >= 1 && S >= 1 && B <= (1 << 20) && L <= (1 << 24) && S <= (1 << 24) &&
         B * L <= ((int64_t)1 << 28);
}

bool heads_ok(const msgla_heads* t, int es) {
  auto stride = [es](int64_t s) { return s >= 0 && s * es % 16 == 0; };
  return t && t->data && aligned16(t->data) && stride(t->stride_b) && stride(t->stride_t) && stride(t->stride_h);
}
// the step's tensors of one position: stride_t is not read
bool heads_t_ok(const msgla_heads* t, int es) {
  if (!t) return false;
  msgla_heads u = *t;
  u.stride_t = 0;
  return heads_ok(&u, es);
}
bool i32_ok(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

BlkHeads heads_of(const msgla_heads* t, int es) {
  return BlkHeads{static_cast<char*>(t->data), t->stride_b * es, t->stride_t * es, t->stride_h * es};
}

BlkParams blk_params(const msgla_block_config* c, int64_t B, int64_t L, int64_t S) {
  BlkParams P{};
  P.B = (int)B;
  P.L = (int)L;
  P.S = (int)S;
  P.Hq = c->heads_q;
  P.Hkv = c->heads_kv;
  P.G = c->heads_q / c->heads_kv;
  P.dkw = c->d_k;
  P.dvw = c->d_v;
  P.lgT = c->block == 32 ? 5 : c->block == 64 ? 6 : 7;
  P.n = c->n_select;
  P.n_first = c->n_first;
  P.n_recent = c->n_recent;
  P.nb = (int)((S + c->block - 1) / c->block);
  P.scale = c->scale;
  P.QT = P.G <= BLK_ROWS ? BLK_ROWS / P.G : 1;
  P.GT = P.G <= BLK_ROWS ? 1 : cdiv(P.G, BLK_ROWS);
  P.tiles_per_seq = P.GT > 1 ? P.L * P.GT : cdiv(P.L, P.QT);
  P.tiles = B * P.Hkv * (int64_t)P.tiles_per_seq;
  return P;
}

int es_of(const msgla_block_config* c) { return c->dtype == MSGLA_BF16 ? 2 : 4; }

// Tiles that share keys and values, in workgroups; or, for a few queries over long
// sequences, a tile a wave with its blocks dealt, 32 keys at a time, to as many
// waves (parts) as give about 4096, sixteen on a CU.  Calls of the forward of 16 / 4
// heads of 128, shared against dealt: 256 tiles 17 and 32 us, 64 (of 16 blocks at
// 8192 positions) 117 and 53, 128 118 and 90, with the gradient 176 and 152; 8 / 2
// heads of 128 in fp32: 256 tiles 54 and 57, with the gradient 141 and 131, 32 of
// 16 / 4 heads 469 and 70.  Single queries have nothing to share.
bool use_tiles(const BlkParams& P) { return P.L > 1 && P.tiles >= 128 && P.nb <= BLK_TILES_MAX; }
int parts_of(const BlkParams& P) {
  return use_tiles(P) || P.tiles >= 4096 ? 1 : std::min<int>(P.n << (P.lgT - 5), (int)(4096 / P.tiles));
}

struct Take {
  size_t cur = 0;
  size_t operator()(size_t bytes) {
    const size_t o = cur;
    cur += align256(bytes);
    return o;
  }
};

struct FwdWs {
  size_t po, pm, total;
  int parts;
};
FwdWs fwd_ws(const BlkParams& P, Take take = Take()) {
  FwdWs w{};
  w.parts = parts_of(P);
  if (w.parts > 1) {
    w.po = take((size_t)P.tiles * w.parts * BLK_ROWS * blk_dvp(P.dvw) * 4);
    w.pm = take((size_t)P.tiles * w.parts * BLK_ROWS * 8);
  }
  w.total = take.cur;
  return w;
}
void set_fwd(BlkParams& P, const FwdWs& w, void* ws) {
  P.parts = w.parts;
  if (w.parts > 1) {
    P.po = at<float>(ws, w.po);
    P.pm = at<float>(ws, w.pm);
  }
}

struct StepWs {
  size_t sel, key;
  FwdWs fwd;
};
StepWs step_ws(const BlkParams& P) {
  StepWs w{};
  Take take;
  w.sel = take((size_t)P.B * P.Hkv * P.n * 4);
  w.key = take(blk_step_spread(P) ? (size_t)P.B * P.Hkv * P.nb * 8 : 0);
  w.fwd = fwd_ws(P, take);
  return w;
}

struct BwdWs {
  size_t delta, bits, cnt, off, slot, list, items, n_items, part, po, pm, total;
  int parts, seg, W, max_items, max_parts;
};
BwdWs bwd_ws(const BlkParams& P) {
  BwdWs w{};
  Take take;
  const size_t bh = (size_t)P.B * P.Hkv;
  const int64_t pairs = (int64_t)P.L * std::min(P.n, P.nb);
  // about 1536 work items, of 128 to 2048 rows: fewer leave CUs idle, more write partial sums
  const int64_t even = (int64_t)P.B * P.Hkv * pairs / 1536;
  w.seg = (int)std::max<int64_t>(std::max(1, 128 / P.G), std::min<int64_t>(even, std::max(1, 2048 / P.G)));
  w.W = cdiv(P.L, 64);
  w.max_items = (int)(P.nb + pairs / w.seg);
  w.max_parts = (int)std::min<int64_t>(w.max_items, 2 * (pairs / w.seg));  // blocks of more than seg queries
  w.delta = take((size_t)P.B * P.Hq * P.L * 4);
  w.bits = take(bh * w.W * P.nb * 8);
  w.cnt = take(bh * P.nb * 4);
  w.off = take(bh * P.nb * 4);
  w.slot = take(bh * P.nb * 4);
  w.list = take(bh * P.L * P.n * 4);
  w.items = take(bh * w.max_items * 8);
  w.n_items = take(bh * 4);
  w.part = take(((bh * w.max_parts) << P.lgT) * (size_t)(blk_dkp(P.dkw) + blk_dvp(P.dvw)) * 4);
  w.parts = parts_of(P);
  if (w.parts > 1) {  // partial gradients of the queries
    w.po = take((size_t)P.tiles * w.parts * BLK_ROWS * 2 * blk_dkp(P.dkw) * 4);
    w.pm = take((size_t)P.tiles * w.parts * BLK_ROWS * 4);
  }
  w.total = take.cur;
  return w;
}

// The launches of an operator (the step's attention is the forward's).
bool means_grid_ok(const BlkParams& P) { return launch_ok((int64_t)P.B * P.Hkv * P.nb, 64); }
bool select_grid_ok(const BlkParams& P) { return launch_ok((int64_t)P.B * P.Hkv * cdiv(P.L, 16), 256); }
bool step_grid_ok(const BlkParams& P) { return launch_ok((int64_t)P.B * P.Hkv, 512); }
bool tiles_grid_ok(const BlkParams& P, int es, bool gradient, int parts) {
  if (!use_tiles(P)) return launch_ok(P.tiles * std::max(parts, parts > 1 ? BLK_ROWS : 1), 64);
  const TileShape s = tile_shape(es, blk_dkp(P.dkw), blk_dvp(P.dvw), gradient, 1 << P.lgT, P.tiles >= BLK_TILES_MANY);
  return launch_ok(tile_grid(s.tiles, P.tiles_per_seq, (int64_t)P.B * P.Hkv), 64 * (s.tiles + 1));
}
bool bwd_grid_ok(const BlkParams& P, const BwdWs& w) {
  const int64_t bh = (int64_t)P.B * P.Hkv;
  return launch_ok(bh * P.nb, 256) && launch_ok(bh * w.W, 256) &&
         launch_ok(bh * w.max_items << (P.lgT > 6 ? 1 : 0), P.lgT == 5 ? 128 : 256);
}

}  // namespace

extern "C" {

size_t msgla_block_attention_workspace_bytes(const msgla_block_config* cfg, int64_t B, int64_t L, int64_t S) {
  return blk_config_ok(cfg) && blk_sizes_ok(B, L, S) ? fwd_ws(blk_params(cfg, B, L, S)).total : BAD;
}

size_t msgla_block_attention_backward_workspace_bytes(const msgla_block_config* cfg, int64_t B, int64_t L,
                                                      int64_t S) {
  return blk_config_ok(cfg) && blk_sizes_ok(B, L, S) ? bwd_ws(blk_params(cfg, B, L, S)).total : BAD;
}

size_t msgla_block_attention_step_workspace_bytes(const msgla_block_config* cfg, int64_t B, int64_t S) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, 1, S)) return BAD;
  return step_ws(blk_params(cfg, B, 1, S)).fwd.total;
}

msgla_status msgla_block_means(const msgla_block_config* cfg, const msgla_heads* k,
                               const int32_t* lens, const int32_t* from, int64_t B, int64_t S,
                               float* means, void* stream) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, 1, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(k, es) || !means || !aligned16(means) || !i32_ok(lens) || !i32_ok(from)) return MSGLA_ERR_INVALID_ARG;
  BlkParams P = blk_params(cfg, B, 1, S);
  if (!means_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  P.k = heads_of(k, es);
  P.lens = lens;
  P.from = from;
  P.means = means;
  HIP_TRY(launch_block_means(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_block_select(const msgla_block_config* cfg, const msgla_heads* q,
                                const float* means, const int32_t* start, const int32_t* lens,
                                int64_t B, int64_t L, int64_t S, int32_t* sel, void* stream) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !means || !aligned16(means) || !sel || !i32_ok(sel) || !i32_ok(start) || !i32_ok(lens))
    return MSGLA_ERR_INVALID_ARG;
  BlkParams P = blk_params(cfg, B, L, S);
  if (!select_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  P.q = heads_of(q, es);
  P.means = const_cast<float*>(means);
  P.start = start;
  P.lens = lens;
  P.sel_out = sel;
  HIP_TRY(launch_block_select(P, es == 2, static_cast<hipStream_t>(stream)));
  return MSGLA_OK;
}

msgla_status msgla_block_attention(const msgla_block_config* cfg, const msgla_heads* q,
                                   const msgla_heads* k, const msgla_heads* v, const int32_t* sel,
                                   const int32_t* start, const int32_t* lens, int64_t B, int64_t L,
                                   int64_t S, const msgla_heads* out, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  if (!heads_ok(q, es) || !heads_ok(k, es) || !heads_ok(v, es) || !heads_ok(out, es) || !sel || !i32_ok(sel) ||
      !i32_ok(start) || !i32_ok(lens) || !i32_ok(lse))
    return MSGLA_ERR_INVALID_ARG;
  BlkParams P = blk_params(cfg, B, L, S);
  const FwdWs w = fwd_ws(P);
  if (w.total && (!workspace || !aligned16(workspace))) return MSGLA_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  if (!tiles_grid_ok(P, es, false, w.parts)) return MSGLA_ERR_UNSUPPORTED;
  P.q = heads_of(q, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out, es);
  P.sel = sel;
  P.start = start;
  P.lens = lens;
  P.lse = lse;
  set_fwd(P, w, workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (use_tiles(P)) HIP_TRY(launch_block_tiles(P, false, es == 2, st));
  else HIP_TRY(launch_block_forward(P, es == 2, st));
  return MSGLA_OK;
}

msgla_status msgla_block_attention_backward(const msgla_block_config* cfg, const msgla_heads* q,
                                            const msgla_heads* k, const msgla_heads* v,
                                            const int32_t* sel, const int32_t* start,
                                            const int32_t* lens, const msgla_heads* out,
                                            const float* lse, const msgla_heads* dout, int64_t B,
                                            int64_t L, int64_t S, const msgla_heads* dq,
                                            const msgla_heads* dk, const msgla_heads* dv,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, L, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  for (const msgla_heads* t : {q, k, v, out, dout, dq, dk, dv})
    if (!heads_ok(t, es)) return MSGLA_ERR_INVALID_ARG;
  if (!sel || !i32_ok(sel) || !i32_ok(start) || !i32_ok(lens) || !lse || !i32_ok(lse) || !workspace ||
      !aligned16(workspace))
    return MSGLA_ERR_INVALID_ARG;
  BlkParams P = blk_params(cfg, B, L, S);
  const BwdWs w = bwd_ws(P);
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  if (!tiles_grid_ok(P, es, true, w.parts) || !bwd_grid_ok(P, w)) return MSGLA_ERR_UNSUPPORTED;
  P.q = heads_of(q, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out, es);
  P.dout = heads_of(dout, es);
  P.dq = heads_of(dq, es);
  P.dk = heads_of(dk, es);
  P.dv = heads_of(dv, es);
  P.sel = sel;
  P.start = start;
  P.lens = lens;
  P.lse_in = lse;
  P.parts = w.parts;
  if (w.parts > 1) {
    P.po = at<float>(workspace, w.po);
    P.pm = at<float>(workspace, w.pm);
  }
  P.delta = at<float>(workspace, w.delta);
  P.bits = at<uint64_t>(workspace, w.bits);
  P.cnt = at<int32_t>(workspace, w.cnt);
  P.off = at<int32_t>(workspace, w.off);
  P.slot = at<int32_t>(workspace, w.slot);
  P.list = at<int32_t>(workspace, w.list);
  P.items = at<int2>(workspace, w.items);
  P.n_items = at<int32_t>(workspace, w.n_items);
  P.part = at<float>(workspace, w.part);
  P.seg = w.seg;
  P.W = w.W;
  P.max_items = w.max_items;
  P.max_parts = w.max_parts;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (use_tiles(P)) HIP_TRY(launch_block_tiles(P, true, es == 2, st));
  else HIP_TRY(launch_block_dq(P, es == 2, st));
  HIP_TRY(launch_block_dkdv(P, es == 2, st));
  return MSGLA_OK;
}

msgla_status msgla_block_attention_step(const msgla_block_config* cfg, const msgla_heads* q_t,
                                        const msgla_heads* k_t, const msgla_heads* v_t,
                                        const int32_t* pos, int64_t B, int64_t S,
                                        const msgla_heads* k, const msgla_heads* v, float* means,
                                        const msgla_heads* out_t, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (!blk_config_ok(cfg) || !blk_sizes_ok(B, 1, S)) return MSGLA_ERR_INVALID_ARG;
  const int es = es_of(cfg);
  for (const msgla_heads* t : {q_t, k_t, v_t, out_t})
    if (!heads_t_ok(t, es)) return MSGLA_ERR_INVALID_ARG;
  if (!heads_ok(k, es) || !heads_ok(v, es) || !pos || !i32_ok(pos) || !means || !aligned16(means) || !workspace ||
      !aligned16(workspace))
    return MSGLA_ERR_INVALID_ARG;
  BlkParams P = blk_params(cfg, B, 1, S);
  const StepWs s = step_ws(P);
  const FwdWs& w = s.fwd;
  if (workspace_bytes < w.total) return MSGLA_ERR_WORKSPACE;
  if (!tiles_grid_ok(P, es, false, w.parts) || !step_grid_ok(P)) return MSGLA_ERR_UNSUPPORTED;
  P.q = heads_of(q_t, es);
  P.kt = heads_of(k_t, es);
  P.vt = heads_of(v_t, es);
  P.k = heads_of(k, es);
  P.v = heads_of(v, es);
  P.o = heads_of(out_t, es);
  P.means = means;
  P.start = pos;
  P.sel_out = at<int32_t>(workspace, s.sel);
  P.bits = at<uint64_t>(workspace, s.key);
  P.sel = P.sel_out;
  set_fwd(P, w, workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  HIP_TRY(launch_block_step(P, es == 2, st));
  HIP_TRY(launch_block_forward(P, es == 2, st));
  return MSGLA_OK;
}

}  // extern "C"
