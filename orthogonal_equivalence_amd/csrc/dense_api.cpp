// C ABI of the dense linear with its epilogue (poetx_dense_fwd / _bwd):
// argument validation, workspace planning and the order of kernel launches.
// Declarations and the contract are in include/poetx.h. Validation touches no
// HIP API, so every argument error is reported before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_util.h"
#include "dense_plan.h"
#include "kernels.h"
#include "poetx.h"

using poetx::Activation;
using poetx::DType;
using poetx::TileProduct;
using namespace poetx::api;

namespace {

constexpr int64_t kMaxTokens = 1 << 30, kMaxWidth = 1 << 22;

DType dtype_of(const poetx_dense_desc* d) {
  return d->act == POETX_BF16 ? DType::BF16 : DType::F32;
}
bool int8_weight(const poetx_dense_desc* d) { return d->w_scale != nullptr; }

int check_desc(const poetx_dense_desc* d) {
  if (!d) return POETX_ERR_NULL;
  if (d->act != POETX_F32 && d->act != POETX_BF16) return POETX_ERR_DTYPE;
  if (d->tokens < 1 || d->d_in < 1 || d->d_out < 1) return POETX_ERR_SHAPE;
  if (d->tokens > kMaxTokens || d->d_in > kMaxWidth || d->d_out > kMaxWidth) return POETX_ERR_SHAPE;
  if (d->activation < POETX_ACT_NONE || d->activation > POETX_ACT_SILU || d->flags != 0 ||
      d->reserved != 0)
    return POETX_ERR_SHAPE;
  // (tile counts are ints)
  if (ceil_div(d->tokens, 64) * ceil_div(std::max(d->d_in, d->d_out), 64) > INT32_MAX)
    return POETX_ERR_SHAPE;
  if (d->w_scale && ((reinterpret_cast<uintptr_t>(d->w_scale) & 15) || d->d_in % 8))
    return POETX_ERR_ALIGN;
  const int v = act_vec(d->act);
  if (d->d_in % v || d->d_out % v) return POETX_ERR_ALIGN;
  return POETX_OK;
}

size_t weight_bytes(const poetx_dense_desc* d) {
  return (size_t)d->d_out * d->d_in * (int8_weight(d) ? 1 : act_size(d->act));
}
size_t widened_bytes(const poetx_dense_desc* d) {
  return int8_weight(d) ? align_up((size_t)d->d_out * d->d_in * act_size(d->act)) : 0;
}

struct FwdPlan : poetx::FwdChoice {
  size_t wq, part, total;
};
FwdPlan plan_fwd(const poetx_dense_desc* d) {
  FwdPlan p = {};
  static_cast<poetx::FwdChoice&>(p) =
      poetx::choose_fwd(dtype_of(d), int8_weight(d), d->tokens, d->d_in, d->d_out);
  if (p.stream) return p;
  p.part = p.widen ? widened_bytes(d) : 0;
  p.total = p.part + (p.dense ? 0 : align_up(p.tile.part_floats * sizeof(float)));
  return p;
}

struct BwdPlan : poetx::BwdChoice {
  size_t gu, bias, wq, part, total;
};
// whether the products take g_u from the workspace (else g_y is g_u)
bool forms_gu(const poetx_dense_desc* d) {
  return d->activation != POETX_ACT_NONE || int8_weight(d);
}
BwdPlan plan_bwd(const poetx_dense_desc* d) {
  BwdPlan p = {};
  static_cast<poetx::BwdChoice&>(p) =
      poetx::choose_bwd(dtype_of(d), int8_weight(d), d->tokens, d->d_in, d->d_out);
  size_t off = 0;
  p.gu = off;
  if (forms_gu(d)) off += align_up((size_t)d->tokens * d->d_out * act_size(d->act));
  p.bias = off;
  off += align_up((size_t)poetx::act_grad_splits(d->tokens) * d->d_out * sizeof(float));
  p.wq = off;
  off += widened_bytes(d);
  p.part = off;
  size_t part = p.gx.part_floats;
  if (!int8_weight(d)) part = std::max(part, p.gw.part_floats);
  if (p.paired) part = std::max(part, p.pair.gx.part_floats + p.pair.gw.part_floats);
  off += align_up(part * sizeof(float));
  p.total = off;
  return p;
}

bool any_overlap(const Range* outs, int nout, const Range* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}
Range opt_range(const void* p, size_t bytes) { return range_of(p, p ? bytes : 0); }

}  // namespace

#define POETX_TRY(expr)                            \
  do {                                             \
    if ((expr) != hipSuccess) return POETX_ERR_HIP; \
  } while (0)

extern "C" {

size_t poetx_dense_fwd_workspace_size(const poetx_dense_desc* d) {
  return check_desc(d) == POETX_OK ? plan_fwd(d).total : 0;
}

size_t poetx_dense_bwd_workspace_size(const poetx_dense_desc* d) {
  return check_desc(d) == POETX_OK ? plan_bwd(d).total : 0;
}

int poetx_dense_fwd(const poetx_dense_desc* d, const void* x, const void* W, const float* bias,
                    const void* residual, void* y, void* u_save, void* ws, size_t ws_bytes,
                    void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (!x || !W || !y) return POETX_ERR_NULL;
  for (const void* p : {x, W, (const void*)bias, residual, (const void*)y, (const void*)u_save})
    if (p && !aligned16(p)) return POETX_ERR_ALIGN;
  const FwdPlan plan = plan_fwd(d);
  if (!plan.launchable()) return POETX_ERR_SHAPE;
  if (plan.total && (!ws || ws_bytes < plan.total)) return POETX_ERR_WORKSPACE;
  if (plan.total && !aligned16(ws)) return POETX_ERR_ALIGN;
  const size_t es = act_size(d->act), out = (size_t)d->tokens * d->d_out * es;
  const Range outs[] = {range_of(y, out), opt_range(u_save, out),
                        opt_range(plan.total ? ws : nullptr, plan.total)};
  const Range ins[] = {range_of(x, (size_t)d->tokens * d->d_in * es), range_of(W, weight_bytes(d)),
                       opt_range(bias, (size_t)d->d_out * 4), opt_range(residual, out),
                       opt_range(d->w_scale, (size_t)d->d_out * 4)};
  if (any_overlap(outs, 3, ins, 5)) return POETX_ERR_ALIAS;

  const DType t = dtype_of(d);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  poetx::Epilogue ep;
  ep.scale = d->w_scale;
  ep.bias = bias;
  ep.residual = residual;
  ep.y = y;
  ep.u = u_save;
  ep.ld = d->d_out;
  ep.act = d->activation;
  if (plan.stream) {
    poetx::StreamProduct p;
    p.x = x;
    p.W = W;
    p.M = (int)d->tokens; p.N = (int)d->d_out; p.K = (int)d->d_in;
    p.ep = ep;
    POETX_TRY(poetx::launch_stream_product(t, int8_weight(d), p, s));
    return POETX_OK;
  }
  const void* B = W;
  if (plan.widen) {
    POETX_TRY(poetx::launch_widen_codes(t, static_cast<const int8_t*>(W), d->d_out, d->d_in,
                                        d->d_in, w + plan.wq, plan.w_tiled, s));
    B = w + plan.wq;
  }
  if (plan.dense) {
    poetx::DenseProduct p;
    p.A = x; p.lda = d->d_in;
    p.B = B; p.ldb = d->d_in;
    p.M = (int)d->tokens; p.N = (int)d->d_out; p.K = (int)d->d_in;
    p.b_tiled = plan.w_tiled;
    p.ep = ep;
    POETX_TRY(poetx::launch_dense_epilogue(p, s));
    return POETX_OK;
  }
  TileProduct p;
  p.A = x; p.lda = d->d_in;
  p.B = B; p.ldb = d->d_in;
  p.M = (int)d->tokens; p.N = (int)d->d_out; p.K = (int)d->d_in;
  p.b_int8 = int8_weight(d) && !plan.widen;
  p.part = reinterpret_cast<float*>(w + plan.part);
  p.ep = ep;
  POETX_TRY(poetx::launch_tile_product(t, plan.tile, p, true, true, s));
  return POETX_OK;
}

int poetx_dense_bwd(const poetx_dense_desc* d, const void* g_y, const void* x, const void* W,
                    const void* u_saved, void* g_x, void* g_W, float* g_bias, void* ws,
                    size_t ws_bytes, void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (!g_y || (!g_x && !g_W && !g_bias)) return POETX_ERR_NULL;
  if ((g_x && !W) || (g_W && !x)) return POETX_ERR_NULL;
  if (d->activation != POETX_ACT_NONE && !u_saved) return POETX_ERR_NULL;
  if (g_W && int8_weight(d)) return POETX_ERR_DTYPE;  // codes have no gradient
  // (what this choice of outputs does not read is not looked at)
  if (!g_x) W = nullptr;
  if (!g_W) x = nullptr;
  if (d->activation == POETX_ACT_NONE) u_saved = nullptr;
  for (const void* p : {g_y, x, W, u_saved, (const void*)g_x, (const void*)g_W,
                        (const void*)g_bias})
    if (p && !aligned16(p)) return POETX_ERR_ALIGN;
  const BwdPlan plan = plan_bwd(d);
  if ((g_x && !plan.gx_launchable()) || (g_W && !plan.gw_launchable())) return POETX_ERR_SHAPE;
  if (!ws || ws_bytes < plan.total) return POETX_ERR_WORKSPACE;
  if (!aligned16(ws)) return POETX_ERR_ALIGN;
  const size_t es = act_size(d->act);
  const size_t out = (size_t)d->tokens * d->d_out * es, in = (size_t)d->tokens * d->d_in * es;
  const Range outs[] = {opt_range(g_x, in), opt_range(g_W, weight_bytes(d)),
                        opt_range(g_bias, (size_t)d->d_out * 4), range_of(ws, plan.total)};
  const Range ins[] = {range_of(g_y, out), opt_range(x, in), opt_range(W, weight_bytes(d)),
                       opt_range(u_saved, out), opt_range(d->w_scale, (size_t)d->d_out * 4)};
  if (any_overlap(outs, 4, ins, 5)) return POETX_ERR_ALIAS;

  const DType t = dtype_of(d);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const bool products = g_x || g_W, pair = plan.paired && g_x && g_W;
  // (g_u in the dense kernel's fastest layout, which g_W's product cannot read)
  const bool gu_tiled = plan.dense && forms_gu(d) && g_x && !g_W &&
                        d->tokens % poetx::kTileRows == 0;
  const void* gu = g_y;
  if ((forms_gu(d) && products) || g_bias) {
    poetx::ActGrad a;
    a.g_y = g_y;
    a.u = u_saved;
    a.scale = d->w_scale;
    a.g_u = forms_gu(d) && products ? w + plan.gu : nullptr;
    a.g_bias = g_bias;
    a.part = reinterpret_cast<float*>(w + plan.bias);
    a.rows = d->tokens;
    a.d = (int)d->d_out;
    a.act = static_cast<Activation>(d->activation);
    a.gu_tiled = gu_tiled;
    POETX_TRY(poetx::launch_act_grad(t, a, s));
    if (a.g_u) gu = a.g_u;
  }
  float* part = reinterpret_cast<float*>(w + plan.part);
  TileProduct gx, gw;
  if (g_x) {  // g_x = g_u W: B(n, k) = W[k][n]
    const void* B = W;
    if (int8_weight(d)) {
      POETX_TRY(poetx::launch_widen_codes(t, static_cast<const int8_t*>(W), d->d_out, d->d_in,
                                          d->d_in, w + plan.wq, false, s));
      B = w + plan.wq;
    }
    gx.A = gu; gx.lda = d->d_out;
    gx.B = B; gx.ldb = d->d_in;
    gx.M = (int)d->tokens; gx.N = (int)d->d_in; gx.K = (int)d->d_out;
    gx.part = part;
    gx.ep.y = g_x;
    gx.ep.ld = d->d_in;
  }
  if (g_W) {  // g_W = g_u^T x: A(m, k) = g_u[k][m], B(n, k) = x[k][n]
    gw.A = gu; gw.lda = d->d_out;
    gw.B = x; gw.ldb = d->d_in;
    gw.M = (int)d->d_out; gw.N = (int)d->d_in; gw.K = (int)d->tokens;
    gw.part = pair ? part + plan.pair.gx.part_floats : part;
    gw.ep.y = g_W;
    gw.ep.ld = d->d_in;
  }
  if (pair) {
    POETX_TRY(poetx::launch_tile_pair(t, plan.pair, gx, gw, s));
    return POETX_OK;
  }
  if (g_x && plan.dense)
    POETX_TRY(poetx::launch_dense(gu, gx.B, g_x, d->tokens, d->d_in, d->d_out, d->d_out, d->d_in,
                                  d->d_in, false, gu_tiled, false, s));
  else if (g_x)
    POETX_TRY(poetx::launch_tile_product(t, plan.gx, gx, true, false, s));
  if (g_W) POETX_TRY(poetx::launch_tile_product(t, plan.gw, gw, false, false, s));
  return POETX_OK;
}

}  // extern "C"
