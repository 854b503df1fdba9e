// C ABI of the losses over a vocabulary whose logits are not kept
// (poetx_cross_entropy_fwd / _bwd, poetx_distill_fwd / _bwd): argument
// validation, workspace planning and the order of kernel launches. Declarations
// and the contract are in include/poetx.h. Validation touches no HIP API, so
// every argument error is reported before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "kernels.h"
#include "poetx.h"
#include "vocab_plan.h"

using poetx::DType;
using poetx::TileProduct;
using poetx::VocabList;
using poetx::VocabProduct;
using poetx::VocabRow;
using namespace poetx::api;

namespace {

constexpr int64_t kMaxTokens = 1 << 24, kMaxWidth = 1 << 22, kMaxTop = 1024;
constexpr int64_t kMaxValues = INT64_C(1) << 35;  // of x or W
DType dtype_of(const poetx_vocab_desc* d) {
  return d->act == POETX_BF16 ? DType::BF16 : DType::F32;
}

int check_desc(const poetx_vocab_desc* d) {
  if (!d) return POETX_ERR_NULL;
  if (d->act != POETX_F32 && d->act != POETX_BF16) return POETX_ERR_DTYPE;
  if (d->tokens < 1 || d->d < 1 || d->vocab < 1) return POETX_ERR_SHAPE;
  if (d->tokens > kMaxTokens || d->d > kMaxWidth || d->vocab > kMaxWidth) return POETX_ERR_SHAPE;
  if (d->top < 0 || d->top > kMaxTop || d->flags != 0 || d->reserved != 0)
    return POETX_ERR_SHAPE;
  if (d->top == 0) {
    if (d->teacher != 0 || d->temperature != 1.0f) return POETX_ERR_SHAPE;
  } else {
    if (d->teacher != POETX_F32 && d->teacher != POETX_BF16) return POETX_ERR_DTYPE;
    // (so that it, its square and its inverse are ordinary numbers)
    if (!(d->temperature >= 1e-6f && d->temperature <= 1e6f)) return POETX_ERR_SHAPE;
  }
  // (the gradients' tiles fit a launch, their counts an int)
  if (std::max(d->tokens, d->vocab) * d->d > kMaxValues) return POETX_ERR_SHAPE;
  if (d->d % act_vec(d->act)) return POETX_ERR_ALIGN;
  return POETX_OK;
}

size_t x_bytes(const poetx_vocab_desc* d) { return (size_t)d->tokens * d->d * act_size(d->act); }
size_t w_bytes(const poetx_vocab_desc* d) { return (size_t)d->vocab * d->d * act_size(d->act); }
size_t list_entries(const poetx_vocab_desc* d) { return (size_t)d->tokens * std::max(d->top, 1); }

VocabList list_of(const poetx_vocab_desc* d, const int64_t* ids, const void* teacher) {
  VocabList l;
  l.ids = ids;
  l.teacher = teacher;
  l.type = d->teacher == POETX_BF16 ? DType::BF16 : DType::F32;
  l.top = std::max(d->top, 1);
  l.vocab = d->vocab;
  l.temperature = d->temperature;
  return l;
}
// rows [row, ..) of a list
VocabList list_at(VocabList l, int64_t row) {
  l.ids += row * l.top;
  if (l.teacher)
    l.teacher = static_cast<const char*>(l.teacher) + row * l.top * (l.type == DType::BF16 ? 2 : 4);
  return l;
}
poetx::VocabSizes sizes_of(const poetx_vocab_desc* d) {
  return {dtype_of(d), d->tokens, d->d, d->vocab, d->top};
}
float scale_of(const poetx_vocab_desc* d) { return 1.44269504088896341f / d->temperature; }

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
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

#define POETX_TRY(expr)                            \
  do {                                             \
    if ((expr) != hipSuccess) return POETX_ERR_HIP; \
  } while (0)

// Both forwards: z is the output of a distillation (its targets' logits go to
// the workspace otherwise).
int forward(const poetx_vocab_desc* d, const void* x, const void* W, const int64_t* ids,
            const void* teacher, float* loss, float* lse, float* z, void* ws, size_t ws_bytes,
            void* stream) {
  if (!x || !W || !ids || !loss || !lse || (d->top && (!teacher || !z))) return POETX_ERR_NULL;
  if (!aligned16(x) || !aligned16(W) || !aligned_to(ids, 8) || !aligned_to(loss, 4) ||
      !aligned_to(lse, 4) || !aligned_to(z, 4) || !aligned_to(teacher, act_size(d->teacher)))
    return POETX_ERR_ALIGN;
  const poetx::VocabFwdPlan plan = poetx::plan_vocab_fwd(sizes_of(d));
  if (!ws || ws_bytes < plan.total) return POETX_ERR_WORKSPACE;
  if (!aligned16(ws)) return POETX_ERR_ALIGN;
  const size_t rows4 = (size_t)d->tokens * 4, n = list_entries(d);
  const Range outs[] = {range_of(loss, rows4), range_of(lse, rows4), opt_range(z, n * 4),
                        range_of(ws, plan.total)};
  const Range ins[] = {range_of(x, x_bytes(d)), range_of(W, w_bytes(d)), range_of(ids, n * 8),
                       opt_range(teacher, n * act_size(d->teacher))};
  if (any_overlap(outs, 4, ins, 4)) return POETX_ERR_ALIAS;

  const DType t = dtype_of(d);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const VocabList list = list_of(d, ids, teacher);
  if (!z) z = reinterpret_cast<float*>(w + plan.z);
  float2* part = reinterpret_cast<float2*>(w + plan.part);
  // (targets' logits come out of the products)
  const bool beside = teacher && !plan.cells && plan.cols.dense == 0 &&
                      list_entries(d) <= (size_t)1 << 24;  // (and few beside a launch's limit)
  if (teacher && !plan.cells && !beside)
    POETX_TRY(poetx::launch_listed_logits(t, x, W, list, d->tokens, (int)d->d, z, s));
  if (plan.copied) {
    poetx::VocabCopies c;
    c.W = W;
    c.W_last = w + plan.last;
    POETX_TRY(poetx::launch_vocab_last_rows(t, d->vocab, (int)d->d, c, s));
  }
  for (int64_t at = 0; at < d->tokens; at += plan.rows) {
    const int64_t rows = std::min(plan.rows, d->tokens - at);
    // (the dense tiles take 256 rows at least: the last range begins early, and
    // forms some rows' sums again)
    const int64_t r = plan.cols.dense ? std::min(at, std::max(d->tokens - poetx::kTileRows, INT64_C(0))) : at;
    VocabProduct p;
    p.x = static_cast<const char*>(x) + r * d->d * act_size(d->act);
    p.W = W;
    p.M = (int)(at + rows - r); p.N = (int)plan.cols.dense; p.K = (int)d->d;
    p.scale = scale_of(d);
    const int64_t* targets = teacher ? nullptr : ids + r;
    const int64_t dense = plan.cols.dense, rest = d->vocab - dense;
    poetx::VocabCells cells[2];
    for (int i = 0; plan.cells && i < 2; ++i) {
      const int64_t from = i ? dense : 0, n = i ? rest : dense;
      if (n == 0) continue;
      const poetx::CellShape shape =
          i ? poetx::vocab_tile_cells(t, plan.cols.tile) : poetx::vocab_dense_cells();
      int* offsets = reinterpret_cast<int*>(w + plan.offsets[i]);
      uint32_t* entries = reinterpret_cast<uint32_t*>(w + plan.entries[i]);
      POETX_TRY(poetx::launch_vocab_cells(list_at(list, r), p.M, from, n, shape, offsets, entries,
                                          z + r * list.top, i == 1 || rest == 0, s));
      cells[i].offsets = offsets;
      cells[i].entries = entries;
      cells[i].bins = (int)shape.bins(n);
      cells[i].per_cell = shape.rows * list.top;
      cells[i].top = list.top;
      cells[i].z = z + r * list.top;
    }
    if (p.N) POETX_TRY(poetx::launch_vocab_lse_dense(p, w + plan.last, part, p.M, targets, z + r, cells[0],
                                              s));
    if (plan.cols.dense < d->vocab) {
      p.col0 = p.N;
      p.W = static_cast<const char*>(W) + p.col0 * d->d * act_size(d->act);
      p.N = (int)(d->vocab - p.col0);
      POETX_TRY(poetx::launch_vocab_lse_tile(t, plan.cols.tile, p, part + p.col0 / 128 * (int64_t)p.M,
                                             p.M, targets, z + r * list.top, cells[1],
                                             beside ? list_at(list, r) : VocabList(), s));
    }
    POETX_TRY(poetx::launch_vocab_loss(part, p.M, plan.slots, list_at(list, r), p.M,
                                       z + r * list.top, loss + r, lse + r, s));
  }
  return POETX_OK;
}

int backward(const poetx_vocab_desc* d, const float* g_loss, const float* g_lse, const void* x,
             const void* W, const int64_t* ids, const void* teacher, const float* lse,
             const float* z, void* g_x, void* g_W, void* ws, size_t ws_bytes, void* stream) {
  if (!g_loss || !x || !W || !ids || !lse || (!g_x && !g_W) || (d->top && (!teacher || !z)))
    return POETX_ERR_NULL;
  if (!aligned16(x) || !aligned16(W) || !aligned16(g_x) || !aligned16(g_W) || !aligned_to(ids, 8) ||
      !aligned_to(g_loss, 4) || !aligned_to(g_lse, 4) || !aligned_to(lse, 4) || !aligned_to(z, 4) ||
      !aligned_to(teacher, act_size(d->teacher)))
    return POETX_ERR_ALIGN;
  const poetx::VocabBwdPlan plan = poetx::plan_vocab_bwd(sizes_of(d), g_W != nullptr);
  if (!ws || ws_bytes < plan.total) return POETX_ERR_WORKSPACE;
  if (!aligned16(ws)) return POETX_ERR_ALIGN;
  const size_t rows4 = (size_t)d->tokens * 4, n = list_entries(d);
  const Range outs[] = {opt_range(g_x, x_bytes(d)), opt_range(g_W, w_bytes(d)),
                        range_of(ws, plan.total)};
  const Range ins[] = {range_of(x, x_bytes(d)), range_of(W, w_bytes(d)), range_of(ids, n * 8),
                       range_of(g_loss, rows4), opt_range(g_lse, rows4), range_of(lse, rows4),
                       opt_range(z, n * 4), opt_range(teacher, n * act_size(d->teacher))};
  if (any_overlap(outs, 3, ins, 8)) return POETX_ERR_ALIAS;

  const DType t = dtype_of(d);
  const int64_t es = (int64_t)act_size(d->act);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const VocabList list = list_of(d, ids, teacher);
  VocabRow* rows = reinterpret_cast<VocabRow*>(w + plan.rows);
  // (the dense products read x out of its tiled copy too)
  void* xs = g_W || plan.dense ? w + plan.xs : nullptr;
  char* gz = w + plan.gz;
  float* acc = reinterpret_cast<float*>(w + plan.acc);
  const int parts = plan.two ? 2 : 1;
  const int64_t low = !plan.two ? 0 : plan.dense ? poetx::kPairLow : d->tokens * plan.ldg;
  const int64_t dense_rows = sizes_of(d).dense_rows();
  const bool ragged = plan.dense && d->vocab % poetx::kTileRows != 0;
  poetx::VocabCopies copies;
  copies.x = x;
  copies.xs = xs;
  copies.tiled = plan.dense;
  copies.twice = plan.two && !plan.dense;
  if (plan.two && plan.dense && g_W) copies.pairs = w + plan.pairs;
  copies.W = W;
  copies.W_last = ragged ? w + plan.last : nullptr;
  if (g_W && !plan.dense && plan.few) {
    copies.xs = nullptr;
    copies.xt = w + plan.xs;
    copies.xt_rows = poetx::few_padded(t, (int)d->tokens);
  }
  POETX_TRY(poetx::launch_vocab_rows(t, list, d->tokens, plan.padded, g_loss, g_lse, lse, rows,
                                     (int)d->d, copies, s));
  for (int64_t c = 0; c < d->vocab; c += plan.piece) {
    const int64_t cols = std::min(plan.piece, d->vocab - c);
    const char* Wc = static_cast<const char*>(W) + c * d->d * es;
    const void* last = ragged && c + cols == d->vocab ? copies.W_last : nullptr;
    char* gWc = g_W ? static_cast<char*>(g_W) + c * d->d * es : nullptr;
    // the gradient of the piece's logits
    const poetx::VocabColumns split = poetx::plan_vocab_columns(sizes_of(d), plan, cols);
    VocabProduct p;
    p.x = xs;
    p.W = Wc;
    p.M = (int)plan.padded; p.N = (int)split.dense; p.K = (int)d->d;
    p.col0 = (int)c;
    p.scale = 1.0f / d->temperature;
    if (p.N) POETX_TRY(poetx::launch_vocab_grad_dense(p, last, rows, gz, plan.ldg, plan.two, s));
    if (split.dense < cols) {
      p.x = x;
      p.W = Wc + split.dense * d->d * es;
      p.M = (int)d->tokens; p.N = (int)(cols - split.dense);
      p.col0 = (int)(c + split.dense);
      POETX_TRY(poetx::launch_vocab_grad_tile(t, split.tile, p, rows,
                                              gz + split.dense * poetx::kTileRows * es, plan.ldg,
                                              plan.dense, low, s));
    }
    if (teacher)
      POETX_TRY(poetx::launch_vocab_listed_grad(t, list, d->tokens, rows, z, gz, plan.ldg,
                                                plan.dense, low, (int)c, (int)cols, s));
    if (plan.dense) {
      if (g_x)
        POETX_TRY(poetx::launch_vocab_gx_dense(
            gz, plan.ldg, Wc, last, dense_rows, (int)d->d, (int)cols,
            (int)ceil_div(cols, plan.kchunk), plan.kchunk, acc, c > 0,
            plan.summed() ? nullptr : g_x, s));
      if (g_W)
        POETX_TRY(poetx::launch_vocab_gw_dense(gz, plan.ldg, plan.two ? copies.pairs : xs,
                                               ceil_div(dense_rows, 32) * 32, (int)d->d, (int)cols,
                                               gWc, s));
      continue;
    }
    const poetx::VocabProducts tiles = poetx::plan_vocab_products(sizes_of(d), cols);
    float* part = reinterpret_cast<float*>(w + plan.part);
    TileProduct qx, qw;
    qx.blocked = qw.blocked = true;
    // g_x += g_z W: B(n, k) = W[k][n]
    qx.A = gz; qx.lda = plan.ldg;
    qx.B = Wc; qx.ldb = d->d;
    qx.M = (int)d->tokens * parts; qx.N = (int)d->d; qx.K = (int)cols;
    qx.part = part;
    qx.halves = parts;
    qx.ep.y = g_x;
    qx.ep.add = c > 0 ? acc : nullptr;
    qx.ep.sum = c + cols < d->vocab ? acc : nullptr;
    qx.ep.ld = d->d;
    // g_W = g_z^T x: A(m, k) = g_z[k][m], B(n, k) = xs[k][n]
    qw.A = gz; qw.lda = plan.ldg;
    qw.B = xs; qw.ldb = d->d;
    qw.M = (int)cols; qw.N = (int)d->d; qw.K = (int)d->tokens * parts;
    qw.part = g_x && tiles.paired ? part + tiles.pair.gx.part_floats : part;
    qw.ep.y = gWc;
    qw.ep.ld = d->d;
    if (g_x && g_W && tiles.paired && !copies.xt) {
      POETX_TRY(poetx::launch_tile_pair(t, tiles.pair, qx, qw, s));
      continue;
    }
    if (g_x) POETX_TRY(poetx::launch_tile_product(t, tiles.gx, qx, true, false, s));
    // (after g_x, which finds W in the caches)
    if (g_W && copies.xt)
      POETX_TRY(poetx::launch_few_gw(t, gz, plan.ldg, copies.xt, (int)d->tokens, (int)cols,
                                     (int)d->d, gWc, s));
    else if (g_W)
      POETX_TRY(poetx::launch_tile_product(t, tiles.gw, qw, false, false, s));
  }
  if (plan.dense && g_x && plan.summed())
    POETX_TRY(poetx::launch_sum_slabs(t, acc, plan.splits, d->tokens, (int)d->d, g_x, plan.two, s));
  return POETX_OK;
}

}  // namespace

extern "C" {

size_t poetx_vocab_fwd_workspace_size(const poetx_vocab_desc* d) {
  return check_desc(d) == POETX_OK ? poetx::plan_vocab_fwd(sizes_of(d)).total : 0;
}

size_t poetx_vocab_bwd_workspace_size(const poetx_vocab_desc* d) {
  if (check_desc(d) != POETX_OK) return 0;
  return std::max(poetx::plan_vocab_bwd(sizes_of(d), false).total,
                  poetx::plan_vocab_bwd(sizes_of(d), true).total);
}

int poetx_cross_entropy_fwd(const poetx_vocab_desc* d, const void* x, const void* W,
                            const int64_t* targets, float* loss, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (d->top != 0) return POETX_ERR_SHAPE;
  return forward(d, x, W, targets, nullptr, loss, lse, nullptr, ws, ws_bytes, stream);
}

int poetx_cross_entropy_bwd(const poetx_vocab_desc* d, const float* g_loss, const float* g_lse,
                            const void* x, const void* W, const int64_t* targets, const float* lse,
                            void* g_x, void* g_W, void* ws, size_t ws_bytes, void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (d->top != 0) return POETX_ERR_SHAPE;
  return backward(d, g_loss, g_lse, x, W, targets, nullptr, lse, nullptr, g_x, g_W, ws, ws_bytes,
                  stream);
}

int poetx_distill_fwd(const poetx_vocab_desc* d, const void* x, const void* W, const int64_t* ids,
                      const void* teacher, float* loss, float* lse, float* z, void* ws,
                      size_t ws_bytes, void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (d->top == 0) return POETX_ERR_SHAPE;
  return forward(d, x, W, ids, teacher, loss, lse, z, ws, ws_bytes, stream);
}

int poetx_distill_bwd(const poetx_vocab_desc* d, const float* g_loss, const void* x, const void* W,
                      const int64_t* ids, const void* teacher, const float* lse, const float* z,
                      void* g_x, void* g_W, void* ws, size_t ws_bytes, void* stream) {
  const int st = check_desc(d);
  if (st != POETX_OK) return st;
  if (d->top == 0) return POETX_ERR_SHAPE;
  return backward(d, g_loss, nullptr, x, W, ids, teacher, lse, z, g_x, g_W, ws, ws_bytes, stream);
}

}  // extern "C"
