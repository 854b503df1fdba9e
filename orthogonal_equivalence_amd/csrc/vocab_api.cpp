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
#include "dense_plan.h"
#include "kernels.h"
#include "poetx.h"

using poetx::DType;
using poetx::TilePlan;
using poetx::TileProduct;
using poetx::VocabList;
using poetx::VocabProduct;
using poetx::VocabRow;
using namespace poetx::api;

namespace {

constexpr int64_t kMaxTokens = 1 << 24, kMaxWidth = 1 << 22, kMaxTop = 1024;
constexpr int64_t kMaxValues = INT64_C(1) << 35;  // of x or W
// What the logits' pieces may take in the workspace: the forward's partial
// sums of a range of rows, the backward's gradient of a range of columns (every
// piece adds to g_x's float32 sums; 8192 x 131072 x 4096 in pieces of 128 MB 19300
// us, 256 19150, 512 18880, 1024 19100).
constexpr int64_t kPartBytes = INT64_C(128) << 20, kPieceBytes = INT64_C(512) << 20;
constexpr int64_t kTile = 256;  // rows and columns of a piece, where there is more than one

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
float scale_of(const poetx_vocab_desc* d) { return 1.44269504088896341f / d->temperature; }

// The time (us) of `tiles` 256 x 256 tiles of the products of vocab_dense.hip
// over K: a round of the 256 CUs is 1.35 us for each 64 of K and 10 for its end
// (measured: logits 52.7 and 93 a round at K = 2048 and 4096, with their gradient
// 54.8 and 97.5, g_W 29, 101 and 194 at 1024, 4096 and 8192).
float dense_cost(int64_t tiles, int64_t K) {
  return 3.0f + (float)ceil_div(tiles, 256) * (10.0f + 1.35f * (float)K / 64);
}

// Columns of the logits of `rows` rows on the 256 x 256 tiles; the rest, if any, go
// to the tile kernel: what a last round of the CUs that would be nearly empty
// holds (777 x 50001 x 2048 forward 217 -> 174 us), or what is left of the
// last tile where the copy of W's rows that it would take (`copy` us) costs more.
struct Columns {
  int64_t dense;
  TilePlan tile;
  float cost;
};
Columns split_columns(DType t, int64_t rows, int64_t cols, int64_t K, float copy) {
  Columns best = {0, plan_tile_product(t, rows, cols, K, false, 1), 0.0f};
  best.cost = best.tile.nsplit ? best.tile.cost : 1e30f;
  if (t != DType::BF16 || !poetx::vocab_dense_supported(rows, cols, K)) return best;
  const int64_t rt = ceil_div(rows, kTile), panels = cols / kTile;
  const int64_t whole = rt * panels / 256 * 256 / rt;  // (in whole rounds)
  for (int64_t n : {ceil_div(cols, kTile), panels, whole}) {
    if (n < 1) continue;
    Columns c = {std::min(n * kTile, cols), {}, dense_cost(rt * n, K)};
    if (c.dense % kTile) c.cost += copy;
    if (c.dense < cols) {
      c.tile = plan_tile_product(t, rows, cols - c.dense, K, false, 1);
      c.cost += c.tile.nsplit ? c.tile.cost : 1e30f;
    }
    if (c.cost < best.cost) best = c;
  }
  return best;
}

// The forward's partial sums: `rows` rows at a time, so that they stay within
// kPartBytes.
// A teacher's ids get their logits out of the products (`cells`, two launches'
// at most) where reading W's rows for each of them again would take longer than
// sorting them into the waves' cells and picking them out of the accumulators
// (4096 x 65536 x 2048, 64 ids a row: 116 us against 11 and about 40).
struct FwdPlan {
  Columns cols;
  int64_t rows, slots;
  bool copied;  // W_last
  bool cells;
  size_t z, last, part, offsets[2], entries[2], total;
};
struct CellSizes {
  size_t offsets, entries;  // bytes
  bool possible;
};
CellSizes cell_sizes(const poetx::CellShape& c, int64_t rows, int64_t cols, int top) {
  const int64_t n = c.row_cells(rows), bins = c.bins(cols);
  return {align_up((size_t)(n * (bins + 1) * 4)), align_up((size_t)(n * c.rows * top * 4)),
          bins <= poetx::kMaxBins};
}
FwdPlan plan_fwd(const poetx_vocab_desc* d) {
  FwdPlan p = {};
  const DType t = dtype_of(d);
  p.rows = d->tokens;
  for (;;) {
    p.cols = split_columns(t, p.rows, d->vocab, d->d, 5.0f);
    p.slots = 2 * ceil_div(p.cols.dense, kTile);
    if (p.cols.dense < d->vocab)
      p.slots += p.cols.tile.nsplit
                     ? poetx::vocab_tile_slots(t, p.cols.tile, d->vocab - p.cols.dense)
                     : INT32_MAX;
    if (p.slots * p.rows * 8 <= kPartBytes || p.rows <= kTile) break;
    p.rows = (p.rows / 2 + kTile - 1) / kTile * kTile;
  }
  p.last = d->top ? 0 : align_up((size_t)d->tokens * 4);  // (the targets' logits)
  p.copied = p.cols.dense % kTile != 0;
  p.part = p.last + (p.copied ? align_up((size_t)(kTile * d->d) * act_size(d->act)) : 0);
  p.total = p.part + align_up((size_t)(p.slots * p.rows * 8));
  const double read = (double)list_entries(d) * d->d * act_size(d->act) / 9.0e6;  // us
  if (d->top && read > 20.0) {
    const int64_t rest = d->vocab - p.cols.dense;
    CellSizes c[2] = {{0, 0, true}, {0, 0, true}};
    if (p.cols.dense) c[0] = cell_sizes(poetx::vocab_dense_cells(), p.rows, p.cols.dense, d->top);
    if (rest)
      c[1] = cell_sizes(poetx::vocab_tile_cells(t, p.cols.tile), p.rows, rest, d->top);
    p.cells = c[0].possible && c[1].possible;
    for (int i = 0; p.cells && i < 2; ++i) {
      p.offsets[i] = p.total;
      p.entries[i] = p.offsets[i] + c[i].offsets;
      p.total = p.entries[i] + c[i].entries;
    }
  }
  return p;
}

// The backward: `piece` columns of the vocabulary at a time.
struct BwdPlan {
  bool dense;
  int64_t padded;       // rows of xs and gz
  int64_t piece, pieces, ldg;
  int splits, kchunk;   // dense: of g_x's reduction over a piece
  size_t rows, last, xs, gz, acc, part, total;
  bool summed() const { return pieces > 1 || splits > 1; }
};
// g_z's two products of a piece of n columns on the tile kernel, each by itself
// or (few launches where they are what costs) in one
struct TileProducts {
  TilePlan gx, gw;
  poetx::TilePairPlan pair;
  bool paired;
  bool few;  // g_W on its own kernel for few tokens
  size_t part_floats() const {
    const size_t alone = std::max(gx.part_floats, gw.part_floats);
    return paired ? std::max(alone, pair.gx.part_floats + pair.gw.part_floats) : alone;
  }
};
TileProducts tile_products(const poetx_vocab_desc* d, int64_t n) {
  const DType t = dtype_of(d);
  TileProducts p;
  p.gx = plan_tile_product(t, d->tokens, d->d, n, false, poetx::kManySplits);
  p.gw = plan_tile_product(t, n, d->d, d->tokens, false);
  p.pair = plan_tile_pair(t, d->tokens, d->d, n, poetx::kManySplits);
  // a launch for the turned copy of x and one that stores g_W
  const float few = 6.0f + (float)(n * d->d * (int64_t)act_size(d->act)) / 3.2e6f;
  p.few = d->tokens <= poetx::kFewTokens &&
          few < std::min(p.gw.cost, std::max(p.pair.cost - p.gx.cost, 0.0f));
  p.paired = !p.few && p.pair.gx.nsplit != 0 && p.pair.cost < p.gx.cost + p.gw.cost;
  return p;
}
void set_pieces(const poetx_vocab_desc* d, BwdPlan& p) {
  const int64_t es = (int64_t)act_size(d->act);
  const int64_t most = std::max(kTile, kPieceBytes / (p.padded * es) / kTile * kTile);
  p.pieces = ceil_div(d->vocab, most);
  p.piece = p.pieces == 1 ? d->vocab : ceil_div(ceil_div(d->vocab, p.pieces), kTile) * kTile;
  p.pieces = ceil_div(d->vocab, p.piece);
  p.ldg = ceil_div(p.piece, kTile) * kTile;
}
// g_x's tiles are few where tokens and d are: its reduction, the vocabulary, is
// split so that they fill the CUs
float split_gx(const poetx_vocab_desc* d, BwdPlan& p) {
  const int64_t tiles = p.padded / kTile * ceil_div(d->d, kTile);
  float best = 1e30f;
  for (int s = 1; s <= 128; s += s < 16 ? 1 : 8) {
    const int64_t chunk = ceil_div(ceil_div(p.piece, s), kTile) * kTile;
    const int64_t n = ceil_div(p.piece, chunk);
    // (a slab is written and read once more)
    const float cost = dense_cost(tiles * n, chunk) +
                       (n > 1 ? 3.0f + (float)(8 * n * d->tokens * d->d) / 5e6f : 0.0f);
    if (cost >= best) continue;
    best = cost;
    p.splits = (int)n;
    p.kchunk = (int)chunk;
  }
  return best;
}
BwdPlan plan_bwd(const poetx_vocab_desc* d) {
  BwdPlan p = {};
  const DType t = dtype_of(d);
  const int64_t es = (int64_t)act_size(d->act);
  p.splits = 1;
  if (t == DType::BF16 && poetx::vocab_dense_supported(d->tokens, d->vocab, d->d)) {
    p.padded = ceil_div(d->tokens, kTile) * kTile;
    set_pieces(d, p);
    const float dense = split_columns(t, p.padded, p.piece, d->d, 1.0f).cost + split_gx(d, p) +
                        dense_cost(ceil_div(p.piece, kTile) * ceil_div(d->d, kTile), d->tokens);
    const float tile = plan_tile_product(t, d->tokens, p.piece, d->d, false, 1).cost +
                       plan_tile_product(t, d->tokens, d->d, p.piece, false, poetx::kManySplits).cost +
                       plan_tile_product(t, p.piece, d->d, d->tokens, false).cost;
    p.dense = dense < tile;
  }
  if (!p.dense) {
    p.padded = d->tokens;
    p.splits = 1;
    set_pieces(d, p);
  }
  size_t off = 0;
  p.rows = off;
  off += align_up((size_t)p.padded * sizeof(VocabRow));
  p.last = off;
  if (p.dense && d->vocab % kTile) off += align_up((size_t)(kTile * d->d * es));
  p.xs = off;
  const int64_t copied = p.dense || d->tokens > poetx::kFewTokens
                             ? p.padded
                             : poetx::few_padded(t, (int)d->tokens);
  off += align_up((size_t)(copied * d->d * es));
  p.gz = off;
  off += align_up((size_t)(p.padded * p.ldg * es));
  p.acc = off;
  if (p.summed()) off += align_up((size_t)d->tokens * d->d * 4 * p.splits);
  p.part = off;
  if (!p.dense) {
    const size_t rest = tile_products(d, d->vocab - (p.pieces - 1) * p.piece).part_floats();
    off += align_up(std::max(tile_products(d, p.piece).part_floats(), rest) * 4);
  }
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
  const FwdPlan plan = plan_fwd(d);
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
  if (teacher && !plan.cells)
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
    const int64_t r = plan.cols.dense ? std::min(at, std::max(d->tokens - kTile, INT64_C(0))) : at;
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
                                             p.M, targets, z + r, cells[1], s));
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
  const BwdPlan plan = plan_bwd(d);
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
  const bool ragged = plan.dense && d->vocab % kTile != 0;
  poetx::VocabCopies copies;
  copies.x = x;
  copies.xs = xs;
  copies.tiled = plan.dense;
  copies.W = W;
  copies.W_last = ragged ? w + plan.last : nullptr;
  if (g_W && !plan.dense && tile_products(d, std::min(plan.piece, d->vocab)).few) {
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
    Columns split = {0, {}, 0.0f};
    if (plan.dense) split = split_columns(t, plan.padded, cols, d->d, 1.0f);
    VocabProduct p;
    p.x = xs;
    p.W = Wc;
    p.M = (int)plan.padded; p.N = (int)split.dense; p.K = (int)d->d;
    p.col0 = (int)c;
    p.scale = scale_of(d);
    if (p.N) POETX_TRY(poetx::launch_vocab_grad_dense(p, last, rows, gz, plan.ldg, s));
    if (split.dense < cols) {
      p.x = x;
      p.W = Wc + split.dense * d->d * es;
      p.M = (int)d->tokens; p.N = (int)(cols - split.dense);
      p.col0 = (int)(c + split.dense);
      POETX_TRY(poetx::launch_vocab_grad_tile(
          t, plan_tile_product(t, p.M, p.N, d->d, false, 1), p, rows,
          gz + split.dense * kTile * es, plan.ldg, plan.dense, s));
    }
    if (teacher)
      POETX_TRY(poetx::launch_vocab_listed_grad(t, list, d->tokens, rows, z, gz, plan.ldg,
                                                plan.dense, (int)c, (int)cols, s));
    if (plan.dense) {
      if (g_x)
        POETX_TRY(poetx::launch_vocab_gx_dense(
            gz, plan.ldg, Wc, last, d->tokens, (int)d->d, (int)cols,
            (int)ceil_div(cols, plan.kchunk), plan.kchunk, acc, c > 0,
            plan.summed() ? nullptr : g_x, s));
      if (g_W)
        POETX_TRY(poetx::launch_vocab_gw_dense(gz, plan.ldg, xs, ceil_div(d->tokens, 32) * 32,
                                               (int)d->d, (int)cols, gWc, s));
      continue;
    }
    const TileProducts tiles = tile_products(d, cols);
    float* part = reinterpret_cast<float*>(w + plan.part);
    TileProduct qx, qw;
    // g_x += g_z W: B(n, k) = W[k][n]
    qx.A = gz; qx.lda = plan.ldg;
    qx.B = Wc; qx.ldb = d->d;
    qx.M = (int)d->tokens; qx.N = (int)d->d; qx.K = (int)cols;
    qx.part = part;
    qx.ep.y = g_x;
    qx.ep.add = c > 0 ? acc : nullptr;
    qx.ep.sum = c + cols < d->vocab ? acc : nullptr;
    qx.ep.ld = d->d;
    // g_W = g_z^T x: A(m, k) = g_z[k][m], B(n, k) = xs[k][n]
    qw.A = gz; qw.lda = plan.ldg;
    qw.B = xs; qw.ldb = d->d;
    qw.M = (int)cols; qw.N = (int)d->d; qw.K = (int)d->tokens;
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
    POETX_TRY(poetx::launch_sum_slabs(t, acc, plan.splits, d->tokens, (int)d->d, g_x, s));
  return POETX_OK;
}

}  // namespace

extern "C" {

size_t poetx_vocab_fwd_workspace_size(const poetx_vocab_desc* d) {
  return check_desc(d) == POETX_OK ? plan_fwd(d).total : 0;
}

size_t poetx_vocab_bwd_workspace_size(const poetx_vocab_desc* d) {
  return check_desc(d) == POETX_OK ? plan_bwd(d).total : 0;
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
