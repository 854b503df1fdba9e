// Which kernels the losses over a vocabulary take, their pieces and workspaces:
// estimates of times from the sizes alone. Host code, no HIP call.
#include "vocab_plan.h"

#include <algorithm>

#include "api_util.h"

namespace poetx {

using api::align_up;
using api::ceil_div;

namespace {
// rows, columns, wave rows and wave columns of a tile, by shape (launch_end in
// vocab_tile.hip)
constexpr int kBf16Tiles[][4] = {{256, 128, 4, 2}, {128, 128, 2, 4}, {128, 64, 4, 2},
                                 {64, 64, 2, 2},   {32, 64, 1, 4},   {128, 64, 4, 2}};
constexpr int kF32Tiles[][4] = {{64, 64, 2, 2}, {32, 64, 1, 4}};
const int* tile_of(DType t, const TilePlan& plan) {
  return t == DType::F32 ? kF32Tiles[plan.shape] : kBf16Tiles[plan.shape];
}
}  // namespace

int64_t vocab_tile_slots(DType t, const TilePlan& plan, int64_t N) {
  const int* h = tile_of(t, plan);
  return (N + h[1] - 1) / h[1] * h[3];
}

CellShape vocab_tile_cells(DType t, const TilePlan& plan) {
  const int* h = tile_of(t, plan);
  return CellShape{h[0] / h[2], h[1] / h[3], false};
}

int few_padded(DType t, int tokens) {
  const int k = t == DType::BF16 ? 32 : 16;
  return (tokens + k - 1) / k * k;
}

namespace {

// What the logits' pieces may take in the workspace: the forward's partial
// sums of a range of rows, the backward's gradient of a range of columns (every
// piece adds to g_x's float32 sums; 8192 x 131072 x 4096 in pieces of 128 MB 19300
// us, 256 19150, 512 18880, 1024 19100).
constexpr int64_t kPartBytes = INT64_C(128) << 20, kPieceBytes = INT64_C(512) << 20;
constexpr int64_t kTile = 256;  // rows and columns of a piece, where there is more than one

// The time (us) of `tiles` 256 x 256 tiles of the products of vocab_dense.hip
// over K: a round of the 256 CUs is 1.35 us for each 64 of K and 10 for its end
// (measured: logits 52.7 and 93 a round at K = 2048 and 4096, with their gradient
// 54.8 and 97.5, g_W 29, 101 and 194 at 1024, 4096 and 8192).
float dense_cost(int64_t tiles, int64_t K) {
  return 3.0f + (float)ceil_div(tiles, 256) * (10.0f + 1.35f * (float)K / 64);
}

VocabColumns split_columns(DType t, int64_t rows, int64_t cols, int64_t K, float copy) {
  VocabColumns best = {0, plan_tile_product(t, rows, cols, K, false, 1), 0.0f};
  best.cost = best.tile.nsplit ? best.tile.cost : 1e30f;
  if (t != DType::BF16 || !vocab_dense_supported(rows, cols, K)) return best;
  const int64_t rt = ceil_div(rows, kTile), panels = cols / kTile;
  const int64_t whole = rt * panels / 256 * 256 / rt;  // (in whole rounds)
  for (int64_t n : {ceil_div(cols, kTile), panels, whole}) {
    if (n < 1) continue;
    VocabColumns c = {std::min(n * kTile, cols), {}, dense_cost(rt * n, K)};
    if (c.dense % kTile) c.cost += copy;
    if (c.dense < cols) {
      c.tile = plan_tile_product(t, rows, cols - c.dense, K, false, 1);
      c.cost += c.tile.nsplit ? c.tile.cost : 1e30f;
    }
    if (c.cost < best.cost) best = c;
  }
  return best;
}

struct CellSizes {
  size_t offsets, entries;  // bytes
  bool possible;
};
CellSizes cell_sizes(const CellShape& c, int64_t rows, int64_t cols, int top) {
  const int64_t n = c.row_cells(rows), bins = c.bins(cols);
  return {align_up((size_t)(n * (bins + 1) * 4)), align_up((size_t)(n * c.rows * top * 4)),
          bins <= kMaxBins};
}

}  // namespace

VocabFwdPlan plan_vocab_fwd(const VocabSizes& v) {
  VocabFwdPlan p = {};
  p.rows = v.tokens;
  for (;;) {
    p.cols = split_columns(v.t, p.rows, v.vocab, v.d, 5.0f);
    p.slots = 2 * ceil_div(p.cols.dense, kTile);
    if (p.cols.dense < v.vocab)
      p.slots += p.cols.tile.nsplit
                     ? vocab_tile_slots(v.t, p.cols.tile, v.vocab - p.cols.dense)
                     : INT32_MAX;
    if (p.slots * p.rows * 8 <= kPartBytes || p.rows <= kTile) break;
    p.rows = (p.rows / 2 + kTile - 1) / kTile * kTile;
  }
  p.last = v.top ? 0 : align_up((size_t)v.tokens * 4);  // (the targets' logits)
  p.copied = p.cols.dense % kTile != 0;
  p.part = p.last + (p.copied ? align_up((size_t)(kTile * v.d) * v.es()) : 0);
  p.total = p.part + align_up((size_t)(p.slots * p.rows * 8));
  const double read = (double)v.tokens * v.top * v.d * v.es() / 9.0e6;  // us
  if (v.top && read > 20.0) {
    const int64_t rest = v.vocab - p.cols.dense;
    CellSizes c[2] = {{0, 0, true}, {0, 0, true}};
    if (p.cols.dense) c[0] = cell_sizes(vocab_dense_cells(), p.rows, p.cols.dense, v.top);
    if (rest)
      c[1] = cell_sizes(vocab_tile_cells(v.t, p.cols.tile), p.rows, rest, v.top);
    p.cells = c[0].possible && c[1].possible;
    for (int i = 0; p.cells && i < 2; ++i) {
      p.offsets[i] = p.total;
      p.entries[i] = p.offsets[i] + c[i].offsets;
      p.total = p.entries[i] + c[i].entries;
    }
  }
  return p;
}

namespace {
// a launch for the turned copy of x and one that stores g_W, by its products' steps (us a
// MB, from 131072 x 4096 bf16: 1 token 211 us, 64 275, 96 323, 128 454; rows that are not
// whole lines take longer)
float few_cost(const VocabSizes& v, int64_t n) {
  if (v.tokens > few_tokens(v.t)) return 1e30f;
  constexpr float kStep[4] = {0.191f, 0.251f, 0.295f, 0.417f};
  const int step = few_padded(v.t, (int)v.tokens) / few_padded(v.t, 1) - 1;
  const float mb = (float)n * (float)(v.d * v.es()) / 1e6f;
  const float rate = v.parts() == 2 ? kStep[step] : 0.19f + 0.0013f * v.tokens;
  return 6.0f + mb * rate * (v.d * v.es() % 128 ? 1.2f : 1.0f);
}
float gw_cost(const VocabSizes& v, int64_t n) {
  return std::min(few_cost(v, n), plan_tile_product(v.t, n, v.d, v.tokens * v.parts(), false).cost);
}
}  // namespace

VocabProducts plan_vocab_products(const VocabSizes& v, int64_t n) {
  VocabProducts p;
  const int64_t rows = v.tokens * v.parts();
  p.gx = plan_tile_product(v.t, rows, v.d, n, false, kManySplits);
  p.gw = plan_tile_product(v.t, n, v.d, rows, false);
  p.pair = plan_tile_pair(v.t, rows, v.d, n, kManySplits);
  if (v.parts() == 2)  // (summed by the join even where the reduction is whole)
    for (TilePlan* gx : {&p.gx, &p.pair.gx})
      if (gx->nsplit == 1) gx->part_floats = (size_t)(rows * v.d);
  p.few = few_cost(v, n) < std::min(p.gw.cost, std::max(p.pair.cost - p.gx.cost, 0.0f));
  p.paired = !p.few && p.pair.gx.nsplit != 0 && p.pair.cost < p.gx.cost + p.gw.cost;
  return p;
}

namespace {

void set_pieces(const VocabSizes& v, VocabBwdPlan& p) {
  const int64_t es = v.es();
  const int64_t most = std::max(kTile, kPieceBytes / (p.padded * v.parts() * es) / kTile * kTile);
  p.pieces = ceil_div(v.vocab, most);
  p.piece = p.pieces == 1 ? v.vocab : ceil_div(ceil_div(v.vocab, p.pieces), kTile) * kTile;
  p.pieces = ceil_div(v.vocab, p.piece);
  p.ldg = ceil_div(p.piece, kTile) * kTile;
}
// g_x's tiles are few where tokens and d are: its reduction, the vocabulary, is
// split so that they fill the CUs
float split_gx(const VocabSizes& v, VocabBwdPlan& p) {
  const int64_t tiles = p.padded * v.parts() / kTile * ceil_div(v.d, kTile);
  float best = 1e30f;
  for (int s = 1; s <= 128; s += s < 16 ? 1 : 8) {
    const int64_t chunk = ceil_div(ceil_div(p.piece, s), kTile) * kTile;
    const int64_t n = ceil_div(p.piece, chunk);
    // (a slab is written and read once more)
    const float cost = dense_cost(tiles * n, chunk) +
                       (n > 1 || v.parts() == 2
                            ? 3.0f + (float)(8 * n * v.dense_rows() * v.d) / 5e6f
                            : 0.0f);
    if (cost >= best) continue;
    best = cost;
    p.splits = (int)n;
    p.kchunk = (int)chunk;
  }
  return best;
}

}  // namespace

VocabBwdPlan plan_vocab_bwd(const VocabSizes& v, bool weight) {
  VocabBwdPlan p = {};
  const int64_t es = v.es();
  p.splits = 1;
  // Fewer rows than a tile's 256 are padded, from where g_W has its kernel for few
  // tokens on. (160 tokens, on tiles and padded, us: 131072 x 4096 1484, 1162, 50257 x 2048
  // 324, 305, 32000 x 4096 397, 329; W frozen 764, 678, 154, 166, 185, 190, 32000 x 1024 70, 77:
  // there the tiles' estimate is a tenth too high.)
  p.padded = ceil_div(v.tokens, kTile) * kTile;
  p.two = v.parts() == 2;
  if (v.t == DType::BF16 && v.tokens > few_tokens(v.t) &&
      vocab_dense_supported(p.padded, v.vocab, v.d)) {
    set_pieces(v, p);
    float dense = split_columns(v.t, p.padded, p.piece, v.d, 1.0f).cost + split_gx(v, p);
    float tile = plan_tile_product(v.t, v.tokens, p.piece, v.d, false, 1).cost +
                 plan_vocab_products(v, p.piece).gx.cost;
    if (weight) {
      dense += dense_cost(ceil_div(p.piece, kTile) * ceil_div(v.d, kTile), v.dense_rows());
      tile += gw_cost(v, p.piece);
    }
    if (!weight && v.tokens < kTile) tile *= 0.9f;
    p.dense = dense < tile;
  }
  if (!p.dense) {
    p.padded = v.tokens;
    p.splits = 1;
    set_pieces(v, p);
  }
  size_t off = 0;
  p.rows = off;
  off += align_up((size_t)p.padded * sizeof(VocabRow));
  p.last = off;
  if (p.dense && v.vocab % kTile) off += align_up((size_t)(kTile * v.d * es));
  p.xs = off;
  int64_t copied = p.dense ? p.padded : p.padded * v.parts();
  if (v.tokens <= few_tokens(v.t)) copied = std::max<int64_t>(copied, few_padded(v.t, (int)v.tokens));
  off += align_up((size_t)(copied * v.d * es));
  p.pairs = off;
  if (p.dense && p.two && weight) off += align_up((size_t)(2 * p.padded * v.d * es));
  p.gz = off;
  off += align_up((size_t)(p.padded * v.parts() * p.ldg * es));
  p.acc = off;
  if (p.summed())
    off += align_up((size_t)(p.dense ? v.dense_rows() : v.tokens) * v.d * 4 * p.splits);
  p.part = off;
  if (!p.dense) {
    const size_t rest = plan_vocab_products(v, v.vocab - (p.pieces - 1) * p.piece).part_floats();
    off += align_up(std::max(plan_vocab_products(v, p.piece).part_floats(), rest) * 4);
  }
  p.total = off;
  p.few = !p.dense && plan_vocab_products(v, std::min(p.piece, v.vocab)).few;
  return p;
}

VocabColumns plan_vocab_columns(const VocabSizes& v, const VocabBwdPlan& p, int64_t cols) {
  if (!p.dense)
    return {0, plan_tile_product(v.t, v.tokens, cols, v.d, false, 1), 0.0f};
  return split_columns(v.t, p.padded, cols, v.d, 1.0f);
}

}  // namespace poetx
