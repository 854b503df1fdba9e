// What the losses over a vocabulary launch (vocab_api.cpp), and their workspaces,
// from the types and sizes alone. Host code, no HIP call.
#pragma once

#include <algorithm>

#include "kernels.h"

namespace poetx {

struct VocabSizes {
  DType t;
  int64_t tokens, d, vocab;
  int top;  // 0: cross entropy
  int64_t es() const { return t == DType::BF16 ? 2 : 4; }
  // The rows of g_z a token. One entry often makes most of a row (the target's), and its
  // rounding to bf16 shifts the whole row of g_x, and of g_W, by up to half a step; over
  // hundreds of tokens that averages to a rounding beside the result's own, over few it
  // may be 2.5 times that. There g_z has a second row, of what rounding took off the
  // first (and the products' bytes, which bound them, stay as they are).
  int parts() const { return t == DType::BF16 && tokens < kTileRows ? 2 : 1; }
  // rows of the dense products' tiled g_z
  int64_t dense_rows() const { return parts() == 2 ? pair_rows(tokens) : tokens; }
};

// Columns of the logits of `rows` rows on the 256 x 256 tiles; the rest, if any, go
// to the tile kernel: what a last round of the CUs that would be nearly empty
// holds (777 x 50001 x 2048 forward 217 -> 174 us), or what is left of the
// last tile where the copy of W's rows that it would take (`copy` us) costs more.
struct VocabColumns {
  int64_t dense;
  TilePlan tile;
  float cost;
};

// The forward, `rows` rows at a time, so that its partial sums stay small. A
// teacher's ids get their logits out of the products (`cells`, two launches'
// at most) where reading W's rows for each of them again would take longer than
// sorting them into the waves' cells and picking them out of the accumulators
// (4096 x 65536 x 2048, 64 ids a row: 116 us against 11 and about 40).
struct VocabFwdPlan {
  VocabColumns cols;
  int64_t rows, slots;
  bool copied;  // W_last
  bool cells;
  size_t z, last, part, offsets[2], entries[2], total;
};
VocabFwdPlan plan_vocab_fwd(const VocabSizes& v);

// The backward: `piece` columns of the vocabulary at a time. weight: g_W too (the
// workspace is that of the larger of the two).
struct VocabBwdPlan {
  bool dense;
  int64_t padded;       // rows of xs and gz (row-major: of each part)
  int64_t piece, pieces, ldg;
  bool few;             // g_W on the kernel for few tokens
  int splits, kchunk;   // dense: of g_x's reduction over a piece
  size_t rows, last, xs, pairs, gz, acc, part, total;
  bool two;  // rows of g_z a token
  bool summed() const { return pieces > 1 || splits > 1 || (dense && two); }
};
VocabBwdPlan plan_vocab_bwd(const VocabSizes& v, bool weight);
// of a piece's logits
VocabColumns plan_vocab_columns(const VocabSizes& v, const VocabBwdPlan& p, int64_t cols);

// g_z's two products of a piece of n columns on the tile kernel, each by itself
// or (few launches where they are what costs) in one
struct VocabProducts {
  TilePlan gx, gw;
  TilePairPlan pair;
  bool paired;
  bool few;  // g_W on its own kernel for few tokens
  size_t part_floats() const {
    const size_t alone = std::max(gx.part_floats, gw.part_floats);
    return paired ? std::max(alone, pair.gx.part_floats + pair.gw.part_floats) : alone;
  }
};
VocabProducts plan_vocab_products(const VocabSizes& v, int64_t n);

}  // namespace poetx
