// Which kernel, tile shape and split of the reduction a dense linear's products
// take: estimates of their times from the sizes alone. Host code, no HIP call.
#include "dense_plan.h"

#include <algorithm>

#include "api_util.h"

namespace poetx {

using api::ceil_div;

namespace {

// The tile shapes: workgroups that fit a CU, what one step of 128 bytes of k
// costs there (us) with one of them on it and with all, and what a workgroup
// costs beside its steps (the first loads, the last products, the epilogue).
// These and the constants below are fitted to the times of 600 random
// products on an MI355X under every shape and split (9 .. 4096 tokens, widths
// 128 .. 14336) and 250 of a model's sizes: the estimates are within 11% (one
// standard deviation), and the plans chosen by them cost 1.0 to 1.2% (forward)
// and 2.3% (backward pair) more than the best plan of each product, on average
// over others like them. Without the fixed costs, which decide the short
// reductions of g_W at few tokens, 5 and 9%, up to 1.9 times.
struct Shape {
  int bm, bn, threads, per_cu;
  float alone, full, fixed;
  bool int8;  // B may be INT8 codes
};
constexpr Shape kBf16Shapes[] = {{256, 128, 512, 1, 0.83f, 0.83f, 6.3f, true},
                                 {128, 128, 512, 1, 0.50f, 0.50f, 3.5f, true},
                                 {128, 64, 512, 1, 0.37f, 0.37f, 3.0f, false},
                                 {64, 64, 256, 2, 0.25f, 0.455f, 2.55f, true},
                                 {32, 64, 256, 2, 0.19f, 0.37f, 2.0f, true},
                                 // in a ring of three steps, which leaves
                                 // room for two: 422 x 2248 x 1440 backward
                                 // 21.7 -> 16.4 us, 232 x 5216 x 2776 51.8 ->
                                 // 39.0; 2714 x 128 x 5376 forward 27.2 ->
                                 // 22.5; but 777 x 2048 x 2048, one on a CU,
                                 // 19.2 against 15.3 in a ring of four
                                 {128, 64, 512, 2, 0.42f, 0.70f, 2.1f, false}};
constexpr int kPairFirst = 1;  // (256 x 128: large products, which fill the chip)
constexpr int kOneOn = 2;      // 128 x 64, one on a CU: no pair takes it
constexpr int kTwoOn = 5;      // and two: only where there are two
// float32 is bound by its matrix rate (a 64 x 64 step is 1024 cycles of it),
// so small shapes, which fill the chip most evenly, serve all sizes
constexpr Shape kF32Shapes[] = {{64, 64, 256, 2, 0.59f, 0.95f, 2.8f, false},
                                {32, 64, 256, 3, 0.275f, 0.76f, 1.7f, false}};
int64_t tiles_of(const Shape& h, int64_t M, int64_t N) {
  return ((M + h.bm - 1) / h.bm) * ((N + h.bn - 1) / h.bn);
}
constexpr int kCus = 256;
// (above kFewSplits: only where a caller allows them, for long reductions
// into small outputs)
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
static_assert(kSplits[7] == kFewSplits, "the default of max_split");
constexpr int kMinSteps = 4;               // of a split's part
constexpr float kInt8Step = 1.4f;          // a step with B's codes widened
constexpr float kLaunch = 2.1f;            // us of a launch
constexpr float kFinish = 2.75f;           // and of the pass that joins the partial tiles
constexpr float kPartBytesPerUs = 6.75e6f; // which are written and read near the cores
constexpr float kHbmBytesPerUs = 6.2e6f;
// operands that come from HBM rather than a cache lengthen the steps by about
// this share of their transfer time
constexpr float kCold = 0.38f;

}  // namespace

// Every shape and a few splits of the reduction, by rounds of workgroups
// times steps times the step's cost, the operands' transfer and the partial
// tiles'. What it decides, measured: 777 x 2048 x 2048 128 x 64 tiles 15.1 us,
// 64 x 64 16.8, 128 x 128 21.0; 1024 x 4096 x 4096 39 us on 128 x 128, 53 on
// 128 x 64, 56 on 256 x 128; 2048 x 4096 x 4096 69 us on 256 x 128, 75 on 128
// x 128; 16 x 4096 x 14336 26.7 us on 32 x 64, 28.7 on 64 x 64; 16 x 14336 x
// 4096 25.3 us on 32 x 64 in 8 splits, 27.0 in 4, 32.0 in 3.
TilePlan plan_tile_product(DType t, int64_t M, int64_t N, int64_t K, bool b_int8, int max_split) {
  const bool bf16 = t == DType::BF16;
  const Shape* shapes = bf16 ? kBf16Shapes : kF32Shapes;
  const int nshapes = (int)((bf16 ? sizeof(kBf16Shapes) : sizeof(kF32Shapes)) / sizeof(Shape));
  const int bk = bf16 ? 64 : 32, es = bf16 ? 2 : 4;
  const int steps = (int)((K + bk - 1) / bk);
  const float hbm = (float)(M * K * es + N * K * (b_int8 ? 1 : es)) / kHbmBytesPerUs;
  TilePlan best = {};
  best.cost = 1e30f;
  for (int i = 0; i < nshapes; ++i) {
    const Shape& h = shapes[i];
    if (b_int8 && !h.int8) continue;
    const int64_t tiles = tiles_of(h, M, N);
    if (tiles * h.threads > kMaxWorkItems) continue;
    const int64_t slots = (int64_t)kCus * h.per_cu;
    for (int want : kSplits) {
      if (want > max_split) break;
      const int per = (steps + want - 1) / want, split = (steps + per - 1) / per;
      // (28 x 2560 x 256 in 8 splits of five steps 6.8 us, in 4 7.9; none is
      // made of tiles that fill the chip anyway)
      if (split != want || (split > 1 && (per < kMinSteps || tiles >= slots))) continue;
      const int64_t wgs = tiles * split, rest = wgs % slots;
      if (bf16 && i == kTwoOn && wgs <= kCus) continue;
      float rounds = (float)(wgs / slots), step = rounds * h.full;
      if (rest) {
        rounds += 1.0f;
        step += h.per_cu == 1 ? h.full
                              : h.alone + (h.full - h.alone) * (float)((rest - 1) / kCus) /
                                              (float)(h.per_cu - 1);
      }
      const float busy = step * (float)per * (b_int8 ? kInt8Step : 1.0f) + rounds * h.fixed;
      float cost = kLaunch + std::max(busy + kCold * hbm, hbm);
      if (split > 1) cost += kFinish + (float)(2 * split * M * N * 4) / kPartBytesPerUs;
      if (cost < best.cost)
        best = TilePlan{i, split, per * bk, split > 1 ? (size_t)split * M * N : 0, cost};
    }
  }
  return best;
}

// The two products of a backward in one launch: for each shape and pair of
// splits, the steps of both over the chip, or the longer one's chain if that
// is more, by the same constants.
TilePairPlan plan_tile_pair(DType t, int64_t tokens, int64_t d_in, int64_t d_out, int max_split) {
  const bool bf16 = t == DType::BF16;
  const Shape* shapes = bf16 ? kBf16Shapes : kF32Shapes;
  const int nshapes = (int)((bf16 ? sizeof(kBf16Shapes) : sizeof(kF32Shapes)) / sizeof(Shape));
  const int bk = bf16 ? 64 : 32, es = bf16 ? 2 : 4;
  const int64_t M[2] = {tokens, d_out}, N = d_in, K[2] = {d_out, tokens};
  const float hbm = (float)((2 * tokens * d_in + tokens * d_out + 2 * d_in * d_out) * es) /
                    kHbmBytesPerUs;
  TilePairPlan best = {};
  best.cost = 1e30f;
  constexpr int kNumSplits = (int)(sizeof(kSplits) / sizeof(kSplits[0]));
  for (int i = bf16 ? kPairFirst : 0; i < nshapes; ++i) {
    if (bf16 && i == kOneOn) continue;
    const Shape& h = shapes[i];
    const float slots = (float)(kCus * h.per_cu);
    struct Option {
      int split, per;
      float work, extra;  // us of the whole chip; of joining the parts
    } opt[2][kNumSplits];
    int nopt[2] = {0, 0};
    for (int q = 0; q < 2; ++q) {
      const int64_t tiles = tiles_of(h, M[q], N);
      const int steps = (int)((K[q] + bk - 1) / bk);
      for (int want : kSplits) {
        if (want > max_split) break;
        const int per = (steps + want - 1) / want, split = (steps + per - 1) / per;
        if (split != want || (split > 1 && (per < kMinSteps || tiles >= (int64_t)slots))) continue;
        const float extra =
            split > 1 ? kFinish + (float)(2 * split * M[q] * N * 4) / kPartBytesPerUs : 0.0f;
        opt[q][nopt[q]++] = Option{
            split, per, (float)(tiles * split) * ((float)per * h.full + h.fixed) / slots, extra};
      }
    }
    for (int x = 0; x < nopt[0]; ++x) {
      for (int w = 0; w < nopt[1]; ++w) {
        const Option &ox = opt[0][x], &ow = opt[1][w];
        // (7: the first product's workgroups, rounded up to the XCDs)
        if ((tiles_of(h, M[0], N) * ox.split + 7 + tiles_of(h, M[1], N) * ow.split) * h.threads >
            kMaxWorkItems)
          continue;
        // (the chip full throughout, and half a short workgroup's time of tail)
        const float busy =
            std::max(ox.work + ow.work + 0.44f * (float)std::min(ox.per, ow.per) * h.alone,
                     (float)std::max(ox.per, ow.per) * h.alone + h.fixed);
        const float cost = kLaunch + busy + kCold * hbm + ox.extra + ow.extra;
        if (cost >= best.cost) continue;
        best.cost = cost;
        best.gx = TilePlan{i, ox.split, ox.per * bk,
                           ox.split > 1 ? (size_t)ox.split * M[0] * N : 0, 0.0f};
        best.gw = TilePlan{i, ow.split, ow.per * bk,
                           ow.split > 1 ? (size_t)ow.split * M[1] * N : 0, 0.0f};
      }
    }
  }
  return best;
}

namespace {

// The dense kernel's time for an M x N x K product, as the tile kernel's plan
// estimates its own: rounds of 256 x 256 tiles over the CUs (1.38 us a round
// and 64 of k, 6 us for a round's epilogue). One estimate for the forward's
// paired copies and g_x's plain ones; without activation, measured and (estimated):
// 4096 x 4096 x 4096 forward 104 us, g_x 103 (97); 8192 x 14336 x 4096 674 (663),
// its g_x 665 (633); 2048 x 8192 x 2048 57 (53); 4096 x 4096 x 1024 36 (31).
float dense_cost(int64_t M, int64_t N, int64_t K) {
  const int64_t rounds = ceil_div(ceil_div(M, 256) * ceil_div(N, 256), 256);
  return 3.0f + (float)rounds * (1.38f * (float)K / 64 + 6.0f);
}
// Whether an M x N product of K-major A takes that kernel.
bool use_dense(DType t, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
               const TilePlan& tile) {
  return t == DType::BF16 && dense_supported(M, N, K, lda, ldb, ldc) &&
         dense_cost(M, N, K) < tile.cost;
}
constexpr float kWidenLaunch = 3.0f, kWidenBytesPerUs = 4.5e6f;

}  // namespace

FwdChoice choose_fwd(DType t, bool int8, int64_t tokens, int64_t d_in, int64_t d_out) {
  FwdChoice p = {};
  // few tokens: the weight read once, straight into the products
  p.stream = tokens <= kStreamRows && !(int8 && t == DType::F32);
  if (p.stream) return p;
  const int64_t M = tokens, N = d_out, K = d_in;
  p.tile = plan_tile_product(t, M, N, K, false);
  p.dense = use_dense(t, M, N, K, K, K, N, p.tile);
  p.widen = int8;
  if (int8 && t == DType::BF16 && K % 16 == 0) {
    // the tile kernel can take the codes themselves: worth it while widening
    // them (a byte read, two written) costs more than the products gain
    const TilePlan direct = plan_tile_product(t, M, N, K, true);
    const float widened = (p.dense ? dense_cost(M, N, K) : p.tile.cost) + kWidenLaunch +
                          (float)(3 * N * K) / kWidenBytesPerUs;
    if (direct.cost < widened) {
      p.tile = direct;
      p.dense = p.widen = false;
    }
  }
  p.w_tiled = p.dense && p.widen && N % kTileRows == 0;
  return p;
}

BwdChoice choose_bwd(DType t, bool int8, int64_t tokens, int64_t d_in, int64_t d_out) {
  BwdChoice p = {};
  const int64_t M = tokens, N = d_in, K = d_out;
  p.gx = plan_tile_product(t, M, N, K, false);
  p.dense = use_dense(t, M, N, K, K, N, N, p.gx);
  if (p.dense) {
    p.gx.part_floats = 0;
    p.gx.cost = dense_cost(M, N, K);
  }
  p.gw = plan_tile_product(t, K, N, M, false);
  p.pair = plan_tile_pair(t, M, N, K);
  p.paired = !int8 && p.pair.gx.nsplit != 0 && p.pair.cost < p.gx.cost + p.gw.cost;
  return p;
}

}  // namespace poetx
