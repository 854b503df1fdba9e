// The logits of a piece of the vocabulary on the tile products' main loop
// (tile_core.h), for any number of rows and columns; the logits stay in
// registers. Two ends:
//
//   forward   per row the maximum and the sum of exponentials over the wave's
//             columns: with c = log2(e) / temperature, m = max z_j and
//             s = sum 2^(c (z_j - m)). 32 lanes' worth of columns of one row lie in four
//             lanes (16 apart), so a row costs its exponentials and four
//             exchanges. (m, s) goes to part[slot][row]: nothing is read again
//             but 8 bytes for every 16 to 64 columns.
//   backward  g_z = a exp(z / temperature - lse), less b at the row's target: in x's
//             type, the operand of the two products that follow (bf16 of few tokens in
//             two parts, VocabSizes::parts()).
//
// Few rows are bound by W's bytes: 1 token, 131072 x 4096 bf16 167 us (6.4 TB/s).
// float32: 100 x 5003 x 1024 27 us, one round of workgroups; 2048 x 32000 x 2048 1.94 ms
// (138 TFLOP/s); 6508 x 80128 x 168 2.5 ms (70), where a tile's six steps are followed by
// its exponentials.
#include "tile_core.h"
#include "vocab.h"

namespace poetx {
namespace {

// fragment (f / FN, f % FN) of the accumulators, f wave-uniform (copied by name:
// as an index it would put them into memory)
template <int FM, int FN>
__device__ __forceinline__ floatx4 pick(const floatx4 (&acc)[FM][FN], int f) {
  floatx4 v{0.0f, 0.0f, 0.0f, 0.0f};
  for_each<FM * FN>([&](auto n) POETX_INLINE {
    constexpr int F = decltype(n)::value;
    if (f == F) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x;
        asm volatile("v_mov_b32 %0, %1" : "=v"(x) : "v"(acc[F / FN][F % FN][e]));
        v[e] = x;
      }
    }
  });
  return v;
}

struct LseEnd {
  static constexpr bool kBeside = true, kBlocked = true;
  float2* part;
  int64_t part_ld;
  float scale;
  const int64_t* targets;
  float* z;
  int col0;
  VocabCells cells;
  VocabList list;  // of workgroups past the tiles (`beside`): its logits, into z
  int64_t beside;
  template <typename T, int FM, int FN>
  __device__ __forceinline__ void run(const TileProduct& p, const floatx4 (&acc)[FM][FN], int m_at,
                                      int n_at, int, int wave_col, int lane) const {
    float2* out = part + (int64_t)wave_col * part_ld;
    // (a wave past the rows or columns has no cell)
    const bool listed = cells.offsets && m_at < p.M && n_at < p.N;
    OwnCell cell = {};
    if (listed) cell = read_cell(cells, m_at / (16 * FM), n_at / (16 * FN), lane);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      float v[4 * FN];
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[4 * j + e] = n_at + 16 * j + 4 * (lane >> 4) + e < p.N ? acc[i][j][e] : -INFINITY;
      const float2 ms = row_max_sum<4 * FN>(v, scale);
      const int m = m_at + 16 * i + (lane & 15);
      if (lane < 16 && m < p.M) out[m] = ms;
      if (!targets) continue;
      // the row's target, where it is among the wave's columns
      const int64_t at = m < p.M ? targets[m] - (col0 + n_at) : -1;
      if (!__any(at >= 0 && at < 16 * FN)) continue;
      const int own = at >= 0 && at < 16 * FN ? (int)at - 4 * (lane >> 4) : -1;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (own == 16 * j + e) z[m] = acc[i][j][e];
    }
    if (listed)
      store_cell(cells, cell, m_at, lane,
                 [&](int i, int j) POETX_INLINE { return pick(acc, i * FN + j); });
  }
};

struct GradEnd {
  static constexpr bool kBeside = false, kBlocked = true;
  const VocabRow* rows;
  void* gz;
  int64_t ldg;
  int tiled, col0;
  float scale;
  int64_t low;
  template <typename T, int FM, int FN>
  __device__ __forceinline__ void run(const TileProduct& p, const floatx4 (&acc)[FM][FN], int m_at,
                                      int n_at, int, int, int lane) const {
    // (the tiled layout's reductions run over whole K tiles of 32 rows, 16 of pairs)
    const int whole = low ? 15 : 31;
    const int m_end = tiled ? (p.M + whole) & ~whole : p.M, n_end = (p.N + 255) / 256 * 256;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m_at + 16 * i + (lane & 15);
      if (m >= m_end) continue;
      const VocabRow r = m < p.M ? rows[m] : VocabRow{0.0f, 0.0f, 0.0f, -1};
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = n_at + 16 * j + 4 * (lane >> 4);
        if (n >= n_end) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = n + e < p.N ? logit_gradient<T>(r, acc[i][j][e], scale, col0 + n + e) : 0.0f;
        T* out = static_cast<T*>(gz) +
                 (tiled ? tiled_offset(low ? pair_row(m) : m, n, ldg) : m * ldg + n);
        Quad<T>::store(out, v);
        if constexpr (sizeof(T) == 2) {
          if (!low) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = low_part(v[e], bf16_to_f32(f32_to_bf16(v[e])));
          Quad<T>::store(out + low, v);
        }
      }
    }
  }
};

template <typename T, int BM, int BN, int WM, int WN, int NS, typename End>
__global__ void __launch_bounds__(64 * WM * WN, 2)
vocab_tile_kernel(const TileProduct p, const End end) {
  __shared__ __attribute__((aligned(1024))) char ring[ring_bytes<T, T, BM, BN, WM * WN, NS>()];
  if constexpr (End::kBeside) {
    const int64_t tiles = (int64_t)gridDim.x - end.beside;
    if ((int64_t)blockIdx.x >= tiles) {
      listed_logits(static_cast<const T*>(p.A), static_cast<const T*>(p.B), end.list, p.M, p.K, end.z,
                    ((int64_t)blockIdx.x - tiles) * (WM * WN) + (threadIdx.x >> 6),
                    threadIdx.x & 63);
      return;
    }
  }
  tile_body<T, T, BM, BN, WM, WN, true, true, NS>(p, blockIdx.x, 0, ring, end);
}

template <typename T, int BM, int BN, int WM, int WN, int NS, typename End>
hipError_t launch_cfg(const TileProduct& p, const End& end, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  End e = end;
  int64_t grid = tiles;
  if constexpr (End::kBeside) {
    if (end.list.ids)
      e.beside = (listed_waves(p.M, end.list.top) + WM * WN - 1) / (WM * WN);
    grid += e.beside;
  }
  if (grid * 64 * WM * WN > kMaxWorkItems) return hipErrorInvalidValue;
  hipLaunchKernelGGL((vocab_tile_kernel<T, BM, BN, WM, WN, NS, End>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, s, p, e);
  return hipGetLastError();
}

// the shapes of dense_plan.cpp, with their rings as in tilegemm.hip (their waves:
// vocab_plan.cpp's tables too)
template <typename End>
hipError_t launch_end(DType t, const TilePlan& plan, const VocabProduct& v, const End& end,
                      hipStream_t s) {
  if (plan.nsplit != 1) return hipErrorInvalidValue;
  TileProduct p;
  p.A = v.x; p.lda = v.K;
  p.B = v.W; p.ldb = v.K;
  p.M = v.M; p.N = v.N; p.K = v.K;
  p.kchunk = plan.kchunk;
  if (t == DType::F32) {
    switch (plan.shape) {
      case 0: return launch_cfg<float, 64, 64, 2, 2, 4>(p, end, s);
      case 1: return launch_cfg<float, 32, 64, 1, 4, 4>(p, end, s);
    }
  } else {
    switch (plan.shape) {
      case 0: return launch_cfg<bf16_t, 256, 128, 4, 2, 3>(p, end, s);
      case 1: return launch_cfg<bf16_t, 128, 128, 2, 4, 4>(p, end, s);
      case 2: return launch_cfg<bf16_t, 128, 64, 4, 2, 4>(p, end, s);
      case 3: return launch_cfg<bf16_t, 64, 64, 2, 2, 4>(p, end, s);
      case 4: return launch_cfg<bf16_t, 32, 64, 1, 4, 6>(p, end, s);
      case 5: return launch_cfg<bf16_t, 128, 64, 4, 2, 3>(p, end, s);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_vocab_lse_tile(DType t, const TilePlan& plan, const VocabProduct& p, float2* part,
                                 int64_t part_ld, const int64_t* targets, float* z,
                                 const VocabCells& cells, const VocabList& list, hipStream_t s) {
  return launch_end(t, plan, p, LseEnd{part, part_ld, p.scale, targets, z, p.col0, cells, list, 0}, s);
}

hipError_t launch_vocab_grad_tile(DType t, const TilePlan& plan, const VocabProduct& p,
                                  const VocabRow* rows, void* gz, int64_t ldg, bool tiled,
                                  int64_t low, hipStream_t s) {
  return launch_end(t, plan, p, GradEnd{rows, gz, ldg, (int)tiled, p.col0, p.scale, low}, s);
}

}  // namespace poetx
