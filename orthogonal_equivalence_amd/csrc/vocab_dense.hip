// The four large bf16 products of the losses over a vocabulary on the 256 x 256
// tile loop of dense_core.h: the forward's logits ending in partial sums of
// exponentials, the backward's ending in the gradient g_z of the logits, and
// g_z's own products with W and x.
//
// No end stages its tile in LDS, so the ring is free as soon as the last
// products have run and the next tile's first four K tiles are copied into it
// behind the epilogue. g_z leaves as 16-byte stores straight from the
// registers: a lane holds four consecutive columns of a row of each 16 x 16
// fragment, and one v_permlane16_swap of a pair of neighbouring fragments makes
// that eight; in the tiled layout (kernels.h) the wave's 16 rows x 32 columns
// are then 1 KB of consecutive bytes. Both of g_z's products read whole
// 128-byte lines of that layout, K-major (g_x = g_z W) and M-major (g_W = g_z^T x).
#include <algorithm>

#include "dense_core.h"
#include "epilogue.h"
#include "vocab.h"

namespace poetx {
namespace {

// the panel of W's rows n0 .. n0 + 255 less n0 rows: of the vocabulary, or of the
// zero-padded copy of its last rows
__device__ __forceinline__ const bf16_t* panel(const bf16_t* W, const bf16_t* W_last, int n0, int N,
                                               int K) {
  return n0 + BN <= N ? W : W_last - (int64_t)n0 * K;
}
// The persistent loop: products, then the next tile's first copies, then
// end(m0, n0, q, nt) of this one, for the tiles of nq products side by side (their
// panels through set(q, m0, n0)). end returns whether it has issued at least
// LATE vector memory instructions, for which the next products then do not
// wait before their copies.
// What an end reads from memory is loaded by before(m0, n0, nt), ahead of the
// products, and is there at there(), behind them: a wait for a load after the next
// tile's copies would be one for the copies too (the counter is in order, and the
// compiler does not know of them).
// SHORT: reductions of fewer than the 8 K tiles that mainloop_late() takes occur.
template <int LATE, bool SHORT = false, typename D, typename Set, typename Before, typename There,
          typename End>
__device__ __forceinline__ void tile_loop(D& d, int num_mt, int num_nt, int nq, int m_last,
                                          int n_last, const Set& set, const Before& before,
                                          const There& there, const End& end) {
  const int total = num_mt * num_nt * nq;
  int tile = blockIdx.x, mt, nt, q, ntiles;
  bool late = false;
  if (tile >= total) return;
  auto go = [&]() __attribute__((always_inline)) {
    // (wave-uniform; said again where the loop's phis have lost it)
    d.lds0 = __builtin_amdgcn_readfirstlane(d.lds0);
    d.wave = __builtin_amdgcn_readfirstlane(d.wave);
    int ntb;
    xcd_grouped_tile_at(tile, total, num_mt, num_nt * nq, mt, ntb);
    q = ntb / num_nt;
    nt = ntb - q * num_nt;
    ntiles = set(q, min(mt * BM, m_last), min(nt * BN, n_last));
    d.prefetch(ntiles);
  };
  go();
  for (;;) {
    const int m0 = min(mt * BM, m_last), n0 = min(nt * BN, n_last), nt0 = nt, q0 = q;
    before(m0, n0, nt0);
    if (SHORT && ntiles < 8) {
      d.start(ntiles);
      d.mainloop(ntiles);
    } else {
      d.template start_late<LATE>(late);
      d.template mainloop_late<LATE>(ntiles, late);
    }
    d.settle();
    there();
    wait_lds();
    barrier_nofence();  // every wave is done with the ring
    tile += (int)gridDim.x;
    const bool more = tile < total;
    if (more) go();
    late = end(m0, n0, q0, nt0);
    if (!more) break;
  }
}

// (opaque: keeps the compiler from hoisting the epilogue's address arithmetic
// out of the tile loop)
template <typename D> __device__ __forceinline__ int opaque_lane(const D& d) {
  int ln = d.lane;
  asm volatile("" : "+v"(ln));
  return ln;
}

// The end of the logits' forward: for each of the wave's 128 rows the maximum and
// the sum of exponentials over its 128 columns, in two passes over the
// accumulators, so that the eight rows of a lane are exchanged together; and the
// targets' logits, which few waves hold any of.
// LISTED: `cells` in the place of targets.
// Bound by the matrix units at the clock that the chip's power leaves (a launch under the
// profiler): 8192 x 131072 x 4096 5.86 ms (1.5 PFLOP/s), units busy 74% at 1.76 GHz; 4096 x
// 65536 x 2048 with 64 listed logits a row 0.90 ms (64%), 0.86 without them.
template <bool LISTED>
__global__ void __launch_bounds__(NT)
vocab_lse_kernel(const bf16_t* __restrict__ x, const bf16_t* __restrict__ W,
                 const bf16_t* __restrict__ W_last, int M, int N, int K, float scale, int col0,
                 float2* __restrict__ part, int64_t part_ld, const int64_t* __restrict__ targets,
                 float* __restrict__ z, const VocabCells cells) {
  typedef Dense<true, true> D;
  D d;
  d.init(K, K, false, false);
  const int ntiles = K / BK;
  int64_t target[FM] = {};
  OwnCell cell = {};
  tile_loop<FM>(
      d, (M + BM - 1) / BM, (N + BN - 1) / BN, 1, M - BM, N,
      [&](int, int m0, int n0) __attribute__((always_inline)) {
        d.set_tile(x, panel(W, W_last, n0, N, K), K, K, m0, n0);
        return ntiles;
      },
      [&](int m0, int n0, int nt) __attribute__((always_inline)) {
        if constexpr (LISTED) {
          if (cells.offsets)
            cell = read_cell(cells, 2 * ((m0 + BM - 1) / BM) + d.wm, 2 * nt + d.wn, d.lane);
        } else {
#pragma unroll
          for (int i = 0; i < FM; ++i)
            target[i] = targets[m0 + d.wm * 128 + 16 * i + (d.lane & 15)];
        }
      },
      [&]() __attribute__((always_inline)) {
        if constexpr (LISTED) {
          asm volatile("" : "+v"(cell.first));
        } else {
#pragma unroll
          for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(target[i]));
        }
      },
      [&](int m0, int n0, int, int nt) __attribute__((always_inline)) {
        const int ln = opaque_lane(d);
        const int m = m0 + d.wm * 128 + (ln & 15), n = n0 + d.wn * 128;
        if (n + 128 > N) {  // (the last panel, padded)
          const int left = N - n - 4 * (ln >> 4);
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool out = 16 * j + e >= left;
#pragma unroll
              for (int i = 0; i < FM; ++i) d.acc[i][j][e] = out ? -INFINITY : d.acc[i][j][e];
              if (e == 3) d.in_agprs();
            }
        }
        d.in_agprs();
        float mx[FM], sum[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          float v = d.acc[i][0][0];
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) v = fmaxf(v, d.acc[i][j][e]);
          mx[i] = v;
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) mx[i] = quad_max(mx[i]);
        d.in_agprs();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const float at = exponent_base(mx[i]);
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[e] += __builtin_amdgcn_exp2f((d.acc[i][j][e] - at) * scale);
          sum[i] = (s[0] + s[1]) + (s[2] + s[3]);
          __builtin_amdgcn_sched_barrier(0);
        }
        float2* out = part + (int64_t)(2 * nt + d.wn) * part_ld + m;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          sum[i] = quad_sum(sum[i]);
          if (ln < 16) out[16 * i] = make_float2(mx[i], sum[i]);
        }
        if constexpr (!LISTED) {
          d.in_agprs();
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            const int64_t at = target[i] - (col0 + n);
            if (!__any(at >= 0 && at < 128)) continue;
            const int own = at >= 0 && at < 128 ? (int)at - 4 * (ln >> 4) : -1;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (own == 16 * j + e) z[m + 16 * i] = d.acc[i][j][e];
          }
        }
        if constexpr (LISTED)
          store_cell(cells, cell, m0 + d.wm * 128, ln,
                     [&](int i, int j) __attribute__((always_inline)) { return d.pick(8 * i + j); });
        return true;  // (the eight stores)
      });
}

// The end of the logits' backward. A row's target is one column of the
// vocabulary: few waves hold any, and the others only scale exponentials.
// 8192 x 32768 x 4096 1.55 ms (1.42 PFLOP/s), matrix units busy 70% at 1.89 GHz.
// g_z is rounded to bf16, the products' operand (gradients 0.0024 off, 2-norm, where the
// result's rounding alone gives 0.0017; a second part from 256 tokens on would add
// two products to three). PAIRS: what the rounding takes off g_z too, rows by pair_row().
template <bool PAIRS>
__global__ void __launch_bounds__(NT)
vocab_grad_kernel(const bf16_t* __restrict__ xs, const bf16_t* __restrict__ W,
                  const bf16_t* __restrict__ W_last, int M, int N, int K, float scale, int col0,
                  const VocabRow* __restrict__ rows, bf16_t* __restrict__ gz, int64_t ldg) {
  typedef Dense<true, true> D;
  D d;
  d.init(K, K, true, false);
  const int ntiles = K / BK;
  VocabRow row[FM];
  tile_loop<FM * FN / 2>(
      d, M / BM, (N + BN - 1) / BN, 1, M, N,
      [&](int, int m0, int n0) __attribute__((always_inline)) {
        d.set_tile(xs, panel(W, W_last, n0, N, K), K, K, m0, n0);
        return ntiles;
      },
      [&](int m0, int, int) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i) row[i] = rows[m0 + d.wm * 128 + 16 * i + (d.lane & 15)];
      },
      [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
          asm volatile("" : "+v"(row[i].a), "+v"(row[i].lse), "+v"(row[i].b), "+v"(row[i].target));
      },
      [&](int m0, int n0, int, int) __attribute__((always_inline)) {
        const int ln = opaque_lane(d);
        // (the wave's first block of 32 columns, this lane's place in it)
        constexpr int kRows = PAIRS ? 2 : 1;  // of gz a row
        bf16_t* out = gz + tiled_offset(kRows * (m0 + d.wm * 128), n0 + d.wn * 128, ldg) +
                      (ln & 15) * kTileCols + pair_column(ln);
        const int col = col0 + n0 + d.wn * 128;
        const bool padded = n0 + BN > N;
        int left = N - n0 - d.wn * 128 - 4 * (ln >> 4);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          d.in_agprs();
          const VocabRow r = row[i];
          const int own = r.target - col - 4 * (ln >> 4);  // (this lane's: 16 j + e)
          const bool rare = __any((unsigned)(r.target - col) < 128u) || padded;
          asm volatile("" : "+v"(left));
#pragma unroll
          for (int j = 0; j < FN; j += 2) {
            uint2 w[2], low[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = r.a == 0.0f ? 0.0f : r.a * softmax_at<bf16_t>(d.acc[i][j + h][e], scale, r.lse);
              if (rare) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (own == 16 * (j + h) + e) v[e] -= r.b;
                  if (16 * (j + h) + e >= left) v[e] = 0.0f;
                }
              }
              w[h] = Quad<bf16_t>::pack(v);
              if constexpr (PAIRS) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  v[e] = low_part(v[e], bf16_to_f32(f32_to_bf16(v[e])));
                low[h] = Quad<bf16_t>::pack(v);
              }
            }
            bf16_t* at = out + i * kRows * 16 * kTileCols + j / 2 * TILE;
            *reinterpret_cast<uint4*>(at) = swap_pair(w[0], w[1]);
            if constexpr (PAIRS) *reinterpret_cast<uint4*>(at + kPairLow) = swap_pair(low[0], low[1]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        return true;
      });
}

// g_x: `splits` ranges of the piece's columns (kchunk each) side by side, each
// into its own float32 slab [rows][N], added to what is there with `add`; or,
// with y, one range whose result is g_x itself.
// LAST: the piece ends inside a K tile (a choice of the source at every copy:
// 8192 x 131072 x 4096 backward 19150 us with it in every piece, 18890 without),
// or one of its ranges is shorter than 256.
// 8192 x 4096 x 32768 1.50 ms (1.47 PFLOP/s), busy 76%; LDS bank conflicts (W's rows
// read across) in 10% of the cycles.
template <bool WHOLE, bool LAST>
__global__ void __launch_bounds__(NT)
vocab_gx_kernel(const bf16_t* __restrict__ gz, const bf16_t* __restrict__ W,
                const bf16_t* __restrict__ W_last, int rows, int M, int N, int K, int64_t ldg,
                int splits, int kchunk, float* __restrict__ slabs, int add, bf16_t* __restrict__ y) {
  typedef Dense<false, false, true, false, LAST> D;
  D d;
  d.init(ldg, N, true, false);
  tile_loop<FM * FN / 2, LAST>(d, M / BM, (N + BN - 1) / BN, splits, M, N - BN,
            [&](int q, int m0, int n0) __attribute__((always_inline)) {
              // (the tiled layout's blocks of 32 columns lie one behind another)
              d.set_tile(gz + (int64_t)q * kchunk * BM, W + (int64_t)q * kchunk * N, ldg, N, m0, n0);
              const int n = min(K, (q + 1) * kchunk) - q * kchunk;
              d.last_t = n % BK ? n / BK : -1;
              d.last_b = W_last + n0;
              return (n + BK - 1) / BK;
            },
            [](int, int, int) {}, []() {},
            [&](int m0, int n0, int q, int nt) __attribute__((always_inline)) {
              const int ln = opaque_lane(d);
              const int m = m0 + d.wm * 128 + (ln & 15);
              if constexpr (WHOLE) {
                bf16_t* out = y + (int64_t)m * N + n0 + d.wn * 128 + pair_column(ln);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                  d.in_agprs();
#pragma unroll
                  for (int j = 0; j < FN; j += 2) {
                    uint2 w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const float v[4] = {d.acc[i][j + h][0], d.acc[i][j + h][1],
                                          d.acc[i][j + h][2], d.acc[i][j + h][3]};
                      w[h] = Quad<bf16_t>::pack(v);
                    }
                    const uint4 v = swap_pair(w[0], w[1]);
                    if (m + 16 * i < rows)
                      *reinterpret_cast<uint4*>(out + (int64_t)16 * i * N + 16 * j) = v;
                  }
                }
                return m0 + BM <= rows;
              }
              const int n = d.wn * 128 + 4 * (ln >> 4);
              float* out = slabs + ((int64_t)q * rows + m) * N + n0 + n;
              // (a tile shifted back repeats columns of its neighbour, which
              // are added once)
              const int first = nt * BN - n0;
#pragma unroll
              for (int i = 0; i < FM; ++i) {
                d.in_agprs();
                if (m + 16 * i < rows) {
                  float4 was[FN];
#pragma unroll
                  for (int j = 0; j < FN; ++j)
                    was[j] = add ? *reinterpret_cast<const float4*>(out + 16 * j)
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                  for (int j = 0; j < FN; ++j) {
                    if (n + 16 * j < first) continue;
                    *reinterpret_cast<float4*>(out + 16 * j) =
                        make_float4(d.acc[i][j][0] + was[j].x, d.acc[i][j][1] + was[j].y,
                                    d.acc[i][j][2] + was[j].z, d.acc[i][j][3] + was[j].w);
                  }
                }
                out += (int64_t)16 * N;
                asm volatile("" : "+v"(out));
                __builtin_amdgcn_sched_barrier(0);
              }
              return m0 + BM <= rows && first == 0;
            });
}

// g_W of the piece: both operands tiled, their rows (tokens) the reduction (256 of
// them at least). 32768 x 4096 x 8192 1.58 ms (1.39 PFLOP/s), busy 71%, bank
// conflicts in 18% of the cycles; 50001 x 2048 x 1000 0.205 ms: seven rounds for 6.1 of
// tiles, of 23 us and 6 for what is not products.
__global__ void __launch_bounds__(NT)
vocab_gw_kernel(const bf16_t* __restrict__ gz, const bf16_t* __restrict__ xs, int M, int N, int K,
                int64_t ldg, bf16_t* __restrict__ g_W) {
  typedef Dense<false, false, false, true> D;
  D d;
  d.init(ldg, N, true, true);
  const int ntiles = K / BK;
  tile_loop<FM * FN / 2>(d, (M + BM - 1) / BM, (N + BN - 1) / BN, 1, M, N - BN,
            [&](int, int m0, int n0) __attribute__((always_inline)) {
              d.set_tile(gz, xs, ldg, N, m0, n0);
              return ntiles;
            },
            [](int, int, int) {}, []() {},
            [&](int m0, int n0, int, int) __attribute__((always_inline)) {
              const int ln = opaque_lane(d);
              const int m = m0 + d.wm * 128 + (ln & 15);
              bf16_t* out = g_W + (int64_t)m * N + n0 + d.wn * 128 + pair_column(ln);
#pragma unroll
              for (int i = 0; i < FM; ++i) {
                d.in_agprs();
#pragma unroll
                for (int j = 0; j < FN; j += 2) {
                  uint2 w[2];
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const float v[4] = {d.acc[i][j + h][0], d.acc[i][j + h][1], d.acc[i][j + h][2],
                                        d.acc[i][j + h][3]};
                    w[h] = Quad<bf16_t>::pack(v);
                  }
                  const uint4 v = swap_pair(w[0], w[1]);
                  if (m + 16 * i < M)  // (gz is padded to whole tiles)
                    *reinterpret_cast<uint4*>(out + (int64_t)16 * i * N + 16 * j) = v;
                }
              }
              return m0 + BM <= M;
            });
}

constexpr int kLongK = 8 * BK;  // of mainloop_late()

const bf16_t* b16(const void* p) { return static_cast<const bf16_t*>(p); }

}  // namespace

hipError_t launch_vocab_lse_dense(const VocabProduct& p, const void* W_last, float2* part,
                                  int64_t part_ld, const int64_t* targets, float* z,
                                  const VocabCells& cells, hipStream_t s) {
  if (!vocab_dense_supported(p.M, p.N, p.K) || (p.N % BN != 0 && !W_last))
    return hipErrorInvalidValue;
  int grid = 0;
  const hipError_t e = dense_grid(p.M, p.N, &grid);
  if (e != hipSuccess) return e;
  const auto kernel = targets ? vocab_lse_kernel<false> : vocab_lse_kernel<true>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(NT), 0, s, b16(p.x), b16(p.W), b16(W_last), p.M, p.N,
                     p.K, p.scale, p.col0, part, part_ld, targets, z, cells);
  return hipGetLastError();
}

hipError_t launch_vocab_grad_dense(const VocabProduct& p, const void* W_last, const VocabRow* rows,
                                   void* gz, int64_t ldg, bool pairs, hipStream_t s) {
  if (!vocab_dense_supported(p.M, p.N, p.K) || (p.N % BN != 0 && !W_last) || p.M % BM != 0 ||
      ldg % BN != 0 || ldg < p.N)
    return hipErrorInvalidValue;
  int grid = 0;
  const hipError_t e = dense_grid(p.M, p.N, &grid);
  if (e != hipSuccess) return e;
  const auto kernel = pairs ? vocab_grad_kernel<true> : vocab_grad_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(NT), 0, s, b16(p.x), b16(p.W), b16(W_last),
                     p.M, p.N, p.K, p.scale, p.col0, rows, static_cast<bf16_t*>(gz), ldg);
  return hipGetLastError();
}

hipError_t launch_vocab_gx_dense(const void* gz, int64_t ldg, const void* W, const void* W_last,
                                 int64_t rows, int d, int cols, int splits, int kchunk,
                                 float* slabs, bool add, void* y, hipStream_t s) {
  const int64_t M = (rows + BM - 1) / BM * BM;
  if (!vocab_dense_supported(M, cols, d) || (cols % BK != 0 && !W_last) || ldg % BN != 0 ||
      ldg < cols || splits < 1 || kchunk % BK != 0 || kchunk < BK ||
      (int64_t)(splits - 1) * kchunk >= cols || (int64_t)splits * kchunk < cols ||
      (y ? splits != 1 || add : !slabs))
    return hipErrorInvalidValue;
  int grid = 0;
  const hipError_t e = dense_grid(M, (int64_t)(d + BN - 1) / BN * BN * splits, &grid);
  if (e != hipSuccess) return e;
  const bool cut = cols % BK != 0;
  const bool ragged = cut || std::min(kchunk, cols - (splits - 1) * kchunk) < kLongK;
  // (its rows from the last whole K tile on)
  const bf16_t* last = cut ? b16(W_last) + (int64_t)(cols / BK * BK % BN) * d : nullptr;
#define POETX_GX(WHOLE, LAST)                                                                  \
  hipLaunchKernelGGL((vocab_gx_kernel<WHOLE, LAST>), dim3(grid), dim3(NT), 0, s, b16(gz),      \
                     b16(W), last, (int)rows, (int)M, d, cols, ldg, splits, kchunk, slabs,     \
                     (int)add, static_cast<bf16_t*>(y))
  if (y && ragged) POETX_GX(true, true);
  else if (y) POETX_GX(true, false);
  else if (ragged) POETX_GX(false, true);
  else POETX_GX(false, false);
#undef POETX_GX
  return hipGetLastError();
}

hipError_t launch_vocab_gw_dense(const void* gz, int64_t ldg, const void* xs, int64_t padded, int d,
                                 int cols, void* g_W, hipStream_t s) {
  if (!vocab_dense_supported(256, cols, d) || ldg % BN != 0 || ldg < cols || padded % BK != 0 ||
      padded < kLongK)
    return hipErrorInvalidValue;
  int grid = 0;
  const hipError_t e = dense_grid(cols, d, &grid);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(vocab_gw_kernel, dim3(grid), dim3(NT), 0, s, b16(gz), b16(xs), cols, d,
                     (int)padded, ldg, static_cast<bf16_t*>(g_W));
  return hipGetLastError();
}

}  // namespace poetx
