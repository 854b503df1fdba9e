// Matrix products of the dense linear with its epilogue, for any number of
// rows: one workgroup of four or eight waves computes a BM x BN tile of
//   C(m, n) = sum_k A(m, k) B(n, k),
//   A(m, k) = A[m lda + k] (K-major) or A[k lda + m] (M-major), B likewise,
// and ends with the float32 accumulators in registers, so that scale, bias,
// activation and residual cost no pass of their own (epilogue.h). With a
// split reduction axis each workgroup leaves its float32 partial tile in the
// workspace and finish_kernel sums them in split order and applies the
// epilogue.
// The main loop is tile_core.h's.
#include <algorithm>

#include "tile_core.h"

namespace poetx {
namespace {

constexpr int NT = 256;

// the plain end: the epilogue, or a split's partial tile
template <bool BLOCKED> struct StoreEnd {
  static constexpr bool kBlocked = BLOCKED;
  template <typename T, int FM, int FN>
  __device__ __forceinline__ void run(const TileProduct& p, const floatx4 (&acc)[FM][FN], int m_at,
                                      int n_at, int part_k, int, int lane) const {
    float* part = p.part ? p.part + (int64_t)part_k * p.M * p.N : nullptr;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m_at + 16 * i + (lane & 15);
      if (m >= p.M) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = n_at + 16 * j + 4 * (lane >> 4);
        if (n >= p.N) continue;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if (part) Quad<float>::store(part + (int64_t)m * p.N + n, v);
        else epilogue4<T>(p.ep, m, n, v);
      }
    }
  }
};

template <typename T, typename TB, int BM, int BN, int WM, int WN, bool A_KMAJ, bool B_KMAJ, int NS,
          bool BLOCKED = false>
__global__ void __launch_bounds__(64 * WM * WN, 2) tile_kernel(const TileProduct p) {
  __shared__ __attribute__((aligned(1024))) char ring[ring_bytes<T, TB, BM, BN, WM * WN, NS>()];
  tile_body<T, TB, BM, BN, WM, WN, A_KMAJ, B_KMAJ, NS>(p, blockIdx.x, blockIdx.y, ring,
                                                      StoreEnd<BLOCKED>{});
}

// The backward's two products, which are independent, in one launch: g_x = g_u
// W (gx: A K-major, B N-major) and g_W = g_u^T x (gw: both M-, N-major). The
// product with the longer reduction comes first, so that its tiles do not
// start last. padded: its workgroups, rounded up to the 8 XCDs (the ones past
// its tiles return at once).
template <typename T, int BM, int BN, int WM, int WN, int NS, bool BLOCKED>
__global__ void __launch_bounds__(64 * WM * WN, 2)
tile_pair_kernel(const TileProduct gx, const TileProduct gw, int gx_tiles, int gw_tiles, int gx_wgs,
                 int gw_wgs, int padded, int gx_first) {
  __shared__ __attribute__((aligned(1024))) char ring[ring_bytes<T, T, BM, BN, WM * WN, NS>()];
  const bool first = (int)blockIdx.x < padded;
  const int wg = first ? blockIdx.x : blockIdx.x - padded;
  if (first == (gx_first != 0)) {
    if (wg >= gx_wgs) return;
    tile_body<T, T, BM, BN, WM, WN, true, false, NS>(gx, wg % gx_tiles, wg / gx_tiles, ring,
                                                     StoreEnd<BLOCKED>{});
  } else {
    if (wg >= gw_wgs) return;
    tile_body<T, T, BM, BN, WM, WN, false, false, NS>(gw, wg % gw_tiles, wg / gw_tiles, ring,
                                                      StoreEnd<BLOCKED>{});
  }
}

// sum of the partial tiles in split order, then the epilogue; four columns a
// thread. PAIRS: the tiles' rows are pair_row()'s.
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(NT)
finish_kernel(const float* __restrict__ part, int nsplit, int64_t rows, int64_t stride, int N,
              Epilogue ep) {
  const int quads = N / 4;
  const int64_t total = rows * quads;
  for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < total; i += (int64_t)gridDim.x * NT) {
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* p = part + (PAIRS ? pair_row(m) : m) * N + n;
    int s = 0;
    if constexpr (PAIRS) {
      for (; s < nsplit; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[4];
          Quad<float>::load(p + s * stride + (int64_t)16 * h * N, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += w[e];
        }
    }
    for (; s + 4 <= nsplit; s += 4) {  // four loads in flight
      float w[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) Quad<float>::load(p + (s + q) * stride, w[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += w[q][e];
    }
    for (; s < nsplit; ++s) {
      float w[4];
      Quad<float>::load(p + s * stride, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += w[e];
    }
    epilogue4<T>(ep, m, n, v);
  }
}

// NS, NS8: ring depth, and with INT8 codes. The step of 32 x 64 tiles is short
// against a load's latency. bf16 six deep against four, 16 tokens of 14336 x
// 4096 (d_in x d_out) 27.0 us against 29.1, 4096 x 14336 28.2 against 29.5, 4096
// x 4096 11.6 against 12.3, but 2048 x 2048 7.7 against 7.4 and 1008 x 5000 6.6
// against 6.2; 9, 30 and 60 tokens alike. INT8 codes, half the bytes a step and
// more work on them, four deep against six: 20.9 against 22.2, 23.9 against
// 22.8, 11.7 against 12.2, 7.9 against 7.9, 7.5 against 8.3.
template <typename T, int BM, int BN, int WM, int WN, int NS, int NS8 = NS>
hipError_t launch_cfg(bool ak, bool bk, const TileProduct& p, int nsplit, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  if (nsplit < 1 || tiles * 64 * WM * WN > kMaxWorkItems) return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, nsplit), block(64 * WM * WN);
  if (p.b_int8) {
    // (64 bytes a row and step: a shape whose waves each copy some of them)
    if constexpr (sizeof(T) == 2 && BN * 64 >= 1024 * WM * WN) {
      if (ak && bk && p.K % 16 == 0) {
        hipLaunchKernelGGL((tile_kernel<T, int8_t, BM, BN, WM, WN, true, true, NS8>), grid, block,
                           0, s, p);
        return hipGetLastError();
      }
    }
    return hipErrorInvalidValue;
  }
  if constexpr (sizeof(T) == 4) {
    if (p.blocked) {
      if (bk) return hipErrorInvalidValue;  // (no caller)
      const auto kernel = ak ? tile_kernel<T, T, BM, BN, WM, WN, true, false, NS, true>
                             : tile_kernel<T, T, BM, BN, WM, WN, false, false, NS, true>;
      hipLaunchKernelGGL(kernel, grid, block, 0, s, p);
      return hipGetLastError();
    }
  }
  if (ak && bk)
    hipLaunchKernelGGL((tile_kernel<T, T, BM, BN, WM, WN, true, true, NS>), grid, block, 0, s, p);
  else if (ak)
    hipLaunchKernelGGL((tile_kernel<T, T, BM, BN, WM, WN, true, false, NS>), grid, block, 0, s, p);
  else if (!bk)
    hipLaunchKernelGGL((tile_kernel<T, T, BM, BN, WM, WN, false, false, NS>), grid, block, 0, s, p);
  else
    return hipErrorInvalidValue;  // no caller has an M-major A with a K-major B
  return hipGetLastError();
}

template <typename T, int BM, int BN, int WM, int WN, int NS>
hipError_t launch_pair_cfg(const TileProduct& gx, int gx_split, const TileProduct& gw, int gw_split,
                           hipStream_t s) {
  const int64_t tx = (int64_t)((gx.M + BM - 1) / BM) * ((gx.N + BN - 1) / BN);
  const int64_t tw = (int64_t)((gw.M + BM - 1) / BM) * ((gw.N + BN - 1) / BN);
  const bool gx_first = gx.kchunk >= gw.kchunk;
  const int64_t first = gx_first ? tx * gx_split : tw * gw_split;
  const int64_t padded = (first + 7) / 8 * 8;
  const int64_t grid = padded + (gx_first ? tw * gw_split : tx * gx_split);
  if (gx_split < 1 || gw_split < 1 || grid * 64 * WM * WN > kMaxWorkItems)
    return hipErrorInvalidValue;
  const auto kernel = sizeof(T) == 4 && gx.blocked
                          ? tile_pair_kernel<T, BM, BN, WM, WN, NS, sizeof(T) == 4>
                          : tile_pair_kernel<T, BM, BN, WM, WN, NS, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, gx, gw, (int)tx, (int)tw,
                     (int)(tx * gx_split), (int)(tw * gw_split), (int)padded, (int)gx_first);
  return hipGetLastError();
}

// joins a split product's partial tiles
hipError_t join(DType t, int nsplit, const TileProduct& p, bool pairs, hipStream_t s) {
  const int64_t groups = (int64_t)p.M * (p.N / 4);
  const int grid = (int)std::min<int64_t>((groups + NT - 1) / NT, 4096);
  const int64_t stride = (pairs ? pair_rows(p.M) : (int64_t)p.M) * p.N;
  const auto kernel = t == DType::F32 ? finish_kernel<float, false>
                      : pairs         ? finish_kernel<bf16_t, true>
                                      : finish_kernel<bf16_t, false>;
  if (pairs && t == DType::F32) return hipErrorInvalidValue;  // (no caller)
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(NT), 0, s, p.part, nsplit, (int64_t)p.M, stride, p.N,
                     p.ep);
  return hipGetLastError();
}

hipError_t finish(DType t, const TilePlan& plan, TileProduct p, hipStream_t s) {
  // (a partial tile of two halves is two partial tiles of the output)
  p.M /= p.halves;
  const int parts = plan.nsplit * p.halves;
  return parts == 1 ? hipSuccess : join(t, parts, p, false, s);
}

// p as `plan` has it; false: a split without room for its partial tiles
bool apply_plan(const TilePlan& plan, TileProduct& p) {
  p.kchunk = plan.kchunk;
  const bool whole = plan.nsplit == 1 && p.halves == 1;
  if (whole) p.part = nullptr;
  return (whole || p.part) && p.M % p.halves == 0;
}

}  // namespace

hipError_t launch_sum_slabs(DType t, const float* slabs, int nsplit, int64_t rows, int N, void* out,
                            bool pairs, hipStream_t s) {
  TileProduct p;
  p.M = (int)rows; p.N = N;
  p.part = const_cast<float*>(slabs);
  p.ep.y = out;
  p.ep.ld = N;
  return join(t, nsplit, p, pairs, s);
}

hipError_t launch_tile_pair(DType t, const TilePairPlan& plan, TileProduct gx, TileProduct gw,
                            hipStream_t s) {
  if (!apply_plan(plan.gx, gx) || !apply_plan(plan.gw, gw) || plan.gx.shape != plan.gw.shape)
    return hipErrorInvalidValue;
  const int sx = plan.gx.nsplit, sw = plan.gw.nsplit;
  hipError_t e = hipErrorInvalidValue;
  if (t == DType::F32) {
    switch (plan.gx.shape) {  // kF32Shapes (dense_plan.cpp)
      case 0: e = launch_pair_cfg<float, 64, 64, 2, 2, 4>(gx, sx, gw, sw, s); break;
      case 1: e = launch_pair_cfg<float, 32, 64, 1, 4, 4>(gx, sx, gw, sw, s); break;
    }
  } else {
    switch (plan.gx.shape) {  // kBf16Shapes (dense_plan.cpp)
      case 1: e = launch_pair_cfg<bf16_t, 128, 128, 2, 4, 4>(gx, sx, gw, sw, s); break;
      case 3: e = launch_pair_cfg<bf16_t, 64, 64, 2, 2, 4>(gx, sx, gw, sw, s); break;
      case 4: e = launch_pair_cfg<bf16_t, 32, 64, 1, 4, 6>(gx, sx, gw, sw, s); break;
      case 5: e = launch_pair_cfg<bf16_t, 128, 64, 4, 2, 3>(gx, sx, gw, sw, s); break;
    }
  }
  if (e == hipSuccess) e = finish(t, plan.gx, gx, s);
  return e == hipSuccess ? finish(t, plan.gw, gw, s) : e;
}

hipError_t launch_tile_product(DType t, const TilePlan& plan, TileProduct p, bool a_kmajor,
                               bool b_kmajor, hipStream_t s) {
  if (!apply_plan(plan, p)) return hipErrorInvalidValue;
  hipError_t e = hipErrorInvalidValue;
  if (t == DType::F32) {
    switch (plan.shape) {  // kF32Shapes (dense_plan.cpp)
      case 0: e = launch_cfg<float, 64, 64, 2, 2, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 1: e = launch_cfg<float, 32, 64, 1, 4, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
    }
  } else {
    switch (plan.shape) {  // kBf16Shapes (dense_plan.cpp)
      case 0: e = launch_cfg<bf16_t, 256, 128, 4, 2, 3>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 1: e = launch_cfg<bf16_t, 128, 128, 2, 4, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 2: e = launch_cfg<bf16_t, 128, 64, 4, 2, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 3: e = launch_cfg<bf16_t, 64, 64, 2, 2, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 4: e = launch_cfg<bf16_t, 32, 64, 1, 4, 6, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
      case 5: e = launch_cfg<bf16_t, 128, 64, 4, 2, 3>(a_kmajor, b_kmajor, p, plan.nsplit, s); break;
    }
  }
  return e == hipSuccess ? finish(t, plan, p, s) : e;
}

}  // namespace poetx
