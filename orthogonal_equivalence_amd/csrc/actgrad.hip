// The elementwise half of the dense linear's backward and its bias gradient
// in one pass over the token-major gradient:
//   g_u = g_y act'(u),  g_bias[n] = sum over tokens of g_u,
// and with an INT8 weight diag(s) q the product's operand g_u diag(s).
// Memory bound: g_y and u are read once, g_u written once.
//
// A workgroup takes 32 column vectors of 16 bytes (256 bf16 or 128 float32
// columns) and one range of rows, eight rows at a time; each thread sums its
// column vector in float32 over an eighth of it, the eight row lanes are joined
// in LDS, in float32 too, and the ranges' sums by bias_reduce_kernel in float64,
// in range order: no atomics, the same bits every time. A range is 32 rows (up
// to 64 rows are one, whose float32 sum is g_bias; past 2^20 rows ranges grow,
// to 2^15 rows at 2^30). The sums take the unrounded g_u.
#include <algorithm>

#include "common.h"
#include "epilogue.h"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int NT = 256, kVecs = 32, kLanes = NT / kVecs;
// rows of one range: four a thread, all of whose loads are in flight at once
// (two a thread and twice the ranges: 4.6 us against 4.8 for g_bias of 1000 x
// 2048 gelu, with a longer join); more only where the ranges would pass the
// grid's limit
constexpr int kRows = 4 * kLanes, kMaxSplits = 32768;
// so few rows are one range, whose sums are the bias gradient itself: one
// launch less where launches are what costs (g_bias of d = 2048 silu, in one
// range against ranges of 32: bf16 48 rows 4.1 us against 5.3, 64 rows 4.5
// against 5.4, 96 rows 5.7 against 5.5, 128 rows 6.9 against 5.5; float32 64
// rows 5.3 against 5.7, 96 rows 6.8 against 5.7; d = 256 and 8192 alike)
constexpr int kOneRange = 64;
int rows_per_split(int64_t rows) {
  if (rows <= kOneRange) return (int)rows;
  return (int)(kRows * ((rows + (int64_t)kRows * kMaxSplits - 1) / ((int64_t)kRows * kMaxSplits)));
}

template <typename T> struct Vec;  // one 16-byte vector as float32
template <> struct Vec<bf16_t> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const bf16_t* p, float v[8]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(bf16_t* p, const float v[8]) {
    union { bf16_t h[8]; uint4 w; } o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.h[e] = f32_to_bf16(v[e]);
    *reinterpret_cast<uint4*>(p) = o.w;
  }
};
template <> struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const float* p, float v[4]) { Quad<float>::load(p, v); }
  static __device__ __forceinline__ void store(float* p, const float v[4]) { Quad<float>::store(p, v); }
};

// g_u may be null (only the column sums are wanted), part too (no bias
// gradient); a whole pass over `rows` in one range writes g_bias itself.
template <typename T, Activation ACT>
__global__ void __launch_bounds__(NT)
act_grad_kernel(const T* __restrict__ g_y, const T* __restrict__ u, const float* __restrict__ scale,
                T* __restrict__ g_u, float* __restrict__ part, int64_t rows, int d,
                int rows_per_split, int gu_tiled) {
  constexpr int E = Vec<T>::E;
  const int vec = threadIdx.x & (kVecs - 1), lane = threadIdx.x / kVecs;
  const int n = (blockIdx.x * kVecs + vec) * E;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_split;
  const int64_t r1 = min(rows, r0 + rows_per_split);
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.0f;
  if (n < d) {
    float sc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sc[e] = scale ? scale[n + e] : 1.0f;
    for (int64_t r = r0 + lane; r < r1; r += 4 * kLanes) {
      float g[4][E], w[4][E];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (rows past the range are read as its last one and left out below)
        const int64_t at = min(r + q * kLanes, r1 - 1) * d + n;
        Vec<T>::load(g_y + at, g[q]);
        if constexpr (ACT != Activation::None) Vec<T>::load(u + at, w[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t rq = r + q * kLanes;
        if (rq >= r1) break;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (ACT != Activation::None)
            g[q][e] = activation_gradient<T, ACT>(g[q][e], w[q][e]);
          sum[e] += g[q][e];
          g[q][e] *= sc[e];
        }
        if (g_u) Vec<T>::store(g_u + (gu_tiled ? tiled_offset(rq, n, d) : rq * d + n), g[q]);
      }
    }
  }
  if (!part) return;
  __shared__ float s[kLanes][kVecs * E + 4];
#pragma unroll
  for (int e = 0; e < E; ++e) s[lane][vec * E + e] = sum[e];
  __syncthreads();
  const int col = threadIdx.x, nn = blockIdx.x * kVecs * E + col;
  if (col < kVecs * E && nn < d) {
    float t = 0.0f;
#pragma unroll
    for (int l = 0; l < kLanes; ++l) t += s[l][col];
    part[(int64_t)blockIdx.y * d + nn] = t;
  }
}

// 64 columns a workgroup; its four waves take every fourth range, eight loads
// in flight each, and are joined in wave order
__global__ void __launch_bounds__(NT)
bias_reduce_kernel(const float* __restrict__ part, int nsplit, int d, float* __restrict__ g_bias) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + lane;
  double t = 0.0;
  if (n < d) {
    const float* p = part + n;
    for (int s = wave; s < nsplit; s += 32) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = p[(int64_t)min(s + 4 * q, nsplit - 1) * d];
#pragma unroll
      for (int q = 0; q < 8; ++q) t += s + 4 * q < nsplit ? (double)v[q] : 0.0;
    }
  }
  __shared__ double sums[NT / 64][64];
  sums[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && n < d)
    g_bias[n] = (float)(((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane]);
}

template <typename T>
hipError_t launch_typed(const ActGrad& a, float* part, hipStream_t s) {
  const dim3 grid((a.d / Vec<T>::E + kVecs - 1) / kVecs, act_grad_splits(a.rows));
#define POETX_ACT_GRAD(A)                                                                     \
  case Activation::A:                                                                         \
    hipLaunchKernelGGL((act_grad_kernel<T, Activation::A>), grid, dim3(NT), 0, s,             \
                       static_cast<const T*>(a.g_y), static_cast<const T*>(a.u), a.scale,     \
                       static_cast<T*>(a.g_u), part, a.rows, a.d, rows_per_split(a.rows),     \
                       (int)a.gu_tiled);                                                     \
    break;
  switch (a.act) {
    POETX_ACT_GRAD(None)
    POETX_ACT_GRAD(Relu)
    POETX_ACT_GRAD(Gelu)
    POETX_ACT_GRAD(GeluTanh)
    POETX_ACT_GRAD(Silu)
  }
#undef POETX_ACT_GRAD
  return hipGetLastError();
}

}  // namespace

int act_grad_splits(int64_t rows) {
  const int64_t per = rows_per_split(rows);
  return (int)((rows + per - 1) / per);
}

hipError_t launch_act_grad(DType t, const ActGrad& a, hipStream_t s) {
  if (a.gu_tiled && (t != DType::BF16 || a.rows % kTileRows != 0 || a.d % kTileCols != 0))
    return hipErrorInvalidValue;
  const int nsplit = act_grad_splits(a.rows);
  float* part = !a.g_bias ? nullptr : nsplit == 1 ? a.g_bias : a.part;
  hipError_t e = t == DType::BF16 ? launch_typed<bf16_t>(a, part, s) : launch_typed<float>(a, part, s);
  if (e != hipSuccess || !a.g_bias || nsplit == 1) return e;
  hipLaunchKernelGGL(bias_reduce_kernel, dim3((a.d + 63) / 64), dim3(NT), 0, s, part, nsplit,
                     a.d, a.g_bias);
  return hipGetLastError();
}

}  // namespace poetx
