// Device functions shared by the kernels that turn logits into a loss and its
// gradient (vocab_tile.hip, vocab.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace poetx {
namespace {

// The maximum and the sum over the four lanes that are 16 apart, in all four:
// two exchanges of rows of 16 lanes, in the vector unit (through LDS, as
// __shfl_xor goes, each costs its latency).
__device__ __forceinline__ float quad_max(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// what the exponents of a row's sum are taken from: its maximum, or 0 where
// that is not finite (the sum is then 0 for -inf alone and +inf with a +inf
// among the values; a NaN reaches it either way)
__device__ __forceinline__ float exponent_base(float m) { return fabsf(m) < INFINITY ? m : 0.0f; }

// The maximum m of c v over a row's values, this lane's NV and those of the
// lanes 16, 32 and 48 further on, and the sum of 2^(c v - m), in all four
// lanes.
template <int NV> __device__ __forceinline__ float2 row_max_sum(const float (&v)[NV], float c) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < NV; ++q) m = fmaxf(m, v[q]);
  m = quad_max(m) * c;
  const float at = exponent_base(m);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < NV; ++q) s[q & 3] += __builtin_amdgcn_exp2f(fmaf(v[q], c, -at));
  return make_float2(m, quad_sum((s[0] + s[1]) + (s[2] + s[3])));
}

// Two 16 x 16 fragments that are neighbours along the columns (lane l: row l % 16,
// columns 4 (l / 16) .. + 3 of each), four values packed, as this lane's 16 bytes: columns
// pair_column() .. + 7 of the pair's 32.
__device__ __forceinline__ uint4 swap_pair(uint2 a, uint2 b) {
  const auto lo = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
  return make_uint4(lo[0], hi[0], lo[1], hi[1]);
}
__device__ __forceinline__ int pair_column(int ln) {
  return 16 * ((ln >> 4) & 1) + 8 * (ln >> 5);
}

// g_z at a logit z of the vocabulary's column `col` (VocabRow)
__device__ __forceinline__ float logit_gradient(const VocabRow& r, float z, float c, int col) {
  const float q = r.a == 0.0f ? 0.0f : r.a * __builtin_amdgcn_exp2f(fmaf(z, c, -r.lse2));
  return col == r.target ? q - r.b : q;
}

}  // namespace
}  // namespace poetx
