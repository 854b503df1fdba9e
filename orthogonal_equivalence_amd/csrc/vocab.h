// Device functions shared by the kernels that turn logits into a loss and its
// gradient (vocab_tile.hip, vocab.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace poetx {
namespace {

// The maximum m of c v over a row's values, this lane's NV and those of the
// lanes 16, 32 and 48 further on, and the sum of 2^(c v - m), in all four
// lanes. Where m is not finite the sum is that of 2^(c v): 0 for -inf alone,
// +inf with a +inf among them; a NaN reaches it either way.
template <int NV> __device__ __forceinline__ float2 row_max_sum(const float (&v)[NV], float c) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < NV; ++q) m = fmaxf(m, v[q]);
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32)) * c;
  const float at = fabsf(m) < INFINITY ? m : 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < NV; ++q) s += __builtin_amdgcn_exp2f(fmaf(v[q], c, -at));
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  return make_float2(m, s);
}

// g_z at a logit z of the vocabulary's column `col` (VocabRow)
__device__ __forceinline__ float logit_gradient(const VocabRow& r, float z, float c, int col) {
  const float q = r.a == 0.0f ? 0.0f : r.a * __builtin_amdgcn_exp2f(fmaf(z, c, -r.lse2));
  return col == r.target ? q - r.b : q;
}

}  // namespace
}  // namespace poetx
