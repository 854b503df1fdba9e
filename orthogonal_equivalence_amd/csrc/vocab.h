// Device functions shared by the kernels that turn logits into a loss and its
// gradient (vocab_tile.hip, vocab.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace poetx {
namespace {

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
};
template <> struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const float* p, float v[4]) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// The logits at a row's listed ids, four entries a wave (the `at`-th of
// listed_waves()): x's piece is loaded once for four rows of W. The products are
// summed in float32 per lane (K / 64 of them), the lanes as a tree.
constexpr int kEntries = 4;
__host__ __device__ inline int64_t listed_waves(int64_t rows, int top) {
  return rows * ((top + kEntries - 1) / kEntries);
}
template <typename T>
__device__ __forceinline__ void listed_logits(const T* __restrict__ x, const T* __restrict__ W,
                                              const VocabList& l, int64_t rows, int K,
                                              float* __restrict__ z, int64_t at, int lane) {
  constexpr int E = Vec<T>::E;
  const int groups = (l.top + kEntries - 1) / kEntries;
  const int64_t row = at / groups;
  const int k0 = (int)(at - row * groups) * kEntries;
  if (row >= rows) return;
  int64_t id[kEntries];
  bool any = false;
#pragma unroll
  for (int q = 0; q < kEntries; ++q) {
    id[q] = k0 + q < l.top ? l.ids[row * l.top + k0 + q] : -1;
    any |= id[q] >= 0 && id[q] < l.vocab;
  }
  float acc[kEntries] = {};
  if (any) {
    const T* w[kEntries];
#pragma unroll
    for (int q = 0; q < kEntries; ++q)
      w[q] = W + (id[q] >= 0 && id[q] < l.vocab ? id[q] : 0) * (int64_t)K;
#pragma unroll 2
    for (int k = lane * E; k < K; k += 64 * E) {
      float xv[E], wv[kEntries][E];
      Vec<T>::load(x + row * K + k, xv);
#pragma unroll
      for (int q = 0; q < kEntries; ++q) Vec<T>::load(w[q] + k, wv[q]);
#pragma unroll
      for (int q = 0; q < kEntries; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[q] = fmaf(xv[e], wv[q][e], acc[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < kEntries; ++q) {
    const float v = wave_sum(acc[q]);
    if (lane == 0 && k0 + q < l.top)
      z[row * l.top + k0 + q] = id[q] < 0 ? 0.0f : id[q] >= l.vocab ? NAN : v;
  }
}

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

// The maximum m of a row's values, this lane's NV and those of the lanes 16, 32
// and 48 further on, and the sum of 2^(c (v - m)), in all four lanes. (The
// difference before the product: the maximum's own term is then exactly 1 and
// what a term loses goes by its distance from the maximum. As 2^(c v - c m), one
// instruction less, it went by |m|, and one to two steps of lse were lost; 8192 x
// 131072 x 4096 5940 us that way, 5965 this.)
template <int NV> __device__ __forceinline__ float2 row_max_sum(const float (&v)[NV], float c) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < NV; ++q) m = fmaxf(m, v[q]);
  m = quad_max(m);
  const float at = exponent_base(m);
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < NV; ++q) s[q & 3] += __builtin_amdgcn_exp2f((v[q] - at) * c);
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

// the value of lane l ^ 8
__device__ __forceinline__ uint32_t ror8(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, false);  // row_ror:8
}
__device__ __forceinline__ uint4 ror8(uint4 v) {
  return make_uint4(ror8(v.x), ror8(v.y), ror8(v.z), ror8(v.w));
}

__device__ __forceinline__ uint4 choose(bool c, uint4 a, uint4 b) {
  return make_uint4(c ? a.x : b.x, c ? a.y : b.y, c ? a.z : b.z, c ? a.w : b.w);
}
// what is left of v where bf16 keeps `high` of it (less than 2^-16 of it is nothing
// beside the result's rounding, and left out: a g_z that is a bf16 value but for the
// rounding of lse stays one)
__device__ __forceinline__ float low_part(float v, float high) {
  const float low = v - high;
  return fabsf(low) > 0x1p-16f * fabsf(high) && fabsf(high) < INFINITY ? low : 0.0f;
}
// The entries of one wave's cell: their range and the first 64 of them, read
// well before their logits are stored (each read waits for the L2, one for the
// other).
struct OwnCell {
  const uint32_t* entries;
  int begin, end;
  uint32_t first;  // this lane's of the first 64
};
__device__ __forceinline__ OwnCell read_cell(const VocabCells& cells, int64_t row_cell, int bin,
                                             int lane) {
  OwnCell c;
  // (a uniform address: read through the scalar cache)
  typedef const __attribute__((address_space(4))) int* ConstInts;
  const ConstInts at = (ConstInts)(cells.offsets + row_cell * (cells.bins + 1) + bin);
  c.begin = __builtin_amdgcn_readfirstlane(at[0]);
  c.end = __builtin_amdgcn_readfirstlane(at[1]);
  c.entries = cells.entries + row_cell * cells.per_cell;
  c.first = c.begin + lane < c.end ? c.entries[c.begin + lane] : 0;
  return c;
}
// Stores their logits (z's row of the cell's first row: `m`): pick(i, j) is the
// wave's fragment (i, j), wave-uniform; entries are taken one by one.
template <typename Pick>
__device__ __forceinline__ void store_cell(const VocabCells& cells, const OwnCell& c, int64_t m,
                                           int lane, const Pick& pick) {
  auto store = [&](uint32_t own, int n) __attribute__((always_inline)) {
    for (int q = 0; q < n; ++q) {
      const uint32_t w = __builtin_amdgcn_readlane(own, q);
      const int row = w & 127, col = (w >> 7) & 127;
      const floatx4 v = pick(row >> 4, col >> 4);
      const int k = col & 3;
      const float z = k < 2 ? (k == 0 ? v[0] : v[1]) : (k == 2 ? v[2] : v[3]);
      if (lane == (row & 15) + 16 * ((col >> 2) & 3))
        cells.z[(m + row) * cells.top + (w >> 14)] = z;
    }
  };
  store(c.first, min(64, c.end - c.begin));
  for (int e = c.begin + 64; e < c.end; e += 64)  // (few cells; these wait for their loads)
    store(e + lane < c.end ? c.entries[e + lane] : 0, min(64, c.end - e));
}

// exp(z / T - lse), inv = 1 / T. (In base 2 from the start, 2^(c z - log2(e) lse), it
// lost a rounding of lse; this loses one of the difference, where 1 / T is exact.)
// float32 also takes back what the product with log2(e) lost, x 2^-24 of the value
// (bf16's rounding is far above it).
template <typename T> __device__ __forceinline__ float softmax_at(float z, float inv, float lse) {
  constexpr float kHigh = 1.44269502162933349609375f, kLow = 1.92596299112661768e-8f;  // log2(e)
  const float x = fmaf(z, inv, -lse), t = x * kHigh, e = __builtin_amdgcn_exp2f(t);
  if constexpr (sizeof(T) == 2) return e;
  const float left = fmaf(x, kLow, fmaf(x, kHigh, -t)) * 0.693147180559945309f;
  return fabsf(t) < 126.0f ? fmaf(e, left, e) : e;
}
// g_z at a logit z of the vocabulary's column `col` (VocabRow)
template <typename T>
__device__ __forceinline__ float logit_gradient(const VocabRow& r, float z, float inv, int col) {
  const float q = r.a == 0.0f ? 0.0f : r.a * softmax_at<T>(z, inv, r.lse);
  return col == r.target ? q - r.b : q;
}

}  // namespace
}  // namespace poetx
