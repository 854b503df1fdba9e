// g_W = g_z^T x for few tokens (up to kFewTokens): each element of g_W is a sum of
// at most 64 products, so the store of g_W is all there is to it (131072 x 4096
// bf16 1.07 GB), and tiles that load, wait, multiply once and store spend most of
// their time on the first two.
//
// One wave takes 32 rows of g_W (ids): their g_z, at most 64 tokens, are the
// products' operand and stay in registers; it walks along d with one 16-byte load a
// lane for 16 columns, 32 columns ahead, out of a copy of x with the tokens
// innermost (xt [d][tokens padded]; it stays in the L2), and stores 64-byte pieces of
// 16 rows. No LDS, no barrier. 16 tokens, 131072 x 4096: 360 us, 3.0 TB/s of
// stores alone; 30 tokens, 56370 x 2256: 63 us, on 64 x 64 tiles 113. Stores past
// the caches (half lines) 194 us there; 16 ids a wave 75; walks of 1024 columns 71.
#include "epilogue.h"
#include "vocab.h"

namespace poetx {
namespace {

constexpr int NT = 256, NWAVES = NT / 64;
constexpr int VF = 2;            // fragments of 16 ids a wave
constexpr int kRows = 16 * VF;   // ids a wave
constexpr int kChunk = 512;      // columns a workgroup walks along

template <typename T> struct Few;
template <> struct Few<bf16_t> {
  typedef bf16x8_t Frag;
  static constexpr int K = 32, E = 8;  // tokens a product and a fragment's lane takes
  static __device__ __forceinline__ floatx4 mma(const Frag& a, const Frag& b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Few<float> {
  typedef floatx4 Frag;
  static constexpr int K = 16, E = 4;  // (four products of 4 tokens)
  static __device__ __forceinline__ floatx4 mma(const Frag& a, const Frag& b, floatx4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

// STEPS: K tokens each
template <typename T, int STEPS>
__global__ void __launch_bounds__(NT)
few_gw_kernel(const T* __restrict__ gz, int64_t ldg, const T* __restrict__ xt, int tokens, int cols,
              int d, T* __restrict__ g_W) {
  typedef Few<T> F;
  typedef typename F::Frag Frag;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * NWAVES + (threadIdx.x >> 6)) * kRows;
  if (v0 >= cols) return;
  Frag a[VF][STEPS];
#pragma unroll
  for (int f = 0; f < VF; ++f) {
    const int64_t v = min(v0 + 16 * f + r, (int64_t)cols - 1);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      union { T e[F::E]; Frag v; } u;
#pragma unroll
      for (int e = 0; e < F::E; ++e) {
        const int t = s * F::K + g * F::E + e;
        const T z = gz[min(t, tokens - 1) * ldg + v];
        u.e[e] = t < tokens ? z : T{};
      }
      a[f][s] = u.v;
    }
  }
  constexpr int kPad = STEPS * F::K;
  const int c0 = blockIdx.y * kChunk, c1 = min(d, c0 + kChunk);
  Frag next[2][STEPS];  // of the 32 columns after the current ones
  auto load = [&](int n0) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        next[j][s] = *reinterpret_cast<const Frag*>(
            xt + (int64_t)min(n0 + 16 * j + r, d - 1) * kPad + s * F::K + g * F::E);
  };
  load(c0);
  for (int n0 = c0; n0 < c1; n0 += 32) {
    Frag b[2][STEPS];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) b[j][s] = next[j][s];
    load(n0 + 32);
#pragma unroll
    for (int f = 0; f < VF; ++f) {
      floatx4 c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < STEPS; ++s) c[j] = F::mma(b[j][s], a[f][s], c[j]);
      }
      // (lane l: id l % 16, columns 4 (l / 16) .. + 3 of each fragment)
      const int64_t v = v0 + 16 * f + r;
      if constexpr (sizeof(T) == 2) {
        uint2 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float q[4] = {c[j][0], c[j][1], c[j][2], c[j][3]};
          w[j] = Quad<bf16_t>::pack(q);
        }
        const uint4 out = swap_pair(w[0], w[1]);
        const int n = n0 + pair_column(lane);
        if (v < cols && n < d) *reinterpret_cast<uint4*>(g_W + v * d + n) = out;
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = n0 + 16 * j + 4 * g;
          if (v < cols && n < d)
            *reinterpret_cast<uint4*>(g_W + v * d + n) = __builtin_bit_cast(uint4, c[j]);
        }
      }
    }
  }
}

template <typename T, int STEPS>
hipError_t launch_steps(const void* gz, int64_t ldg, const void* xt, int tokens, int cols, int d,
                        void* g_W, hipStream_t s) {
  const dim3 grid((unsigned)((cols + kRows * NWAVES - 1) / (kRows * NWAVES)),
                  (unsigned)((d + kChunk - 1) / kChunk));
  hipLaunchKernelGGL((few_gw_kernel<T, STEPS>), grid, dim3(NT), 0, s, static_cast<const T*>(gz), ldg,
                     static_cast<const T*>(xt), tokens, cols, d, static_cast<T*>(g_W));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_gw(DType t, const void* gz, int64_t ldg, const void* xt, int tokens, int cols,
                         int d, void* g_W, hipStream_t s) {
  if (tokens < 1 || tokens > kFewTokens || cols < 1 || d < 1 || d > (1 << 22))
    return hipErrorInvalidValue;
  const int steps = few_padded(t, tokens) / (t == DType::BF16 ? 32 : 16);
  if (t == DType::BF16)
    return steps == 1 ? launch_steps<bf16_t, 1>(gz, ldg, xt, tokens, cols, d, g_W, s)
                      : launch_steps<bf16_t, 2>(gz, ldg, xt, tokens, cols, d, g_W, s);
  switch (steps) {
    case 1: return launch_steps<float, 1>(gz, ldg, xt, tokens, cols, d, g_W, s);
    case 2: return launch_steps<float, 2>(gz, ldg, xt, tokens, cols, d, g_W, s);
    case 3: return launch_steps<float, 3>(gz, ldg, xt, tokens, cols, d, g_W, s);
    default: return launch_steps<float, 4>(gz, ldg, xt, tokens, cols, d, g_W, s);
  }
}

}  // namespace poetx
