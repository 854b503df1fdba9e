// The dense linear's forward for a few tokens (decoding): the weight's bytes
// are all that counts, so each is read once, straight into the registers that
// the matrix instructions take it from, and nothing else is read from HBM
// twice:
//   u(m, n) = scale[n] sum_k x(m, k) W(n, k) + bias[n],  y = act(u) + residual.
//
// A workgroup owns 16 rows of W (output columns) for all tokens (kStreamRows at
// most, of the 16 that a product has room for); its
// eight waves take interleaved pieces of k, so that the workgroup reads whole
// 128-byte lines of each row, kUnroll loads of 16 bytes a lane in flight a
// wave. The fragments need no LDS: lane l of a 16 x 16 x 32 product holds k =
// 8 (l / 16) .. + 7 of row l % 16 of both operands, which is one 16-byte load
// of W's row and one of x's (rows past the last token read the last one; their
// results are dropped). The waves' sums meet in LDS, added in wave order, and
// one thread per four columns ends them with the epilogue: one launch, no
// workspace.
//
// x comes from the caches, once per 16 rows of W: half as many bytes as the
// weight at 8 tokens and as many at 16, which is why more than kStreamRows go to
// the tile kernel, whose workgroups share x among 64 rows and more (measured at
// kStreamRows).
//
// INT8 codes are widened in registers: code + 128 as an unsigned byte to
// float32, less 128, to bf16, all exact.
#include <type_traits>

#include "common.h"
#include "epilogue.h"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int kWaves = 8, NT = 64 * kWaves, kUnroll = 4;

// One lane's eight (bf16 products) or four (float32) consecutive k.
template <typename TX> struct Chunk;
template <> struct Chunk<bf16_t> {
  typedef bf16x8_t V;
  static constexpr int E = 8, STEP = 32;
};
template <> struct Chunk<float> {
  typedef floatx4 V;
  static constexpr int E = 4, STEP = 16;
};

// What one lane loads of a row of W for one step: kParts chunks.
template <typename TW, typename TX> struct Weight {  // W in the activation type
  typedef typename Chunk<TX>::V Raw;
  static constexpr int kParts = 1;
  static __device__ __forceinline__ Raw widen(const Raw& r, int) { return r; }
};
// INT8 codes, eight or (rows of whole 16 bytes) sixteen of them
template <int BYTES> struct Codes;
template <> struct Codes<8> { typedef uint2 Raw; };
template <> struct Codes<16> { typedef uint4 Raw; };
template <int BYTES> struct Weight<Codes<BYTES>, bf16_t> {
  typedef typename Codes<BYTES>::Raw Raw;
  static constexpr int kParts = BYTES / 8;
  static __device__ __forceinline__ bf16x8_t widen(const Raw& r, int part) {
    union { Raw r; uint32_t w[BYTES / 4]; } in;
    in.r = r;
    union { bf16_t h[8]; bf16x8_t v; } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = in.w[2 * part + (i >> 2)] ^ 0x80808080u;
      o.h[i] = f32_to_bf16((float)((w >> (8 * (i & 3))) & 0xffu) - 128.0f);
    }
    return o.v;
  }
};

__device__ __forceinline__ floatx4 mma(const bf16x8_t& a, const bf16x8_t& b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mma(const floatx4& a, const floatx4& b, floatx4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

template <typename TW, typename TX>
__global__ void __launch_bounds__(NT)
stream_kernel(const TX* __restrict__ x, const char* __restrict__ W, int64_t row_bytes, int M, int N,
              int K, const Epilogue ep) {
  typedef Weight<TW, TX> Wt;
  typedef typename Wt::Raw Raw;
  typedef typename Chunk<TX>::V Frag;
  constexpr int P = Wt::kParts, E = Chunk<TX>::E * P, STEP = Chunk<TX>::STEP * P;
  constexpr int WB = sizeof(Raw) / E;  // bytes of a weight
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  // lane l takes E consecutive k of every step, from E (l / 16) on, for both
  // operands (with two parts the products take a half of them each: the order
  // of k inside a step is the same on both sides)
  const char* wrow = W + min(n0 + r, N - 1) * row_bytes + WB * E * g;
  const TX* xrow = x + (int64_t)min(r, M - 1) * K + E * g;
  floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};

  // pieces of kUnroll steps of k, interleaved over the waves; a piece's loads
  // are in flight while the one before it is multiplied
  constexpr int PIECE = STEP * kUnroll, STRIDE = kWaves * PIECE;
  Raw w[2][kUnroll];
  Frag v[2][kUnroll][P];
  auto load = [&](auto buf, int k) __attribute__((always_inline)) {
    constexpr int b = decltype(buf)::value;
#pragma unroll
    for (int s = 0; s < kUnroll; ++s)
      w[b][s] = *reinterpret_cast<const Raw*>(wrow + (int64_t)(k + STEP * s) * WB);
#pragma unroll
    for (int s = 0; s < kUnroll; ++s)
#pragma unroll
      for (int p = 0; p < P; ++p)
        v[b][s][p] = *reinterpret_cast<const Frag*>(xrow + k + STEP * s + E / P * p);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](auto buf) __attribute__((always_inline)) {
    constexpr int b = decltype(buf)::value;
#pragma unroll
    for (int s = 0; s < kUnroll; ++s)
#pragma unroll
      for (int p = 0; p < P; ++p) acc = mma(Wt::widen(w[b][s], p), v[b][s][p], acc);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> kA{};
  constexpr std::integral_constant<int, 1> kB{};
  int k = wave * PIECE;
  if (k + PIECE <= K) load(kA, k);
  for (; k + PIECE <= K; k += 2 * STRIDE) {
    const bool second = k + STRIDE + PIECE <= K;
    if (second) load(kB, k + STRIDE);
    multiply(kA);
    if (!second) {
      k += STRIDE;
      break;
    }
    if (k + 2 * STRIDE + PIECE <= K) load(kA, k + 2 * STRIDE);
    multiply(kB);
  }
  // this wave's last piece, cut by K: chunks past the end are zeros in both
  for (; k < K; k += STEP) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = k + E * g + E / P * p;  // (K is a multiple of E)
      Frag a = {}, b = {};
      if (at < K) {
        a = Wt::widen(*reinterpret_cast<const Raw*>(wrow + (int64_t)k * WB), p);
        b = *reinterpret_cast<const Frag*>(xrow + k + E / P * p);
      }
      acc = mma(a, b, acc);
    }
  }

  // lane l: token l % 16, columns 4 (l / 16) .. + 3
  __shared__ floatx4 sums[kWaves][64];
  sums[wave][lane] = acc;
  __syncthreads();
  const int n = n0 + 4 * g;
  if (wave != 0 || r >= M || n >= N) return;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const floatx4 p = sums[w][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] += p[e];
  }
  epilogue4<TX>(ep, r, n, t);
}

template <typename TW, typename TX>
hipError_t launch_typed(const StreamProduct& p, int weight_bytes, hipStream_t s) {
  hipLaunchKernelGGL((stream_kernel<TW, TX>), dim3((p.N + 15) / 16), dim3(NT), 0, s,
                     static_cast<const TX*>(p.x), static_cast<const char*>(p.W),
                     (int64_t)p.K * weight_bytes, p.M, p.N, p.K, p.ep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_stream_product(DType t, bool int8, const StreamProduct& p, hipStream_t s) {
  if (p.M > kStreamRows || (int8 && t != DType::BF16)) return hipErrorInvalidValue;
  if (t == DType::F32) return launch_typed<float, float>(p, 4, s);
  if (!int8) return launch_typed<bf16_t, bf16_t>(p, 2, s);
  return p.K % 16 == 0 ? launch_typed<Codes<16>, bf16_t>(p, 1, s)
                       : launch_typed<Codes<8>, bf16_t>(p, 1, s);
}

}  // namespace poetx
