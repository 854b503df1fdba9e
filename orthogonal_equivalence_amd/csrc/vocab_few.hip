// g_W = g_z^T x for few tokens (up to few_tokens()): each element of g_W is a sum of
// at most 128 products, so the store of g_W is all there is to it (131072 x 4096
// bf16 1.07 GB, 180 us at what stores alone reach), and tiles that load, wait, multiply
// once and store spend most of their time on the first two.
//
// bf16: g_z in two parts, the second what rounding took off the first, both times the
// same x.
//
// One wave takes 32 or 64 rows of g_W (ids): their g_z are the products' operand and
// stay in registers; it walks along d with one 16-byte load a lane for 16 columns
// and K tokens, 128 bytes of columns ahead, out of a copy of x with the tokens
// innermost (xt [d][tokens padded]; it stays in the L2), and stores 8 rows' whole
// lines at a time. No LDS, no barrier. Workgroups in the order of g_W's rows, not of its
// columns: what is stored at one time then lies together (stores alone of 1.07 GB
// 181 us, the other way 235).
// us:                      1 token   64   96  128
//   131072 x 4096, bf16      211  275  323  454     (with one part of g_z 211, 245, 300, 385)
//   32000 x 4096              55   64
// From 33 tokens on 64 ids a wave (32 ids: a third more at 64 tokens, a sixth at 96, alike at
// 128); up to 32 tokens 32 ids (56370 x 2256, 16 tokens: 232 us a backward, 64 ids 239). Stores of
// 16 rows' half lines: a third more. Past 128 tokens the registers are spent.
#include "epilogue.h"
#include "vocab.h"

namespace poetx {
namespace {

constexpr int NT = 256, NWAVES = NT / 64;
// fragments of 16 ids a wave: the more, the less often x's copy is read
template <int STEPS> constexpr int kFrags = STEPS == 1 ? 2 : 4;
// Columns a workgroup walks along: as many as pay for its g_z, while there are
// workgroups enough (131072 x 4096, both gradients, us: 64 tokens 743 with 512, 706 with
// 1024, 782 with 2048; 96 tokens 890, 854, 872; 128 tokens 1244, 1075, 1017).
template <typename T, int STEPS>
constexpr int kChunk = sizeof(T) == 4 || STEPS == 1 ? 512 : STEPS == 4 ? 2048 : 1024;
constexpr int kGroups = 128;
// a g_W larger than this goes past the caches, where its rows are whole lines, and W
// stays in them for the next pass (backward of 64 tokens: 32000 x 4096 227 -> 172 us,
// 131072 x 4096 833 -> 768; 32000 x 1024 float32, 131 MB, alike; rows of 4512 bytes 60 -> 160)
constexpr int64_t kCacheBytes = INT64_C(128) << 20;

template <typename T> struct Few;
template <> struct Few<bf16_t> {
  typedef bf16x8_t Frag;
  static constexpr int K = 32, E = 8;  // tokens a product and a fragment's lane takes
  static constexpr int kParts = 2;     // of g_z
  static __device__ __forceinline__ floatx4 mma(const Frag& a, const Frag& b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Few<float> {
  typedef floatx4 Frag;
  static constexpr int K = 16, E = 4;  // (four products of 4 tokens)
  static constexpr int kParts = 1;
  static __device__ __forceinline__ floatx4 mma(const Frag& a, const Frag& b, floatx4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
};

template <bool PAST> __device__ __forceinline__ void store16(void* p, uint4 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 w{v.x, v.y, v.z, v.w};
  if constexpr (PAST) __builtin_nontemporal_store(w, static_cast<u32x4*>(p));
  else *static_cast<u32x4*>(p) = w;
}

// 64 bytes of columns (bf16: two fragments, float32 one): this lane's 16 of them in
// row l % 16, columns pair_column() or 4 (l / 16) on
template <typename T, int STEPS>
__device__ __forceinline__ uint4 half(const typename Few<T>::Frag (*b)[STEPS],
                                      const typename Few<T>::Frag (&a)[STEPS][Few<T>::kParts]) {
  constexpr int N = sizeof(T) == 2 ? 2 : 1;
  floatx4 c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    c[j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int h = 0; h < Few<T>::kParts; ++h) c[j] = Few<T>::mma(b[j][s], a[s][h], c[j]);
  }
  if constexpr (sizeof(T) == 2) {
    const float p[4] = {c[0][0], c[0][1], c[0][2], c[0][3]};
    const float q[4] = {c[1][0], c[1][1], c[1][2], c[1][3]};
    return swap_pair(Quad<bf16_t>::pack(p), Quad<bf16_t>::pack(q));
  } else {
    return __builtin_bit_cast(uint4, c[0]);
  }
}

// STEPS: K tokens each. PAST: stores past the caches.
template <typename T, int STEPS, bool PAST>
__global__ void __launch_bounds__(NT)
few_gw_kernel(const T* __restrict__ gz, int64_t ldg, const T* __restrict__ xt, int tokens, int cols,
              int d, int chunks, int walk, T* __restrict__ g_W) {
  typedef Few<T> F;
  typedef typename F::Frag Frag;
  // fragments and columns of one step along d: 128 bytes
  constexpr int kStep = 128 / sizeof(T), NF = kStep / 16;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  constexpr int VF = kFrags<STEPS>, kRows = 16 * VF;
  const unsigned group = blockIdx.x / (unsigned)chunks, chunk = blockIdx.x - group * chunks;
  const int64_t v0 = ((int64_t)group * NWAVES + (threadIdx.x >> 6)) * kRows;
  if (v0 >= cols) return;
  Frag a[VF][STEPS][F::kParts];
#pragma unroll
  for (int f = 0; f < VF; ++f) {
    const int64_t v = min(v0 + 16 * f + r, (int64_t)cols - 1);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int h = 0; h < F::kParts; ++h) {
        union { T e[F::E]; Frag v; } u;
#pragma unroll
        for (int e = 0; e < F::E; ++e) {
          const int t = s * F::K + g * F::E + e;
          const T z = gz[(h * tokens + min(t, tokens - 1)) * ldg + v];
          u.e[e] = t < tokens ? z : T{};
        }
        a[f][s][h] = u.v;
      }
  }
  constexpr int kPad = STEPS * F::K;
  const int c0 = (int)chunk * walk, c1 = min(d, c0 + walk);
  Frag next[NF][STEPS];  // of the kStep columns after the current ones
  auto load = [&](int n0) {
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        next[j][s] = *reinterpret_cast<const Frag*>(
            xt + (int64_t)min(n0 + 16 * j + r, d - 1) * kPad + s * F::K + g * F::E);
  };
  load(c0);
  const bool upper = r >= 8;
  // this lane's first column of a step
  const int at = (upper ? kStep / 2 : 0) + (sizeof(T) == 2 ? pair_column(lane) : 4 * g);
  for (int n0 = c0; n0 < c1; n0 += kStep) {
    Frag b[NF][STEPS];
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) b[j][s] = next[j][s];
    load(n0 + kStep);
#pragma unroll
    for (int f = 0; f < VF; ++f) {
      // this lane's 16 bytes of row r, of either half of the columns
      const uint4 w0 = half<T, STEPS>(&b[0], a[f]), w1 = half<T, STEPS>(&b[NF / 2], a[f]);
      // rows 8 .. 15 of the first half for rows 0 .. 7 of the second: a store then
      // covers 8 rows by both halves, whole 128-byte lines
      const uint4 got = ror8(choose(upper, w0, w1));
      const uint4 lo = choose(upper, got, w0), hi = choose(upper, w1, got);
      const int n = n0 + at;
      const int64_t v = v0 + 16 * f + (r & 7);
      if (n < d) {
        if (v < cols) store16<PAST>(g_W + v * d + n, lo);
        if (v + 8 < cols) store16<PAST>(g_W + (v + 8) * d + n, hi);
      }
    }
  }
}

template <typename T, int STEPS>
hipError_t launch_steps(const void* gz, int64_t ldg, const void* xt, int tokens, int cols, int d,
                        void* g_W, hipStream_t s) {
  constexpr int kRows = 16 * kFrags<STEPS>;
  const int64_t groups = ((int64_t)cols + kRows * NWAVES - 1) / (kRows * NWAVES);
  int walk = kChunk<T, STEPS>;
  while (walk > 512 && groups * ((d + walk - 1) / walk) < kGroups) walk /= 2;
  const int chunks = (d + walk - 1) / walk;
  const int64_t blocks = groups * chunks;
  if (blocks >= INT64_C(1) << 24) return hipErrorInvalidValue;  // (2^32 work items)
  const int64_t row = d * (int64_t)sizeof(T);
  const auto kernel = row % 128 == 0 && cols * row > kCacheBytes
                          ? few_gw_kernel<T, STEPS, true>
                          : few_gw_kernel<T, STEPS, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(NT), 0, s, static_cast<const T*>(gz), ldg,
                     static_cast<const T*>(xt), tokens, cols, d, chunks, walk, static_cast<T*>(g_W));
  return hipGetLastError();
}

template <typename T>
hipError_t launch_type(int steps, const void* gz, int64_t ldg, const void* xt, int tokens, int cols,
                       int d, void* g_W, hipStream_t s) {
  switch (steps) {
    case 1: return launch_steps<T, 1>(gz, ldg, xt, tokens, cols, d, g_W, s);
    case 2: return launch_steps<T, 2>(gz, ldg, xt, tokens, cols, d, g_W, s);
    case 3: return launch_steps<T, 3>(gz, ldg, xt, tokens, cols, d, g_W, s);
    default: return launch_steps<T, 4>(gz, ldg, xt, tokens, cols, d, g_W, s);
  }
}

}  // namespace

hipError_t launch_few_gw(DType t, const void* gz, int64_t ldg, const void* xt, int tokens, int cols,
                         int d, void* g_W, hipStream_t s) {
  if (tokens < 1 || tokens > few_tokens(t) || cols < 1 || d < 1 || d > (1 << 22))
    return hipErrorInvalidValue;
  const int steps = few_padded(t, tokens) / (t == DType::BF16 ? 32 : 16);
  return t == DType::BF16 ? launch_type<bf16_t>(steps, gz, ldg, xt, tokens, cols, d, g_W, s)
                          : launch_type<float>(steps, gz, ldg, xt, tokens, cols, d, g_W, s);
}

}  // namespace poetx
