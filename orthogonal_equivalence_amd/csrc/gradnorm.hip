// Global gradient norm over many tensors and clipping by it.
//   norm = sqrt(sum over every value of g^2),  out = g min(1, max_norm / norm).
//
// Two passes over the data, each a grid of workgroups that walk 16 KB chunks
// of the runs: the first leaves one float64 partial sum per workgroup, the
// second joins the partials (every workgroup for itself, in the same order)
// and scales. The norm has to be known before the first value is scaled, so
// the values are read twice; the second pass takes the chunks from last to
// first, whose values the first pass read last and the memory-side cache may
// still hold.
//
// Squares and sums are float64: float32 squares overflow from 1.8e19 and
// vanish below 1e-23, and the float64 rate is far above what the loads feed.
// The factor is not rounded to float32 (Factor): that would be a rounding of
// its own, loses bits below 2^-126 and is zero below 2^-150, which finite
// gradients and an ordinary max_norm reach.
// The partials' places and the order of every sum follow from the sizes and
// the runs' alignment alone: no atomics, the same bits every time.
//
// The runs' addresses and sizes travel in the kernel arguments (kMaxRuns a
// launch), so a call needs no device table, no copy and no allocation, and a
// captured graph holds them by value.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace poetx {
namespace {

constexpr int NT = 256;
constexpr int kMaxRuns = 120;        // 3.5 KB of the 4 KB of kernel arguments
constexpr int kChunkBytes = 16384;   // four 16-byte loads a thread
constexpr int kMaxParts = 2048;      // workgroups of a pass: eight per CU

constexpr int kFewRuns = 16;         // a short list's arguments: 0.5 KB a launch

template <int N> struct Batch {
  const void* grad[N];
  void* out[N];
  int64_t n[N];
  int32_t first[N + 1];  // chunks before run i
  int8_t bf16[N];
  int count;
};
static_assert(sizeof(Batch<kMaxRuns>) < 3900, "kernel argument space");

int64_t chunks_of(const GradRun& r) {
  const int64_t per = kChunkBytes / (r.dtype == DType::BF16 ? 2 : 4);
  return (r.n + per - 1) / per;
}

// the run that holds `chunk`
template <int N> __device__ __forceinline__ int find_run(const Batch<N>& b, int chunk) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// sum over the workgroup, the same value in every thread
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[NT / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = s[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) t += s[w];
  return t;
}

// the 16-byte vector's values as float32
template <typename T> __device__ __forceinline__ void unpack(uint4 w, float v[16 / sizeof(T)]) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(a[i]);
    } else {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void add_square(double& acc, float v) {
  const double d = (double)v;
  acc = fma(d, d, acc);
}

template <typename T> __device__ __forceinline__ void add_squares(double& acc, uint4 w) {
  float f[16 / sizeof(T)];
  unpack<T>(w, f);
#pragma unroll
  for (int e = 0; e < (int)(16 / sizeof(T)); ++e) add_square(acc, f[e]);
}

// one thread's share of a chunk that is cut by its run's end or not aligned
template <typename T>
__device__ __forceinline__ double cut_sumsq(const T* p, int64_t n, int64_t at) {
  constexpr int E = 16 / sizeof(T), PER = kChunkBytes / sizeof(T);
  const int len = (int)min((int64_t)PER, n - at);
  const T* src = p + at;
  double acc = 0.0;
  int i0 = 0;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const int nv = len / E;
    for (int i = threadIdx.x; i < nv; i += NT)
      add_squares<T>(acc, reinterpret_cast<const uint4*>(src)[i]);
    i0 = nv * E;
  }
  for (int i = i0 + threadIdx.x; i < len; i += NT) add_square(acc, ElemTraits<T>::to_f32(src[i]));
  return acc;
}

// A store that the caches need not keep: 334 M float32 values, clipped into
// another buffer, took 742 us with plain stores and 714 with these (what the
// first pass read last stays in the memory-side cache for the second).
__device__ __forceinline__ void store_nt(uint4* p, uint4 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

// max_norm / norm <= 1 as (hi + lo) 2^e, hi in [1/2, 1) its first 24 bits and lo
// < 2^-24 the rest, so that a value times the factor is off by its one rounding
// and 2^-46 relative. Three float32 operations a value: 10.4 M values 24.7 us,
// with float64 products 26.2, with one float32 factor 24.5. lo is never 0 (2^-60
// is below every rounding), so that an infinity stays one; a factor of 0 is 0.
struct Factor {
  float hi, lo;
  int e;
  __device__ __forceinline__ explicit Factor(double k) {
    const double m = frexp(k, &e);
    hi = (float)m;
    if ((double)hi > m) hi = __uint_as_float(__float_as_uint(hi) - 1u);
    lo = m > 0.0 ? fmaxf((float)(m - (double)hi), 0x1p-60f) : 0.0f;
  }
  __device__ __forceinline__ float times(float v) const { return ldexpf(fmaf(v, hi, v * lo), e); }
};

// (grad and out may be the same memory: each value is read, then written, by
// one thread)
template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int64_t n, int64_t at, const Factor& k) {
  constexpr int E = 16 / sizeof(T), PER = kChunkBytes / sizeof(T), Q = PER / E / NT;
  const int len = (int)min((int64_t)PER, n - at);
  const T* src = p + at;
  T* dst = o + at;
  auto scaled = [&](uint4 w) {
    float f[E];
    unpack<T>(w, f);
    union { T h[E]; uint4 u; } r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.h[e] = ElemTraits<T>::from_f32(k.times(f[e]));
    return r.u;
  };
  int i0 = 0;
  if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    const uint4* v = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    if (len == PER) {
      uint4 w[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) w[q] = v[q * NT + threadIdx.x];
#pragma unroll
      for (int q = 0; q < Q; ++q) store_nt(d + q * NT + threadIdx.x, scaled(w[q]));
      return;
    }
    const int nv = len / E;
    for (int i = threadIdx.x; i < nv; i += NT) d[i] = scaled(v[i]);
    i0 = nv * E;
  }
  for (int i = i0 + threadIdx.x; i < len; i += NT)
    dst[i] = ElemTraits<T>::from_f32(k.times(ElemTraits<T>::to_f32(src[i])));
}

// a whole chunk's 16-byte vectors of one thread, or null: a cut or unaligned
// chunk
template <int N>
__device__ __forceinline__ const uint4* whole_chunk(const Batch<N>& b, int chunk, int* bf16) {
  const int i = find_run(b, chunk);
  const int64_t at = (int64_t)(chunk - b.first[i]) * kChunkBytes;
  const char* p = static_cast<const char*>(b.grad[i]);
  *bf16 = b.bf16[i];
  const bool whole = (reinterpret_cast<uintptr_t>(p) & 15) == 0 &&
                     at + kChunkBytes <= b.n[i] * (b.bf16[i] ? 2 : 4);
  return whole ? reinterpret_cast<const uint4*>(p + at) + threadIdx.x : nullptr;
}

template <int N>
__global__ void __launch_bounds__(NT) sumsq_kernel(const Batch<N> b, double* __restrict__ part) {
  constexpr int Q = kChunkBytes / 16 / NT;
  const int total = b.first[b.count];
  double acc = 0.0;
  // a chunk's loads are in flight while the one before it is summed
  uint4 w[2][Q];
  int bf16[2] = {};
  const uint4* src = whole_chunk(b, blockIdx.x, &bf16[0]);
  if (src)
#pragma unroll
    for (int q = 0; q < Q; ++q) w[0][q] = src[q * NT];
  bool whole = src != nullptr;
  auto one = [&](auto buf, int c) __attribute__((always_inline)) {
    constexpr int k = decltype(buf)::value;
    const int next = c + gridDim.x;
    const uint4* ns = next < total ? whole_chunk(b, next, &bf16[k ^ 1]) : nullptr;
    if (ns)
#pragma unroll
      for (int q = 0; q < Q; ++q) w[k ^ 1][q] = ns[q * NT];
    if (whole) {
      if (bf16[k]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) add_squares<bf16_t>(acc, w[k][q]);
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) add_squares<float>(acc, w[k][q]);
      }
    } else {
      const int i = find_run(b, c);
      const int64_t at = c - b.first[i];
      acc += b.bf16[i] ? cut_sumsq(static_cast<const bf16_t*>(b.grad[i]), b.n[i], at * (kChunkBytes / 2))
                       : cut_sumsq(static_cast<const float*>(b.grad[i]), b.n[i], at * (kChunkBytes / 4));
    }
    whole = ns != nullptr;
  };
  for (int c = blockIdx.x; c < total; c += 2 * gridDim.x) {
    one(std::integral_constant<int, 0>{}, c);
    if (c + (int)gridDim.x >= total) break;
    one(std::integral_constant<int, 1>{}, c + gridDim.x);
  }
  const double t = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = t;
}

__device__ __forceinline__ double parts_sum(const double* part, int nparts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < nparts; i += NT) v += part[i];
  return block_sum(v);
}

__global__ void __launch_bounds__(NT)
norm_kernel(const double* __restrict__ part, int nparts, float* __restrict__ norm) {
  const double t = parts_sum(part, nparts);
  if (threadIdx.x == 0) *norm = (float)sqrt(t);
}

template <int N>
__global__ void __launch_bounds__(NT)
scale_kernel(const Batch<N> b, const double* part, int nparts, const float* norm_in, float max_norm,
             float* norm_out) {
  const double norm = part ? sqrt(parts_sum(part, nparts)) : (double)*norm_in;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // (factor 1 for a norm that is NaN, infinite or past float32's range, as the
  // caller reads it)
  const bool clip = norm > (double)max_norm && (float)norm < INFINITY;
  const Factor k(clip ? (double)max_norm / norm : 1.0);
  const int total = b.first[b.count];
  for (int c = total - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = find_run(b, c);
    if (!clip && b.grad[i] == b.out[i]) continue;  // nothing to change
    const int64_t q = c - b.first[i];
    if (b.bf16[i])
      chunk_scale(static_cast<const bf16_t*>(b.grad[i]), static_cast<bf16_t*>(b.out[i]), b.n[i],
                  q * (kChunkBytes / 2), k);
    else
      chunk_scale(static_cast<const float*>(b.grad[i]), static_cast<float*>(b.out[i]), b.n[i],
                  q * (kChunkBytes / 4), k);
  }
}

constexpr int kMinParts = 64;        // of a launch, however many there are
int64_t launches_of(int64_t count) { return (count + kMaxRuns - 1) / kMaxRuns; }
int parts_per_launch(int count) {
  return std::max(kMinParts, kMaxParts / (int)std::max<int64_t>(1, launches_of(count)));
}

// The runs in launches of at most kMaxRuns, in order. fn(batch, workgroups).
template <int N, typename F>
hipError_t for_batches_of(const GradRun* runs, int count, F fn) {
  const int cap = parts_per_launch(count);
  Batch<N> b;
  for (int i = 0; i < count;) {
    b.count = 0;
    int64_t chunks = 0;
    b.first[0] = 0;
    for (; i < count && b.count < N; ++i, ++b.count) {
      b.grad[b.count] = runs[i].grad;
      b.out[b.count] = runs[i].out;
      b.n[b.count] = runs[i].n;
      b.bf16[b.count] = runs[i].dtype == DType::BF16;
      chunks += chunks_of(runs[i]);
      if (chunks > INT32_MAX) return hipErrorInvalidValue;
      b.first[b.count + 1] = (int32_t)chunks;
    }
    const hipError_t e = fn(b, (int)std::min<int64_t>(cap, chunks));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename F> hipError_t for_batches(const GradRun* runs, int count, F fn) {
  return count <= kFewRuns ? for_batches_of<kFewRuns>(runs, count, fn)
                           : for_batches_of<kMaxRuns>(runs, count, fn);
}

}  // namespace

// (of fewer runs too: neighbours are joined)
int64_t grad_partials_max(int64_t count) {
  return std::max<int64_t>(kMaxParts, kMinParts * launches_of(count));
}

hipError_t launch_grad_sumsq(const GradRun* runs, int count, double* part, int* nparts,
                             hipStream_t s) {
  *nparts = 0;
  return for_batches(runs, count, [&](const auto& b, int wgs) {
    hipLaunchKernelGGL(sumsq_kernel, dim3(wgs), dim3(NT), 0, s, b, part + *nparts);
    *nparts += wgs;
    return hipGetLastError();
  });
}

hipError_t launch_grad_norm(const double* part, int nparts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(NT), 0, s, part, nparts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradRun* runs, int count, const double* part, int nparts,
                             const float* norm_in, float max_norm, float* norm_out,
                             hipStream_t s) {
  return for_batches(runs, count, [&](const auto& b, int wgs) {
    hipLaunchKernelGGL(scale_kernel, dim3(wgs), dim3(NT), 0, s, b, part, nparts, norm_in, max_norm,
                       norm_out);
    norm_out = nullptr;  // the first launch stores it
    return hipGetLastError();
  });
}

}  // namespace poetx
