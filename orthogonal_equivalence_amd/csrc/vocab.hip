// Everything of the losses over a vocabulary but their matrix products: the
// logits at listed ids, the join of the forward's partial sums with the loss,
// the rows' parts in the backward, and a teacher's entries in the gradient of
// the logits. All are small beside the products (8192 x 131072 logits: 67 MB of
// partial sums against 8.8 TFLOP).
//
//   L    = log sum_i s_i 2^((m_i - M) log2(e) / T), (m_i, s_i) the slots' parts
//          and M the largest of the m_i;  lse = M / T + L
//   loss = L + (M - z[target]), or with p the softmax of the listed teacher
//          logits over T: T^2 sum_k p_k (log p_k + (M - z_k) / T + L)
// The sum holds M's own term, 1, so L >= 0, and M - z is a difference of two
// logits: a loss is off by roundings of its own size, however large the logits
// are, and not below 0. (lse - z loses a step of lse.)
#include <algorithm>

#include "lds_dma.h"
#include "vocab.h"

namespace poetx {
namespace {

constexpr int NT = 256, NWAVES = NT / 64;
constexpr int kMaxTop = 1024;  // entries of a row's list
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

template <typename T>
__global__ void __launch_bounds__(NT)
listed_logits_kernel(const T* __restrict__ x, const T* __restrict__ W, const VocabList l,
                     int64_t rows, int K, float* __restrict__ z) {
  listed_logits(x, W, l, rows, K, z, (int64_t)blockIdx.x * NWAVES + (threadIdx.x >> 6),
                threadIdx.x & 63);
}

// One workgroup a row of cells: counts of its entries by cell in LDS, their sums,
// and the entries dealt out. (The order within a cell is the atomics'; each
// entry's logit is stored at its own place, so results do not depend on it. 4096 rows
// of 64 entries: 12 us, two reads of the ids and the latency of LDS.)
constexpr int kCellThreads = 1024;
__global__ void __launch_bounds__(kCellThreads)
cells_kernel(const VocabList l, int64_t M, int64_t col0, int64_t N, const CellShape shape, int bins,
             int per_cell, int* __restrict__ offsets, uint32_t* __restrict__ entries,
             float* __restrict__ z, int own) {
  extern __shared__ int count[];  // [bins]
  __shared__ int sums[kCellThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t cell = blockIdx.x;
  const int64_t m0 = shape.dense ? min(cell / 2 * 256, M - 256) + (cell & 1) * 128
                                 : cell * shape.rows;
  const int n = (int)min((int64_t)shape.rows, M - m0) * l.top;
  const int64_t* ids = l.ids + m0 * l.top;
  for (int b = tid; b < bins; b += kCellThreads) count[b] = 0;
  __syncthreads();
  for (int e = tid; e < n; e += kCellThreads) {
    const int64_t id = ids[e], at = id - col0;
    if (at >= 0 && at < N) atomicAdd(&count[(int)at / shape.cols], 1);
    if (own && (id < 0 || id >= l.vocab)) z[m0 * l.top + e] = id < 0 ? 0.0f : NAN;
  }
  __syncthreads();
  // counts to first places: a run of cells a thread, the runs' sums by waves
  const int run = (bins + kCellThreads - 1) / kCellThreads;
  const int b0 = min(bins, tid * run), b1 = min(bins, b0 + run);
  int own_sum = 0;
  for (int b = b0; b < b1; ++b) own_sum += count[b];
  int before = own_sum;
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const int v = __shfl_up(before, k);
    if (lane >= k) before += v;
  }
  if (lane == 63) sums[wave] = before;
  __syncthreads();
  before -= own_sum;
  for (int w = 0; w < wave; ++w) before += sums[w];
  int* out = offsets + cell * (bins + 1);
  for (int b = b0; b < b1; ++b) {
    const int c = count[b];
    count[b] = out[b] = before;
    before += c;
  }
  if (tid == kCellThreads - 1) out[bins] = before;
  __syncthreads();
  uint32_t* to = entries + cell * per_cell;
  for (int e = tid; e < n; e += kCellThreads) {
    const int64_t at = ids[e] - col0;
    if (at < 0 || at >= N) continue;
    const int b = (int)at / shape.cols, row = e / l.top;
    to[atomicAdd(&count[b], 1)] =
        (uint32_t)(row | ((int)at - b * shape.cols) << 7 | (e - row * l.top) << 14);
  }
}

// One row's teacher distribution, by one wave: entry k of lane k % 64. An
// entry takes part with an id >= 0 and a logit above -inf.
struct Teacher {
  float top, total;  // maximum logit, sum of exp((t - top) / T)
  bool any, bad;     // whether an entry takes part; an id past the vocabulary among them
};
__device__ __forceinline__ float teacher_logit(const VocabList& l, int64_t at) {
  return l.type == DType::BF16 ? bf16_to_f32(static_cast<const bf16_t*>(l.teacher)[at])
                               : static_cast<const float*>(l.teacher)[at];
}
__device__ __forceinline__ bool takes_part(int64_t id, float t) { return id >= 0 && !(t == -INFINITY); }
__device__ __forceinline__ float teacher_exp(float t, float top, float rt) {
  return __builtin_amdgcn_exp2f((t - top) * rt);
}
// The row's list is read once, into LDS: ids (-1 where an entry takes no part or is
// past the vocabulary) and logits (-inf where it takes none), padded to a multiple
// of 4.
__device__ __forceinline__ Teacher read_teacher(const VocabList& l, int64_t row, float rt, int lane,
                                                int* ids, float* t) {
  Teacher w;
  float top = -INFINITY;
  bool any = false, bad = false;
  for (int k = lane; k < (l.top + 3) / 4 * 4; k += 64) {
    int64_t id = -1;
    float v = -INFINITY;
    if (k < l.top) {
      id = l.ids[row * l.top + k];
      v = teacher_logit(l, row * l.top + k);
    }
    const bool in = takes_part(id, v), past = in && id >= l.vocab;
    any |= in;
    bad |= past;
    ids[k] = in && !past ? (int)id : -1;
    t[k] = in ? v : -INFINITY;
    if (in) top = fmaxf(top, v);
  }
  w.top = wave_max(top);
  w.any = __any(any);
  w.bad = __any(bad);
  float e = 0.0f;
  for (int k = lane; k < l.top; k += 64)  // (its own entries)
    if (!(t[k] == -INFINITY)) e += teacher_exp(t[k], w.top, rt);
  w.total = wave_sum(e);
  return w;
}

// The loss of one row, by one wave, from M = base and L = log_sum: log p_k =
// (t_k - top) / T - log total; an entry whose p is 0 adds nothing. Its lse is stored
// with it.
__device__ __forceinline__ void distill_loss(const VocabList& l, int64_t row, float base,
                                             float log_sum, const float* __restrict__ z, float* loss,
                                             float* lse, int lane, int* ids, float* t) {
  const float inv = 1.0f / l.temperature, rt = kLog2e / l.temperature;
  const Teacher w = read_teacher(l, row, rt, lane, ids, t);
  const float log_total = logf(w.total);
  float sum = 0.0f;
  for (int k = lane; k < l.top; k += 64) {
    if (t[k] == -INFINITY) continue;
    const float p = teacher_exp(t[k], w.top, rt) / w.total;
    if (p == 0.0f) continue;
    sum += p * (((t[k] - w.top) + (base - z[row * l.top + k])) * inv - log_total + log_sum);
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    loss[row] = !w.any ? 0.0f : w.bad ? NAN : l.temperature * l.temperature * sum;
    lse[row] = w.any ? base * inv + log_sum : 0.0f;
  }
}
// (join_kernel left M in loss and L in lse)
__global__ void __launch_bounds__(NT)
distill_loss_kernel(const VocabList l, int64_t rows, const float* __restrict__ z, float* loss,
                    float* lse) {
  __shared__ int ids[NWAVES][kMaxTop];
  __shared__ float ts[NWAVES][kMaxTop];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * NWAVES + wave;
  if (row >= rows) return;
  distill_loss(l, row, loss[row], lse[row], z, loss, lse, lane, ids[wave], ts[wave]);
}

// R rows a workgroup, their slots dealt over NT / R threads each (R a power of
// two: 32 where there are rows enough to read part in whole lines, 1 where there
// are few: 32 rows of 5408 slots 39.4 us with 32, 9.1 with 1); the threads' parts
// are joined in order. Targets: the loss too; a teacher's where a wave has a row or
// less (kJoinLoss: a launch less), else it has a kernel of its own.
enum Join { kTargets, kTeacher, kJoinLoss };
template <Join JOIN>
__global__ void __launch_bounds__(NT)
join_kernel(const float2* __restrict__ part, int64_t part_ld, int64_t slots, int R, const VocabList l,
            int64_t rows, const float* __restrict__ z, float* __restrict__ loss,
            float* __restrict__ lse) {
  const int r = threadIdx.x & (R - 1), g = threadIdx.x / R, groups = NT / R;
  const int64_t row = (int64_t)blockIdx.x * R + r;
  const float scale = kLog2e / l.temperature;
  float m = -INFINITY, s = 0.0f;
  auto scaled = [&](float2 v, float to) { return v.y * __builtin_amdgcn_exp2f((v.x - to) * scale); };
  auto add = [&](float2 v) {
    const float top = fmaxf(m, v.x), to = exponent_base(top);
    // (a part of -inf alone is 0 2^-inf; NaN sums stay)
    s = scaled(make_float2(m, s), to) + scaled(v, to);
    m = top;
  };
  if (row < rows) {
    const float2* p = part + row;
    int64_t i = g;
    for (; i + 7 * groups < slots; i += 8 * groups) {  // eight loads in flight
      float2 v[8];
      float top = m;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = p[(i + q * groups) * part_ld];
        top = fmaxf(top, v[q].x);
      }
      const float to = exponent_base(top);
      s = scaled(make_float2(m, s), to);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += scaled(v[q], to);
      m = top;
    }
    for (; i < slots; i += groups) add(p[i * part_ld]);
  }
  __shared__ float2 sums[NT];
  sums[threadIdx.x] = make_float2(m, s);
  for (int half = groups / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (g < half) {
      add(sums[threadIdx.x + half * R]);
      sums[threadIdx.x] = make_float2(m, s);
    }
  }
  if constexpr (JOIN == kJoinLoss) {
    __shared__ float2 own[NWAVES];
    if (g == 0 && r < NWAVES) own[r] = make_float2(exponent_base(m), logf(s));
    __shared__ int ids[NWAVES][kMaxTop];
    __shared__ float ts[NWAVES][kMaxTop];
    __syncthreads();
    const int wave = threadIdx.x >> 6;
    const int64_t mine = (int64_t)blockIdx.x * R + wave;
    if (wave < R && mine < rows)
      distill_loss(l, mine, own[wave].x, own[wave].y, z, loss, lse, threadIdx.x & 63, ids[wave],
                   ts[wave]);
    return;
  }
  if (g != 0 || row >= rows) return;
  const float base = exponent_base(m), log_sum = logf(s);
  if constexpr (JOIN == kTargets) {
    const bool part_of = l.ids[row] >= 0;
    lse[row] = part_of ? base + log_sum : 0.0f;
    loss[row] = !part_of ? 0.0f : l.ids[row] >= l.vocab ? NAN : log_sum + (base - z[row]);
  } else {
    loss[row] = base;
    lse[row] = log_sum;
  }
}

// Whether the row takes part (one wave; *bad: an id past the vocabulary)
__device__ __forceinline__ bool row_takes_part(const VocabList& l, int64_t row, int lane, bool* bad) {
  bool any = false, out = false;
  if (l.teacher) {
    for (int k = lane; k < l.top; k += 64) {
      const int64_t id = l.ids[row * l.top + k];
      if (!takes_part(id, teacher_logit(l, row * l.top + k))) continue;
      any = true;
      out |= id >= l.vocab;
    }
    any = __any(any);
    out = __any(out);
  } else {
    const int64_t id = l.ids[row];
    any = id >= 0;
    out = id >= l.vocab;
  }
  *bad = out;
  return any;
}

// Whether a row is in the copies of x: a row that takes no part, or whose gradients
// to loss and lse are zero, has g_z = 0 whatever its x holds, and 0 times an
// infinity there must not reach g_W.
__device__ __forceinline__ bool has_gradient(float a, float b) { return a != 0.0f || b != 0.0f; }

// 16 bytes at p, or zeros (as a choice of two values the compiler loads through an
// address that may be the zeros' in scratch memory)
__device__ __forceinline__ uint4 load16_if(bool c, const void* p) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (c) v = *static_cast<const uint4*>(p);
  return v;
}

// Four rows a workgroup, one wave each: the row's part in the gradient, and
// its copy of x; then the copy of W's last rows. (8192 rows of 4096: 29 us, 4.6 TB/s.)
constexpr int kLastRows = kTileRows;
template <typename T>
__global__ void __launch_bounds__(NT)
rows_kernel(const VocabList l, int64_t rows, int64_t padded, const float* __restrict__ g_loss,
            const float* __restrict__ g_lse, const float* __restrict__ lse,
            VocabRow* __restrict__ out, int K, const VocabCopies c) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * NWAVES + (threadIdx.x >> 6);
  if (row >= padded) {
    const int64_t last = row - padded, from = l.vocab / kLastRows * kLastRows + last;
    if (!c.W_last || last >= kLastRows) return;
    const T* w = static_cast<const T*>(c.W) + from * K;
    T* out_w = static_cast<T*>(c.W_last) + last * K;
    for (int k = lane * Vec<T>::E; k < K; k += 64 * Vec<T>::E)
      *reinterpret_cast<uint4*>(out_w + k) = load16_if(from < l.vocab, w + k);
    return;
  }
  float a = 0.0f, b = 0.0f, own = 0.0f;
  int target = -1;
  if (row < rows) {
    bool bad;
    const bool any = row_takes_part(l, row, lane, &bad);
    own = lse[row];
    if (l.teacher) {
      a = any ? g_loss[row] * l.temperature : 0.0f;
    } else {
      b = any ? g_loss[row] : 0.0f;
      a = any && g_lse ? b + g_lse[row] : b;
      target = any && !bad ? (int)l.ids[row] : -1;
    }
    if (bad) a = NAN;
  }
  if (lane == 0) out[row] = VocabRow{a, own, b, target};
  T* xs = static_cast<T*>(c.xs);
  if (!xs) return;
  const T* x = static_cast<const T*>(c.x);
  for (int k = lane * Vec<T>::E; k < K; k += 64 * Vec<T>::E) {
    const uint4 v = load16_if(has_gradient(a, b), x + row * K + k);
    *reinterpret_cast<uint4*>(xs + (c.tiled ? tiled_offset(row, k, K) : row * K + k)) = v;
    if (c.twice) *reinterpret_cast<uint4*>(xs + (padded + row) * K + k) = v;
    if (c.pairs) {
      T* two = static_cast<T*>(c.pairs) + tiled_offset(pair_row(row), k, K);
      *reinterpret_cast<uint4*>(two) = v;
      *reinterpret_cast<uint4*>(two + kPairLow) = v;
    }
  }
}

// x's copy with the rows innermost, for few rows (after their parts): a workgroup
// takes 64 columns, reads them row by row into LDS and writes them turned.
template <typename T>
__global__ void __launch_bounds__(NT)
turned_copy_kernel(const VocabRow* __restrict__ parts, int rows, int K, const VocabCopies c) {
  constexpr int E = Vec<T>::E;
  __shared__ T tile[few_tokens(sizeof(T) == 2 ? DType::BF16 : DType::F32)][64 + E];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k0 = blockIdx.x * 64;
  const T* x = static_cast<const T*>(c.x);
  for (int row = wave; row < c.xt_rows; row += NWAVES) {
    const bool any = row < rows && has_gradient(parts[row].a, parts[row].b);
    tile[row][lane] = any && k0 + lane < K ? x[(int64_t)row * K + k0 + lane] : T{};
  }
  __syncthreads();
  const int n = min(64, K - k0) * c.xt_rows / E;  // 16-byte pieces
  T* out = static_cast<T*>(c.xt) + (int64_t)k0 * c.xt_rows;
  for (int i = threadIdx.x; i < n; i += NT) {
    const int k = i * E / c.xt_rows, row = i * E % c.xt_rows;
    union { T e[E]; uint4 v; } u;
#pragma unroll
    for (int e = 0; e < E; ++e) u.e[e] = tile[row + e][k];
    reinterpret_cast<uint4*>(out)[i] = u.v;
  }
}

// One wave a row: where the row's id j lies in the piece,
//   g_z[j] = a (exp(z_j / T - lse) - the sum of p over the entries with that id).
// The entries' p are in LDS, so that each finds its id's other entries (an id
// listed twice: both write the same value). 4096 rows of 64 entries 12 us.
template <typename T>
__global__ void __launch_bounds__(NT)
listed_grad_kernel(const VocabList l, int64_t rows, const VocabRow* __restrict__ r,
                   const float* __restrict__ z, T* __restrict__ gz, int64_t ldg, int tiled,
                   int64_t low, int col0, int N) {
  __shared__ __attribute__((aligned(16))) int ids[NWAVES][kMaxTop];
  __shared__ __attribute__((aligned(16))) float p[NWAVES][kMaxTop];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * NWAVES + wave;
  if (row >= rows) return;
  const VocabRow own = r[row];
  if (own.a == 0.0f) return;  // (whose gradient is zero)
  const float inv = 1.0f / l.temperature, rt = kLog2e / l.temperature;
  const Teacher w = read_teacher(l, row, rt, lane, ids[wave], p[wave]);
  const int padded = (l.top + 3) / 4 * 4;
  for (int k = lane; k < padded; k += 64) {
    const float t = p[wave][k];
    p[wave][k] = t == -INFINITY ? 0.0f : teacher_exp(t, w.top, rt) / w.total;
  }
  // (a wave reads its own row's entries only)
  asm volatile("" ::: "memory");
  wait_lds();
  asm volatile("" ::: "memory");
  for (int k = lane; k < l.top; k += 64) {
    const int id = ids[wave][k];
    if (id < col0 || id >= col0 + N) continue;
    float sum = 0.0f;
    for (int q = 0; q < padded; q += 4) {
      const int4 i = *reinterpret_cast<const int4*>(&ids[wave][q]);
      const float4 v = *reinterpret_cast<const float4*>(&p[wave][q]);
      sum += i.x == id ? v.x : 0.0f;
      sum += i.y == id ? v.y : 0.0f;
      sum += i.z == id ? v.z : 0.0f;
      sum += i.w == id ? v.w : 0.0f;
    }
    const float e = softmax_at<T>(z[row * l.top + k], inv, own.lse);
    const int64_t at = tiled ? tiled_offset(low ? pair_row(row) : row, id - col0, ldg)
                             : row * ldg + (id - col0);
    const float v = own.a * (e - sum);
    store_as(gz + at, v);
    if constexpr (sizeof(T) == 2) {
      if (low) store_as(gz + at + low, low_part(v, bf16_to_f32(f32_to_bf16(v))));
    }
  }
}

bool fits(int64_t blocks) { return blocks * NT <= kMaxWorkItems; }

}  // namespace

hipError_t launch_listed_logits(DType t, const void* x, const void* W, const VocabList& l,
                                int64_t rows, int K, float* z, hipStream_t s) {
  // (as many rows a launch as it takes)
  const int64_t most = (kMaxWorkItems - NT) / 64 / listed_waves(1, l.top);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    const int64_t blocks = (listed_waves(n, l.top) + NWAVES - 1) / NWAVES;
    if (!fits(blocks)) return hipErrorInvalidValue;
    VocabList at = l;
    at.ids += r * l.top;  // (the teacher's logits are not read)
    float* to = z + r * l.top;
    if (t == DType::BF16)
      hipLaunchKernelGGL(listed_logits_kernel<bf16_t>, dim3((unsigned)blocks), dim3(NT), 0, s,
                         static_cast<const bf16_t*>(x) + r * K, static_cast<const bf16_t*>(W), at, n,
                         K, to);
    else
      hipLaunchKernelGGL(listed_logits_kernel<float>, dim3((unsigned)blocks), dim3(NT), 0, s,
                         static_cast<const float*>(x) + r * K, static_cast<const float*>(W), at, n, K,
                         to);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_vocab_cells(const VocabList& l, int64_t M, int64_t col0, int64_t N,
                              const CellShape& shape, int* offsets, uint32_t* entries, float* z,
                              bool own, hipStream_t s) {
  const int64_t bins = shape.bins(N), cells = shape.row_cells(M);
  if (bins < 1 || bins > kMaxBins || shape.rows > 128 || shape.cols > 128 || l.top > kMaxTop ||
      cells * kCellThreads > kMaxWorkItems || (shape.dense && M < 256))
    return hipErrorInvalidValue;
  hipLaunchKernelGGL(cells_kernel, dim3((unsigned)cells), dim3(kCellThreads),
                     (unsigned)(bins * sizeof(int)), s, l, M, col0, N, shape, (int)bins,
                     shape.rows * l.top, offsets, entries, z, (int)own);
  return hipGetLastError();
}

hipError_t launch_vocab_loss(const float2* part, int64_t part_ld, int64_t slots, const VocabList& l,
                             int64_t rows, const float* z, float* loss, float* lse, hipStream_t s) {
  int R = 1;
  while (R < 32 && R * 256 <= rows) R *= 2;
  const int64_t blocks = (rows + R - 1) / R, loss_blocks = (rows + NWAVES - 1) / NWAVES;
  if (!fits(blocks) || !fits(loss_blocks)) return hipErrorInvalidValue;
  const auto kernel = !l.teacher     ? join_kernel<kTargets>
                      : R <= NWAVES ? join_kernel<kJoinLoss>
                                    : join_kernel<kTeacher>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(NT), 0, s, part, part_ld, slots, R, l, rows,
                     z, loss, lse);
  if (l.teacher && R > NWAVES)
    hipLaunchKernelGGL(distill_loss_kernel, dim3((unsigned)loss_blocks), dim3(NT), 0, s, l, rows, z,
                       loss, lse);
  return hipGetLastError();
}

hipError_t launch_vocab_rows(DType t, const VocabList& l, int64_t rows, int64_t padded,
                             const float* g_loss, const float* g_lse, const float* lse,
                             VocabRow* out, int K, const VocabCopies& c, hipStream_t s) {
  const int64_t blocks = (padded + (c.W_last ? kLastRows : 0) + NWAVES - 1) / NWAVES;
  if (!fits(blocks)) return hipErrorInvalidValue;
  if (t == DType::BF16)
    hipLaunchKernelGGL(rows_kernel<bf16_t>, dim3((unsigned)blocks), dim3(NT), 0, s, l, rows, padded,
                       g_loss, g_lse, lse, out, K, c);
  else
    hipLaunchKernelGGL(rows_kernel<float>, dim3((unsigned)blocks), dim3(NT), 0, s, l, rows, padded,
                       g_loss, g_lse, lse, out, K, c);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (c.xt) {
    if (rows > few_tokens(t) || c.xt_rows > few_tokens(t) || c.xt_rows < rows ||
        c.xt_rows != few_padded(t, (int)rows))
      return hipErrorInvalidValue;
    const dim3 grid((unsigned)((K + 63) / 64));
    if (t == DType::BF16)
      hipLaunchKernelGGL(turned_copy_kernel<bf16_t>, grid, dim3(NT), 0, s, out, (int)rows, K, c);
    else
      hipLaunchKernelGGL(turned_copy_kernel<float>, grid, dim3(NT), 0, s, out, (int)rows, K, c);
  }
  return hipGetLastError();
}

hipError_t launch_vocab_last_rows(DType t, int64_t vocab, int K, const VocabCopies& c,
                                  hipStream_t s) {
  VocabList l;
  l.vocab = vocab;
  return launch_vocab_rows(t, l, 0, 0, nullptr, nullptr, nullptr, nullptr, K, c, s);
}

hipError_t launch_vocab_listed_grad(DType t, const VocabList& l, int64_t rows, const VocabRow* r,
                                    const float* z, void* gz, int64_t ldg, bool tiled, int64_t low,
                                    int col0, int N, hipStream_t s) {
  const int64_t blocks = (rows + NWAVES - 1) / NWAVES;
  if (!fits(blocks) || l.top > kMaxTop || (tiled && low && low != kPairLow)) return hipErrorInvalidValue;
  if (t == DType::BF16)
    hipLaunchKernelGGL(listed_grad_kernel<bf16_t>, dim3((unsigned)blocks), dim3(NT), 0, s, l, rows,
                       r, z, static_cast<bf16_t*>(gz), ldg, (int)tiled, low, col0, N);
  else
    hipLaunchKernelGGL(listed_grad_kernel<float>, dim3((unsigned)blocks), dim3(NT), 0, s, l, rows,
                       r, z, static_cast<float*>(gz), ldg, (int)tiled, low, col0, N);
  return hipGetLastError();
}

}  // namespace poetx
