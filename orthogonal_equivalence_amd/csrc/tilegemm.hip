// Matrix products of the dense linear with its epilogue, for any number of
// rows: one workgroup of four waves computes a BM x BN tile of
//   C(m, n) = sum_k A(m, k) B(n, k),
//   A(m, k) = A[m lda + k] (K-major) or A[k lda + m] (M-major), B likewise,
// and ends with the float32 accumulators in registers, so that scale, bias,
// activation and residual cost no pass of their own (epilogue.h). With a
// split reduction axis each workgroup leaves its float32 partial tile in the
// workspace and finish_kernel sums them in split order and applies the
// epilogue.
//
// The reduction runs in steps of 128 bytes (64 bf16, 32 float32) through a
// ring of kStages LDS slots filled by global_load_lds_dwordx4, kStages - 1
// steps ahead: at the mid sizes this kernel serves (a few tiles per CU, often
// one) nothing else hides the latency of the loads. Rows past the end are
// read as the last row and never stored; a last step that is not full is
// zeroed in LDS past its end, in both operands.
//
// LDS tiles, 16-byte chunks XOR-swizzled against bank conflicts (64 banks of
// 4 bytes; a fragment read takes 256 bytes per clock):
//   K-major  [rows][128 bytes]: chunk c of row r at c ^ ((r >> 1) & 7): the
//            16 rows of a fragment read fill two rows' worth of banks once;
//   MN-major [k][rows]: bf16 is read by ds_read_b64_tr_b16, 32-byte pieces
//            of k rows 8 g + 0..3 (g = lane / 16), float32 by 4-byte reads,
//            64-byte pieces of k rows 4 g + j; the swizzle spreads those rows
//            over the banks (mn_swz).
// float32 products run on v_mfma_f32_16x16x4_f32: a lane's 16-byte chunk
// holds 4 consecutive k, and product j takes element j of both operands'
// chunks, so the order of k inside a step of 16 differs from memory order in
// the same way for both.
#include <algorithm>

#include "common.h"
#include "epilogue.h"
#include "kernels.h"
#include "lds_dma.h"

namespace poetx {
namespace {

constexpr int NT = 256;
constexpr int kRowBytes = 128;

template <typename T> struct Elem;
template <> struct Elem<bf16_t> {
  static constexpr int E = 8, BK = 64;  // elements per 16-byte chunk, per step
  typedef bf16x8_t Frag;
};
template <> struct Elem<float> {
  static constexpr int E = 4, BK = 32;
  typedef floatx4 Frag;
};

__device__ __forceinline__ int k_swz(int row) { return (row >> 1) & 7; }

// chunk XOR of row k of an MN-major tile of ROWS elements per k
template <typename T, int ROWS> __device__ __forceinline__ int mn_swz(int k) {
  if constexpr (sizeof(T) == 4) return ((k >> 2) & 3) << 2;  // 64-byte pieces
  if constexpr (ROWS >= 128) return ((k & 3) | (((k >> 3) & 1) << 2)) << 1;  // 32-byte pieces
  return (((k >> 1) & 1) | (((k >> 3) & 1) << 1)) << 1;  // (k & 1 picks the half of the banks)
}

// One operand's tile: ROWS rows (m or n), one step of k.
template <typename T, int ROWS, bool KMAJ>
struct Operand {
  static constexpr int E = Elem<T>::E, BK = Elem<T>::BK;
  static constexpr int BYTES = ROWS * kRowBytes;
  static constexpr int PIECES = BYTES / 1024 / 4;  // 1 KB copies per wave and step
  static constexpr int CPR = ROWS / E;             // chunks per k row (MN-major)
  static_assert(PIECES >= 1, "a tile is at least 4 KB");

  const T* base;  // K-major: row r0; MN-major: column r0
  int64_t ld;
  int rows, K;  // rows of the operand from r0 on; whole reduction length

  __device__ __forceinline__ void init(const T* p, int64_t ld_, int r0, int total, int K_) {
    ld = ld_;
    K = K_;
    rows = total - r0;
    base = KMAJ ? p + (int64_t)r0 * ld : p + r0;
  }
  // this wave's copies of step k0 into `slot`
  __device__ __forceinline__ void issue(char* slot, int k0, int wave, int lane) const {
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const int q = wave + 4 * j;
      const int c16 = q * 64 + lane;  // 16-byte chunk of the tile, in LDS order
      const T* src;
      if (KMAJ) {
        const int r = c16 >> 3, c = (c16 & 7) ^ k_swz(r);
        src = base + (int64_t)min(r, rows - 1) * ld + min(k0 + c * E, K - E);
      } else {
        const int k = c16 / CPR, c = (c16 % CPR) ^ mn_swz<T, ROWS>(k);
        src = base + (int64_t)min(k0 + k, K - 1) * ld + min(c * E, rows - E);
      }
      dma16(src, reinterpret_cast<const bf16_t*>(slot + q * 1024));
    }
  }
  // zeros from k = kleft on (the whole workgroup)
  __device__ __forceinline__ void zero_tail(char* slot, int kleft, int tid) const {
    for (int c16 = tid; c16 < BYTES / 16; c16 += NT) {
      bool out;
      if (KMAJ) {
        const int r = c16 >> 3, c = (c16 & 7) ^ k_swz(r);
        out = c * E >= kleft;
      } else {
        out = c16 / CPR >= kleft;
      }
      if (out) *reinterpret_cast<uint4*>(slot + 16 * c16) = make_uint4(0, 0, 0, 0);
    }
  }
  // fragment of rows r0 .. r0 + 15 (tile-relative), half-step s (0, 1): lane
  // l holds row l % 16, chunk 4 s + l / 16
  __device__ __forceinline__ typename Elem<T>::Frag read(const char* slot, int r0, int s,
                                                         int lane) const {
    const int r = r0 + (lane & 15), g = lane >> 4;
    if constexpr (KMAJ) {
      return *reinterpret_cast<const typename Elem<T>::Frag*>(
          slot + r * kRowBytes + (((4 * s + g) ^ k_swz(r)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      // transposing read: lane j of 16 addresses 8 bytes at (k + j / 4, 4 (j % 4))
      const int i = lane & 15;
      union { short4_t h[2]; bf16x8_t v; } u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 32 * s + 8 * g + 4 * h + (i >> 2), n = r0 + 4 * (i & 3);
        const int c = (n / E) ^ mn_swz<T, ROWS>(k);
        u.h[h] = ds_read_tr4(reinterpret_cast<const bf16_t*>(slot) + k * ROWS + c * E + (n & 7));
      }
      return u.v;
    } else {
      floatx4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 16 * s + 4 * g + j;
        const int c = (r / E) ^ mn_swz<T, ROWS>(k);
        v[j] = reinterpret_cast<const float*>(slot)[k * ROWS + c * E + (r & 3)];
      }
      return v;
    }
  }
};

__device__ __forceinline__ floatx4 mma(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mma(floatx4 a, floatx4 b, floatx4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// at most `n` steps of LPW copies still in flight
template <int LPW, int NS> __device__ __forceinline__ void wait_steps(int n) {
  static_assert(NS >= 2 && NS <= 4, "ring depth");
  if (NS > 3 && n >= 2) wait_vm<2 * LPW>();
  else if (NS > 2 && n >= 1) wait_vm<LPW>();
  else wait_vm<0>();
}

template <typename T, int BM, int BN, bool A_KMAJ, bool B_KMAJ, int NS>
__global__ void __launch_bounds__(NT) tile_kernel(const TileProduct p) {
  typedef Operand<T, BM, A_KMAJ> OpA;
  typedef Operand<T, BN, B_KMAJ> OpB;
  constexpr int BK = Elem<T>::BK;
  constexpr int TM = BM / 2, TN = BN / 2;  // 2 x 2 waves
  constexpr int FM = TM / 16, FN = TN / 16;
  constexpr int SLOT = OpA::BYTES + OpB::BYTES;
  constexpr int LPW = OpA::PIECES + OpB::PIECES;
  __shared__ __attribute__((aligned(1024))) char ring[NS * SLOT];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  int mt, nt;
  xcd_grouped_tile((p.M + BM - 1) / BM, (p.N + BN - 1) / BN, mt, nt);
  const int m0 = mt * BM, n0 = nt * BN;
  const int kbeg = blockIdx.y * p.kchunk, kend = min(p.K, kbeg + p.kchunk);
  const int steps = (kend - kbeg + BK - 1) / BK;

  OpA oa;
  OpB ob;
  oa.init(static_cast<const T*>(p.A), p.lda, m0, p.M, p.K);
  ob.init(static_cast<const T*>(p.B), p.ldb, n0, p.N, p.K);

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int t = 0; t < NS - 1; ++t)
    if (t < steps) {
      oa.issue(ring + t * SLOT, kbeg + t * BK, wave, lane);
      ob.issue(ring + t * SLOT + OpA::BYTES, kbeg + t * BK, wave, lane);
    }
  int slot = 0;
  for (int t = 0; t < steps; ++t) {
    char* sa = ring + slot * SLOT;
    char* sb = sa + OpA::BYTES;
    // this wave's copies of step t have landed and its reads of step t - 1
    // are done; after the barrier that holds for every wave
    wait_steps<LPW, NS>(steps - 1 - t);
    wait_lds();
    barrier_nofence();
    const int kleft = kend - kbeg - t * BK;
    if (kleft < BK) {
      oa.zero_tail(sa, kleft, tid);
      ob.zero_tail(sb, kleft, tid);
      wait_lds();
      barrier_nofence();
    }
    if (t + NS - 1 < steps) {  // into the slot of step t - 1
      char* nx = ring + (slot == 0 ? NS - 1 : slot - 1) * SLOT;
      oa.issue(nx, kbeg + (t + NS - 1) * BK, wave, lane);
      ob.issue(nx + OpA::BYTES, kbeg + (t + NS - 1) * BK, wave, lane);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      typename Elem<T>::Frag fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = oa.read(sa, wm * TM + 16 * i, s, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = ob.read(sb, wn * TN + 16 * j, s, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mma(fb[j], fa[i], acc[i][j]);
    }
    slot = slot + 1 == NS ? 0 : slot + 1;
  }

  // (operand roles swapped: lane l holds row 16 i + l % 16, columns
  // 16 j + 4 (l / 16) .. + 3 of its wave's tile)
  float* part = p.part ? p.part + (int64_t)blockIdx.y * p.M * p.N : nullptr;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + wm * TM + 16 * i + (lane & 15);
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + wn * TN + 16 * j + 4 * (lane >> 4);
      if (n >= p.N) continue;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if (part) Quad<float>::store(part + (int64_t)m * p.N + n, v);
      else epilogue4<T>(p.ep, m, n, v);
    }
  }
}

// sum of the partial tiles in split order, then the epilogue; four columns a
// thread
template <typename T>
__global__ void __launch_bounds__(NT)
finish_kernel(const float* __restrict__ part, int nsplit, int64_t rows, int N, Epilogue ep) {
  const int quads = N / 4;
  const int64_t total = rows * quads, stride = rows * N;
  for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < total; i += (int64_t)gridDim.x * NT) {
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < nsplit; ++s) {
      float w[4];
      Quad<float>::load(part + s * stride + m * N + n, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += w[e];
    }
    epilogue4<T>(ep, m, n, v);
  }
}

template <typename T, int BM, int BN, int NS>
hipError_t launch_cfg(bool ak, bool bk, const TileProduct& p, int nsplit, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, nsplit);
  if (ak && bk)
    hipLaunchKernelGGL((tile_kernel<T, BM, BN, true, true, NS>), grid, dim3(NT), 0, s, p);
  else if (ak)
    hipLaunchKernelGGL((tile_kernel<T, BM, BN, true, false, NS>), grid, dim3(NT), 0, s, p);
  else if (!bk)
    hipLaunchKernelGGL((tile_kernel<T, BM, BN, false, false, NS>), grid, dim3(NT), 0, s, p);
  else
    return hipErrorInvalidValue;  // no caller has an M-major A with a K-major B
  return hipGetLastError();
}

int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) {
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

}  // namespace

TilePlan plan_tile_product(DType t, int64_t M, int64_t N, int64_t K) {
  const int bk = t == DType::BF16 ? 64 : 32;
  TilePlan r;
  r.big = tiles_of(M, N, 128, 128) >= 192;
  const int64_t tiles = r.big ? tiles_of(M, N, 128, 128) : tiles_of(M, N, 64, 64);
  int64_t split = 1;
  if (tiles < 192) split = std::min<int64_t>((256 + tiles - 1) / tiles, K / (8 * bk));
  split = std::max<int64_t>(1, split);
  const int64_t steps = (K + bk - 1) / bk;
  const int64_t per = (steps + split - 1) / split;
  r.kchunk = (int)(per * bk);
  r.nsplit = (int)((steps + per - 1) / per);
  r.part_floats = r.nsplit > 1 ? (size_t)r.nsplit * M * N : 0;
  return r;
}

hipError_t launch_tile_product(DType t, const TilePlan& plan, TileProduct p, bool a_kmajor,
                               bool b_kmajor, hipStream_t s) {
  p.kchunk = plan.kchunk;
  if (plan.nsplit == 1) p.part = nullptr;
  else if (!p.part) return hipErrorInvalidValue;
  hipError_t e;
  if (t == DType::BF16)
    e = plan.big ? launch_cfg<bf16_t, 128, 128, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s)
                 : launch_cfg<bf16_t, 64, 64, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s);
  else
    e = plan.big ? launch_cfg<float, 128, 128, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s)
                 : launch_cfg<float, 64, 64, 4>(a_kmajor, b_kmajor, p, plan.nsplit, s);
  if (e != hipSuccess || plan.nsplit == 1) return e;
  const int64_t groups = (int64_t)p.M * (p.N / 4);
  const int grid = (int)std::min<int64_t>((groups + NT - 1) / NT, 4096);
  if (t == DType::BF16)
    hipLaunchKernelGGL(finish_kernel<bf16_t>, dim3(grid), dim3(NT), 0, s, p.part, plan.nsplit,
                       (int64_t)p.M, p.N, p.ep);
  else
    hipLaunchKernelGGL(finish_kernel<float>, dim3(grid), dim3(NT), 0, s, p.part, plan.nsplit,
                       (int64_t)p.M, p.N, p.ep);
  return hipGetLastError();
}

}  // namespace poetx
