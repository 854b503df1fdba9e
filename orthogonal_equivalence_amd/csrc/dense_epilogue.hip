// The large products of the dense linear's forward: C = A B^T on the
// 256 x 256 tile loop of dense_core.h (bf16, both operands K-major), whose
// accumulators end in
//   u = C scale[n] + bias[n],  y = act(u) + residual
// instead of being stored. At 8192 x 14336 x 4096 the loop runs at ~1.4
// PFLOP/s; a separate pass for the activation would read u and write y once
// more (470 MB, ~90 us at the copy rate).
//
// Each lane holds four consecutive columns of one row for each of its 64
// 16 x 16 fragments. Fragments are taken column by column, so that a column's
// bias and scale are loaded once for eight fragments and the next column's
// residual values (8 bytes a lane) are in flight while this one's are used.
// u, where it is kept, leaves through the staging tile first, while y waits
// in the 128 registers that the loop's operand fragments leave free.
#include "dense_core.h"
#include "epilogue.h"

namespace poetx {
namespace {

template <Activation ACT, bool SAVE_U>
struct DenseEpilogue {
  // this lane's column of fragment column j
  static __device__ __forceinline__ int column(const Dense<true, true>& d, int j, int ln) {
    return d.wn * 128 + 16 * j + 4 * (ln >> 4);
  }
  static __device__ __forceinline__ int row(const Dense<true, true>& d, int i, int ln) {
    return d.wm * 128 + 16 * i + (ln & 15);
  }
  static __device__ __forceinline__ void load_column(const Epilogue& ep, int n, float4& sc,
                                                     float4& bi) {
    sc = ep.scale ? *reinterpret_cast<const float4*>(ep.scale + n)
                  : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    bi = ep.bias ? *reinterpret_cast<const float4*>(ep.bias + n)
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  static __device__ __forceinline__ void stage(int m, int n, uint2 v) {
    *reinterpret_cast<uint2*>(g_dense_lds + stage_off(m, n)) = v;
  }

  static __device__ __forceinline__ void run(Dense<true, true>& d, const Epilogue& ep, int m0, int n0) {
    // opaque copies of the lane and thread ids: keeps the compiler from
    // hoisting the epilogue's address arithmetic out of the tile loop
    int ln = d.lane, tid = (int)threadIdx.x;
    asm volatile("" : "+v"(ln), "+v"(tid));
    const bf16_t* res = static_cast<const bf16_t*>(ep.residual);
    uint2 r[2][FM];
    uint2 keep[SAVE_U ? FN : 1][SAVE_U ? FM : 1];
    auto load_residual = [&](int j) {
      const bf16_t* p = res + (int64_t)(m0 + row(d, 0, ln)) * ep.ld + n0 + column(d, j, ln);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        r[j & 1][i] = *reinterpret_cast<const uint2*>(p + 16 * i * ep.ld);
    };
    if (res) load_residual(0);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = column(d, j, ln);
      float4 sc, bi;
      load_column(ep, n0 + n, sc, bi);
      if (res && j + 1 < FN) load_residual(j + 1);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        float v[4] = {fmaf(d.acc[i][j][0], sc.x, bi.x), fmaf(d.acc[i][j][1], sc.y, bi.y),
                      fmaf(d.acc[i][j][2], sc.z, bi.z), fmaf(d.acc[i][j][3], sc.w, bi.w)};
        if constexpr (SAVE_U) stage(row(d, i, ln), n, Quad<bf16_t>::pack(v));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = activate<bf16_t, ACT>(v[e]);
        if (res) {
          const uint2 w = r[j & 1][i];
          v[0] += __uint_as_float(w.x << 16);
          v[1] += __uint_as_float(w.x & 0xffff0000u);
          v[2] += __uint_as_float(w.y << 16);
          v[3] += __uint_as_float(w.y & 0xffff0000u);
        }
        if constexpr (SAVE_U) keep[j][i] = Quad<bf16_t>::pack(v);
        else stage(row(d, i, ln), n, Quad<bf16_t>::pack(v));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_lds();
    barrier_nofence();
    if constexpr (SAVE_U) {
      d.store_staged(static_cast<bf16_t*>(ep.u), ep.ld, m0, n0, tid);
      wait_lds();
      barrier_nofence();  // every wave has read the staged u
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) stage(row(d, i, ln), column(d, j, ln), keep[j][i]);
      wait_lds();
      barrier_nofence();
    }
    d.store_staged(static_cast<bf16_t*>(ep.y), ep.ld, m0, n0, tid);
    wait_lds();
    barrier_nofence();
  }
};

template <Activation ACT, bool SAVE_U>
__global__ void __launch_bounds__(NT)
dense_epilogue_kernel(const bf16_t* __restrict__ A, const bf16_t* __restrict__ B, int M, int N,
                      int K, int64_t lda, int64_t ldb, int b_tiled, const Epilogue ep) {
  const int num_mt = (M + BM - 1) / BM, num_nt = (N + BN - 1) / BN;
  const int total = num_mt * num_nt;
  const int ntiles = K / BK;
  Dense<true, true> d;
  d.init(lda, ldb, false, b_tiled != 0);
  for (int tile = blockIdx.x; tile < total; tile += (int)gridDim.x) {
    int mt, nt;
    xcd_grouped_tile_at(tile, total, num_mt, num_nt, mt, nt);
    const int m0 = min(mt * BM, M - BM), n0 = min(nt * BN, N - BN);
    d.set_tile(A, B, lda, ldb, m0, n0);
    d.prefetch(ntiles);
    d.start(ntiles);
    d.mainloop(ntiles);
    wait_lds();
    barrier_nofence();  // every wave is done with the ring
    DenseEpilogue<ACT, SAVE_U>::run(d, ep, m0, n0);
  }
}

template <Activation ACT>
hipError_t launch_act(const DenseProduct& p, int grid, hipStream_t s) {
  const bf16_t* a = static_cast<const bf16_t*>(p.A);
  const bf16_t* b = static_cast<const bf16_t*>(p.B);
  if (p.ep.u)
    hipLaunchKernelGGL((dense_epilogue_kernel<ACT, true>), dim3(grid), dim3(NT), 0, s, a, b, p.M,
                       p.N, p.K, p.lda, p.ldb, (int)p.b_tiled, p.ep);
  else
    hipLaunchKernelGGL((dense_epilogue_kernel<ACT, false>), dim3(grid), dim3(NT), 0, s, a, b, p.M,
                       p.N, p.K, p.lda, p.ldb, (int)p.b_tiled, p.ep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_epilogue(const DenseProduct& p, hipStream_t s) {
  if (!dense_supported(p.M, p.N, p.K, p.lda, p.ldb, p.ep.ld)) return hipErrorInvalidValue;
  if (p.b_tiled && (p.N % BN != 0 || p.ldb != p.K)) return hipErrorInvalidValue;
  int grid = 0;
  const hipError_t e = dense_grid(p.M, p.N, &grid);
  if (e != hipSuccess) return e;
  switch (static_cast<Activation>(p.ep.act)) {
    case Activation::None: return launch_act<Activation::None>(p, grid, s);
    case Activation::Relu: return launch_act<Activation::Relu>(p, grid, s);
    case Activation::Gelu: return launch_act<Activation::Gelu>(p, grid, s);
    case Activation::GeluTanh: return launch_act<Activation::GeluTanh>(p, grid, s);
    case Activation::Silu: return launch_act<Activation::Silu>(p, grid, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace poetx
