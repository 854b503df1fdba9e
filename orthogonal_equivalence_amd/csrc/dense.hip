// The dense W0 products of the POET-X layer on bf16 MFMA: the forward
// Z = U W0^T (W0 is [d_out][d_in], so both operands are K-contiguous) and the
// backward g_U = g_Z W0 (W0 read along its rows, i.e. N-contiguous). W0 is
// the frozen weight of the layer (gist.science technical summary of "POET-X:
// Memory-efficient LLM Training by Scaling Orthogonal Transformation",
// section 2 Methodik); these two products carry almost all of the layer's
// arithmetic.
//
// C[M][N] = A[M][K] B(n, k) with B(n, k) = B[n][k] (K-major) or B[k][n]
// (N-major); bf16 in and out, float32 accumulation.
//
// One workgroup of four waves, one per SIMD, computes a 256 x 256 tile; each
// wave owns a 128 x 128 quarter as 8 x 8 tiles of v_mfma_f32_16x16x32_bf16
// whose 256 accumulator registers live in AGPRs. A 128 x 128 wave tile is
// the largest the register file allows and reads the fewest operand bytes
// from LDS per product (64 KB per 32-deep K tile for the workgroup, against
// 96 KB for eight 128 x 64 waves). Measured on gfx950 at one wave per SIMD:
// a back-to-back 16x16x32 stream issues every 16.2 cycles, and every
// ds_read_b128 interleaved with it costs about 8 more, so operand bytes read
// into registers, not the products, set the pace; the fewer of them, the
// less power the LDS draws, and the chip's clock under this load is power
// limited.
//
// K tiles of 32 are copied from global memory straight into a 4-slot LDS
// ring with global_load_lds_dwordx4 (no register staging, no LDS store
// instructions), three tiles ahead of the products. Every wave issues its
// share of the copies, one 1 KB piece after each row of eight products, so
// the address unit sees a steady stream rather than a burst that would block
// the issuing wave (in-order issue: a blocked copy holds back the products
// behind it). Per K tile: the first row of products runs on registers, then
// one barrier publishes the next K tile and frees the slot of the current
// one, then the other seven rows run while the next tile's fragments are
// read, two per row, into the second register set.
//
// The products are inline asm with the accumulator tied to an AGPR operand:
// with the compiler's builtin the register allocator rotated the
// accumulators between AGPRs on every iteration (hundreds of
// v_accvgpr_mov per K tile). The first K tile uses a zero addend, so the
// accumulators are never cleared by VALU writes. The compiler does not see
// the asm products, so the wait states before the epilogue reads them are
// explicit.
//
// LDS layouts (16-byte chunks XOR-swizzled so that the fragment reads are
// free of bank conflicts):
//   K-major tile  [256 rows][32 k]  (64-byte rows): chunk c of row r at
//                 c ^ ((r >> 1) & 3). Measured on gfx950 (whose LDS returns
//                 256 bytes per clock for these reads): this pattern of
//                 ds_read_b128 fragment reads streams 234 B/clk per CU, while
//                 c ^ (((r >> 1) & 3) ^ ((r >> 3) & 1)), r & 3, (r >> 2) & 3
//                 or no swizzle all give 128 B/clk (two-way conflicts);
//   N-major tile  [32 k][256 n]     (512-byte rows): chunk c of row k at
//                 c ^ 2 (k & 3), read with the transposing ds_read_b64_tr_b16;
//   epilogue      [256 m][256 n] bf16 (the whole ring): chunk c of row m at
//                 c ^ (m & 15).
// The products are issued as D' = B A^T (the operand roles swapped), so each
// lane ends up holding four consecutive output columns of one row and stages
// them with one 8-byte LDS write; the staged tile leaves as 16-byte stores of
// whole 512-byte row segments.
//
// A may also be in the tiled layout (kernels.h): each 256 x 32 piece of the
// matrix one contiguous 16 KB block, so a K tile of a 256-row panel is one
// block and every copy reads 1 KB of consecutive bytes (eight whole 128-byte
// lines), where the row-major layout gives each copy 16 half lines of 64
// bytes; on the 8B MLP-up shapes the forward took 7 % less time and the
// backward 4 % less. A K-major B may be tiled the same way (the forward's
// weight, where a caller widens INT8 codes into a buffer of its own).
//
// M and N must be at least 256 and K a multiple of 32: a tile that would
// cross the end of M or N is shifted back to end there (it recomputes, and
// rewrites with identical values, part of its neighbour), so no load or
// store needs a bounds test. The kernel is persistent: workgroup g computes
// tiles g, g + G, ... (G = grid size, a multiple of 8, so each workgroup
// stays on one XCD's share of the grouped tile order).
#include "dense_core.h"

namespace poetx {
namespace {

// nbatch independent products of the same shape, product q at A + q sA,
// B + q sB, C + q sC (the block-diagonal products of b >= 512 blocks run as
// one batched launch); their output tiles form one grid of num_mt x
// (nbatch num_nt) tiles, products side by side along N.
template <bool B_KMAJ, bool FUSE_R = false, bool KEEP_Z = true>
__global__ void __launch_bounds__(NT)
dense_kernel(const bf16_t* __restrict__ A, const bf16_t* __restrict__ B, bf16_t* __restrict__ C,
             int M, int N, int K, int64_t lda, int64_t ldb, int64_t ldc,
             const bf16_t* __restrict__ R, bf16_t* __restrict__ Y, int64_t ldy, int nbatch,
             int64_t sA, int64_t sB, int64_t sC, int a_tiled, int b_tiled) {
  const int num_mt = (M + BM - 1) / BM, num_nt = (N + BN - 1) / BN;
  const int total = num_mt * num_nt * nbatch;
  const int ntiles = K / BK;
  int tile = blockIdx.x;
  if (tile >= total) return;

  Dense<B_KMAJ> d;
  d.init(lda, ldb, a_tiled != 0, B_KMAJ && b_tiled != 0);
  for (;;) {
    int mt, ntb;
    xcd_grouped_tile_at(tile, total, num_mt, num_nt * nbatch, mt, ntb);
    const int q = ntb / num_nt, nt = ntb - q * num_nt;
    const int m0 = min(mt * BM, M - BM), n0 = min(nt * BN, N - BN);
    d.set_tile(A + q * sA, B + q * sB, lda, ldb, m0, n0);
    d.prefetch(ntiles);
    d.start(ntiles);
    d.mainloop(ntiles);
    wait_lds();
    barrier_nofence();  // every wave is done with the ring
    if constexpr (FUSE_R)
      d.template epilogue_fused<KEEP_Z>(C, ldc, m0, n0, R + (int64_t)(n0 / 256) * 256 * 256, Y,
                                        ldy);
    else
      d.epilogue(C + q * sC, ldc, m0, n0);
    tile += (int)gridDim.x;
    if (tile >= total) break;
  }
}

}  // namespace

hipError_t dense_grid(int64_t M, int64_t N, int* grid_out) {
  const int tiles = (int)(((M + BM - 1) / BM) * ((N + BN - 1) / BN));
  // one workgroup per CU (the register and LDS footprints allow no more),
  // rounded down to a multiple of the 8 XCDs
  static thread_local int cached_dev = -1, cached_cus = 0;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev != cached_dev) {
    e = hipDeviceGetAttribute(&cached_cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    cached_dev = dev;
  }
  int grid = cached_cus >= 8 ? cached_cus & ~7 : cached_cus;
  if (grid > tiles) grid = tiles;
  if (grid < 1) grid = 1;
  *grid_out = grid;
  return hipSuccess;
}

hipError_t launch_dense(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
                        int64_t lda, int64_t ldb, int64_t ldc, bool b_kmajor, bool a_tiled,
                        bool b_tiled, hipStream_t s) {
  if (a_tiled && (M % BM != 0 || lda != K)) return hipErrorInvalidValue;
  if (b_tiled && (!b_kmajor || N % BN != 0 || ldb != K)) return hipErrorInvalidValue;
  int grid = 0;
  hipError_t e = dense_grid(M, N, &grid);
  if (e != hipSuccess) return e;
  const bf16_t* a = static_cast<const bf16_t*>(A);
  const bf16_t* b = static_cast<const bf16_t*>(B);
  bf16_t* c = static_cast<bf16_t*>(C);
  if (b_kmajor)
    hipLaunchKernelGGL((dense_kernel<true, false>), dim3(grid), dim3(NT), 0, s, a, b, c, (int)M,
                       (int)N, (int)K, lda, ldb, ldc, nullptr, nullptr, (int64_t)0, 1, (int64_t)0,
                       (int64_t)0, (int64_t)0, (int)a_tiled, (int)b_tiled);
  else
    hipLaunchKernelGGL((dense_kernel<false, false>), dim3(grid), dim3(NT), 0, s, a, b, c, (int)M,
                       (int)N, (int)K, lda, ldb, ldc, nullptr, nullptr, (int64_t)0, 1, (int64_t)0,
                       (int64_t)0, (int64_t)0, (int)a_tiled, (int)b_tiled);
  return hipGetLastError();
}

hipError_t launch_dense_batched(const void* A, const void* B, void* C, int64_t M, int64_t N,
                                int64_t K, int64_t lda, int64_t ldb, int64_t ldc, bool b_kmajor,
                                int64_t nbatch, int64_t sA, int64_t sB, int64_t sC,
                                hipStream_t s) {
  if (nbatch < 1 || nbatch * ((N + BN - 1) / BN) * ((M + BM - 1) / BM) > INT32_MAX)
    return hipErrorInvalidValue;
  int grid = 0;
  hipError_t e = dense_grid(M, N * nbatch, &grid);
  if (e != hipSuccess) return e;
  const bf16_t* a = static_cast<const bf16_t*>(A);
  const bf16_t* b = static_cast<const bf16_t*>(B);
  bf16_t* c = static_cast<bf16_t*>(C);
  if (b_kmajor)
    hipLaunchKernelGGL((dense_kernel<true, false>), dim3(grid), dim3(NT), 0, s, a, b, c, (int)M,
                       (int)N, (int)K, lda, ldb, ldc, nullptr, nullptr, (int64_t)0, (int)nbatch,
                       sA, sB, sC, 0, 0);
  else
    hipLaunchKernelGGL((dense_kernel<false, false>), dim3(grid), dim3(NT), 0, s, a, b, c, (int)M,
                       (int)N, (int)K, lda, ldb, ldc, nullptr, nullptr, (int64_t)0, (int)nbatch,
                       sA, sB, sC, 0, 0);
  return hipGetLastError();
}

bool dense_fused_r_supported(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                             int64_t ldc, int64_t ldy) {
  return dense_supported(M, N, K, lda, ldb, ldc) && N % 256 == 0 && ldy % 8 == 0;
}

hipError_t launch_dense_fused_r(const void* A, const void* B, void* C, int64_t M, int64_t N,
                                int64_t K, int64_t lda, int64_t ldb, int64_t ldc, const void* R,
                                void* Y, int64_t ldy, bool a_tiled, bool b_tiled, hipStream_t s) {
  if (a_tiled && (M % BM != 0 || lda != K)) return hipErrorInvalidValue;
  if (b_tiled && (N % BN != 0 || ldb != K)) return hipErrorInvalidValue;
  int grid = 0;
  hipError_t e = dense_grid(M, N, &grid);
  if (e != hipSuccess) return e;
  if (C)
    hipLaunchKernelGGL((dense_kernel<true, true>), dim3(grid), dim3(NT), 0, s,
                       static_cast<const bf16_t*>(A), static_cast<const bf16_t*>(B),
                       static_cast<bf16_t*>(C), (int)M, (int)N, (int)K, lda, ldb, ldc,
                       static_cast<const bf16_t*>(R), static_cast<bf16_t*>(Y), ldy, 1, (int64_t)0,
                       (int64_t)0, (int64_t)0, (int)a_tiled, (int)b_tiled);
  else
    hipLaunchKernelGGL((dense_kernel<true, true, false>), dim3(grid), dim3(NT), 0, s,
                       static_cast<const bf16_t*>(A), static_cast<const bf16_t*>(B), nullptr,
                       (int)M, (int)N, (int)K, lda, ldb, ldc, static_cast<const bf16_t*>(R),
                       static_cast<bf16_t*>(Y), ldy, 1, (int64_t)0, (int64_t)0, (int64_t)0,
                       (int)a_tiled, (int)b_tiled);
  return hipGetLastError();
}

}  // namespace poetx
