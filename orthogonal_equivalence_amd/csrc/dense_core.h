// The main loop of the dense bf16 products on one 256 x 256 output tile, its
// operand copies, LDS layouts and plain epilogues, shared by the kernels of
// dense.hip (the W0 products, whose comment describes the design) and
// dense_epilogue.hip (the same loop ending with bias, activation and
// residual).
#pragma once

#include "common.h"
#include "kernels.h"
#include "lds_dma.h"

namespace poetx {
namespace {

constexpr int BM = 256, BN = 256, BK = 32;
constexpr int NW = 4, NT = 64 * NW;        // one wave per SIMD
constexpr int FM = 8, FN = 8;              // 16-row / 16-column fragments per wave
constexpr int TILE = BM * BK;              // bf16 elements of one operand tile (16 KB)
constexpr int SLOT = 2 * TILE;             // A and B tiles
constexpr int NSLOT = 4;
constexpr int RING = NSLOT * SLOT;         // 128 KB, also the epilogue's staging tile
constexpr int PPW = TILE * 2 / 1024 / NW;  // 1 KB pieces per wave per operand tile
constexpr int LPW = 2 * PPW;               // copies per wave per K tile
static_assert(RING == BM * BN, "the epilogue stages the whole output tile in the ring");
static_assert(BM == 256 && BN == 256 && BK == 32, "dense_supported (kernels.h)");
static_assert(PPW == 4 && LPW == 8, "one copy after each of the eight rows of products");

// 1 KB alignment: the fragment addressing XORs bits 4..6 of element offsets
__shared__ __attribute__((aligned(1024))) bf16_t g_dense_lds[RING];

__device__ __forceinline__ int kmaj_swz(int row) { return (row >> 1) & 3; }
__device__ __forceinline__ int nmaj_swz(int k) { return (k & 3) << 1; }
__device__ __forceinline__ int nmaj_off(int k, int n) {
  return k * BN + ((((n >> 3) ^ nmaj_swz(k))) << 3) + (n & 7);
}
__device__ __forceinline__ int stage_off(int m, int n) {
  return m * BN + ((((n >> 3) ^ (m & 15))) << 3) + (n & 7);
}

// One global_load_lds_dwordx4 in the scalar-base form: lane l copies the 16
// bytes at sbase + voff into LDS at m0 + 16 l.
__device__ __forceinline__ void dma16_sb(const void* sbase, uint32_t voff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(m0), "v"(voff), "s"(sbase)
               : "memory", "m0");
}

__device__ __forceinline__ const bf16_t* uniform_ptr(const bf16_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const bf16_t*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// PAIR (both operands K-major and row-major in memory): a K tile is 64 bytes
// of each row, half a 128-byte line, and by the next tile's copies the lines
// have left the 32 KB L1, so every line crossed from the L2 twice. Paired, the
// copies of an even tile and of the odd one behind it are issued together,
// piece by piece, during every second tile; a line's second half then finds it
// in the L1.
//
// MN_TILED (A_KMAJ and B_KMAJ false: C(m, n) = sum_k A[k][m] B[k][n]): both
// operands are M- or N-major out of the tiled layout (kernels.h), whose rows are k:
// a K tile is 32 rows of eight blocks, 64 bytes of a row in each, and the next
// tile lies 32 rows further on in the blocks, the ninth in the next panel.
// LAST_B: the B rows of K tile last_t come from last_b instead (an N-major B
// whose rows end inside that tile, of which last_b is a padded copy).
template <bool B_KMAJ, bool PAIR = false, bool A_KMAJ = true, bool MN_TILED = false,
          bool LAST_B = false>
struct Dense {
  const bf16_t* last_b;
  int last_t;
  const bf16_t* baseA;  // wave-uniform bases of the current tile's A and B panels
  const bf16_t* baseB;
  int64_t stepA, stepB; // elements between consecutive K tiles of A and of B
  bool a_tiled;         // A in the tiled layout (then M % 256 == 0 and lda == K)
                        // (a tiled K-major B likewise: N % 256 == 0, ldb == K)
  uint32_t offA, offB;  // per-lane byte offsets of this wave's first piece at k = 0
  uint32_t strA, strB;  // bytes between this wave's consecutive pieces
  uint32_t lds0;        // LDS byte address of the ring, wave-uniform
  int wave, lane, wm, wn;
  int rdA, rdB;         // per-lane element offsets of fragment 0 within a tile
  floatx4 acc[FM][FN];
  bf16x8_t fa[2][FM], fb[2][FN];

  __device__ __forceinline__ void init(int64_t lda, int64_t ldb, bool tiled, bool b_tiled) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    wm = wave & 1;
    wn = wave >> 1;
    lds0 = __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)g_dense_lds)));
    a_tiled = tiled;
    stepA = tiled ? (int64_t)BM * BK : BK;
    stepB = B_KMAJ ? (b_tiled ? (int64_t)BN * BK : BK) : (int64_t)BK * ldb;
    const int r = lane & 15;
    if constexpr (A_KMAJ) rdA = (wm * 128 + r) * BK + (((lane >> 4) ^ kmaj_swz(r)) << 3);
    else rdA = nmaj_off(8 * (lane >> 4) + (r >> 2), wm * 128 + 4 * (r & 3));
    if (B_KMAJ) {
      rdB = (wn * 128 + r) * BK + (((lane >> 4) ^ kmaj_swz(r)) << 3);
    } else {
      // fragment j adds 16 j columns: chunk index + 2 j, which the swizzle
      // turns into an XOR of the element offset with 16 j
      const int k = 8 * (lane >> 4) + (r >> 2);
      rdB = nmaj_off(k, wn * 128 + 4 * (r & 3));
    }
    // wave w copies pieces q = w + 4 j (j < 4) of each operand tile: K-major
    // piece q holds rows 16 q .. 16 q + 15, N-major piece q holds k rows
    // 2 q, 2 q + 1; either way the swizzle of a lane's data is the same for
    // all of its pieces
    const int row = 16 * wave + (lane >> 2);
    const int c = (lane & 3) ^ kmaj_swz(row);
    if constexpr (MN_TILED) {
      static_assert(!A_KMAJ && !B_KMAJ, "both operands are read alike");
      const int k = 2 * wave + (lane >> 5);
      const int cn = (lane & 31) ^ nmaj_swz(k);
      offA = offB = (uint32_t)((cn >> 2) * TILE + k * BK + 8 * (cn & 3)) * 2u;
      strA = strB = 2 * NW * BK * 2;
      stepA = 256 * lda;  // (between panels)
      stepB = 256 * ldb;
      return;
    }
    // (tiled: the rows of a K tile are 32 elements apart within its block)
    const int64_t rsa = tiled ? BK : lda;
    offA = (uint32_t)(row * rsa + 8 * c) * 2u;
    strA = (uint32_t)(16 * NW * rsa) * 2u;
    if (B_KMAJ) {
      const int64_t rsb = b_tiled ? BK : ldb;
      offB = (uint32_t)(row * rsb + 8 * c) * 2u;
      strB = (uint32_t)(16 * NW * rsb) * 2u;
    } else {
      const int k = 2 * wave + (lane >> 5);
      const int cn = (lane & 31) ^ nmaj_swz(k);
      offB = (uint32_t)(k * ldb + 8 * cn) * 2u;
      strB = (uint32_t)(2 * NW * ldb) * 2u;
    }
  }

  // panels of the output tile at (m0, n0) (wholly inside M x N)
  __device__ __forceinline__ void set_tile(const bf16_t* A, const bf16_t* B, int64_t lda,
                                           int64_t ldb, int m0, int n0) {
    // (tiled: the panel's blocks start at row m0 of the row-major count,
    // since a panel of 256 rows holds 256 lda elements)
    if constexpr (MN_TILED) {  // (m0, n0 multiples of 32)
      baseA = uniform_ptr(A + (int64_t)m0 * 256);
      baseB = uniform_ptr(B + (int64_t)n0 * 256);
      return;
    }
    baseA = uniform_ptr(A + (int64_t)m0 * lda);
    baseB = uniform_ptr(B_KMAJ ? B + (int64_t)n0 * ldb : B + n0);
  }

  // piece J of K tile t of operand OP (0: A, 1: B) into ring slot S
  template <int S, int OP, int J>
  __device__ __forceinline__ void dma(int t) {
    const uint32_t m = lds0 + (uint32_t)(S * SLOT * 2 + OP * TILE * 2 + (wave + NW * J) * 1024);
    if constexpr (MN_TILED) {
      const int64_t at = (int64_t)(t & 7) * (32 * BK);
      if (OP == 0)
        dma16_sb(uniform_ptr(baseA + (t >> 3) * stepA + at), offA + J * strA, m);
      else
        dma16_sb(uniform_ptr(baseB + (t >> 3) * stepB + at), offB + J * strB, m);
      return;
    }
    if (OP == 0)
      dma16_sb(uniform_ptr(baseA + (int64_t)t * stepA), offA + J * strA, m);
    else if (LAST_B)
      dma16_sb(uniform_ptr(t == last_t ? last_b : baseB + (int64_t)t * stepB), offB + J * strB, m);
    else
      dma16_sb(uniform_ptr(baseB + (int64_t)t * stepB), offB + J * strB, m);
  }
  template <int S>
  __device__ __forceinline__ void issue(int t) {
    dma<S, 0, 0>(t); dma<S, 0, 1>(t); dma<S, 0, 2>(t); dma<S, 0, 3>(t);
    dma<S, 1, 0>(t); dma<S, 1, 1>(t); dma<S, 1, 2>(t); dma<S, 1, 3>(t);
  }

  // the copies of tiles t (slot S) and t + 1 (slot S + 1), piece by piece
  template <int S>
  __device__ __forceinline__ void issue_pair(int t) {
    dma<S, 0, 0>(t); dma<S + 1, 0, 0>(t + 1); dma<S, 0, 1>(t); dma<S + 1, 0, 1>(t + 1);
    dma<S, 0, 2>(t); dma<S + 1, 0, 2>(t + 1); dma<S, 0, 3>(t); dma<S + 1, 0, 3>(t + 1);
    dma<S, 1, 0>(t); dma<S + 1, 1, 0>(t + 1); dma<S, 1, 1>(t); dma<S + 1, 1, 1>(t + 1);
    dma<S, 1, 2>(t); dma<S + 1, 1, 2>(t + 1); dma<S, 1, 3>(t); dma<S + 1, 1, 3>(t + 1);
  }

  // A fragment I (rows 16 I .. of this wave's 128; lane l holds row l % 16,
  // k = 8 (l / 16) .. +7) from ring slot S into set P
  template <int S, int P, int I>
  __device__ __forceinline__ void read_a() {
    if constexpr (A_KMAJ) {
      fa[P][I] = *reinterpret_cast<const bf16x8_t*>(g_dense_lds + S * SLOT + rdA + 512 * I);
    } else {
      const bf16_t* sa = g_dense_lds + S * SLOT;
      const int o = rdA ^ (16 * I);
      union { short4_t h[2]; bf16x8_t v; } u;
      u.h[0] = ds_read_tr4(sa + o);
      u.h[1] = ds_read_tr4(sa + o + 4 * BM);
      fa[P][I] = u.v;
    }
  }
  // B fragment J (16 of this wave's columns) likewise
  template <int S, int P, int J>
  __device__ __forceinline__ void read_b() {
    const bf16_t* sb = g_dense_lds + S * SLOT + TILE;
    if (B_KMAJ) {
      fb[P][J] = *reinterpret_cast<const bf16x8_t*>(sb + rdB + 512 * J);
    } else {
      const int o = rdB ^ (16 * J);
      union { short4_t h[2]; bf16x8_t v; } u;
      u.h[0] = ds_read_tr4(sb + o);
      u.h[1] = ds_read_tr4(sb + o + 4 * BN);
      fb[P][J] = u.v;
    }
  }

  // acc[I][J] += B fragment J x A fragment I (D' = B A^T: lane l holds
  // output row 16 I + l % 16, columns 16 J + 4 (l / 16) .. +3)
  template <int P, int I, int J, bool FIRST>
  __device__ __forceinline__ void mma() {
    if (FIRST)
      asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0"
                   : "=a"(acc[I][J])
                   : "v"(fb[P][J]), "v"(fa[P][I]));
    else
      asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
                   : "+a"(acc[I][J])
                   : "v"(fb[P][J]), "v"(fa[P][I]));
  }
  template <int P, int I, bool FIRST>
  __device__ __forceinline__ void mma_row() {
    mma<P, I, 0, FIRST>(); mma<P, I, 1, FIRST>(); mma<P, I, 2, FIRST>(); mma<P, I, 3, FIRST>();
    mma<P, I, 4, FIRST>(); mma<P, I, 5, FIRST>(); mma<P, I, 6, FIRST>(); mma<P, I, 7, FIRST>();
  }

  // K tile t, held in ring slot S, its fragments in set P. STEADY: tiles
  // t+1 .. t+4 all exist, so every step below is taken. FIRST: t == 0.
  // LATE (t < 3): with `late`, at least LATE vector memory instructions (the
  // stores of the output tile before) were issued behind the copies of the first
  // four K tiles, and need not have completed for those.
  template <int S, int P, bool STEADY, bool FIRST = false, int LATE = 0>
  __device__ __forceinline__ void tile(int t, int ntiles, bool late = false) {
    constexpr int S1 = (S + 1) & 3;
    const bool more = STEADY || t + 1 < ntiles;
    // paired: an odd tile issues the copies of tiles t + 3 and t + 4
    constexpr bool ODD = (S & 1) != 0;
    const bool iss = (!PAIR || ODD) && (STEADY || t + 4 < ntiles);
    const bool iss3 = PAIR && ODD && (STEADY || t + 3 < ntiles);
    constexpr int S3 = (S + 3) & 3;
    mma_row<P, 0, FIRST>();
    __builtin_amdgcn_sched_barrier(0);
    if (more) {
      // this wave's part of tile t+1 landed (tiles t+2, t+3 may still be in
      // flight) and its reads of tile t are done; after the barrier every
      // part has landed and slot S is free
      // (paired, odd t: of the pair t + 1, t + 2 only the last copy may be)
      if constexpr (LATE > 0) {
        static_assert(STEADY && LATE <= 40, "vmcnt range");
        constexpr int kLeft = PAIR && ODD ? 1 : 2 * LPW;
        if (late) wait_vm<(kLeft + LATE < 63 ? kLeft + LATE : 63)>();
        else wait_vm<kLeft>();
      } else if constexpr (PAIR && ODD) {
        if (STEADY || t + 2 < ntiles) wait_vm<1>();
        else wait_vm<0>();
      } else {
        if (STEADY || t + 3 < ntiles) wait_vm<2 * LPW>();
        else if (t + 2 < ntiles) wait_vm<LPW>();
        else wait_vm<0>();
      }
      wait_lds();
      barrier_nofence();
    }
    if (iss3) dma<S3, 0, 0>(t + 3);
    if (iss) dma<S, 0, 0>(t + 4);
    __builtin_amdgcn_sched_barrier(0);
#define POETX_DENSE_ROW(I)                                                          \
  mma_row<P, I, FIRST>();                                                           \
  if (iss3) dma<S3, (I) / 4, (I) % 4>(t + 3);                                       \
  if (iss) dma<S, (I) / 4, (I) % 4>(t + 4);                                         \
  if (more) { read_a<S1, P ^ 1, (I) - 1>(); read_b<S1, P ^ 1, (I) - 1>(); }         \
  __builtin_amdgcn_sched_barrier(0);
    POETX_DENSE_ROW(1) POETX_DENSE_ROW(2) POETX_DENSE_ROW(3) POETX_DENSE_ROW(4)
    POETX_DENSE_ROW(5) POETX_DENSE_ROW(6) POETX_DENSE_ROW(7)
#undef POETX_DENSE_ROW
    if (more) { read_a<S1, P ^ 1, 7>(); read_b<S1, P ^ 1, 7>(); }
  }

  // copies of the first (up to) four K tiles of the current output tile
  __device__ __forceinline__ void prefetch(int ntiles) {
    if constexpr (PAIR) {
      if (ntiles > 1) issue_pair<0>(0);
      else issue<0>(0);
      if (ntiles > 3) issue_pair<2>(2);
      else if (ntiles > 2) issue<2>(2);
      return;
    }
    issue<0>(0);
    if (ntiles > 1) issue<1>(1);
    if (ntiles > 2) issue<2>(2);
    if (ntiles > 3) issue<3>(3);
  }

  // every part of K tile 0 landed (this wave's earlier stores too: the
  // count is conservative); its fragments read
  __device__ __forceinline__ void start(int ntiles) {
    // (paired: tile 1 with it)
    if (ntiles > 3) wait_vm<(PAIR ? 2 : 3) * LPW>();
    else if (ntiles > 2) wait_vm<(PAIR ? 1 : 2) * LPW>();
    else if (ntiles > 1) wait_vm<(PAIR ? 0 : 1) * LPW>();
    else wait_vm<0>();
    barrier_nofence();
    read_a<0, 0, 0>(); read_a<0, 0, 1>(); read_a<0, 0, 2>(); read_a<0, 0, 3>();
    read_a<0, 0, 4>(); read_a<0, 0, 5>(); read_a<0, 0, 6>(); read_a<0, 0, 7>();
    read_b<0, 0, 0>(); read_b<0, 0, 1>(); read_b<0, 0, 2>(); read_b<0, 0, 3>();
    read_b<0, 0, 4>(); read_b<0, 0, 5>(); read_b<0, 0, 6>(); read_b<0, 0, 7>();
  }

  // start() and mainloop() with LATE's waits; ntiles >= 8
  template <int LATE>
  __device__ __forceinline__ void start_late(bool late) {
    constexpr int kLeft = (PAIR ? 2 : 3) * LPW;
    if (late) wait_vm<(kLeft + LATE < 63 ? kLeft + LATE : 63)>();
    else wait_vm<kLeft>();
    barrier_nofence();
    read_a<0, 0, 0>(); read_a<0, 0, 1>(); read_a<0, 0, 2>(); read_a<0, 0, 3>();
    read_a<0, 0, 4>(); read_a<0, 0, 5>(); read_a<0, 0, 6>(); read_a<0, 0, 7>();
    read_b<0, 0, 0>(); read_b<0, 0, 1>(); read_b<0, 0, 2>(); read_b<0, 0, 3>();
    read_b<0, 0, 4>(); read_b<0, 0, 5>(); read_b<0, 0, 6>(); read_b<0, 0, 7>();
  }
  template <int LATE>
  __device__ __forceinline__ void mainloop_late(int ntiles, bool late) {
    tile<0, 0, true, true, LATE>(0, ntiles, late);
    tile<1, 1, true, false, LATE>(1, ntiles, late);
    tile<2, 0, true, false, LATE>(2, ntiles, late);
    int t = 3;
    for (; t + 8 <= ntiles; t += 4) {
      tile<3, 1, true>(t, ntiles);
      tile<0, 0, true>(t + 1, ntiles);
      tile<1, 1, true>(t + 2, ntiles);
      tile<2, 0, true>(t + 3, ntiles);
    }
    // the last 4 .. 7 tiles
    tile<3, 1, false>(t, ntiles);
    tile<0, 0, false>(t + 1, ntiles);
    tile<1, 1, false>(t + 2, ntiles);
    tile<2, 0, false>(t + 3, ntiles);
    t += 4;
    if (t < ntiles) tile<3, 1, false>(t++, ntiles);
    if (t < ntiles) tile<0, 0, false>(t++, ntiles);
    if (t < ntiles) tile<1, 1, false>(t++, ntiles);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void mainloop(int ntiles) {
    // tile 0 writes the accumulators; then slots 1, 2, 3, 0, 1, ...
    if (ntiles > 4) tile<0, 0, true, true>(0, ntiles);
    else tile<0, 0, false, true>(0, ntiles);
    int t = 1;
    for (; t + 8 <= ntiles; t += 4) {  // branch-free steady state
      tile<1, 1, true>(t, ntiles);
      tile<2, 0, true>(t + 1, ntiles);
      tile<3, 1, true>(t + 2, ntiles);
      tile<0, 0, true>(t + 3, ntiles);
    }
    // the last 0 .. 7 tiles
    if (t < ntiles) tile<1, 1, false>(t++, ntiles);
    if (t < ntiles) tile<2, 0, false>(t++, ntiles);
    if (t < ntiles) tile<3, 1, false>(t++, ntiles);
    if (t < ntiles) tile<0, 0, false>(t++, ntiles);
    if (t < ntiles) tile<1, 1, false>(t++, ntiles);
    if (t < ntiles) tile<2, 0, false>(t++, ntiles);
    if (t < ntiles) tile<3, 1, false>(t++, ntiles);
    // wait states between the last products and the VALU reads of their
    // results in the epilogue (more than any 16x16x32 product needs)
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // The wait states again, tied to the accumulators: without the tie the
  // compiler, to which the products are no matrix instructions, may copy an
  // accumulator right behind the last product, ahead of mainloop()'s waits (it
  // did, at the join of the last tiles' branches, where the code that follows
  // takes VGPRs).
  __device__ __forceinline__ void settle() {
    asm volatile("s_nop 15\n\ts_nop 15"
                 : "+a"(acc[FM - 1][0]), "+a"(acc[FM - 1][1]), "+a"(acc[FM - 1][2]),
                   "+a"(acc[FM - 1][3]), "+a"(acc[FM - 1][4]), "+a"(acc[FM - 1][5]),
                   "+a"(acc[FM - 1][6]), "+a"(acc[FM - 1][7])
                 :
                 : "memory");
    in_agprs();
  }
  // the accumulators in their AGPRs at this place (an epilogue that reads them
  // twice would otherwise keep copies, more than the VGPRs hold)
  __device__ __forceinline__ void in_agprs() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      asm volatile(""
                   : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]),
                     "+a"(acc[i][4]), "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
    __builtin_amdgcn_sched_barrier(0);
  }

  // the accumulator of fragment (f / 8, f % 8), f wave-uniform (reads by name:
  // the compiler would otherwise copy all accumulators to VGPRs first)
  __device__ __forceinline__ floatx4 pick(int f) {
    float a = 0.0f, b = 0.0f, c = 0.0f, e = 0.0f;
#define POETX_PICK(F)                                                                   \
  case F:                                                                               \
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(a) : "a"(acc[(F) / 8][(F) % 8][0])); \
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(b) : "a"(acc[(F) / 8][(F) % 8][1])); \
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(c) : "a"(acc[(F) / 8][(F) % 8][2])); \
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(e) : "a"(acc[(F) / 8][(F) % 8][3])); \
    break;
    switch (f) {
      POETX_PICK(0) POETX_PICK(1) POETX_PICK(2) POETX_PICK(3)
      POETX_PICK(4) POETX_PICK(5) POETX_PICK(6) POETX_PICK(7)
      POETX_PICK(8) POETX_PICK(9) POETX_PICK(10) POETX_PICK(11)
      POETX_PICK(12) POETX_PICK(13) POETX_PICK(14) POETX_PICK(15)
      POETX_PICK(16) POETX_PICK(17) POETX_PICK(18) POETX_PICK(19)
      POETX_PICK(20) POETX_PICK(21) POETX_PICK(22) POETX_PICK(23)
      POETX_PICK(24) POETX_PICK(25) POETX_PICK(26) POETX_PICK(27)
      POETX_PICK(28) POETX_PICK(29) POETX_PICK(30) POETX_PICK(31)
      POETX_PICK(32) POETX_PICK(33) POETX_PICK(34) POETX_PICK(35)
      POETX_PICK(36) POETX_PICK(37) POETX_PICK(38) POETX_PICK(39)
      POETX_PICK(40) POETX_PICK(41) POETX_PICK(42) POETX_PICK(43)
      POETX_PICK(44) POETX_PICK(45) POETX_PICK(46) POETX_PICK(47)
      POETX_PICK(48) POETX_PICK(49) POETX_PICK(50) POETX_PICK(51)
      POETX_PICK(52) POETX_PICK(53) POETX_PICK(54) POETX_PICK(55)
      POETX_PICK(56) POETX_PICK(57) POETX_PICK(58) POETX_PICK(59)
      POETX_PICK(60) POETX_PICK(61) POETX_PICK(62) POETX_PICK(63)
      default: break;
    }
#undef POETX_PICK
    return floatx4{a, b, c, e};
  }

  // accumulators -> bf16 staging tile (the whole ring) -> 16-byte stores of
  // whole 512-byte row segments; the ring is free again on return
  __device__ __forceinline__ void epilogue(bf16_t* __restrict__ C, int64_t ldc, int m0, int n0) {
    // opaque copies of the lane and thread ids: keeps the compiler from
    // hoisting the epilogue's address arithmetic out of the tile loop
    int ln = lane, tid = (int)threadIdx.x;
    asm volatile("" : "+v"(ln), "+v"(tid));
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int m = wm * 128 + 16 * i + (ln & 15);
        const int n = wn * 128 + 16 * j + 4 * (ln >> 4);
        union { bf16_t h[4]; uint2 v; } u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u.h[e] = f32_to_bf16(acc[i][j][e]);
        *reinterpret_cast<uint2*>(g_dense_lds + stage_off(m, n)) = u.v;
        __builtin_amdgcn_sched_barrier(0);  // one fragment's registers at a time
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < BM * BN / 8 / NT; ++q) {
      const int c = tid + q * NT;
      const int rl = c >> 5, nl = (c & 31) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(g_dense_lds + stage_off(rl, nl));
      *reinterpret_cast<uint4*>(C + (int64_t)(m0 + rl) * ldc + n0 + nl) = v;
    }
    wait_lds();
    barrier_nofence();
  }

  // ---- forward with the R-apply fused (B K-major, 256 x 256 R blocks) ----
  // Y tile = Z tile R_k^T for the output tile's R block R_k (its 256 columns
  // are one block): the bf16 Z tile staged in the ring is the A operand, R_k's
  // rows are the B fragments (loaded from global memory, the block stays in
  // L2), K = 256 in 8 steps of 32, accumulated in the same AGPRs. Without
  // KEEP_Z only Y leaves the CU (a run-time test there made the compiler
  // spill ~0.5 KB per lane).
  template <int S>
  __device__ __forceinline__ void load_r(const bf16_t* rrow) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[S & 1][j] = *reinterpret_cast<const bf16x8_t*>(rrow + j * 16 * 256 + S * 32);
  }
  template <int S>
  __device__ __forceinline__ void r_step(const bf16_t* rrow, int ln) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fa[S & 1][i] = *reinterpret_cast<const bf16x8_t*>(
          g_dense_lds + stage_off(wm * 128 + 16 * i + (ln & 15), 32 * S + 8 * (ln >> 4)));
    if (S + 1 < 8) load_r<(S + 1) & 7>(rrow);
    mma_row<S & 1, 0, S == 0>(); mma_row<S & 1, 1, S == 0>();
    mma_row<S & 1, 2, S == 0>(); mma_row<S & 1, 3, S == 0>();
    mma_row<S & 1, 4, S == 0>(); mma_row<S & 1, 5, S == 0>();
    mma_row<S & 1, 6, S == 0>(); mma_row<S & 1, 7, S == 0>();
    __builtin_amdgcn_sched_barrier(0);
  }
  // the accumulators -> bf16 -> staging tile (the whole ring)
  __device__ __forceinline__ void stage_acc(int ln) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int m = wm * 128 + 16 * i + (ln & 15);
        const int n = wn * 128 + 16 * j + 4 * (ln >> 4);
        union { bf16_t h[4]; uint2 v; } u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u.h[e] = f32_to_bf16(acc[i][j][e]);
        *reinterpret_cast<uint2*>(g_dense_lds + stage_off(m, n)) = u.v;
        __builtin_amdgcn_sched_barrier(0);
      }
  }
  // the staging tile -> 16-byte stores of whole row segments of C (row stride ldc)
  __device__ __forceinline__ void store_staged(bf16_t* __restrict__ C, int64_t ldc, int m0, int n0,
                                               int tid) {
#pragma unroll
    for (int q = 0; q < BM * BN / 8 / NT; ++q) {
      const int c = tid + q * NT;
      const int rl = c >> 5, nl = (c & 31) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(g_dense_lds + stage_off(rl, nl));
      *reinterpret_cast<uint4*>(C + (int64_t)(m0 + rl) * ldc + n0 + nl) = v;
    }
  }
  template <bool KEEP_Z>
  __device__ __forceinline__ void epilogue_fused(bf16_t* __restrict__ C, int64_t ldc, int m0,
                                                 int n0, const bf16_t* __restrict__ Rk,
                                                 bf16_t* __restrict__ Y, int64_t ldy) {
    int ln = lane, tid = (int)threadIdx.x;
    asm volatile("" : "+v"(ln), "+v"(tid));
    // B fragment (j, step s) of lane l: R_k row wn 128 + 16 j + l % 16,
    // columns 32 s + 8 (l / 16) .. + 7
    const bf16_t* rrow = Rk + (wn * 128 + (ln & 15)) * 256 + 8 * (ln >> 4);
    load_r<0>(rrow);  // in flight while Z is staged
    stage_acc(ln);
    wait_lds();
    barrier_nofence();  // (no memory fence: nothing waits for the loads or stores here)
    r_step<0>(rrow, ln); r_step<1>(rrow, ln); r_step<2>(rrow, ln); r_step<3>(rrow, ln);
    r_step<4>(rrow, ln); r_step<5>(rrow, ln); r_step<6>(rrow, ln); r_step<7>(rrow, ln);
    // wait states before the VALU reads of the products' results
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (KEEP_Z) store_staged(C, ldc, m0, n0, tid);  // Z
    wait_lds();
    barrier_nofence();  // every wave is done reading the staged Z
    stage_acc(ln);
    wait_lds();
    barrier_nofence();  // Z's stores stay in flight
    store_staged(Y, ldy, m0, n0, tid);  // Y
    wait_lds();
    barrier_nofence();
  }
};

}  // namespace
}  // namespace poetx
