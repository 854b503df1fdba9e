// The main loop of the tile products, for any number of rows: one workgroup of
// four or eight waves computes a BM x BN tile of
//   C(m, n) = sum_k A(m, k) B(n, k),
//   A(m, k) = A[m lda + k] (K-major) or A[k lda + m] (M-major), B likewise,
// and hands its float32 accumulators, in registers, to an end of the kernel's
// own (tilegemm.hip, vocab_tile.hip).
//
// The reduction runs in steps of 128 bytes (64 bf16, 32 float32) through a
// ring of NS LDS slots filled by global_load_lds_dwordx4, NS - 1 steps ahead: at
// the mid sizes this kernel serves (a few tiles per CU, often one) nothing
// else hides the latency of the loads. The fragments of one half step are
// read while the products of the other run (read, then multiply, in turn took
// 1400 cycles a step of 128 x 128 tiles whose products take 512). Rows past the end are
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
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "common.h"
#include "epilogue.h"
#include "kernels.h"
#include "lds_dma.h"

namespace poetx {
namespace {

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
  static_assert(ROWS >= 32, "the XOR stays inside a row's chunks");
  if constexpr (sizeof(T) == 4) return ((k >> 2) & (ROWS >= 64 ? 3 : 1)) << 2;  // 64-byte pieces
  if constexpr (ROWS >= 128) return ((k & 3) | (((k >> 3) & 1) << 2)) << 1;  // 32-byte pieces
  if constexpr (ROWS == 64)  // (k & 1 picks the half of the banks)
    return (((k >> 1) & 1) | (((k >> 3) & 1) << 1)) << 1;
  return ((k >> 3) & 1) << 1;  // (k & 3 picks the quarter)
}

// (wave-uniform by construction; said so for the scalar registers)
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// One global_load_lds_dwordx4 in the scalar-base form: lane l copies the 16
// bytes at sbase + voff into LDS at m0 + 16 l.
__device__ __forceinline__ void dma16_at(const char* sbase, uint32_t voff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(m0)), "v"(voff), "s"(uniform(sbase))
               : "memory", "m0");
}

// One operand's tile: ROWS rows (m or n), one step of k; NW waves share its
// copies. The lanes' byte offsets within a step's panel are formed once; a
// step moves the scalar base only.
template <typename T, int ROWS, bool KMAJ, int NW>
struct Operand {
  static constexpr int E = Elem<T>::E, BK = Elem<T>::BK;
  static constexpr int BYTES = ROWS * kRowBytes;
  static constexpr int PIECES = BYTES / 1024 / NW;  // 1 KB copies per wave and step
  static constexpr int CPR = ROWS / E;              // chunks per k row (MN-major)
  static_assert(PIECES >= 1, "every wave copies");
  typedef typename Elem<T>::Frag Raw;  // a fragment as it is read
  static __device__ __forceinline__ const Raw& widen(const Raw& r) { return r; }

  const char* base;  // K-major: row r0, k = 0; MN-major: column r0, k = 0
  int64_t step;      // bytes between steps
  int64_t ld;        // elements
  int rows, K;       // rows of the operand from r0 on; whole reduction length
  uint32_t off[PIECES];

  // 16-byte chunk c16 of the tile (LDS order) in the step at k0: its byte
  // offset from the step's panel, rows and k clamped into the operand
  __device__ __forceinline__ uint32_t offset(int c16, int k0) const {
    if (KMAJ) {
      const int r = c16 >> 3, c = (c16 & 7) ^ k_swz(r);
      return (uint32_t)(min(r, rows - 1) * (int)ld + min(c * E, K - E - k0)) * (uint32_t)sizeof(T);
    }
    const int k = c16 / CPR, c = (c16 % CPR) ^ mn_swz<T, ROWS>(k);
    return (uint32_t)(min(k, K - 1 - k0) * (int)ld + min(c * E, rows - E)) * (uint32_t)sizeof(T);
  }
  __device__ __forceinline__ void init(const T* p, int64_t ld_, int r0, int total, int K_, int wave,
                                       int lane) {
    ld = ld_;
    // (what is contiguous in memory is padded to whole chunks)
    K = KMAJ ? (K_ + E - 1) / E * E : K_;
    rows = (KMAJ ? total : (total + E - 1) / E * E) - r0;
    base = reinterpret_cast<const char*>(KMAJ ? p + (int64_t)r0 * ld : p + r0);
    step = (KMAJ ? (int64_t)BK : (int64_t)BK * ld) * sizeof(T);
    // (of a full step: issue() forms a cut one itself)
#pragma unroll
    for (int j = 0; j < PIECES; ++j) off[j] = offset((wave + NW * j) * 64 + lane, min(0, K - BK));
  }
  // copy J of this wave for step t (k0 = t BK) into the slot at LDS byte
  // `lds`; FULL: the step is known to be
  template <bool FULL, int J>
  __device__ __forceinline__ void issue(uint32_t lds, int t, int wave, int lane) const {
    const int q = wave + NW * J;
    const bool cut = !FULL && (t + 1) * BK > K;  // the operand's last step, not full
    dma16_at(base + t * step, cut ? offset(q * 64 + lane, t * BK) : off[J], lds + q * 1024);
  }
  // zeros from k = kleft on (the whole workgroup)
  __device__ __forceinline__ void zero_tail(char* slot, int kleft, int tid) const {
    for (int c16 = tid; c16 < BYTES / 16; c16 += 64 * NW) {
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

// The INT8 codes of a bf16 product's B, K-major, K a multiple of 16: a step's
// 64 codes of a row are 64 bytes, 16-byte chunk c of row r at
// c ^ ((r >> 1) & 3); widened in registers (code + 128 as an unsigned byte to
// float32, less 128, to bf16, all exact).
template <int ROWS, int NW>
struct Operand<int8_t, ROWS, true, NW> {
  static constexpr int BK = Elem<bf16_t>::BK;
  static constexpr int BYTES = ROWS * 64;
  static constexpr int PIECES = BYTES / 1024 / NW;
  static_assert(PIECES >= 1, "every wave copies");
  typedef uint2 Raw;
  static __device__ __forceinline__ bf16x8_t widen(const Raw& r) {
    union { bf16_t h[8]; bf16x8_t v; } o;
    const uint32_t w[2] = {r.x ^ 0x80808080u, r.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o.h[i] = f32_to_bf16((float)((w[i >> 2] >> (8 * (i & 3))) & 0xffu) - 128.0f);
    return o.v;
  }

  const char* base;
  int64_t ld;
  int rows, K;
  uint32_t off[PIECES];

  static __device__ __forceinline__ int swz(int row) { return (row >> 1) & 3; }
  __device__ __forceinline__ uint32_t offset(int c16, int k0) const {
    const int r = c16 >> 2, c = (c16 & 3) ^ swz(r);
    return (uint32_t)(min(r, rows - 1) * (int)ld + min(c * 16, K - 16 - k0));
  }
  __device__ __forceinline__ void init(const int8_t* p, int64_t ld_, int r0, int total, int K_,
                                       int wave, int lane) {
    ld = ld_;
    K = K_;
    rows = total - r0;
    base = reinterpret_cast<const char*>(p + (int64_t)r0 * ld);
#pragma unroll
    for (int j = 0; j < PIECES; ++j) off[j] = offset((wave + NW * j) * 64 + lane, min(0, K - BK));
  }
  template <bool FULL, int J>
  __device__ __forceinline__ void issue(uint32_t lds, int t, int wave, int lane) const {
    const int q = wave + NW * J;
    const bool cut = !FULL && (t + 1) * BK > K;
    dma16_at(base + t * BK, cut ? offset(q * 64 + lane, t * BK) : off[J], lds + q * 1024);
  }
  __device__ __forceinline__ void zero_tail(char* slot, int kleft, int tid) const {
    for (int c16 = tid; c16 < BYTES / 16; c16 += 64 * NW) {
      const int r = c16 >> 2, c = (c16 & 3) ^ swz(r);
      if (c * 16 >= kleft) *reinterpret_cast<uint4*>(slot + 16 * c16) = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ Raw read(const char* slot, int r0, int s, int lane) const {
    const int r = r0 + (lane & 15), g = lane >> 4;
    return *reinterpret_cast<const Raw*>(slot + r * 64 + (((2 * s + (g >> 1)) ^ swz(r)) << 4) +
                                         8 * (g & 1));
  }
};

// c += a b in VGPRs. Inline asm because with one workgroup per CU the compiler
// otherwise keeps the accumulators in AGPRs and copies them between the half
// steps. It does not see these as matrix instructions: settle() stands
// between them and any other use of their registers.
// mma<J>: product J of a fragment pair (bf16 has one, float32 four).
template <int J> __device__ __forceinline__ void mma(const bf16x8_t& a, const bf16x8_t& b, floatx4& c) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
template <int J> __device__ __forceinline__ void mma(const floatx4& a, const floatx4& b, floatx4& c) {
  asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+v"(c) : "v"(a[J]), "v"(b[J]));
}
// float32 product J alone: c = a b
template <int J> __device__ __forceinline__ void mma_alone(const floatx4& a, const floatx4& b, floatx4& c) {
  asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, 0" : "=&v"(c) : "v"(a[J]), "v"(b[J]));
}
// wait states between VALU writes (of operands, accumulators or EXEC) and the
// products that read them, and between products and VALU reads of their
// results: more than any 16 x 16 product needs
__device__ __forceinline__ void settle_before() { asm volatile("s_nop 4" ::: "memory"); }
__device__ __forceinline__ void settle_after() {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
}

// (lambdas of the unrolled loop: a call would put the fragments into scratch)
#define POETX_INLINE __attribute__((always_inline))

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void for_each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void for_each(F&& f) {
  for_each_of(std::make_integer_sequence<int, N>{}, f);
}

// until at most `n` (0 .. NS - 2) steps of LPW copies are in flight
template <int LPW, int NS> __device__ __forceinline__ void wait_steps(int n) {
  static_assert(NS >= 3 && (NS - 2) * LPW < 64, "ring depth");
  if constexpr (NS > 3) {
    if (n < NS - 2) {
      wait_steps<LPW, NS - 1>(n);
      return;
    }
    wait_vm<(NS - 2) * LPW>();
  } else {
    if (n >= 1) wait_vm<LPW>();
    else wait_vm<0>();
  }
}

// bytes of the ring of a BM x BN shape
template <typename T, typename TB, int BM, int BN, int NW, int NS> constexpr int ring_bytes() {
  return NS * (Operand<T, BM, true, NW>::BYTES + Operand<TB, BN, true, NW>::BYTES);
}

// One accumulator, or (an end with kBlocked, float32) sums of blocks of k that are
// added to it: what a long sum loses goes by the number of additions to the whole.
// A block is a half of each of NS steps (the last steps: of one), whose sums are
// added while the next one's products run. (g_W of 8 tokens, 2440 x 3247, 3.2e-6 off in
// one chain, 0.6e-6 in blocks, 0.4e-6 by a library's products; 2048 tokens, 2048 x
// 32000, forward 1900 us, 1955 in blocks, both gradients 5870, 6070.)
//
// One workgroup's tile (its place `wg` among p's tiles, part `part_k` of a
// split reduction), whose accumulators go to end.run(): lane l holds row
// m + 16 i + l % 16, columns n + 16 j + 4 (l / 16) .. + 3 of its wave's part of
// the tile in acc[i][j] (operand roles swapped); `wave_col` counts the wave
// columns of the whole product.
template <typename T, typename TB, int BM, int BN, int WM, int WN, bool A_KMAJ, bool B_KMAJ, int NS,
          typename End>
__device__ __forceinline__ void tile_body(const TileProduct& p, int wg, int part_k, char* ring,
                                          const End& end) {
  constexpr int NW = WM * WN;
  typedef Operand<T, BM, A_KMAJ, NW> OpA;
  typedef Operand<TB, BN, B_KMAJ, NW> OpB;
  constexpr int BK = Elem<T>::BK;
  constexpr int TM = BM / WM, TN = BN / WN;
  constexpr int FM = TM / 16, FN = TN / 16;
  constexpr int SLOT = OpA::BYTES + OpB::BYTES;
  constexpr int LPW = OpA::PIECES + OpB::PIECES;
  static_assert(NS * SLOT == ring_bytes<T, TB, BM, BN, NW, NS>(), "one ring");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int num_mt = (p.M + BM - 1) / BM, num_nt = (p.N + BN - 1) / BN;
  int mt, nt;
  xcd_grouped_tile_at(wg, num_mt * num_nt, num_mt, num_nt, mt, nt);
  const int m0 = __builtin_amdgcn_readfirstlane(mt * BM);
  const int n0 = __builtin_amdgcn_readfirstlane(nt * BN);
  const int t0 = part_k * (p.kchunk / BK);
  const int steps = (min(p.K, (part_k + 1) * p.kchunk) + BK - 1) / BK - t0;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)ring)));

  OpA oa;
  OpB ob;
  oa.init(static_cast<const T*>(p.A), p.lda, m0, p.M, p.K, wave, lane);
  ob.init(static_cast<const TB*>(p.B), p.ldb, n0, p.N, p.K, wave, lane);

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  constexpr bool kBlocks = End::kBlocked && sizeof(T) == 4;
  floatx4 blk[2][kBlocks ? FM : 1][kBlocks ? FN : 1];  // of the two halves of a step
  for (auto& h : blk)
    for (auto& row : h)
      for (auto& c : row) c = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  // acc += a block's sums, at least a half step after its products
  auto add_block = [&](int h) POETX_INLINE {
    if constexpr (kBlocks) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += blk[h][i][j][e];
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // zeros past the reduction's end where step t is not full
  auto clear_tail = [&](int slot, int t) POETX_INLINE {
    const int kleft = p.K - (t0 + t) * BK;
    if (kleft < BK) {
      oa.zero_tail(ring + slot * SLOT, kleft, tid);
      ob.zero_tail(ring + slot * SLOT + OpA::BYTES, kleft, tid);
      wait_lds();
      barrier_nofence();
    }
  };

  typename Elem<T>::Frag fa[2][FM];
  typename OpB::Raw fb[2][FN];
  // copy J (of LPW) of step t into `slot`
  auto issue = [&](int slot, int t, auto piece, auto full) POETX_INLINE {
    constexpr int J = decltype(piece)::value;
    constexpr bool kFull = decltype(full)::value;
    if constexpr (J < OpA::PIECES)
      oa.template issue<kFull, J>(lds0 + slot * SLOT, t0 + t, wave, lane);
    else if constexpr (J < LPW)
      ob.template issue<kFull, J - OpA::PIECES>(lds0 + slot * SLOT + OpA::BYTES, t0 + t, wave,
                                                lane);
  };
  auto issue_all = [&](int slot, int t) POETX_INLINE {
    for_each<LPW>([&](auto j) POETX_INLINE { issue(slot, t, j, std::false_type{}); });
  };
  auto read = [&](int slot, auto half) POETX_INLINE {
    constexpr int H = decltype(half)::value;
    const char* sa = ring + slot * SLOT;
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[H][i] = oa.read(sa, wm * TM + 16 * i, H, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[H][j] = ob.read(sa + OpA::BYTES, wn * TN + 16 * j, H, lane);
  };
  // the products of one half step, after(r) behind fragment row r (float32:
  // product by product over all pairs, so that no two in a row take the same
  // accumulator)
  // ALONE: they begin a block.
  auto products = [&](auto half, auto alone, auto after) POETX_INLINE {
    constexpr int H = decltype(half)::value;
    constexpr bool ALONE = decltype(alone)::value;
    typename Elem<T>::Frag b[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      b[j] = OpB::widen(fb[H][j]);
      if constexpr (sizeof(TB) == 1) asm volatile("" : "+v"(b[j]));  // widened before settle_before
    }
    settle_before();
    for_each<FM>([&](auto r) POETX_INLINE {
      constexpr int i = decltype(r)::value;
      for_each<FN>([&](auto j) POETX_INLINE {
        if constexpr (kBlocks && ALONE) mma_alone<0>(b[j], fa[H][i], blk[H][i][j]);
        else if constexpr (kBlocks) mma<0>(b[j], fa[H][i], blk[H][i][j]);
        else mma<0>(b[j], fa[H][i], acc[i][j]);
      });
      after(r);
    });
    if constexpr (sizeof(T) == 4)
      for_each<3 * FM * FN>([&](auto q) POETX_INLINE {
        constexpr int e = decltype(q)::value / (FM * FN), ij = decltype(q)::value % (FM * FN);
        if constexpr (kBlocks) mma<1 + e>(b[ij % FN], fa[H][ij / FN], blk[H][ij / FN][ij % FN]);
        else mma<1 + e>(b[ij % FN], fa[H][ij / FN], acc[ij / FN][ij % FN]);
      });
  };
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, 1> kSecond{};
  constexpr int PER_ROW = (LPW + 2 * FM - 1) / (2 * FM);  // copies behind a row of products
  constexpr int FIRST_HALF = PER_ROW * FM < LPW ? PER_ROW * FM : LPW;
  // Step t, whose first half is in registers. Its slot's predecessor is free:
  // step t + NS - 1 is copied into it, spread over the products, since a burst
  // of copies would hold back the products behind it (in-order issue; the
  // address unit takes 16 cycles a copy, for four waves at once). Half way
  // the second half's fragments are in registers too; once this wave's copies
  // of step t + 1 have landed, the barrier makes that hold for every wave.
  // Steady: steps t + 1 .. t + NS - 1 exist and are full; nothing is tested. first,
  // last: of a block.
  auto step = [&](int slot, int t, auto steady, auto first, auto last) POETX_INLINE {
    constexpr bool kSteady = decltype(steady)::value;
    const int prev = slot == 0 ? NS - 1 : slot - 1;
    const int next = slot + 1 == NS ? 0 : slot + 1;
    auto behind = [&](auto half) POETX_INLINE {
      return [&](auto r) POETX_INLINE {
        if constexpr (kSteady) {
          constexpr int row = decltype(half)::value * FM + decltype(r)::value;
          for_each<PER_ROW>([&](auto c) POETX_INLINE {
            issue(prev, t + NS - 1,
                  std::integral_constant<int, row * PER_ROW + decltype(c)::value>{},
                  std::true_type{});
          });
        }
      };
    };
    read(slot, kSecond);
    if (!kSteady && t + NS - 1 < steps) issue_all(prev, t + NS - 1);
    __builtin_amdgcn_sched_barrier(0);
    products(kFirst, first, behind(kFirst));
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(first)::value) add_block(1);  // (of the block before)
    if (kSteady || t + 1 < steps) {
      if constexpr (kSteady) wait_vm<(NS - 3) * LPW + FIRST_HALF>();
      else wait_steps<LPW, NS>(min(NS - 2, steps - 2 - t));
      wait_lds();
      barrier_nofence();
      if constexpr (!kSteady) clear_tail(next, t + 1);
      read(next, kFirst);
    }
    __builtin_amdgcn_sched_barrier(0);
    products(kSecond, first, behind(kSecond));
    if constexpr (decltype(last)::value) add_block(0);
  };

  for_each<NS - 1>([&](auto t) POETX_INLINE {
    if (decltype(t)::value < steps) issue_all(decltype(t)::value, decltype(t)::value);
  });
  wait_steps<LPW, NS>(min(NS - 1, steps) - 1);
  barrier_nofence();
  clear_tail(0, 0);
  read(0, kFirst);
  int t = 0;
  for (; t + 2 * NS - 1 < steps; t += NS)
    for_each<NS>([&](auto q) POETX_INLINE {
      constexpr int Q = decltype(q)::value;
      step(Q, t + Q, std::true_type{}, std::bool_constant<Q == 0>{},
           std::bool_constant<Q == NS - 1>{});
    });
  for (int slot = 0; t < steps; ++t, slot = slot + 1 == NS ? 0 : slot + 1)
    step(slot, t, std::false_type{}, std::true_type{}, std::true_type{});
  __builtin_amdgcn_sched_barrier(0);
  settle_after();
  __builtin_amdgcn_sched_barrier(0);
  add_block(1);

  end.template run<T, FM, FN>(p, acc, m0 + wm * TM, n0 + wn * TN, part_k, nt * WN + wn, lane);
}

}  // namespace
}  // namespace poetx
