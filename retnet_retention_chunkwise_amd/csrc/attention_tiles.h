// Building blocks of the attention kernels: tiles of rows staged from strided
// tensors into LDS, and the 16x16 matrix products on them, for bf16 and fp32
// alike.
//
// Every product is C[r][c] += sum_k A[r][k] B[k][c] on 16x16 accumulators: lane
// l holds C[4 (l / 16) + i][l % 16], i = 0..3.  Operands are eight values per
// lane, A[l % 16][k] and B[k][l % 16] for the lane's eight k.  Which k belong to
// which lane is free as long as A and B agree, and two ways are used:
//   along a row (rows_frag): k = 8 (l / 16) + 0..7, consecutive channels;
//   along tile rows (cols_frag): k = 4 (l / 16) + 0..3 and 16 + the same, which
//   is what two accumulators of a former product hold, so that probabilities
//   become operands without leaving their lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention.h"
#include "common.h"
#include "gfx950.h"
#include "vec_io.h"

namespace ret {

template <typename E>
struct Mma;
template <>
struct Mma<uint16_t> {
  typedef bf16x8 Frag;
  static constexpr bool kSkip = false;
  __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c, int = 32) { return mfma(a, b, c); }
  // Two accumulators as an operand along their rows (round to nearest even).
  __device__ __forceinline__ static Frag pack(f32x4 lo, f32x4 hi) { return pack_bf16x8(lo, hi); }
};
template <>
struct Mma<float> {
  typedef f32x8 Frag;
  // A block of 16 channels is four instructions of 32 clocks: kernels leave out
  // those behind the row (a uniform branch each), n of a product's 32 counting.
  static constexpr bool kSkip = true;
  __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c, int n = 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    if (n > 16) {
#pragma unroll
      for (int i = 4; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    }
    return c;
  }
  __device__ __forceinline__ static Frag pack(f32x4 lo, f32x4 hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// A tile of rows of DIM elements in LDS, in one of two layouts.
//   padded (kDma false): rows LD elements apart, 32 bytes (fp32: 16) more than
//     the row.  With bf16 the 16-byte reads of 16 rows and the transposing reads
//     then both run at 210-220 bytes a clock and compute unit; with 16 bytes more
//     at 120, with none at 32 and 64.
//   swizzled (kDma true, bf16): rows without a gap, as loads straight into LDS
//     leave them, and the row's 16-byte pieces in another order: piece c of row r
//     lies at place c ^ turn(r), turn even.  Transposing reads take two pieces of
//     eight neighbouring rows at a time, which turn puts into different pairs of
//     places.  16-byte reads take one piece of rows 0-3 and 12-15 and the next of
//     rows 4-11 (then the other way round): rows that share a turn are of different
//     sets, and meet different places of their pair.  So both meet every bank once
//     (no conflicts counted; rows at 247 bytes a clock and compute unit, columns at
//     204; with turns that differ in all 16 rows the rows ran at 127).
template <typename E, int DIM, bool kDma>
struct Tile {
  static constexpr int LD = DIM + (kDma ? 0 : sizeof(E) == 2 ? 16 : 4);
  static constexpr int PIECES = DIM * static_cast<int>(sizeof(E)) / 16;
  static_assert(!kDma || sizeof(E) == 2, "the swizzled layout is of bf16 rows");
  static_assert(PIECES >= 8 && (PIECES & (PIECES - 1)) == 0, "a power of two of pieces");
  __device__ __forceinline__ static int turn(int row) {
    return PIECES >= 16 ? (row & 7) << 1 : (row >> 1 & 3) << 1;
  }

  // A[row][channels] of row row0 + lane % 16: bf16 the eight channels from c0 + 8 (lane / 16),
  // fp32 the four from c0 + 4 (lane / 16) and those 16 further.
  __device__ __forceinline__ static typename Mma<E>::Frag rows(const E* tile, int row0, int c0, int lane) {
    const int r = lane & 15;
    if constexpr (kDma) {
      const int at = r * DIM + (((lane >> 4) ^ turn(r)) << 3);
      return *reinterpret_cast<const bf16x8*>(tile + row0 * DIM + (at ^ c0));
    } else {
      const E* p = tile + (row0 + r) * LD + c0 + 16 / static_cast<int>(sizeof(E)) * (lane >> 4);
      if constexpr (sizeof(E) == 2) {
        return *reinterpret_cast<const bf16x8*>(p);
      } else {
        return Mma<float>::pack(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16));
      }
    }
  }

  // A[channel][rows]: of channel c0 + lane % 16, the rows row0 + 4 (lane / 16) + 0..3 and those 16 further.
  __device__ __forceinline__ static typename Mma<E>::Frag cols(const E* tile, int row0, int c0, int lane) {
    const int j = lane & 15, g = lane >> 4;
    if constexpr (kDma) {
      const int r = 4 * g + j / 4, at = r * DIM + (((j >> 1 & 1) ^ turn(r)) << 3) + 4 * (j & 1);
      const uint16_t* p = tile + row0 * DIM + (at ^ c0);
      return join(lds_read_tr(p), lds_read_tr(p + 16 * DIM));
    } else if constexpr (sizeof(E) == 2) {
      const uint16_t* p = tile + (row0 + 4 * g + j / 4) * LD + c0 + 4 * (j % 4);
      return join(lds_read_tr(p), lds_read_tr(p + 16 * LD));
    } else {
      const float* p = tile + (row0 + 4 * g) * LD + c0 + j;
      f32x8 f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = p[e * LD];
        f[4 + e] = p[(16 + e) * LD];
      }
      return f;
    }
  }
};

// A lane's 16 bytes of a row of n elements, nominally from element c on.
// kWhole: rows end with a piece (n a multiple of CE); a piece behind the row
// reads the row's last.  Otherwise a piece that the row ends in is read so far
// back that it ends with the row, and shifted when it is used, with zeros behind
// the row.  No lane leaves the others: with a branch for the lanes of a row's end,
// masks were spilled and the compiler placed a copy of an address in front of the
// instruction that gave the lanes back, which sent stores anywhere.  What a whole
// row's padding holds is left: it meets zeros in the other operand or fills outputs
// that are not stored.
template <typename E, bool kWhole>
struct Piece16 {
  static constexpr int CE = 16 / static_cast<int>(sizeof(E));
  int at, by;
  __device__ __forceinline__ Piece16(int c, int n) : at(min(c, kWhole ? n - CE : max(n - CE, 0))), by(c - at) {}
  // of the row that starts off bytes behind p
  __device__ __forceinline__ u32x4 load(const char* p, unsigned off, int n) const {
    typedef typename RawOf<16, static_cast<int>(sizeof(E))>::at At;
    if (kWhole || n >= CE) return *reinterpret_cast<const At*>(p + (off + at * static_cast<unsigned>(sizeof(E))));
    const E* row = reinterpret_cast<const E*>(p + off);
    E e[CE];
#pragma unroll
    for (int i = 0; i < CE; ++i) {
      const E y = row[i < n ? i : 0];
      e[i] = i < n ? y : E(0);
    }
    u32x4 x;
    __builtin_memcpy(&x, e, 16);
    return x;
  }
  __device__ __forceinline__ u32x4 finish(u32x4 x) const {
    if constexpr (!kWhole) {
      if constexpr (sizeof(E) == 2) {
        const u32x4 y = {x[0] >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16, x[2] >> 16 | x[3] << 16, x[3] >> 16};
        if (by & 1) x = y;
      }
      const int words = by * static_cast<int>(sizeof(E)) / 4;
      if (words & 1) x = u32x4{x[1], x[2], x[3], 0};
      if (words & 2) x = u32x4{x[2], x[3], 0, 0};
      x = zero_behind(x);
    }
    return x;
  }
  __device__ __forceinline__ u32x4 zero_behind(u32x4 x) const { return by >= CE ? u32x4{0, 0, 0, 0} : x; }
};

// ROWS rows of MAPS parts of d elements, each part padded to D, on their way
// from memory to LDS: THREADS threads, 16 bytes a piece.  load() only requests;
// store() waits, and puts zeros for the rows from n on (which load the last row).
template <typename E, int ROWS, int MAPS, int D, int THREADS, bool kWhole>
struct Stage {
  static constexpr int CE = 16 / static_cast<int>(sizeof(E));
  static constexpr int CH = MAPS * D / CE;               // pieces of a row
  static constexpr int STEP = THREADS / CH;              // rows of one round
  static constexpr int N = ROWS / STEP;                  // rounds
  static_assert(THREADS % CH == 0 && ROWS % STEP == 0, "a thread stays in its columns, rounds are full");
  static_assert(ROWS * kMaxTokenStride * sizeof(E) <= 1UL << 32, "a place in the tile has 32 bits");
  u32x4 r[N];
  Piece16<E, kWhole> piece;
  int row, col;  // of the thread's first piece in the tile
  int part;      // elements in front of its part of a row
  __device__ __forceinline__ Stage(int d, int tid)
      : piece((tid % CH - (MAPS > 1 ? tid % CH / (D / CE) : 0) * (D / CE)) * CE, d),
        row(tid / CH),
        col(tid % CH * CE),
        part(MAPS > 1 ? tid % CH / (D / CE) * d : 0) {}

  // Rows row0.. of base, stride (at most kMaxTokenStride) apart; n > row0 rows are
  // readable.  A tile's address is uniform, a thread's place in it 32 bits.
  __device__ __forceinline__ void load(const E* base, long stride, int row0, int n, int d) {
    const char* p = reinterpret_cast<const char*>(base + row0 * stride);
    const unsigned step = static_cast<unsigned>(stride) * sizeof(E);
    unsigned at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] = (row + i * STEP) * step;
    if (row0 + ROWS > n) {
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = min(row + i * STEP, n - 1 - row0) * step;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = piece.load(p, at[i] + part * static_cast<unsigned>(sizeof(E)), d);
  }
  __device__ __forceinline__ void store(E* tile, int row0, int n) {
    if (row0 + ROWS > n) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (row0 + row + i * STEP >= n) r[i] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<u32x4*>(tile + (row + i * STEP) * Tile<E, MAPS * D, false>::LD + col) = piece.finish(r[i]);
  }
};

// Loads straight into LDS: lane l's BYTES (16 or 4) at p + off go to tile + l BYTES.
// Written as assembly, without an output register, because the compiler would wait
// for them to arrive in front of the next read of any tile; the wait is in
// dma_barrier().  m0 holds the LDS address; the wait states cover m0, and the
// pointer where it comes out of a vector register.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0, named as clobbered, is reserved
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* p, unsigned off, const void* tile) {
  static_assert(BYTES == 16 || BYTES == 4, "a piece or a word");
  const unsigned at = static_cast<unsigned>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)(tile)));
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(p) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"(at), "v"(off), "s"(p) : "memory", "m0");
}
#pragma clang diagnostic pop

// ROWS rows of MAPS parts of d elements (16-byte pieces at 16-byte addresses),
// straight into a swizzled tile of MAPS D elements a row, by NW waves.  A wave's
// load fills 64 places in a row; each lane picks the piece that belongs to its
// place.  Rows from n on repeat the last, pieces behind a part the part's last:
// they meet masked scores, or zeros in the other operand.  COUNT loads a wave.
template <int ROWS, int MAPS, int D, int NW>
struct Dma {
  typedef Tile<uint16_t, MAPS * D, true> T;
  static constexpr int COUNT = ROWS * T::PIECES / 64 / NW, STEP = NW * 64 / T::PIECES;  // rows of one round
  static_assert(COUNT >= 1 && COUNT * NW * 64 == ROWS * T::PIECES, "every wave has as many loads");
  static_assert(ROWS * kMaxTokenStride * 2 <= 1L << 32, "a place in the tile has 32 bits");
  int row;
  unsigned piece[COUNT];  // bytes in front of the lane's pieces in their rows
  __device__ __forceinline__ Dma(int d, int wave, int lane) : row((wave * 64 + lane) / T::PIECES) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int c = (lane % T::PIECES) ^ T::turn(row + i * STEP), map = c / (D / 8);
      piece[i] = 2 * (map * d + min(8 * (c - map * (D / 8)), d - 8));
    }
  }
  __device__ __forceinline__ void load(const uint16_t* base, long stride, int row0, int n, uint16_t* tile, int wave) const {
    const uint16_t* p = base + row0 * stride;
    const unsigned step = static_cast<unsigned>(stride) * 2;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      load_to_lds<16>(p, static_cast<unsigned>(min(row + i * STEP, n - 1 - row0)) * step + piece[i],
                      tile + (i * NW + wave) * 512);
  }
};

// Workgroup barrier in front of a tile that was loaded straight into LDS: waits
// until all but this wave's last LATER loads have arrived, and for its LDS reads.
template <int LATER>
__device__ __forceinline__ void dma_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
}

// Walks the tiles first..last-1 of a workgroup through LDS slots that loads fill
// directly: request(i, slot) sends the loads of tile i, use(i, slot) works on it.
// Three slots: one tile in use, one that has been on its way for a tile's time,
// one that is requested now; two where three would keep a second workgroup off
// the compute unit.  Every wave sends COUNT loads for every tile (behind the end
// for the last again), so that the loads that may still be under way at a barrier
// are a constant.  The slots are separate arrays and known in every call, which
// lets the compiler see that reads of one do not wait for loads to another.
template <int SLOTS, int COUNT, typename R, typename U>
__device__ __forceinline__ void walk_tiles(int first, int last, R&& request, U&& use) {
  typedef std::integral_constant<int, 0> C0;
  typedef std::integral_constant<int, 1> C1;
  typedef std::integral_constant<int, 2> C2;
  if (first >= last) return;
  request(first, C0());
  if constexpr (SLOTS == 3) {
    request(min(first + 1, last - 1), C1());
    for (int i = first;; i += 3) {
      dma_barrier<COUNT>();
      request(min(i + 2, last - 1), C2());
      use(i, C0());
      if (i + 1 >= last) break;
      dma_barrier<COUNT>();
      request(min(i + 3, last - 1), C0());
      use(i + 1, C1());
      if (i + 2 >= last) break;
      dma_barrier<COUNT>();
      request(min(i + 4, last - 1), C1());
      use(i + 2, C2());
      if (i + 3 >= last) break;
    }
  } else {
    for (int i = first;; i += 2) {
      dma_barrier<0>();
      request(min(i + 1, last - 1), C1());
      use(i, C0());
      if (i + 1 >= last) break;
      dma_barrier<0>();
      request(min(i + 2, last - 1), C0());
      use(i + 1, C1());
      if (i + 2 >= last) break;
    }
  }
  dma_barrier<0>();  // nothing is on its way to LDS when the workgroup ends
}

// This wave's number in its workgroup, known to be the same in all its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6); }

// B[channels][column]: column col's row of MAPS parts of d elements, padded with
// zeros to D each, channels along a row; zeros where the column is not in (row
// is readable all the same).
template <typename E, int MAPS, int D, bool kWhole>
__device__ __forceinline__ void load_columns(const E* row, bool in, int d, int lane,
                                             typename Mma<E>::Frag (&f)[MAPS * D / 32]) {
  constexpr int CE = 16 / static_cast<int>(sizeof(E));
#pragma unroll
  for (int k = 0; k < MAPS * D / 32; ++k) {
    const int map = k / (D / 32), c = (k - map * (D / 32)) * 32 + CE * (lane >> 4);
    u32x4 x[8 / CE];
#pragma unroll
    for (int i = 0; i < 8 / CE; ++i) {
      const Piece16<E, kWhole> piece(c + i * 16, d);
      x[i] = piece.zero_behind(piece.finish(piece.load(reinterpret_cast<const char*>(row + map * d), 0, d)));
      if (!in) x[i] = u32x4{0, 0, 0, 0};
    }
    __builtin_memcpy(&f[k], x, sizeof(f[k]));
  }
}

// Four consecutive elements of a row of n from element c on; c is a multiple of
// 4, elements from n on are left out.
template <typename E, bool kWhole>
__device__ __forceinline__ void store4(E* row, int c, int n, f32x4 x) {
  if constexpr (kWhole) {
    typename RawOf<4 * sizeof(E), sizeof(E)>::type r;
    if constexpr (sizeof(E) == 4) {
      r = __builtin_bit_cast(u32x4, x);
    } else {
      r[0] = static_cast<uint32_t>(f32_to_bf16(x[0])) | (static_cast<uint32_t>(f32_to_bf16(x[1])) << 16);
      r[1] = static_cast<uint32_t>(f32_to_bf16(x[2])) | (static_cast<uint32_t>(f32_to_bf16(x[3])) << 16);
    }
    if (c < n) *reinterpret_cast<typename RawOf<4 * sizeof(E), sizeof(E)>::at*>(row + c) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < n) Elem<E>::store(row, c + i, x[i]);
  }
}

// The largest of x over lanes l, l^16, l^32, l^48, in each of them.
__device__ __forceinline__ float row4_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float y = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(y), __float_as_uint(y), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// A border the compiler moves no instruction over.  The loops read the operands of
// a stage from LDS one stage ahead of their products; left alone, the compiler
// moves the reads down to their uses to save registers, and every two products
// then wait for an LDS access.  (fp32 products are slow enough without.)
template <typename E>
__device__ __forceinline__ void stage_border() {
  if constexpr (sizeof(E) == 2) __builtin_amdgcn_sched_barrier(0);
}

// Products go before the other wave's exponentials on a SIMD: a product occupies
// the issue for a quarter of its time, the rest is the other wave's.
__device__ __forceinline__ void products_first() { __builtin_amdgcn_s_setprio(1); }
__device__ __forceinline__ void products_done() { __builtin_amdgcn_s_setprio(0); }

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace ret
