// Sums over the LPR threads that hold one row, the same bits in each of them.
// LPR <= 64: consecutive lanes of a wave, DPP inside each 16-lane row and the
// cross-row swaps beyond it, all VALU.  LPR > 64: LPR / 64 consecutive waves,
// their wave sums exchanged through LDS.
#pragma once

#include <hip/hip_runtime.h>

namespace ret {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32 || N == 64, "lanes per row");
  v = dpp_add<0xB1>(v);                     // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);                     // quad_perm [2,3,0,1]
  if constexpr (N >= 8) v = dpp_add<0x141>(v);   // row_half_mirror: the other quad of 8 lanes
  if constexpr (N >= 16) v = dpp_add<0x140>(v);  // row_mirror: the other 8 lanes of 16
  if constexpr (N >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (N >= 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return v;
}

// LDS of one workgroup's exchanges: two slots used in turn, so that one barrier
// per exchange is enough (a slot is written again only after the barrier of
// the exchange in the other slot, which every reader of it has passed).
template <int THREADS>
struct RowExchange {
  float v[2][2][THREADS / 64];
};

// s0 and s1 become their sums over the row.  For LPR > 64 every thread of the
// workgroup calls it the same number of times; phase counts the calls.
template <int LPR, int THREADS>
__device__ __forceinline__ void row_sums(float& s0, float& s1, RowExchange<THREADS>& x, int& phase) {
  if constexpr (LPR <= 64) {
    s0 = lanes_sum<LPR>(s0);
    s1 = lanes_sum<LPR>(s1);
  } else {
    s0 = lanes_sum<64>(s0);
    s1 = lanes_sum<64>(s1);
    const int slot = phase++ & 1, w = threadIdx.x >> 6, first = w / (LPR / 64) * (LPR / 64);
    if ((threadIdx.x & 63) == 0) {
      x.v[slot][0][w] = s0;
      x.v[slot][1][w] = s1;
    }
    __syncthreads();
    s0 = s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < LPR / 64; ++i) {
      s0 += x.v[slot][0][first + i];
      s1 += x.v[slot][1][first + i];
    }
  }
}

}  // namespace ret
