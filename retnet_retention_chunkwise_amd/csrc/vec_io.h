// VEC consecutive elements of a row as fp32, for the streaming kernels: one
// access of VEC * sizeof(element) bytes (at most 16) at any address that is a
// multiple of the element's size (global memory takes unaligned vectors).  All
// accesses are non-temporal: each element is used once per call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace ret {

// type: a value of BYTES bytes; at: the same in memory at multiples of ALIGN bytes.
template <int BYTES, int ALIGN>
struct RawOf;
template <>
struct RawOf<2, 2> {
  typedef uint16_t type;
  typedef uint16_t at;
};
template <>
struct RawOf<4, 2> {
  typedef unsigned int type;
  typedef unsigned int at __attribute__((aligned(2)));
};
template <>
struct RawOf<8, 2> {
  typedef unsigned int type __attribute__((ext_vector_type(2)));
  typedef unsigned int at __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct RawOf<16, 2> {
  typedef unsigned int type __attribute__((ext_vector_type(4)));
  typedef unsigned int at __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct RawOf<4, 4> {
  typedef unsigned int type;
  typedef unsigned int at __attribute__((aligned(4)));
};
template <>
struct RawOf<8, 4> {
  typedef unsigned int type __attribute__((ext_vector_type(2)));
  typedef unsigned int at __attribute__((ext_vector_type(2), aligned(4)));
};
template <>
struct RawOf<16, 4> {
  typedef unsigned int type __attribute__((ext_vector_type(4)));
  typedef unsigned int at __attribute__((ext_vector_type(4), aligned(4)));
};

template <typename E, int VEC>
struct VecIO {
  typedef RawOf<VEC * static_cast<int>(sizeof(E)), static_cast<int>(sizeof(E))> R;
  typedef typename R::type Raw;

  __device__ __forceinline__ static Raw load(const E* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename R::at*>(p));
  }
  __device__ __forceinline__ static void unpack(Raw r, float (&x)[VEC]) {
    if constexpr (sizeof(E) == 4) {
      if constexpr (VEC == 1) {
        x[0] = __uint_as_float(r);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float(r[i]);
      }
    } else {
      if constexpr (VEC == 1) {
        x[0] = bf16_to_f32(r);
      } else if constexpr (VEC == 2) {
        x[0] = __uint_as_float(r << 16);
        x[1] = __uint_as_float(r & 0xffff0000u);
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          x[2 * i] = __uint_as_float(r[i] << 16);
          x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
      }
    }
  }
  // rounds to nearest even for bf16
  __device__ __forceinline__ static void store(E* p, const float (&x)[VEC]) {
    Raw r;
    if constexpr (sizeof(E) == 4) {
      if constexpr (VEC == 1) {
        r = __float_as_uint(x[0]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r[i] = __float_as_uint(x[i]);
      }
    } else {
      if constexpr (VEC == 1) {
        r = f32_to_bf16(x[0]);
      } else if constexpr (VEC == 2) {
        r = static_cast<uint32_t>(f32_to_bf16(x[0])) | (static_cast<uint32_t>(f32_to_bf16(x[1])) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
          r[i] = static_cast<uint32_t>(f32_to_bf16(x[2 * i])) | (static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16);
      }
    }
    __builtin_nontemporal_store(r, reinterpret_cast<typename R::at*>(p));
  }
};

// VEC fp32 parameters (weights and the like), kept in cache.
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
    typedef float f32v4 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) {
      const f32v4 v = *reinterpret_cast<const f32v4*>(p + 4 * k);
      x[4 * k] = v[0]; x[4 * k + 1] = v[1]; x[4 * k + 2] = v[2]; x[4 * k + 3] = v[3];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = p[e];
  }
}

// A thread's piece of a row of n elements (n >= VEC): the VEC elements from c
// on, or, where the row ends inside them, the row's last VEC elements, of which
// the first skip belong to the piece before (it has them too, with the same
// values, and stores them too).
struct Piece {
  int at, skip;
  bool in;
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ Piece(int c, int n, int vec)
      : at(c + vec <= n ? c : c < n ? n - vec : 0), skip(c + vec <= n ? 0 : c < n ? c + vec - n : vec), in(c < n) {}
  // whether element e counts in a sum over the row
  __device__ __forceinline__ bool own(int e) const { return e >= skip; }
};

}  // namespace ret
