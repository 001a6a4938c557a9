// Element types of the row operators (bf16, fp16, fp32): 16-byte pieces of a
// row as float, and back.
#pragma once

#include "common.hpp"

namespace moe {

inline size_t dtype_bytes(int dtype) {
  return dtype == MOE_DT_FP32 ? 4 : dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16 ? 2 : 0;
}

struct Bf16 {
  uint16_t bits;
};
struct Fp16 {
  uint16_t bits;
};

template <typename E>
__device__ __forceinline__ float to_f32(E v);
template <>
__device__ __forceinline__ float to_f32<Bf16>(Bf16 v) {
  return bf16_to_f32(v.bits);
}
template <>
__device__ __forceinline__ float to_f32<Fp16>(Fp16 v) {
  return (float)__builtin_bit_cast(_Float16, v.bits);
}
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}

// One rounding to the element type, to nearest even; infinities and NaN stay
// what they are (f32_to_bf16 of common.hpp is for finite values only).
template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) {
  return Bf16{__builtin_bit_cast(uint16_t, (__bf16)v)};
}
template <>
__device__ __forceinline__ Fp16 from_f32<Fp16>(float v) {
  return Fp16{__builtin_bit_cast(uint16_t, (_Float16)v)};
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// 16 bytes at any element's address, which the hardware takes in one access.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));

// N consecutive elements.  16 bytes pass as one value of four words: element by
// element the compiler joins them to smaller accesses (quantising 65536 rows of
// 2048: 92 us against 74; dispatch of 2048 rows of 4096 to 8 places: 42 against
// 32).
template <typename E, int N = 16 / (int)sizeof(E)>
struct Piece {
  static constexpr int kN = N;
  E e[N];

  __device__ __forceinline__ void load(const E* p) {
    if constexpr (sizeof(e) == 16) {
      const u32x4 w = *(const u32x4*)p;
      __builtin_memcpy(e, &w, 16);
    } else {
      __builtin_memcpy(e, p, sizeof(e));
    }
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (sizeof(e) == 16) {
      u32x4 w;
      __builtin_memcpy(&w, e, 16);
      *(u32x4*)p = w;
    } else {
      __builtin_memcpy(p, e, sizeof(e));
    }
  }
  __device__ __forceinline__ void store_past(E* p) const {  // past the caches (16 bytes)
    u32x4 w;
    static_assert(sizeof(e) == 16, "a whole piece");
    __builtin_memcpy(&w, e, 16);
    __builtin_nontemporal_store(w, (u32x4*)p);
  }
  __device__ __forceinline__ void load_past(const E* p) {
    static_assert(sizeof(e) == 16, "a whole piece");
    const u32x4 w = __builtin_nontemporal_load((const u32x4*)p);
    __builtin_memcpy(e, &w, 16);
  }
  // the first n elements only (n < N); the others are zero
  __device__ __forceinline__ void load_head(const E* p, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = i < n ? p[i] : E{};
  }
  __device__ __forceinline__ void store_head(E* p, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = e[i];
  }
  __device__ __forceinline__ void load_upto(const E* p, int n) {
    if (n >= N)
      load(p);
    else
      load_head(p, n);
  }
  __device__ __forceinline__ void store_upto(E* p, int n) const {
    if (n >= N)
      store(p);
    else
      store_head(p, n);
  }
};

// float sum of the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace moe
