// Device helpers shared by the token operators (layer norm, rotary positions,
// attention): vectors of VEC consecutive values as fp32, rounding to bf16,
// exact division by a launch constant.
#pragma once

#include "internal.h"

namespace st {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// n / d for 0 <= n < 2^31 as (n * m) >> p with p = 31 + ceil(log2 d) and
// m = ceil(2^p / d) < 2^32 (the round-up multiplier: its error stays below
// 1 / d, so the floor is exact)
struct Div31 {
  uint32_t m;
  int32_t p;
  uint32_t d;
};
inline Div31 div31(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  return Div31{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l, d};
}
__device__ __forceinline__ uint32_t quo(uint32_t n, const Div31& f) { return (uint32_t)(((uint64_t)n * f.m) >> f.p); }

// two values rounded to bf16 (nearest even, NaN kept) in one word
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct BF16 { static constexpr int kSize = 2; };
struct F32 { static constexpr int kSize = 4; };

// VEC consecutive values at p (aligned to min(16, VEC * size) bytes)
template <class T, int VEC> __device__ __forceinline__ void load_vec(const char* p, float (&x)[VEC]) {
  if constexpr (T::kSize == 4) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const f32x4_t v = reinterpret_cast<const f32x4_t*>(p)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = reinterpret_cast<const float*>(p)[i];
    }
  } else {
    if constexpr (VEC == 8) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) { x[2 * i] = bf16_lo(w[i]); x[2 * i + 1] = bf16_hi(w[i]); }
    } else if constexpr (VEC == 4) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
      for (int i = 0; i < 2; ++i) { x[2 * i] = bf16_lo(w[i]); x[2 * i + 1] = bf16_hi(w[i]); }
    } else if constexpr (VEC == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      x[0] = bf16_lo(w); x[1] = bf16_hi(w);
    } else {
      static_assert(VEC == 1, "1, 2, 4 or 8 values");
      x[0] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
    }
  }
}

template <class T, int VEC> __device__ __forceinline__ void store_vec(char* p, const float (&x)[VEC]) {
  if constexpr (T::kSize == 4) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i)
        reinterpret_cast<f32x4_t*>(p)[i] = f32x4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) reinterpret_cast<float*>(p)[i] = x[i];
    }
  } else {
    if constexpr (VEC == 8) {
      *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                               pack_bf16(x[6], x[7])};
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    } else if constexpr (VEC == 2) {
      *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(x[0], 0.f);
    }
  }
}

// the same past the caches' reach: for outputs that only a later pass reads
template <class T, int VEC> __device__ __forceinline__ void store_vec_nt(char* p, const float (&x)[VEC]) {
  if constexpr (T::kSize == 4) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i)
        __builtin_nontemporal_store(f32x4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]}, reinterpret_cast<f32x4_t*>(p) + i);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) __builtin_nontemporal_store(x[i], reinterpret_cast<float*>(p) + i);
    }
  } else {
    if constexpr (VEC == 8) {
      __builtin_nontemporal_store(u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                               pack_bf16(x[6], x[7])}, reinterpret_cast<u32x4_t*>(p));
    } else if constexpr (VEC == 4) {
      __builtin_nontemporal_store(u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, reinterpret_cast<u32x2_t*>(p));
    } else if constexpr (VEC == 2) {
      __builtin_nontemporal_store(pack_bf16(x[0], x[1]), reinterpret_cast<uint32_t*>(p));
    } else {
      __builtin_nontemporal_store((uint16_t)pack_bf16(x[0], 0.f), reinterpret_cast<uint16_t*>(p));
    }
  }
}

}  // namespace st
