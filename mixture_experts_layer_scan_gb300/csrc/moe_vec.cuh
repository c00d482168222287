// Vectors of a row: W bytes as one load or store, widened to and rounded from fp32.
#pragma once

#include "moe_device.cuh"

namespace moe {

// W bytes as one load or store
template <int W>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

__device__ __forceinline__ void zero_word(uint4& v) { v = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero_word(uint2& v) { v = make_uint2(0, 0); }
__device__ __forceinline__ void zero_word(uint32_t& v) { v = 0; }
__device__ __forceinline__ void zero_word(uint16_t& v) { v = 0; }

// element e of a vector of W bytes, widened; and packing
template <typename T, int W>
__device__ __forceinline__ void widen(const typename Word<W>::type& v, float (&f)[W / sizeof(T)]) {
  if constexpr (W == 2) {
    f[0] = bf16_bits_to_f32(v);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
        f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
      }
    }
  }
}
template <typename T, int W>
__device__ __forceinline__ typename Word<W>::type narrow(const float (&f)[W / sizeof(T)]) {
  typename Word<W>::type v;
  if constexpr (W == 2) {
    const __nv_bfloat16 b = __float2bfloat16_rn(f[0]);
    v = *reinterpret_cast<const uint16_t*>(&b);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
  return v;
}

// widest vector (bytes) that divides a row
inline int row_word(long row_bytes) {
  return row_bytes % 16 == 0 ? 16 : row_bytes % 8 == 0 ? 8 : row_bytes % 4 == 0 ? 4 : 2;
}

}  // namespace moe
