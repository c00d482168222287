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

// A vector of W bytes (a multiple of 4) widened, and packed again
template <typename T, int W>
__device__ __forceinline__ void widen(const typename Word<W>::type& v, float (&f)[W / sizeof(T)]) {
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
template <typename T, int W>
__device__ __forceinline__ typename Word<W>::type narrow(const float (&f)[W / sizeof(T)]) {
  typename Word<W>::type v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
    else w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

// Pairs of fp32 in one packed instruction, each half one rounding.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(z) : "l"(x), "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(c.x), "=f"(c.y) : "l"(z));
  return c;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(x));
  return a;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace moe
