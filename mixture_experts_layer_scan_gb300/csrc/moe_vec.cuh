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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(x));
  return a;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A vector of W bytes as pairs of fp32 (a single element: the pair's second is 0).
template <typename T, int W>
__device__ __forceinline__ void widen2(const typename Word<W>::type& v, float2 (&f)[(W / sizeof(T) + 1) / 2]) {
  constexpr int N = W / sizeof(T);
  float g[N];
  widen<T, W>(v, g);
#pragma unroll
  for (int i = 0; i < (N + 1) / 2; ++i) f[i] = make_float2(g[2 * i], 2 * i + 1 < N ? g[2 * i + 1 < N ? 2 * i + 1 : 0] : 0.0f);
}
template <typename T, int W>
__device__ __forceinline__ typename Word<W>::type narrow2(const float2 (&f)[(W / sizeof(T) + 1) / 2]) {
  constexpr int N = W / sizeof(T);
  float g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) g[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
  return narrow<T, W>(g);
}

}  // namespace moe
