// Quantisation to e4m3 by blocks: one fp32 scale per row and 128 consecutive columns.
//
//   a = max |x| over the block;  s = max(a * (1/448), 2^-126), 1 where a = 0
//   q = e4m3(x * (1 / s)), round to nearest even, saturating
// with 1/448 a 32-bit constant and both products and the reciprocal 1 / s (once per block) one
// fp32 rounding each.  A
// block that holds a NaN gets a NaN scale, one that holds an infinity an infinite scale, and all
// its codes stand for no finite value: a fault upstream stays visible.  2^-126 keeps 1 / s finite.
//
// The SiLU form quantises h = SiLU(g) * u of a row [g | u] without storing h.  The scatter form
// serves the expert layer: row t's codes and scales go to the expert-sorted rows of its pairs.
//
// Bound by HBM: an element is read once and leaves as one byte.  16 lanes share a block (8
// elements each: 16-byte loads of bf16, 8-byte stores), so its maximum is four shuffles.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kQuantThreads = 256;

struct QuantDev {
  const void* x;
  uint8_t* q;
  float* scale;
  int T, K;           // rows, columns of the result (the SiLU form reads rows of 2 K)
  int nb;             // blocks per row
  const int32_t* inv; // scatter: sorted row of each pair (t * k + j), -1 for a pair left out
  int k;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
    v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <typename TIn, bool SILU, bool SCATTER>
__global__ void __launch_bounds__(kQuantThreads) k_quant_block(const QuantDev p) {
  pdl_enter();
  const int l16 = threadIdx.x & 15;
  const long units = (long)p.T * p.nb;
  const long step = (long)gridDim.x * (kQuantThreads / 16);
  const TIn* x = static_cast<const TIn*>(p.x);
  // (both halves of a warp run the same number of rounds: the shuffles name all 32 lanes)
  const long u0 = (long)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
  for (long base = u0 & ~1l; base < units; base += step) {
    const long u = base + (u0 & 1);
    const bool live = u < units;
    const int t = live ? (int)(u / p.nb) : 0;
    const int b = live ? (int)(u - (long)t * p.nb) : 0;
    const int c = b * 128 + l16 * 8;
    const bool on = live && c < p.K;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
      if constexpr (SILU) {
        float g[8], w[8];
        load8(x + (size_t)t * 2 * p.K + c, g);
        load8(x + (size_t)t * 2 * p.K + p.K + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu(g[i]) * w[i];
      } else {
        load8(x + (size_t)t * p.K + c, v);
      }
    }
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    const float s = block_scale_from_amax(a);
    const float r = 1.0f / s;
    uint2 code;
    code.x = pack_e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
    code.y = pack_e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
    if constexpr (SCATTER) {
      if (live) {
        for (int j = 0; j < p.k; ++j) {
          const int row = p.inv[(size_t)t * p.k + j];
          if (row < 0) continue;
          if (on) *reinterpret_cast<uint2*>(p.q + (size_t)row * p.K + c) = code;
          if (l16 == 0) p.scale[(size_t)row * p.nb + b] = s;
        }
      }
    } else {
      if (on) *reinterpret_cast<uint2*>(p.q + (size_t)t * p.K + c) = code;
      if (live && l16 == 0) p.scale[u] = s;
    }
  }
}

template <typename TIn, bool SILU, bool SCATTER>
cudaError_t launch_inst(const QuantDev& p, cudaStream_t s) {
  const long units = (long)p.T * p.nb;
  const long blocks = (units + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  const int grid = (int)std::min<long>(blocks, 152 * 8);
  MOE_LAUNCH((k_quant_block<TIn, SILU, SCATTER>), dim3(grid), dim3(kQuantThreads), 0, s, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_block(const void* x, bool bf16, bool silu_form, int T, int K, uint8_t* q, float* scale,
                               cudaStream_t s) {
  QuantDev p = {};
  p.x = x;
  p.q = q;
  p.scale = scale;
  p.T = T;
  p.K = K;
  p.nb = (K + 127) / 128;
  if (silu_form) return bf16 ? launch_inst<__nv_bfloat16, true, false>(p, s) : launch_inst<float, true, false>(p, s);
  return bf16 ? launch_inst<__nv_bfloat16, false, false>(p, s) : launch_inst<float, false, false>(p, s);
}

cudaError_t launch_quant_block_scatter(const void* x, int T, int K, int k, const int32_t* inv, uint8_t* q,
                                       float* scale, cudaStream_t s) {
  QuantDev p = {};
  p.x = x;
  p.q = q;
  p.scale = scale;
  p.T = T;
  p.K = K;
  p.nb = (K + 127) / 128;
  p.inv = inv;
  p.k = k;
  return launch_inst<__nv_bfloat16, false, true>(p, s);
}

}  // namespace moe
