// Low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + s[l] B_l (A_l x_t),  l = ids[t];  out[t] = base[t] where ids[t] = -1
//
// Two launches: h = s A x (fp32, in the workspace), then out = base + B h.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

namespace {

struct LoraDev {
  const __nv_bfloat16* x;  // [T][K]
  const __nv_bfloat16* a;  // [L][r][K]
  const __nv_bfloat16* b;  // [L][N][r]
  const int32_t* ids;
  const float* scale;      // [L] or null
  const void* base;        // [T][N] or null
  void* out;
  float* h;                // [T][r]
  int T, K, N, r, L;
  int* status;
};

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  float fa[8], fb[8];
  widen<__nv_bfloat16, 16>(a, fa);
  widen<__nv_bfloat16, 16>(b, fb);
#pragma unroll
  for (int c = 0; c < 8; ++c) acc = fmaf(fa[c], fb[c], acc);
  return acc;
}

// A warp to a token and a row of its A.
__global__ void __launch_bounds__(256) k_lora_shrink(const LoraDev p) {
  pdl_enter();
  const int lane = threadIdx.x & 31, i = blockIdx.y * 8 + (threadIdx.x >> 5);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int l = p.ids[t];
    if (l >= p.L || l < -1) {
      if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, MOE_ERR_DEVICE_INDEX);
      continue;
    }
    if (l < 0 || i >= p.r) continue;
    const uint4* xv = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.K);
    const uint4* av = reinterpret_cast<const uint4*>(p.a + ((size_t)l * p.r + i) * p.K);
    float acc = 0.f;
#pragma unroll 4
    for (int v = lane; v < p.K / 8; v += 32) acc = dot8(xv[v], av[v], acc);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) p.h[(size_t)t * p.r + i] = p.scale ? acc * p.scale[l] : acc;
  }
}

// A thread to a token and an output column.
template <typename T>
__global__ void __launch_bounds__(256) k_lora_expand(const LoraDev p) {
  pdl_enter();
  __shared__ float h[kLoraMaxRank];
  const int n = blockIdx.y * 256 + threadIdx.x;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int l = p.ids[t];
    const bool on = l >= 0 && l < p.L;
    __syncthreads();
    if (on)
      for (int i = threadIdx.x; i < p.r; i += 256) h[i] = p.h[(size_t)t * p.r + i];
    __syncthreads();
    if (n >= p.N) continue;
    const size_t at = (size_t)t * p.N + n;
    float acc = p.base ? to_f32(static_cast<const T*>(p.base)[at]) : 0.f;
    if (on) {
      const uint4* bv = reinterpret_cast<const uint4*>(p.b + ((size_t)l * p.N + n) * p.r);
      float d = 0.f;
      for (int v = 0; v < p.r / 8; ++v) {
        float fb[8];
        widen<__nv_bfloat16, 16>(bv[v], fb);
#pragma unroll
        for (int c = 0; c < 8; ++c) d = fmaf(fb[c], h[8 * v + c], d);
      }
      acc += d;
    }
    if constexpr (sizeof(T) == 4) static_cast<float*>(p.out)[at] = acc;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc);
  }
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int N, int r, int L) {
  (void)K;
  (void)N;
  (void)L;
  return ((size_t)T * r * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) {
  LoraDev p = {};
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.a = static_cast<const __nv_bfloat16*>(a.a);
  p.b = static_cast<const __nv_bfloat16*>(a.b);
  p.ids = a.ids;
  p.scale = a.scale;
  p.base = a.base;
  p.out = a.out;
  p.h = static_cast<float*>(a.workspace);
  p.T = a.T;
  p.K = a.K;
  p.N = a.N;
  p.r = a.r;
  p.L = a.L;
  p.status = a.status;
  const int rows = std::min(a.T, 1 << 16), cols = (a.N + 255) / 256;
  if (cols > 65535) return cudaErrorInvalidValue;
  MOE_LAUNCH(k_lora_shrink, dim3(rows, (a.r + 7) / 8), dim3(256), 0, s, p);
  if (a.out_bf16) MOE_LAUNCH(k_lora_expand<__nv_bfloat16>, dim3(rows, cols), dim3(256), 0, s, p);
  else MOE_LAUNCH(k_lora_expand<float>, dim3(rows, cols), dim3(256), 0, s, p);
  return cudaGetLastError();
}

}  // namespace moe
